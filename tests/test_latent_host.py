"""Rotary positions and the latent cache without a GPU: refusals on the host, the frequencies, and the 64-bit references
against independent facts."""
import ctypes
import math

import pytest
import torch

import latent_ref as ref
from barrier_free_message_gb300 import _build, sfar

INVALID = sfar.SFAR_ERR_INVALID


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sfar.lib()


def ptrs(*values):
    return (ctypes.c_void_p * len(values))(*values)


GOOD = dict(R=2, q_heads=8, latent_dim=512, rope_dim=64, page_tokens=16, pages=4)


@pytest.mark.parametrize("bad", [
    dict(R=0), dict(R=17), dict(q_heads=0), dict(q_heads=65536), dict(latent_dim=128), dict(latent_dim=0), dict(rope_dim=0),
    dict(rope_dim=48), dict(rope_dim=128), dict(page_tokens=8), dict(page_tokens=48), dict(page_tokens=256), dict(pages=0),
    dict(pages=1 << 27), dict(pages=1 << 40)])
def test_create_refuses_bad_shapes(lib, bad):
    c = {**GOOD, **bad}
    caches = ptrs(*[(r + 1) << 44 for r in range(16)])
    h = lib.sfar_latent_create(c["R"], c["q_heads"], c["latent_dim"], c["rope_dim"], c["page_tokens"], c["pages"], caches)
    assert h is None and lib.sfar_last_error() == INVALID


def test_create_refuses_bad_pointers(lib):
    size, base = 4 * 16 * 576 * 2, 1 << 20
    for bad in ((None, base), (base, None), (base, base + 8), (base, base), (base, base + size - 16)):
        assert lib.sfar_latent_create(2, 8, 512, 64, 16, 4, ptrs(*bad)) is None
        assert lib.sfar_last_error() == INVALID, bad
    assert lib.sfar_latent_create(2, 8, 512, 64, 16, 4, None) is None and lib.sfar_last_error() == INVALID
    if not torch.cuda.is_available():       # the same arguments unchanged get as far as the device
        assert lib.sfar_latent_create(2, 8, 512, 64, 16, 4, ptrs(base, base + size)) is None
        assert lib.sfar_last_error() in (sfar.SFAR_ERR_CUDA, sfar.SFAR_ERR_UNSUPPORTED)


def test_null_handles(lib):
    p, one = ptrs(1 << 20, 1 << 21), 1 << 20
    assert lib.sfar_rope(None, p, p, None, None, one, one, 1, 1, 0, 16, *[64] * 8, 0, 1.0, None) == INVALID
    assert lib.sfar_latent_plan(None, *[one] * 10, 1, 1, 1, None) == INVALID
    assert lib.sfar_latent_append(None, p, one, one, one, one, 1, 576, 1e-6, 0, 1.0, None) == INVALID
    assert lib.sfar_latent_gather(None, p, one, one, one, 1, 1, 1, 576, None) == INVALID
    assert lib.sfar_latent_attention(None, p, p, one, one, one, 1, 1, 1, 8, 8, 8, 8, 1, 1.0, None) == INVALID
    assert lib.sfar_latent_prompt(None, p, p, p, p, p, one, one, 1, 1, 1, 64, *[8] * 9, 1, 1.0, None) == INVALID
    assert lib.sfar_latent_status_get(None, None) == INVALID
    assert lib.sfar_latent_reset(None, None) == INVALID
    assert lib.sfar_test_latent_record_failure(None) == INVALID
    lib.sfar_latent_destroy(None)


# ----------------------------------------------------------------- frequencies
def frequencies(*a, **k):
    f, scale = sfar.rope_frequencies(*a, device="cpu", **k)
    return f.double(), scale


def test_frequencies_plain_and_linear(lib):
    f, scale = frequencies(64, base=500000.0)
    want = torch.tensor([500000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64)
    assert scale == 1.0 and (f - want).abs().le(want * 2.0 ** -24).all() and f[0] == 1.0
    g, scale = frequencies(64, base=500000.0, scaling="linear", factor=8.0)
    assert scale == 1.0 and torch.equal(g * 8, f)           # a power of two rounds alike


def test_frequencies_by_wavelength(lib):
    f, _ = frequencies(128, base=500000.0)
    g, scale = frequencies(128, base=500000.0, scaling="wavelength", factor=8.0, trained=8192.0, low=1.0, high=4.0)
    turns = 8192.0 * f / (2 * math.pi)
    assert scale == 1.0
    assert torch.equal(g[turns > 4.001], f[turns > 4.001]) and torch.equal(8 * g[turns < 0.999], f[turns < 0.999])
    mid = (turns > 1.001) & (turns < 3.999)
    s = (turns[mid] - 1) / 3
    assert mid.any() and (g[mid] - ((1 - s) / 8 + s) * f[mid]).abs().le(2.0 ** -22 * f[mid]).all()
    assert (g[:-1] > g[1:]).all()


def test_frequencies_by_ramp(lib):
    f, _ = frequencies(64)
    g, scale = frequencies(64, scaling="ramp", factor=40.0, trained=4096.0, low=1.0, high=32.0)
    # the pair that makes 32 turns of the trained context, and the one that makes 1
    d = [64 * math.log(4096 / (2 * math.pi * n)) / (2 * math.log(10000.0)) for n in (32, 1)]
    lo, hi = math.floor(d[0]), math.ceil(d[1])
    assert 0 < lo < hi < 32
    assert torch.equal(g[:lo + 1], f[:lo + 1]) and (40 * g[hi:] - f[hi:]).abs().le(2.0 ** -22 * f[hi:]).all()
    for i in range(lo, hi):
        s = (i - lo) / (hi - lo)
        assert abs(float(g[i] - (s / 40 + 1 - s) * f[i])) <= 2.0 ** -22 * float(f[i])
    assert scale == pytest.approx(0.1 * math.log(40) + 1, rel=2.0 ** -23)
    same, scale = frequencies(64, scaling="ramp", factor=1.0)
    assert (same - f).abs().le(2.0 ** -22 * f).all() and scale == 1.0


def test_frequencies_refuse(lib):
    for bad in (dict(rot=3), dict(base=1.0), dict(base=float("inf")), dict(scaling="linear", factor=0.5), dict(scaling="ramp", factor=2.0, low=0.0),
                dict(scaling="ramp", factor=2.0, low=2.0, high=2.0), dict(scaling="wavelength", factor=2.0, trained=0.0),
                dict(scaling="wavelength", factor=float("nan")), dict(rot=1 << 20)):
        with pytest.raises(sfar.SfarError):
            frequencies(**{"rot": 64, **bad})
    for bad in (dict(scaling="other"), dict(rot=0), dict(rot=-4)):
        with pytest.raises(ValueError):
            frequencies(**{"rot": 64, **bad})
    out = (ctypes.c_float * 32)()
    assert lib.sfar_rope_frequencies(out, None, 64, 10000.0, 0, 1.0, 1.0, 1.0, 2.0) == INVALID
    assert lib.sfar_rope_frequencies(None, ctypes.byref(ctypes.c_float()), 64, 10000.0, 0, 1.0, 1.0, 1.0, 2.0) == INVALID
    assert lib.sfar_rope_frequencies(out, ctypes.byref(ctypes.c_float()), 64, 10000.0, 4, 1.0, 1.0, 1.0, 2.0) == INVALID


# ------------------------------------------------------------------ references
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_reference_rope(layout):
    g = torch.Generator().manual_seed(0)
    x, pos = torch.randn(5, 3, 16, generator=g), torch.tensor([0, 1, 7, 1000, 1 << 20])
    freq = torch.rand(8, generator=g)
    y, off = ref.rope(x, pos, freq, layout, 2.0)
    assert torch.allclose(y.norm(dim=-1), 2 * x.double().norm(dim=-1)) and torch.equal(y[0], 2 * x[0].double())
    # the product of two rows goes by the difference of their positions alone
    a, _ = ref.rope(x[:1].expand(2, -1, -1), torch.tensor([5, 1005]), freq, layout, 1.0)
    b, _ = ref.rope(x[1:2].expand(2, -1, -1), torch.tensor([3, 1003]), freq, layout, 1.0)
    dots = (a * b).sum(-1)
    assert torch.allclose(dots[0], dots[1], atol=1e-9)
    # a back turn is the turn by the negative angle
    z, _ = ref.rope(y / 2, pos, -freq, layout, 1.0)
    assert torch.allclose(z, x.double(), atol=1e-9) and (off > 0).all()


def test_reference_rows_and_tolerance():
    g = torch.Generator().manual_seed(1)
    q, k = torch.randn(4, 32, generator=g), torch.randn(9, 32, generator=g)
    seen = ref.causal(4, 9, "cpu")
    assert seen.sum(1).tolist() == [6, 7, 8, 9]
    out, off = ref.rows(q, k, k[:, :24], seen, 0.1)
    for i in range(4):
        e = [math.exp(0.1 * float(q[i].double() @ k[j].double())) for j in range(6 + i)]
        want = sum(w * k[j, :24].double() for j, w in enumerate(e)) / sum(e)
        assert torch.allclose(out[i], want)
    for wrong in (ref.rows(q, k, k[:, :24], ref.causal(5, 9, "cpu")[:4], 0.1), ref.rows(q, k, k[:, :24], seen, 0.15),
                  ref.rows(q, k.flip(0), k[:, :24], seen, 0.1)):
        assert ((wrong[0] - out).abs() > off).any()
    none, _ = ref.rows(q, k, k, torch.zeros(4, 9, dtype=torch.bool), 0.1)
    assert (none == 0).all()


def test_reference_append():
    g = torch.Generator().manual_seed(2)
    x, w = torch.randn(3, 24, generator=g), torch.ones(16)
    y, _ = ref.append(x, w, torch.tensor([0, 0, 0]), torch.ones(4), "half", 1.0, 0.0, 16)
    assert torch.allclose(y[:, :16].square().mean(-1), torch.ones(3, dtype=torch.float64)) and torch.equal(y[:, 16:], x[:, 16:].double())
