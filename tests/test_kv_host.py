"""The paged 8-bit operators without a GPU: refusals on the host before any
CUDA call, and the 64-bit references against independent facts."""
import ctypes
import math

import pytest
import torch

import kv_ref
from barrier_free_message_gb300 import _build, sfar


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sfar.lib()


def ptrs(*values):
    return (ctypes.c_void_p * len(values))(*values)


GOOD = dict(R=2, q_heads=8, kv_heads=2, head_dim=64, page_tokens=16, pages=4)


@pytest.mark.parametrize("bad", [
    dict(R=0), dict(R=17), dict(kv_heads=0), dict(q_heads=7), dict(q_heads=0), dict(q_heads=1), dict(head_dim=96),
    dict(head_dim=0), dict(page_tokens=8), dict(page_tokens=48), dict(page_tokens=256), dict(pages=0),
    dict(pages=1 << 27), dict(pages=1 << 40)])
def test_create_refuses_bad_shapes(lib, bad):
    c = {**GOOD, **bad}
    step = 1 << 44
    arrays = [ptrs(*[step * (16 * i + r + 1) for r in range(16)]) for i in range(4)]
    h = lib.sfar_kv_create(c["R"], c["q_heads"], c["kv_heads"], c["head_dim"], c["page_tokens"], c["pages"], *arrays)
    assert h is None and lib.sfar_last_error() == sfar.SFAR_ERR_INVALID


def test_create_refuses_bad_pointers(lib):
    size = 4 * 2 * 16 * 64
    base = 1 << 20

    def arrays(**change):
        p = {"k0": base, "k1": base + size, "v0": base + 2 * size, "v1": base + 3 * size, "a0": base + 4 * size,
             "a1": base + 4 * size + 32, "b0": base + 4 * size + 64, "b1": base + 4 * size + 96, **change}
        return [ptrs(p[n + "0"], p[n + "1"]) for n in "kvab"]

    for change in (dict(k0=None), dict(v1=base + 3 * size + 8), dict(a1=base + 4 * size + 34), dict(b0=None),
                   dict(v0=base), dict(v1=base + size - 16), dict(b1=base + 4 * size + 28), dict(a0=base + 64)):
        assert lib.sfar_kv_create(2, 8, 2, 64, 16, 4, *arrays(**change)) is None
        assert lib.sfar_last_error() == sfar.SFAR_ERR_INVALID, change
    if not torch.cuda.is_available():       # the same arguments unchanged get as far as the device
        assert lib.sfar_kv_create(2, 8, 2, 64, 16, 4, *arrays()) is None
        assert lib.sfar_last_error() in (sfar.SFAR_ERR_CUDA, sfar.SFAR_ERR_UNSUPPORTED)


def test_null_handles(lib):
    p = ptrs(1 << 20, 1 << 21)
    one = 1 << 20
    assert lib.sfar_kv_plan(None, *[one] * 10, 1, 1, 1, None) == sfar.SFAR_ERR_INVALID
    assert lib.sfar_kv_append(None, p, p, one, 1, 8, 8, 8, 8, None) == sfar.SFAR_ERR_INVALID
    assert lib.sfar_kv_attention(None, p, p, one, one, one, 1, 1, 1, 8, 8, 8, 8, 1, 1.0, 0, None) == sfar.SFAR_ERR_INVALID
    assert lib.sfar_kv_status_get(None, None) == sfar.SFAR_ERR_INVALID
    assert lib.sfar_kv_reset(None, None) == sfar.SFAR_ERR_INVALID
    assert lib.sfar_quantize_fp8(None, p, p, p, 1, 1, 1, 1, None) == sfar.SFAR_ERR_INVALID
    assert lib.sfar_rowpar_gemm_fp8(None, p, p, p, p, p, 1, 16, 1, 16, 16, None) == sfar.SFAR_ERR_INVALID
    lib.sfar_kv_destroy(None)


def test_python_layer_refuses_wrong_tensors(lib):
    t = torch.zeros(2, 4, 2, 16, 64, dtype=torch.uint8)
    s = torch.zeros(2, 4, 2)
    for args in ((t.float(), t, s, s), (t, t[:, :, :, :8], s, s), (t, t, s[:, :3], s), (t, t, s, s.double()),
                 (t[..., ::2], t[..., ::2], s, s), ([t[0], t[1][:3]], t, s, s), (t, t[:1], s, s),
                 (t, t, s, s)):                                # on the CPU
        with pytest.raises(ValueError):
            sfar.SfarKv(*args, q_heads=4)


def test_calls_refuse_wrong_tensors(lib):
    """What the module that reads the tensors refuses before it makes the call (a closed handle would be next)."""
    native = sfar._tensors()
    i = torch.zeros(4, dtype=torch.int32)
    bf, f8, f32 = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 64, dtype=torch.uint8), torch.zeros(2, 1, 4)
    for args in (([bf[0]], 2, 3, "bf16"), (bf, 3, 3, "bf16"), (bf, 2, 2, "bf16"), (bf.float(), 2, 3, "bf16"), (f8, 2, 2, "fp32"),
                 (bf, 17, 3, "bf16"), ((bf[0], bf[1, :3]), 2, 3, "bf16"), ([1, 2], 2, 3, "bf16"), (None, 2, 3, "bf16"),
                 (bf, 2, 3, "bf16"), (f8, 2, 2, "byte"), ([f32[0], f32[1]], 2, 2, "fp32")):          # the last three: on the CPU
        with pytest.raises(ValueError):
            native.ranks(*args, "x")
    for call, args in ((native.plan, (4, i, i, i.view(2, 2), i, i[:2], i, i[:2], i, i, i, 0)), (native.plan, (4, *[1] * 10, 0)),
                       (native.append, (2, 2, 64, bf, bf, i, 0)), (native.attention, (2, 2, 64, bf, bf, i.view(2, 2), i, i, 1, 1.0, 0, 0)),
                       (native.quantize_fp8, (2, bf[:, :, 0], f8, f32, 0)), (native.rowpar_gemm_fp8, (2, f8, f32, f8, f32, bf[:, :, 0], 0))):
        with pytest.raises(ValueError):
            call(None, *args)
        with pytest.raises(TypeError):
            call(None, *args[1:])


def test_reference_rounds_as_the_format_does():
    """Every bf16 value of magnitude up to 448 against torch's conversion to e4m3."""
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[x.float().abs() <= 448]
    assert torch.equal(kv_ref.e4m3_round(x.double()), x.to(kv_ref.F8).double())


def test_reference_scale_exponent():
    for amax, e in ((0.0, -100), (448.0, 0), (449.0, 1), (896.0, 1), (1.75, -8), (1.7578125, -7), (2.0 ** -120, -100),
                    (3.3895313892515355e38, 120)):
        assert kv_ref.scale_exponent(amax) == e


def test_reference_plan_by_hand():
    """P = 4; request 0 grows into a page, 1 is dropped, 2 does not fit the pool, 3 needs no page, 4 not its row."""
    got = kv_ref.plan(4, [4, 5, 1, 2, 8], [1, -5, 8, 2, 1], [[7, -1], [3, 5], [2, -1], [1, -1], [9, 8]],
                      [-1] * 8 + [6, 4], [8, 2], 14)
    assert got["lens_out"] == [5, 0, 9, 4, 8][:2] + [1, 4, 8]
    assert got["taken"] == [1, 1, 0, 1, 0]
    assert got["starts"] == [0, 1, 1, 9, 11, 12]
    assert got["slots"] == [24] + [-1] * 8 + [6, 7] + [-1] * 3
    assert got["table"][0] == [7, 6] and got["state_out"] == [9, 3]
    assert got["ring"] == [3, 5] + [-1] * 6 + [6, 4]


def test_reference_attention_of_equal_keys_is_the_mean():
    k = torch.ones(2, 1, 16, 64).to(kv_ref.F8)
    v = torch.arange(32, dtype=torch.float32).view(2, 1, 16, 1).expand(2, 1, 16, 64).to(kv_ref.F8)
    s = torch.ones(2, 1)
    out, _ = kv_ref.attention(torch.ones(2, 1, 64), k, v, s, s, [[1, 0]], [20], [0, 2], 1.0, window=3)
    vals = torch.cat([v[1, 0, :, 0], v[0, 0, :4, 0]]).double()
    assert math.isclose(float(out[0, 0, 0]), float(vals[16:19].mean())) and math.isclose(float(out[1, 0, 5]), float(vals[17:20].mean()))
