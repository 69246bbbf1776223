"""Calls of the latent cache's operators that their headers allow, or refuse, at the edges of what tensors may share."""
import pytest
import torch

import latent_ref as ref
from barrier_free_message_gb300 import _build, sfar
from test_gpu_latent import fine, gen, ints

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def test_append_refuses_what_lies_in_a_cache():
    L, rot, T = 256, 32, 16
    cache = torch.zeros(2, 4, 16, L + rot, dtype=BF, device="cuda")
    kv = sfar.SfarLatent(cache, q_heads=1, rope_dim=rot)
    x, w, f = torch.ones(2, T, L + rot, dtype=BF, device="cuda"), torch.ones(L, dtype=BF, device="cuda"), torch.ones(rot // 2, device="cuda")
    pos, slots = ints([0] * T), ints(list(range(T)))
    good = dict(x=x, weight=w, pos=pos, freq=f, slots=slots)
    kv.append(**good)
    flat = cache.view(-1)
    for bad in (dict(x=cache[:, 2]), dict(x=[x[0], cache[0, 3]]), dict(weight=flat[512:512 + L]), dict(pos=flat.view(torch.int32)[:T]),
                dict(slots=flat.view(torch.int32)[64:64 + T]), dict(freq=flat.view(torch.float32)[-16:])):
        with pytest.raises(sfar.SfarError):
            kv.append(**{**good, **bad})
    # beside the caches is not in them
    line = torch.zeros(flat.numel() + x.numel(), dtype=BF, device="cuda")
    own = sfar.SfarLatent(line[:flat.numel()].view(cache.shape), q_heads=1, rope_dim=rot)
    own.append(line[flat.numel():].view(x.shape).copy_(x), w, pos, f, slots)
    torch.cuda.synchronize()
    fine(kv)
    fine(own)
    assert torch.equal(line[:flat.numel()].view(cache.shape), cache) and (cache[:, 0] != 0).all()
    kv.close()
    own.close()


@pytest.mark.parametrize("B", [1, 2, 33, 700, 8192])
@pytest.mark.parametrize("held", ["first", "last", "both ends", "some", "none"])
def test_gather_of_requests_without_rows(B, held):
    """Requests without rows before, between and after those that have some, and rows past the last one."""
    P, W, pages = 16, 288, 40
    cache = torch.randn(2, pages, P, W, generator=gen(B), device="cuda").to(BF)
    n = [0] * B
    for b in {"first": [0], "last": [B - 1], "both ends": [0, B - 1], "some": range(0, B, max(1, B // 9)), "none": []}[held]:
        n[b] = 1 + (5 * b) % 30
    table = torch.randint(0, pages, (B, 2), generator=gen(B + 1), device="cuda", dtype=torch.int32)
    starts = ref.offsets(n)
    kv = sfar.SfarLatent(cache, q_heads=1, rope_dim=32)
    for pad in (0, 1, 7):
        out = torch.full((2, starts[-1] + pad, W), 5.0, dtype=BF, device="cuda")
        kv.gather(out, table, ints(n), ints(starts))
        torch.cuda.synchronize()
        fine(kv)
        for b, m in enumerate(n):
            for r in range(2 if m else 0):
                assert torch.equal(out[r, starts[b]:starts[b + 1]], ref.held_rows(cache[r], table[b].tolist(), m, P))
        assert (out[:, starts[-1]:] == 5).all()
    kv.close()
