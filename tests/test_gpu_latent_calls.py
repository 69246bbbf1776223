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
