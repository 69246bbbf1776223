"""Outputs of attention whose rows or ranks share memory are refused; every layout whose rows do not is taken."""
import pytest
import torch

from barrier_free_message_gb300 import sfar
from kv_rows import cache, check
from test_gpu_kv import _built, cuda_int, ok  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def test_overlapping_outputs():
    R, Hq, D, T = 2, 4, 64, 3
    cpu, table = cache(R, 2, D, 16, [20], lambda b, i: 0.01, lambda b, i: 0.01, 61)
    kv = sfar.SfarKv(*[t.cuda() for t in cpu], q_heads=Hq)
    q = (torch.randn(R, T, Hq, D, generator=torch.Generator().manual_seed(62)) * 1.5).to(torch.bfloat16)
    args = [cuda_int(table), cuda_int([20]), cuda_int([0, T])]

    def empty(*shape):
        return torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")

    one = empty(T, Hq, D)
    for out in (empty(R, 1, Hq, D).expand(R, T, Hq, D), empty(R, T, 1, D).expand(R, T, Hq, D), empty(1, T, Hq, D).expand(R, T, Hq, D), [one, one],
                [empty(T * Hq * D).as_strided((T, Hq, D), (D, D, 1)) for _ in range(R)],
                [empty(T * Hq * D).as_strided((T, Hq, D), (D // 2, T * D, 1)) for _ in range(R)]):
        with pytest.raises(sfar.SfarError):
            kv.attention(q.cuda(), out, *args, max_q=T)
    for out in (empty(R, T, Hq, D), empty(R, Hq, T, D).transpose(1, 2), empty(T, R, Hq, D).transpose(0, 1), empty(T, Hq, R, D).permute(2, 0, 1, 3),
                [empty(T, 2 * Hq, 2 * D)[:, ::2, :D] for _ in range(R)]):
        kv.attention(q.cuda(), out, *args, max_q=T)
        ok(kv)
        got = torch.stack(list(out)).cpu().double()
        check(got, cpu, table, [20], [0, T], q, D ** -0.5)
    # a single token, or a single head: the stride of that dimension is not used
    single = empty(R, Hq, D).unsqueeze(1)
    kv.attention(q[:, :1].cuda(), single, cuda_int(table), cuda_int([20]), cuda_int([0, 1]), max_q=1)
    ok(kv)
    check(single.cpu().double(), cpu, table, [20], [0, 1], q[:, :1], D ** -0.5)
