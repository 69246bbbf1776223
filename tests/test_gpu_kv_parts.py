"""Attention whose contexts are shared out over many CTAs and joined again: no token is lost or counted twice."""
import pytest
import torch

from kv_ref import F8
from kv_rows import cache, check, offsets
from test_gpu_kv import _built, run_attention  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def segments(cpu, table, lens, P):
    """Values that say where a token stands: the context's d-th part of D holds 256 in element d alone, so that an output
    element is that part's weight, within 2^-8 + 2^-10 of itself."""
    v, D = cpu[1], cpu[1].shape[-1]
    for row, n in zip(table, lens):
        j = torch.arange(n)
        one = torch.zeros(n, D)
        one[j, j * D // n] = 256.0
        for i, page in enumerate(row[:-(-n // P)]):
            part = one[i * P:(i + 1) * P]
            v[:, page, :, :len(part)] = part.to(F8)


@pytest.mark.parametrize("R,H,G,D,P,lens,counts", [
    (1, 1, 16, 128, 32, [60007], [1]), (1, 1, 3, 64, 16, [40000, 17], [1, 1]), (1, 1, 5, 128, 128, [100003], [1]),
    (2, 1, 8, 128, 32, [20011], [1]), (2, 1, 8, 128, 64, [9001, 3, 700, 1, 4096, 64], [1] * 6), (2, 1, 8, 128, 16, [6000, 6000], [2, 3]),
    (1, 2, 8, 64, 64, [9000], [40]), (1, 1, 8, 128, 128, [20000, 300], [17, 2]), (1, 1, 4, 64, 16, [12000, 9000], [200, 1])])
def test_every_token_counts_once(R, H, G, D, P, lens, counts):
    cpu, table = cache(R, H, D, P, lens, lambda b, i: 0.002, lambda b, i: 0.01 * (1 + i % 3), 41)
    segments(cpu, table, lens, P)
    starts = offsets(counts)
    q = (torch.randn(R, starts[-1], H * G, D, generator=torch.Generator().manual_seed(42)) * 1.5).to(torch.bfloat16)
    for _ in range(2):
        got = run_attention(cpu, table, lens, starts, q, H * G, 0.1)
        check(got, cpu, table, lens, starts, q, 0.1, ctx=str(lens))


@pytest.mark.parametrize("B,count,max_q", [(8192, 1, 1), (3000, 2, 64), (2049, 5, 64)])
def test_thousands_of_requests(B, count, max_q):
    """More requests than the kernel for many rows takes, and the most there may be."""
    G, D, P = 8, 64, 16
    lens, counts = [count + b * 7 % 61 for b in range(B)], [count] * B
    cpu, table = cache(1, 1, D, P, lens, lambda b, i: 0.01, lambda b, i: 0.01, 45)
    starts = offsets(counts)
    q = (torch.randn(1, starts[-1], G, D, generator=torch.Generator().manual_seed(46)) * 1.5).to(torch.bfloat16)
    got = run_attention(cpu, table, lens, starts, q, G, 0.125, max_q=max_q)
    check(got, cpu, table, lens, starts, q, 0.125)
