"""Rows of attention by both of its kernels: what other rows and masked tokens hold does not reach them, infinities do."""
import pytest
import torch

from kv_rows import cache, check, offsets
from test_gpu_kv import _built, run_attention  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

FEW, MANY = 1, 512                   # what max_q picks


@pytest.mark.parametrize("form", [FEW, MANY])
@pytest.mark.parametrize("D,G,count,n", [(64, 4, 4, 900), (128, 8, 1, 2000), (128, 4, 40, 700), (64, 8, 30, 5000)])
def test_a_row_does_not_depend_on_other_rows(form, D, G, count, n):
    """Bit for bit: every second query row is replaced by a louder one, then the others."""
    cpu, table = cache(1, 1, D, 32, [n], lambda b, i: 0.01, lambda b, i: 0.01 * 2.0 ** (i % 7), 31)
    g = torch.Generator().manual_seed(32)
    q, other = [(torch.randn(1, count, G, D, generator=g) * sigma).to(torch.bfloat16) for sigma in (1.5, 12.0)]
    rows = torch.arange(count * G).view(count, G)
    whole = run_attention(cpu, table, [n], [0, count], q, G, D ** -0.5, max_q=form)
    for kept in (rows % 2 == 0, rows % 2 == 1, rows == 0, rows == count * G - 1):
        mixed = torch.where(kept[None, :, :, None], q, other)
        got = run_attention(cpu, table, [n], [0, count], mixed, G, D ** -0.5, max_q=form)
        assert torch.equal(got[0][kept], whole[0][kept])


@pytest.mark.parametrize("form", [FEW, MANY])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_a_row_does_not_depend_on_tokens_it_does_not_see(form, D, P):
    """Bit for bit: keys and values behind its position change, and the scales of pages that lie there whole."""
    n, count, G = 1000, 300, 4
    cpu, table = cache(1, 1, D, P, [n], lambda b, i: 0.01, lambda b, i: 0.01, 33)
    q = (torch.randn(1, count, G, D, generator=torch.Generator().manual_seed(34)) * 1.5).to(torch.bfloat16)
    whole = run_attention(cpu, table, [n], [0, count], q, G, D ** -0.5, max_q=form)
    for row, louder in ((0, -0.3), (57, 0.2), (150, 0.0), (299, 0.01)):
        seen = n - count + row + 1                               # tokens that rows 0 .. row see, at most
        changed = [t.clone() for t in cpu]
        for j in range(seen, n):
            for c in changed[:2]:
                c.view(torch.uint8)[0, table[0][j // P], 0, j % P] = (j * 37 + torch.arange(D)) % 0x7f
        for i in range(-(-seen // P), -(-n // P)):
            changed[2][0, table[0][i]] = louder
            changed[3][0, table[0][i]] = -louder
        got = run_attention(changed, table, [n], [0, count], q, G, D ** -0.5, max_q=form)
        assert torch.equal(got[:, :row + 1], whole[:, :row + 1]), row


@pytest.mark.parametrize("form", [FEW, MANY])
def test_infinite_and_nan_queries(form):
    """Such a row is NaN (its largest score is infinite, or none), whatever the signs; the others are as they were."""
    G, D, n = 4, 64, 200
    cpu, table = cache(1, 1, D, 16, [n], lambda b, i: 0.01, lambda b, i: 0.01, 35)
    k = cpu[0].view(torch.uint8)
    k[0, table[0], 0, :, 3] = (k[0, table[0], 0, :, 3] & 0x7f) | 0x80         # negative in every token
    k[0, table[0], 0, :, 3] = torch.where(k[0, table[0], 0, :, 3] == 0x80, 0x81, k[0, table[0], 0, :, 3])
    q = (torch.randn(1, 2, G, D, generator=torch.Generator().manual_seed(36)) * 1.5).to(torch.bfloat16)
    for value in (float("inf"), float("-inf"), float("nan")):
        bad = q.clone()
        bad[0, 0, 1, 3] = value
        bad[0, 1, 2, 40] = value
        got = run_attention(cpu, table, [n], [0, 2], bad, G, 0.125, max_q=form)
        assert torch.isnan(got[0, 0, 1]).all() and torch.isnan(got[0, 1, 2]).all()
        got[0, 0, 1] = got[0, 1, 2] = 0
        clean = run_attention(cpu, table, [n], [0, 2], q, G, 0.125, max_q=form)
        clean[0, 0, 1] = clean[0, 1, 2] = 0
        assert torch.equal(got, clean)
