"""The tolerance of the tests of attention's parts sees a few lost tokens (on the CPU, the loss put into the reference)."""
import pytest
import torch

import kv_ref
from kv_rows import bound, cache, offsets, reference
from test_gpu_kv_parts import segments


@pytest.mark.parametrize("n,D,P", [(60007, 128, 32), (40000, 64, 16), (20011, 128, 32)])
def test_a_hundredth_of_the_context_is_missed(n, D, P):
    cpu, table = cache(1, 1, D, P, [n], lambda b, i: 0.002, lambda b, i: 0.01 * (1 + i % 3), 41)
    segments(cpu, table, [n], P)
    q = (torch.randn(1, 1, 4, D, generator=torch.Generator().manual_seed(42)) * 1.5).to(torch.bfloat16)
    out, mag, top = reference(cpu, 0, table, [n], [0, 1], q, 0.1)
    limit = bound(out, mag, top, n, 0.03)
    for first in (0, n // 3, n - n // 1000):
        for lost in (n // 1000, n // 100, 3 * n // 10):
            short = reference(cpu, 0, table, [n], [0, 1], q, 0.1, lost=(first, first + lost))[0]
            assert ((short - out).abs() > limit).any(), (first, lost)


def test_both_references_agree():
    lens, counts = [100, 0, 33], [3, 0, 5]
    cpu, table = cache(2, 2, 64, 16, lens, lambda b, i: 0.01, lambda b, i: -0.01 if i % 2 else 0.02, 1)
    starts = offsets(counts)
    q = torch.randn(2, 8, 8, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    for window in (0, 5):
        out, mag, _ = reference(cpu, 1, table, lens, starts, q, 0.125, window)
        want, weight = kv_ref.attention(q[1], *[c[1] for c in cpu], table, lens, starts, 0.125, window)
        assert torch.allclose(out, want, rtol=0, atol=1e-12) and torch.allclose(mag, weight, rtol=0, atol=1e-12)
