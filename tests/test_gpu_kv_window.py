"""Windows as wide as numbers go, with requests that have more new tokens than context (their first rows see nothing)."""
import pytest
import torch

from kv_rows import cache, check, offsets
from test_gpu_kv import _built, run_attention  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_q", [1, 512])
@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 30, 1 << 31, 1 << 40, 200, 201, 199])
@pytest.mark.parametrize("lens,counts", [([3, 200, 50], [40, 30, 64]), ([0, 1], [5, 2])])
def test_wide_windows(max_q, window, lens, counts):
    cpu, table = cache(1, 1, 64, 16, lens, lambda b, i: 0.01, lambda b, i: 0.01, 71)
    starts = offsets(counts)
    q = (torch.randn(1, starts[-1], 8, 64, generator=torch.Generator().manual_seed(72)) * 1.5).to(torch.bfloat16)
    got = run_attention(cpu, table, lens, starts, q, 8, 0.125, window=window, max_q=max_q)
    check(got, cpu, table, lens, starts, q, 0.125, window=window)
