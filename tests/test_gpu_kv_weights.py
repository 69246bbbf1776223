"""Attention with weights far below a row's largest."""
import pytest
import torch

from kv_rows import cache, check
from test_gpu_kv import _built, run_attention  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_q", [1, 512])
@pytest.mark.parametrize("gap", [15, 20, 26])
def test_weights_far_below_the_largest(max_q, gap):
    """A first token of value 0 whose score lies `gap` powers of two above 4000 equal others: the result is theirs.  640
    requests of the same context, so that a CTA has contexts whole."""
    B, n, G, D, P = 640, 4000, 2, 64, 16
    scale = 0.125
    cpu, table = cache(1, 1, D, P, [n], lambda b, i: gap * 0.6931471805599453 / (4.0 * 256.0 * scale) if i == 0 else 0.01, lambda b, i: 0.01, 43)
    k, v = [t.view(torch.uint8) for t in cpu[:2]]
    k[:] = 0
    k[0, table[0][0], 0, 0, 0] = 0x78                            # 256
    v[:] = (torch.arange(v.numel()) % 7 + 0x78).view(v.shape).to(torch.uint8)          # 256 to 448
    v[0, table[0][0], 0, 0] = 0
    q = (torch.randn(1, 1, G, D, generator=torch.Generator().manual_seed(44)) * 1.5).to(torch.bfloat16)
    q[..., 0] = 4.0
    got = run_attention(cpu, table * B, [n] * B, list(range(B + 1)), q.expand(1, B, G, D).contiguous(), G, scale, max_q=max_q)
    for b in range(0, B, 37):
        check(got[:, b:b + 1], cpu, table, [n], [0, 1], q, scale, ctx=f"request {b}")
