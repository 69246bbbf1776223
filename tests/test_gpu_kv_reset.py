"""A paged cache's handle after an attention call whose wait ran out (recorded on the host; no wait runs out here)."""
import pytest
import torch

from barrier_free_message_gb300 import sfar
from kv_rows import cache, check, offsets
from test_gpu_kv import _built, cuda_int  # noqa: F401  (a fixture)
from test_gpu_kv_parts import segments

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,counts", [([20011], [1]), ([9001, 300], [40, 2]), ([3000, 70], [1, 1])])
def test_reset_puts_the_workspace_in_order(lens, counts):
    G, D, P = 8, 128, 32
    cpu, table = cache(1, 1, D, P, lens, lambda b, i: 0.002, lambda b, i: 0.01, 51)
    segments(cpu, table, lens, P)
    starts = offsets(counts)
    kv = sfar.SfarKv(*[t.cuda() for t in cpu], q_heads=G)
    for seed in range(3):
        q = (torch.randn(1, starts[-1], G, D, generator=torch.Generator().manual_seed(seed)) * (1 + seed)).to(torch.bfloat16)
        out = torch.empty_like(q, device="cuda")
        kv.attention(q.cuda(), out, cuda_int(table), cuda_int(lens), cuda_int(starts), max_q=max(counts), scale=0.1)
        torch.cuda.synchronize()
        assert kv.status()[0] == sfar.SFAR_OK
        check(out.cpu().double(), cpu, table, lens, starts, q, 0.1, ctx=f"call {seed}")
        assert sfar.lib().sfar_test_kv_record_failure(kv.h) == sfar.SFAR_OK
        code, fault = kv.status()
        assert code == sfar.SFAR_ERR_TIMEOUT and sfar.WAIT_NAMES[fault.where] == "copy"
        side = torch.cuda.Stream()
        kv.reset(stream=side.cuda_stream)
        side.synchronize()
