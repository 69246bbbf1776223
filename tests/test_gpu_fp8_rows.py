"""Row strides of the 8-bit projection's tensors: expanded rows (stride 0) are refused, a single row needs none."""
import pytest
import torch

import kv_ref
from barrier_free_message_gb300 import sfar
from kv_ref import F8
from test_gpu_kv import _built, check_gemm  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture
def h():
    h = sfar.Sfar(2, 1 << 16, "bf16")
    yield h
    h.close()


def test_expanded_rows_are_refused(h):
    m, k, n = 4, 256, 128
    x, x8, sx = torch.ones(2, m, k, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, m, k, dtype=torch.uint8, device="cuda"), torch.ones(2, 2, m, device="cuda")
    w8, sw, y = torch.zeros(2, n, k, dtype=torch.uint8, device="cuda"), torch.ones(2, 1, 2, device="cuda"), torch.zeros(2, m, n, dtype=torch.bfloat16, device="cuda")
    one = {t: v[:, :1].expand(2, v.shape[1], k) for t, v in (("x", x), ("x8", x8), ("w8", w8))}
    as_list = {t: list(v) for t, v in one.items()}
    for e in (one, as_list):
        for call in (lambda: h.quantize_fp8(e["x"], x8, sx), lambda: h.quantize_fp8(x, e["x8"], sx),
                     lambda: h.rowpar_gemm_fp8(e["x8"], sx, w8, sw, y), lambda: h.rowpar_gemm_fp8(x8, sx, e["w8"], sw, y)):
            with pytest.raises(sfar.SfarError):
                call()
    h.quantize_fp8(x, x8, sx)
    h.rowpar_gemm_fp8(x8, sx, w8, sw, y)
    torch.cuda.synchronize()
    assert h.status()[0] == sfar.SFAR_OK


@pytest.mark.parametrize("k,n", [(256, 1), (128, 300), (333, 40)])
def test_single_rows_of_any_stride(h, k, n):
    """One token, or one output: the stride of that row may be anything, 0 too."""
    g = torch.Generator().manual_seed(k)
    x = torch.randn(2, 1, k, generator=g).to(torch.bfloat16)
    w = (torch.randn(2, n, -(-k // 16) * 16, generator=g) * 50).to(F8)
    sw = torch.rand(2, -(-n // 128), -(-k // 128), generator=g) + 0.5
    for stride in (0, 3, 512):
        xd = torch.zeros(2, 1024, dtype=torch.bfloat16, device="cuda").as_strided((2, 1, k), (1024, stride, 1))
        xd.copy_(x)
        x8 = torch.zeros(2, 1024, dtype=torch.uint8, device="cuda").as_strided((2, 1, k), (1024, stride, 1)).view(F8)
        sx, y = torch.empty(2, -(-k // 128), 1, device="cuda"), torch.empty(2, 1, n, dtype=torch.bfloat16, device="cuda")
        h.quantize_fp8(xd, x8, sx)
        h.rowpar_gemm_fp8(x8, sx, w.cuda()[:, :, :k], sw.cuda(), y)
        torch.cuda.synchronize()
        assert h.status()[0] == sfar.SFAR_OK
        for r in range(2):
            q, s = kv_ref.quantize(x[r])
            assert torch.equal(sx[r].cpu().double(), s) and torch.equal(x8[r].cpu().double(), q)
        check_gemm(y.cpu(), x8.cpu(), sx.cpu(), w[:, :, :k], sw)
