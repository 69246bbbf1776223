"""The example's layer: prompts, single tokens, refusals and drops over several
steps.  Every stage is checked against its 64-bit definition on the inputs
that the stage before it really left, and the last one bit for bit."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import kv_ref
import oracle
from barrier_free_message_gb300 import inputs
from gpu_helpers import ensure_built
from test_gpu_kv import check_attention, check_gemm

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    ensure_built()
    spec = importlib.util.spec_from_file_location("paged_decode", os.path.join(ROOT, "examples", "paged_decode.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("R,hidden,Hq,Hk,D,P", [(2, 256, 4, 2, 64, 16), (4, 1024, 8, 1, 128, 32)])
def test_layer(example, R, hidden, Hq, Hk, D, P):
    B, W, pages = 5, 6, 16
    layer = example.PagedLayer(R=R, hidden=hidden, q_heads=Hq, kv_heads=Hk, head_dim=D, page_tokens=P, requests=B, width=W, pages=pages)
    g = torch.Generator().manual_seed(3)
    try:
        for deltas in ([P + 3, 1, 2 * P, 5, 0], [1, 1, 1, 1, 1], [1, -5, 1, 3 * P, 1], [1, 2, -3 * P, 1, 40], [1] * 5, [0, 1, 0, 0, P]):
            T = sum(max(d, 0) for d in deltas)
            b = layer.buffers(T)
            x = torch.randn(T, hidden, generator=g).to(torch.bfloat16)
            res = torch.randn(T, hidden, generator=g).to(torch.bfloat16)
            b["x"].copy_(x.expand(R, T, hidden))
            b["res"].copy_(res.expand(R, T, hidden))
            layer.delta.copy_(torch.tensor(deltas, dtype=torch.int32))
            old = [t.cpu() for t in layer.cache + layer.scales]
            before = {n: getattr(layer, n).tolist() for n in ("lens", "table", "ring", "state")}
            layer.step(b, max_q=max(deltas))
            layer.check()
            c = {k: v.cpu() for k, v in b.items() if k != "T"}
            plan = kv_ref.plan(P, before["lens"], deltas, before["table"], before["ring"], before["state"], T)
            assert layer.lens.tolist() == plan["lens_out"] and layer.table.tolist() == plan["table"] and c["slots"].tolist() == plan["slots"]
            assert layer.ring.tolist() == plan["ring"] and layer.state.tolist() == plan["state_out"]
            for src, q8, sc in (("x", "x8", "sx"), ("o", "o8", "so")):
                for r in range(R):
                    q, s = kv_ref.quantize(c[src][r])
                    assert torch.equal(c[q8][r].double(), q) and torch.equal(c[sc][r].double(), s)
            check_gemm(c["qkv"], c["x8"], c["sx"], layer.w_in.cpu(), layer.s_in.cpu(), "qkv")
            check_gemm(c["y"], c["o8"], c["so"], layer.w_out.cpu(), layer.s_out.cpu(), "out")
            heads = c["qkv"].view(R, T, Hq + 2 * Hk, D)
            for i, new in enumerate((heads[:, :, Hq:Hq + Hk], heads[:, :, Hq + Hk:])):
                for r in range(R):
                    values, scales = kv_ref.append(old[i][r], old[i + 2][r], new[r], plan["slots"])
                    assert torch.equal(layer.cache[i][r].cpu().double(), values) and torch.equal(layer.scales[i][r].cpu().double(), scales)
            # a request that was refused has no place for its new tokens: its rows are not compared
            keep = torch.tensor([plan["taken"][i] for i, d in enumerate(deltas) for _ in range(max(d, 0))], dtype=torch.bool)
            out = c["o"].view(R, T, Hq, D).double()
            cpu = [t.cpu() for t in layer.cache + layer.scales]
            q = heads[:, :, :Hq]
            starts = plan["starts"]
            for i in range(B):
                a, z = starts[i], starts[i + 1]
                if a < z and plan["taken"][i]:
                    check_attention(out[:, a:z], cpu, [plan["table"][i]], [plan["lens_out"][i]], [0, z - a], q[:, a:z], D ** -0.5)
            assert keep.numel() == T
            want_y, want_z = oracle.add_rmsnorm(inputs.to_bits(c["y"].reshape(R, -1)), inputs.to_bits(c["res"].reshape(R, -1)),
                                                inputs.to_bits(layer.norm.cpu()[None])[0], layer.eps, hidden)
            for r in range(R):
                assert np.array_equal(inputs.to_bits(c["z"][r].reshape(-1)), want_z[r])
                assert np.array_equal(inputs.to_bits(c["out"][r].reshape(-1)), want_y[r])
    finally:
        layer.close()


def test_example_runs(example, capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["paged_decode.py", "--ranks", "2", "--hidden", "512", "--requests", "3", "--steps", "4"])
    example.main()
    assert "us per layer step" in capsys.readouterr().out
