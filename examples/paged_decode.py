"""One attention layer of a tensor-parallel decoder over a paged 8-bit cache,
run for a few requests of different lengths: prompts first, then steps of one
token each, the steps as replays of one CUDA graph.

    python examples/paged_decode.py [--ranks 8] [--hidden 8192] [--requests 16] [--steps 32]

Per step, for all R simulated ranks at once:

    plan          pages, slots and offsets from the requests' lengths
    quantize      the normalised hidden state, a scale for each 128 values
    project       to the rank's heads of queries, keys and values (8-bit weights)
    append        the new keys and values into the 8-bit cache
    attention     the new tokens over their contexts
    quantize      the heads' outputs
    project       row-parallel, to partial sums of the hidden state
    AllReduce + residual add + RMSNorm
"""
import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from barrier_free_message_gb300 import sfar

F8 = torch.float8_e4m3fn


def quantize_weight(w):
    """[R, n, k] binary32 -> e4m3 values and a scale for each 128 x 128 block."""
    R, n, k = w.shape
    nb, kb = -(-n // 128), -(-k // 128)
    p = torch.nn.functional.pad(w, (0, kb * 128 - k, 0, nb * 128 - n)).view(R, nb, 128, kb, 128)
    s = (p.abs().amax((2, 4)) / 448).clamp(min=1e-12)
    q = (p / s[:, :, None, :, None]).view(R, nb * 128, kb * 128)[:, :n, :k].to(F8).contiguous()
    return q, s.contiguous()


class PagedLayer:
    """Weights, cache and the state of ``requests`` requests of up to ``width`` pages each; steps of up to ``tokens``
    new tokens."""

    def __init__(self, R=8, hidden=8192, q_heads=8, kv_heads=1, head_dim=128, page_tokens=64, requests=16, width=64, pages=1024,
                 tokens=2048, eps=1e-5, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.R, self.hidden, self.eps, self.width = R, hidden, eps, width
        self.q_heads, self.kv_heads, self.D = q_heads, kv_heads, head_dim
        heads = q_heads + 2 * kv_heads
        new = lambda *s: torch.randn(s, generator=g, device="cuda")                       # noqa: E731
        self.w_in, self.s_in = quantize_weight(new(R, heads * head_dim, hidden) / hidden ** 0.5)
        self.w_out, self.s_out = quantize_weight(new(R, hidden, q_heads * head_dim) / (R * q_heads * head_dim) ** 0.5)
        self.norm = (1 + 0.1 * new(hidden)).to(torch.bfloat16)
        shape = (R, pages, kv_heads, page_tokens, head_dim)
        self.cache = [torch.zeros(shape, dtype=F8, device="cuda") for _ in range(2)]
        self.scales = [torch.zeros(shape[:3], device="cuda") for _ in range(2)]
        self.kv = sfar.SfarKv(*self.cache, *self.scales, q_heads=q_heads)
        self.h = sfar.Sfar(R, tokens * hidden * 2, "bf16")
        whole = lambda v, *s: torch.full(s, v, dtype=torch.int32, device="cuda")          # noqa: E731
        self.lens, self.table = whole(0, requests), whole(-1, requests, width)
        self.ring = torch.arange(pages, dtype=torch.int32, device="cuda")
        self.state = torch.tensor([0, pages], dtype=torch.int32, device="cuda")
        self.starts, self.taken, self.delta = whole(0, requests + 1), whole(0, requests), whole(0, requests)

    def buffers(self, T):
        """What a step of T tokens writes."""
        R, H, D, kb = self.R, self.q_heads + 2 * self.kv_heads, self.D, -(-self.hidden // 128)
        one = lambda dtype, *s: torch.empty(s, dtype=dtype, device="cuda")                # noqa: E731
        k_out = self.q_heads * D
        return {"x": one(torch.bfloat16, R, T, self.hidden), "x8": one(F8, R, T, self.hidden), "sx": one(torch.float32, R, kb, T),
                "qkv": one(torch.bfloat16, R, T, H * D), "slots": one(torch.int32, T), "o": one(torch.bfloat16, R, T, k_out),
                "o8": one(F8, R, T, k_out), "so": one(torch.float32, R, -(-k_out // 128), T),
                "y": one(torch.bfloat16, R, T, self.hidden), "res": one(torch.bfloat16, R, T, self.hidden),
                "z": one(torch.bfloat16, R, T, self.hidden), "out": one(torch.bfloat16, R, T, self.hidden),
                "sum": one(torch.bfloat16, R, T, self.hidden), "T": T}

    def step(self, b, max_q):
        """b: buffers with x (the normalised input) and res (the residual) filled in; self.delta: new tokens of each
        request.  Leaves the layer's normalised output in b["out"], the new residual in b["z"]."""
        R, T, D, Hq, Hk = self.R, b["T"], self.D, self.q_heads, self.kv_heads
        self.kv.plan(self.lens, self.delta, self.table, self.ring, self.state, self.lens, self.state, self.starts, b["slots"], self.taken)
        self.h.quantize_fp8(b["x"], b["x8"], b["sx"])
        self.h.rowpar_gemm_fp8(b["x8"], b["sx"], self.w_in, self.s_in, b["qkv"])
        heads = b["qkv"].view(R, T, Hq + 2 * Hk, D)
        self.kv.append(heads[:, :, Hq:Hq + Hk], heads[:, :, Hq + Hk:], b["slots"])
        self.kv.attention(heads[:, :, :Hq], b["o"].view(R, T, Hq, D), self.table, self.lens, self.starts, max_q=max_q)
        self.h.quantize_fp8(b["o"], b["o8"], b["so"])
        self.h.rowpar_gemm_fp8(b["o8"], b["so"], self.w_out, self.s_out, b["y"])
        ranks = lambda t: [t[r] for r in range(R)]                                         # noqa: E731
        y, res, out, z = [ranks(b[n]) for n in ("y", "res", "out", "z")]
        if T * self.hidden * 2 <= 2 << 20:                       # what the fused call takes
            self.h.allreduce_add_rmsnorm(y, res, self.norm, out, z, self.hidden, self.eps)
        else:
            self.h.allreduce(y, ranks(b["sum"]), "twoshot_tma")
            self.h.add_rmsnorm(ranks(b["sum"]), res, self.norm, out, z, self.hidden, self.eps)

    def check(self):
        torch.cuda.synchronize()
        for what, (code, fault) in (("cache", self.kv.status()), ("ranks", self.h.status())):
            if code != sfar.SFAR_OK:
                raise sfar.SfarError(code, f"{what}: {sfar.WAIT_NAMES.get(fault.where, fault.where)}")

    def close(self):
        self.kv.close()
        self.h.close()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    prompts = [17 + 23 * i % 97 for i in range(a.requests)]
    layer = PagedLayer(R=a.ranks, hidden=a.hidden, requests=a.requests, tokens=max(sum(prompts), a.requests))
    g = torch.Generator(device="cuda").manual_seed(1)

    def fill(b):
        x = torch.randn(b["x"].shape[1:], generator=g, device="cuda").to(torch.bfloat16)
        b["x"].copy_(x.expand_as(b["x"]))                        # every rank holds the same hidden state
        b["res"].copy_(x.expand_as(b["res"]))

    layer.delta.copy_(torch.tensor(prompts, dtype=torch.int32))
    b = layer.buffers(sum(prompts))
    fill(b)
    layer.step(b, max_q=max(prompts))
    layer.check()

    b = layer.buffers(a.requests)
    layer.delta.fill_(1)
    fill(b)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.step(b, max_q=1)                                   # a first step outside the graph
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            layer.step(b, max_q=1)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(a.steps):
            graph.replay()
        end.record()
    layer.check()
    print(f"{a.requests} requests, prompts of {min(prompts)}-{max(prompts)} tokens, now {layer.lens.tolist()} tokens; "
          f"{int(layer.state[1])} pages free; {start.elapsed_time(end) / a.steps * 1e3:.1f} us per layer step")
    layer.close()


if __name__ == "__main__":
    main()
