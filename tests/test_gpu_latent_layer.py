"""The latent cache's operators together, as a layer uses them: prompts expanded from rows read back, then single tokens in
absorbed form replayed from one CUDA graph while requests grow, end and join; streams, devices' state and refusals."""
import pytest
import torch

import latent_ref as ref
from barrier_free_message_gb300 import _build, sfar
from test_gpu_latent import attend, cached, check_attention, check_prompt, expanded, fine, gen, ints, plain_handle, prompt

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
R, H, L, ROT, D, P, W, B = 2, 6, 512, 64, 128, 32, 8, 4
SCALE = (D + ROT) ** -0.5


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


class Layer:
    def __init__(self):
        g = gen(0)
        new = lambda *s: torch.randn(s, generator=g, device="cuda")                       # noqa: E731
        self.u, self.v = [(new(R, H, D, L) / L ** 0.5).to(BF) for _ in range(2)]          # keys U c, values V c
        self.weight = (1 + 0.1 * new(L)).to(BF)
        self.freq, self.mscale = sfar.rope_frequencies(ROT, scaling="ramp", factor=4.0, trained=64.0)
        self.cache = torch.full((R, 24, P, L + ROT), float("nan"), dtype=BF, device="cuda")
        self.kv, self.h = sfar.SfarLatent(self.cache, q_heads=H, rope_dim=ROT), sfar.Sfar(R, 1 << 16, "bf16")
        self.lens, self.delta, self.taken = ints([0] * B), ints([0] * B), ints([0] * B)
        self.table, self.starts = torch.full((B, W), -1, dtype=torch.int32, device="cuda"), ints([0] * (B + 1))
        self.ring, self.state = torch.arange(24, dtype=torch.int32, device="cuda"), ints([0, 24])

    def close(self):
        self.kv.close()
        self.h.close()

    def plan(self, slots):
        self.kv.plan(self.lens, self.delta, self.table, self.ring, self.state, self.lens, self.state, self.starts, slots, self.taken)

    def check_cache(self, x, pos, slots, ctx):
        flat = self.cache.view(R, -1, L + ROT)
        for r in range(R):
            want, off = ref.append(x[r], self.weight, pos, self.freq, "interleaved", self.mscale, 1e-6, L)
            ref.check(flat[r, slots.long()], want, off * 1.01 + want.abs() * ref.HALF[BF], ctx)


def check_rope(before, after, pos, layer):
    for r in range(R):
        want, off = ref.rope(before[r], pos, layer.freq, "interleaved", layer.mscale)
        ref.check(after[r], want, off * 1.01 + want.abs() * ref.HALF[BF], "rope")


def test_prompts_then_replayed_tokens():
    layer = Layer()
    try:
        # prompts of three requests; the fourth joins later
        add = [70, 33, 1, 0]
        T = sum(add)
        g = gen(1)
        x = torch.randn(R, T, L + ROT, generator=g, device="cuda").to(BF)
        q = torch.randn(R, T, H, D + ROT, generator=g, device="cuda").to(BF)
        raw = q.clone()
        layer.delta.copy_(ints(add))
        slots = ints([0] * T)
        layer.plan(slots)
        pos = ints([i for a in add for i in range(a)])
        layer.h.rope(q[..., D:], q[..., D:], pos, layer.freq, layout="interleaved", scale=layer.mscale)
        layer.kv.append(x, layer.weight, pos, layer.freq, slots, layout="interleaved", scale=layer.mscale)
        rows = torch.empty(R, T, L + ROT, dtype=BF, device="cuda")
        layer.kv.gather(rows, layer.table, layer.lens, layer.starts)
        k, v = [torch.einsum("rtl,rhdl->rthd", rows[..., :L].float(), w.float()).to(BF) for w in (layer.u, layer.v)]
        out = torch.empty(R, T, H, D, dtype=BF, device="cuda")
        layer.kv.prompt(q, k, v, rows[..., L:], out, layer.starts, layer.starts, max_q=max(add))
        torch.cuda.synchronize()
        fine(layer.kv)
        assert layer.lens.tolist() == add and torch.equal(raw[..., :D], q[..., :D])
        check_rope(raw[..., D:], q[..., D:], pos, layer)
        layer.check_cache(x, pos, slots, "prompt")
        starts = ref.offsets(add)
        for r in range(R):
            for b, n in enumerate(add):
                s = slice(starts[b], starts[b + 1])
                for h in range(H if n else 0):
                    want, off = ref.rows(q[r, s, h], torch.cat([k[r, s, h], rows[r, s, L:]], -1), v[r, s, h], ref.causal(n, n, "cuda"), SCALE)
                    ref.check(out[r, s, h], want, off, f"prompt {b} head {h}")

        # one captured step of a token of each request; a request of no new token has a row of padding at the end
        x1, q1 = torch.empty(R, B, L + ROT, dtype=BF, device="cuda"), torch.empty(R, B, H, D + ROT, dtype=BF, device="cuda")
        slots1, pos1 = ints([0] * B), ints([0] * B)
        rot, qa = torch.empty(R, B, H, ROT, dtype=BF, device="cuda"), torch.empty(R, B, H, L + ROT, dtype=BF, device="cuda")
        lat = torch.empty(R, B, H, L, dtype=BF, device="cuda")
        index = torch.arange(B, device="cuda")

        def step():
            layer.plan(slots1)
            # row t is of the request whose rows hold it; padding rows have position -1
            of = torch.searchsorted(layer.starts[1:], index, right=True).clamp(max=B - 1)
            pos1.copy_(torch.where(index < layer.starts[B], layer.lens[of] - 1, -1))
            layer.h.rope(q1[..., D:], qa[..., L:], pos1, layer.freq, layout="interleaved", scale=layer.mscale)
            layer.kv.append(x1, layer.weight, pos1, layer.freq, slots1, layout="interleaved", scale=layer.mscale)
            qa[..., :L] = torch.einsum("rthd,rhdl->rthl", q1[..., :D].float(), layer.u.float()).to(BF)
            layer.kv.attention(qa, lat, layer.table, layer.lens, layer.starts, max_q=1, scale=SCALE)

        x1.normal_(generator=g)
        q1.normal_(generator=g)
        layer.delta.zero_()
        qa.zero_()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()                                           # warms torch's own kernels up; nothing is added
        side.synchronize()
        assert layer.lens.tolist() == add and (lat == 0).all()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        lens = list(add)
        for deltas in ([1, 1, 1, 0], [1, 1, 1, 1], [1, 1, -1, 1], [1, -34, 1, 1], [0, 0, 0, 0], [1, 1, 1, 1]):
            x1.normal_(generator=g)
            q1.normal_(generator=g)
            layer.delta.copy_(ints(deltas))
            graph.replay()
            torch.cuda.synchronize()
            fine(layer.kv)
            lens = [max(0, n + d) for n, d in zip(lens, deltas)]
            assert layer.lens.tolist() == lens and layer.taken.tolist() == [1] * B
            new = [b for b, d in enumerate(deltas) if d > 0]
            n = len(new)
            assert pos1.tolist() == [lens[b] - 1 for b in new] + [-1] * (B - n)
            if n:
                check_rope(q1[:, :n, :, D:], qa[:, :n, :, L:], pos1[:n], layer)
                layer.check_cache(x1[:, :n], pos1[:n], slots1[:n], "token")
            table = layer.table.tolist()
            for r in range(R):
                for t, b in enumerate(new):
                    held = ref.held_rows(layer.cache[r], table[b], lens[b], P)
                    want, off = ref.rows(qa[r, t], held, held[:, :L], torch.ones(H, lens[b], dtype=torch.bool, device="cuda"), SCALE)
                    ref.check(lat[r, t], want, off, f"{deltas} request {b}")
            assert (lat[:, n:] == 0).all()
    finally:
        layer.close()


def test_both_forms_agree():
    """The same attention in its two forms: keys U c against queries U^T q, within what rounding k, v, U^T q and the
    results to bf16 allows."""
    g = gen(4)
    n, count = 150, 20
    cache, table = cached(1, L, ROT, P, [n], seed=3)
    u, v = [(torch.randn(H, D, L, generator=g, device="cuda") / L ** 0.5).to(BF) for _ in range(2)]
    q = torch.randn(1, count, H, D + ROT, generator=g, device="cuda").to(BF)
    rows = ref.held_rows(cache[0], table[0], n, P)
    k64, v64 = [torch.einsum("tl,hdl->thd", rows[:, :L].double(), w.double()) for w in (u, v)]
    qa = torch.cat([torch.einsum("thd,hdl->thl", q[0, ..., :D].double(), u.double()).to(BF), q[0, ..., D:]], -1)[None].contiguous()
    kv = sfar.SfarLatent(cache, q_heads=H, rope_dim=ROT)
    lat = torch.empty(1, count, H, L, dtype=BF, device="cuda")
    kv.attention(qa, lat, ints(table), ints([n]), ints([0, count]), max_q=count, scale=SCALE)
    out = torch.empty(1, count, H, D, dtype=BF, device="cuda")
    kv.prompt(q, k64.to(BF)[None], v64.to(BF)[None], rows[None, :, L:].contiguous(), out, ints([0, count]), ints([0, n]), max_q=count)
    torch.cuda.synchronize()
    fine(kv)
    absorbed = torch.einsum("thl,hdl->thd", lat[0].double(), v.double())
    for h in range(H):
        seen = ref.causal(count, n, "cuda")
        exact, off = ref.rows(q[0, :, h], torch.cat([k64[:, h], rows[:, L:].double()], -1), v64[:, h], seen, SCALE)
        # scores off by 2^-8 of their terms on either side; values by 2^-8, latents by 2^-8 of their own size before V
        size = ((q[0, :, h, :D].double().abs() @ k64[:, h].abs().T) * SCALE * seen).amax(-1, keepdim=True)
        qsize = ((qa[0, :, h, :L].double().abs() @ rows[:, :L].double().abs().T) * SCALE * seen).amax(-1, keepdim=True)
        p = torch.softmax((q[0, :, h].double() @ torch.cat([k64[:, h], rows[:, L:].double()], -1).T * SCALE).masked_fill(~seen, -float("inf")), -1)
        mag = p @ v64[:, h].abs()
        latmag = (p @ rows[:, :L].double().abs()) @ v[h].double().abs().T
        assert ((out[0, :, h].double() - exact).abs() <= off + mag * (2 * size * 2.0 ** -8 + 2.0 ** -8) * 1.05).all()
        assert ((absorbed[:, h] - exact).abs() <= latmag * (2 * qsize * 2.0 ** -8 + 3 * 2.0 ** -8) * 1.05).all()
    kv.close()


def test_calls_on_two_streams_and_handles():
    """Two handles' calls on streams of their own, at once, and a call on tensors that another stream made."""
    lens = [900, 2000, 17]
    made = [cached(2, 512, 64, 64, lens, seed=s) for s in (1, 2)]
    handles = [sfar.SfarLatent(c, q_heads=8, rope_dim=64) for c, _ in made]
    x = expanded(2, 3, 128, 64, [700, 300], [400, 300], seed=3)
    px = plain_handle(2, 3, 64)
    qs = [torch.randn(2, 3, 8, 576, generator=gen(s), device="cuda").to(BF) for s in range(2)]
    outs = [[torch.full((2, 3, 8, 512), float("nan"), dtype=BF, device="cuda") for _ in range(4)] for _ in range(2)]
    tabs, ls, st = [ints(t) for _, t in made], ints(lens), ints([0, 1, 2, 3])
    s1, s2 = ints([0, 400, 700]), ints([0, 700, 1000])
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(4):
        for s in range(2):
            handles[s].attention(qs[s], outs[s][i], tabs[s], ls, st, max_q=1, scale=0.07, stream=streams[s].cuda_stream)
        with torch.cuda.stream(streams[2]):
            px.prompt(*x, s1, s2, max_q=400, scale=0.09)
    torch.cuda.synchronize()
    for s in range(2):
        fine(handles[s])
        for i in range(4):
            check_attention(outs[s][i], qs[s], made[s][0], made[s][1], lens, [0, 1, 2, 3], 64)
            assert torch.equal(outs[s][i], outs[s][0])      # the same bits, whichever CTA came last
        handles[s].close()
    check_prompt(x, [700, 300], [400, 300])
    px.close()


def test_reset_puts_the_workspace_in_order():
    lens, count = [9001, 300], [1, 2]
    cache, table = cached(1, 256, 32, 32, lens, seed=5)
    kv = sfar.SfarLatent(cache, q_heads=4, rope_dim=32)
    x = expanded(1, 4, 64, 32, [600], [600], seed=6)
    for _ in range(2):
        out, q, starts = attend(cache, table, lens, count, 4, 32, kv=kv)
        check_attention(out, q, cache, table, lens, starts, 32)
        prompt(kv, x, [600], [600])
        check_prompt(x, [600], [600])
        x[4].fill_(float("nan"))
        assert sfar.lib().sfar_test_latent_record_failure(kv.h) == sfar.SFAR_OK
        code, fault = kv.status()
        assert code == sfar.SFAR_ERR_TIMEOUT and sfar.WAIT_NAMES[fault.where] == "copy"
        side = torch.cuda.Stream()
        kv.reset(stream=side.cuda_stream)
        side.synchronize()
        fine(kv)
    kv.close()


def test_refusals():
    cache = torch.zeros(2, 8, 16, 576, dtype=BF, device="cuda")
    kv = sfar.SfarLatent(cache, q_heads=3)
    w, f, one = torch.ones(512, dtype=BF, device="cuda"), torch.ones(32, device="cuda"), ints([0, 1])
    x = torch.zeros(2, 2, 576, dtype=BF, device="cuda")
    good = dict(x=x, weight=w, pos=one, freq=f, slots=one)
    kv.append(**good)
    for bad in (dict(x=x[..., :568]), dict(x=x.float()), dict(weight=w[:256]), dict(weight=w.float()), dict(freq=f[:16]), dict(pos=one[:1]),
                dict(slots=one.long()), dict(layout="other"), dict(x=[x[0]])):
        with pytest.raises(ValueError):
            kv.append(**{**good, **bad})
    odd = torch.zeros(2 * 2 * 580, dtype=BF, device="cuda").as_strided((2, 2, 576), (1160, 580, 1))
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(scale=float("inf")), dict(x=odd), dict(x=x.as_strided((2, 2, 576), (1152, 8, 1)))):
        with pytest.raises(sfar.SfarError):
            kv.append(**{**good, **bad})

    table, lens, starts = ints([[0, 1]]), ints([20]), ints([0, 2])
    out = torch.empty(2, 2, 576, dtype=BF, device="cuda")
    kv.gather(out, table, lens, starts)
    for bad in (dict(out=out[..., :512]), dict(table=table[0]), dict(lens=ints([1, 2])), dict(starts=ints([0]))):
        with pytest.raises(ValueError):
            kv.gather(**{**dict(out=out, table=table, lens=lens, starts=starts), **bad})
    for bad in (cache[:, 0, :2], out.as_strided((2, 2, 576), (1152, 8, 1)), out[:1].expand(2, 2, 576)):
        with pytest.raises(sfar.SfarError):
            kv.gather(bad, table, lens, starts)

    q, o = torch.zeros(2, 2, 3, 576, dtype=BF, device="cuda"), torch.empty(2, 2, 3, 512, dtype=BF, device="cuda")
    good = dict(q=q, out=o, table=table, lens=lens, starts=starts, max_q=2, scale=0.1)
    kv.attention(**good)
    for bad in (dict(q=q[:, :, :2]), dict(out=q), dict(q=o), dict(max_q=-1), dict(table=lens), dict(lens=starts)):
        with pytest.raises(ValueError):
            kv.attention(**{**good, **bad})
    for bad in (dict(scale=-1.0), dict(scale=float("nan")), dict(out=q[..., :512]), dict(out=o[:, :1].expand(2, 2, 3, 512)),
                dict(out=o[:, :, :1].expand(2, 2, 3, 512)), dict(out=o[:1].expand(2, 2, 3, 512)), dict(out=cache.view(2, -1)[:, :2 * 3 * 512].view(2, 2, 3, 512))):
        with pytest.raises(sfar.SfarError):
            kv.attention(**{**good, **bad})

    qp, k, kr = torch.zeros(2, 2, 3, 192, dtype=BF, device="cuda"), torch.zeros(2, 5, 3, 128, dtype=BF, device="cuda"), torch.zeros(2, 5, 64, dtype=BF, device="cuda")
    op = torch.empty(2, 2, 3, 128, dtype=BF, device="cuda")
    good = dict(q=qp, k=k, v=k, kr=kr, out=op, starts=ints([0, 2]), k_starts=ints([0, 5]), max_q=2)
    kv.prompt(**good)
    for bad in (dict(k=k[..., :64]), dict(v=k[:, :4]), dict(kr=kr[..., :32]), dict(out=qp), dict(starts=ints([0])), dict(k_starts=ints([0, 1, 5])), dict(max_q=-1),
                dict(q=qp[..., :128])):
        with pytest.raises(ValueError):
            kv.prompt(**{**good, **bad})
    p32 = torch.zeros(2, 5, 3, 32, dtype=BF, device="cuda")
    for bad in (dict(scale=-1.0), dict(scale=float("inf")), dict(out=qp[..., :128]), dict(out=op[:, :1].expand(2, 2, 3, 128)), dict(k=k[:, :, :1].expand(2, 5, 3, 128)),
                dict(kr=kr[:, :1].expand(2, 5, 64)), dict(out=k[:, :2]), dict(q=qp[..., :96], k=p32, v=p32, out=op[..., :32])):
        with pytest.raises(sfar.SfarError):
            kv.prompt(**{**good, **bad})
    torch.cuda.synchronize()
    fine(kv)
    kv.close()
    with pytest.raises(sfar.SfarError):
        kv.append(x, w, one, f, one)
    with pytest.raises(ValueError):
        sfar.SfarLatent(cache[..., :568], q_heads=3)
    with pytest.raises(sfar.SfarError):
        sfar.SfarLatent(cache, q_heads=3, rope_dim=32)      # latents of 544


def test_nothing_to_do():
    cache = torch.zeros(1, 2, 16, 576, dtype=BF, device="cuda")
    kv = sfar.SfarLatent(cache, q_heads=3)
    none = lambda *s: torch.zeros(s, dtype=BF, device="cuda")                              # noqa: E731
    w, f = torch.ones(512, dtype=BF, device="cuda"), torch.ones(32, device="cuda")
    kv.append(none(1, 0, 576), w, ints([]), f, ints([]))
    kv.gather(none(1, 0, 576), ints([[0]]), ints([0]), ints([0, 0]))
    kv.attention(none(1, 0, 3, 576), none(1, 0, 3, 512), ints([[0]]), ints([0]), ints([0, 0]), max_q=0, scale=0.1)
    kv.prompt(none(1, 0, 3, 192), none(1, 0, 3, 128), none(1, 0, 3, 128), none(1, 0, 64), none(1, 0, 3, 128), ints([0, 0]), ints([0, 0]), max_q=0)
    h = sfar.Sfar(2, 1 << 16, "bf16")
    h.rope(none(2, 0, 3, 64), none(2, 0, 3, 64), ints([]), f)
    torch.cuda.synchronize()
    fine(kv)
    kv.close()
    h.close()
