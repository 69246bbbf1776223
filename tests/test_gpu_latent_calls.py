"""Calls of the latent cache's operators that their headers allow, or refuse, at the edges of what tensors may share."""
import pytest
import torch

import latent_ref as ref
from barrier_free_message_gb300 import _build, sfar
from test_gpu_latent import fine, gen, ints

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def test_append_refuses_what_lies_in_a_cache():
    L, rot, T = 256, 32, 16
    cache = torch.zeros(2, 4, 16, L + rot, dtype=BF, device="cuda")
    kv = sfar.SfarLatent(cache, q_heads=1, rope_dim=rot)
    x, w, f = torch.ones(2, T, L + rot, dtype=BF, device="cuda"), torch.ones(L, dtype=BF, device="cuda"), torch.ones(rot // 2, device="cuda")
    pos, slots = ints([0] * T), ints(list(range(T)))
    good = dict(x=x, weight=w, pos=pos, freq=f, slots=slots)
    kv.append(**good)
    flat = cache.view(-1)
    for bad in (dict(x=cache[:, 2]), dict(x=[x[0], cache[0, 3]]), dict(weight=flat[512:512 + L]), dict(pos=flat.view(torch.int32)[:T]),
                dict(slots=flat.view(torch.int32)[64:64 + T]), dict(freq=flat.view(torch.float32)[-16:])):
        with pytest.raises(sfar.SfarError):
            kv.append(**{**good, **bad})
    # beside the caches is not in them
    line = torch.zeros(flat.numel() + x.numel(), dtype=BF, device="cuda")
    own = sfar.SfarLatent(line[:flat.numel()].view(cache.shape), q_heads=1, rope_dim=rot)
    own.append(line[flat.numel():].view(x.shape).copy_(x), w, pos, f, slots)
    torch.cuda.synchronize()
    fine(kv)
    fine(own)
    assert torch.equal(line[:flat.numel()].view(cache.shape), cache) and (cache[:, 0] != 0).all()
    kv.close()
    own.close()


@pytest.mark.parametrize("B", [1, 2, 33, 700, 8192])
@pytest.mark.parametrize("held", ["first", "last", "both ends", "some", "none"])
def test_gather_of_requests_without_rows(B, held):
    """Requests without rows before, between and after those that have some, and rows past the last one."""
    P, W, pages = 16, 288, 40
    cache = torch.randn(2, pages, P, W, generator=gen(B), device="cuda").to(BF)
    n = [0] * B
    for b in {"first": [0], "last": [B - 1], "both ends": [0, B - 1], "some": range(0, B, max(1, B // 9)), "none": []}[held]:
        n[b] = 1 + (5 * b) % 30
    table = torch.randint(0, pages, (B, 2), generator=gen(B + 1), device="cuda", dtype=torch.int32)
    starts = ref.offsets(n)
    kv = sfar.SfarLatent(cache, q_heads=1, rope_dim=32)
    for pad in (0, 1, 7):
        out = torch.full((2, starts[-1] + pad, W), 5.0, dtype=BF, device="cuda")
        kv.gather(out, table, ints(n), ints(starts))
        torch.cuda.synchronize()
        fine(kv)
        for b, m in enumerate(n):
            for r in range(2 if m else 0):
                assert torch.equal(out[r, starts[b]:starts[b + 1]], ref.held_rows(cache[r], table[b].tolist(), m, P))
        assert (out[:, starts[-1]:] == 5).all()
    kv.close()


def beside(layout, shape, widths, g):
    """Tensors of these widths beside one another in the last dimension of one tensor, a gap of 8 between them."""
    R, T, H = shape
    wide = torch.randn(R, *((T, H) if layout == "tokens outside" else (H, T)), sum(widths) + 8 * len(widths), generator=g, device="cuda").to(BF)
    out, at = [], 0
    for w in widths:
        x = wide[..., at:at + w]
        out.append(x if layout == "tokens outside" else x.transpose(1, 2))
        at += w + 8
    return wide, out


@pytest.mark.parametrize("layout", ["tokens outside", "heads outside"])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 3), (5, 1), (5, 3)])
def test_results_beside_their_inputs(layout, T, H):
    """Slices of one tensor's last dimension do not meet: the results of slices are those of tensors of their own."""
    g, rot = gen(T + H), 32
    freq, pos = sfar.rope_frequencies(rot)[0], ints(list(range(T)))
    h = sfar.Sfar(2, 1 << 16, "bf16")
    for first in (0, 1):                                    # the output before the input, and after it
        wide, xs = beside(layout, (2, T, H), [rot, rot], g)
        before, own = wide.clone(), torch.empty(2, T, H, rot, dtype=BF, device="cuda")
        h.rope(xs[first].clone(), own, pos, freq)
        h.rope(xs[first], xs[1 - first], pos, freq)
        torch.cuda.synchronize()
        assert torch.equal(xs[1 - first], own) and torch.equal(xs[first].clone(), before[..., 40 * first:40 * first + rot] if
                                                               layout == "tokens outside" else before[..., 40 * first:40 * first + rot].transpose(1, 2))
    L, D = 256, 64
    cache = torch.randn(2, 4, 16, L + rot, generator=g, device="cuda").to(BF)
    kv = sfar.SfarLatent(cache, q_heads=H, rope_dim=rot)
    table, lens, starts = ints([[2, 0, 3, 1]]), ints([50]), ints([0, T])
    for order in (0, 1):
        _, xs = beside(layout, (2, T, H), [L + rot, L] if order else [L, L + rot], g)
        out, q = xs if not order else xs[::-1]
        own = torch.empty(2, T, H, L, dtype=BF, device="cuda")
        kv.attention(q.clone(), own, table, lens, starts, max_q=T, scale=0.07)
        kv.attention(q, out, table, lens, starts, max_q=T, scale=0.07)
        torch.cuda.synchronize()
        assert torch.equal(out, own)
        _, (k, out, q, v) = beside(layout, (2, T, H), [D, D, D + rot, D], g)
        kr, own = cache[:, 0, :T, L:], torch.empty(2, T, H, D, dtype=BF, device="cuda")
        kv.prompt(q.clone(), k.clone(), v.clone(), kr, own, starts, starts, max_q=T)
        kv.prompt(q, k, v, kr, out, starts, starts, max_q=T)
        torch.cuda.synchronize()
        assert torch.equal(out, own)
    fine(kv)
    # by 8 numbers too near, or of a period that the other's rows do not keep
    wide = torch.zeros(2, T, H, L + L + rot, dtype=BF, device="cuda")
    if layout == "heads outside":
        wide = torch.zeros(2, H, T, L + L + rot, dtype=BF, device="cuda").transpose(1, 2)
    with pytest.raises(sfar.SfarError):
        kv.attention(wide[..., :L + rot], wide[..., L + rot - 8:-8], table, lens, starts, max_q=T, scale=0.07)
    with pytest.raises(sfar.SfarError):
        h.rope(wide[..., :rot], wide[..., rot - 8:2 * rot - 8], pos, freq)
    if T * H > 1:
        flat = torch.zeros(2 * 4096, dtype=BF, device="cuda")
        a, b = [flat[at:].as_strided((2, T, H, rot), (4096, H * step, step, 1)) for at, step in ((0, 64), (32, 80))]
        with pytest.raises(sfar.SfarError):
            h.rope(a, b, pos, freq)
    kv.close()
    h.close()


def test_sixteen_ranks():
    R, H, L, rot, D, P, n, count = 16, 2, 256, 32, 64, 16, 70, 40
    g = gen(0)
    cache = torch.full((R, 6, P, L + rot), float("nan"), dtype=BF, device="cuda")
    kv, h = sfar.SfarLatent(cache, q_heads=H, rope_dim=rot), sfar.Sfar(R, 1 << 16, "bf16")
    new = lambda *s: torch.randn(R, *s, generator=g, device="cuda").to(BF)                # noqa: E731
    pages = [4, 1, 5, 0, 2]
    table, pos = ints([pages]), ints(list(range(n)))
    slots = ints([pages[i // P] * P + i % P for i in range(n)])
    freq, weight = sfar.rope_frequencies(rot)[0], torch.ones(L, dtype=BF, device="cuda")
    x, rows, q, k, v = new(n, L + rot), new(n, L + rot), new(count, H, D + rot), new(n, H, D), new(n, H, D)
    kv.append(x, weight, pos, freq, slots, layout="half")
    kv.gather(rows, table, ints([n]), ints([0, n]))
    raw = q.clone()
    h.rope(q[..., D:], q[..., D:], pos[n - count:].clone(), freq)
    qa = new(count, H, L + rot)
    oa, op = [torch.empty(R, count, H, w, dtype=BF, device="cuda") for w in (L, D)]
    kv.attention(qa, oa, table, ints([n]), ints([0, count]), max_q=count, scale=0.07)
    kv.prompt(q, k, v, rows[..., L:], op, ints([0, count]), ints([0, n]), max_q=count, scale=0.09)
    torch.cuda.synchronize()
    fine(kv)
    seen = ref.causal(count, n, "cuda")
    for r in range(R):
        want, off = ref.append(x[r], weight, pos, freq, "half", 1.0, 1e-6, L)
        ref.check(rows[r], want, off * 1.01 + want.abs() * ref.HALF[BF], "append")
        want, off = ref.rope(raw[r, ..., D:], pos[n - count:], freq, "half", 1.0)
        ref.check(q[r, ..., D:], want, off * 1.01 + want.abs() * ref.HALF[BF], "rope")
        for i in range(H):
            ref.check(oa[r, :, i], *ref.rows(qa[r, :, i], rows[r], rows[r, :, :L], seen, 0.07), f"absorbed {r} {i}")
            ref.check(op[r, :, i], *ref.rows(q[r, :, i], torch.cat([k[r, :, i], rows[r, :, L:]], -1), v[r, :, i], seen, 0.09), f"expanded {r} {i}")
    kv.close()
    h.close()


def test_requests_that_share_pages():
    """Two requests with the same first pages, and one whose table names a page twice."""
    L, rot, P, H = 256, 64, 32, 3
    cache = torch.randn(1, 6, P, L + rot, generator=gen(1), device="cuda").to(BF)
    table, lens = [[3, 0, 1, -1], [3, 0, 5, 2], [4, 4, 3, -1]], [70, 128, 96]
    kv = sfar.SfarLatent(cache, q_heads=H, rope_dim=rot)
    q = torch.randn(1, 3, H, L + rot, generator=gen(2), device="cuda").to(BF)
    out = torch.empty(1, 3, H, L, dtype=BF, device="cuda")
    rows = torch.empty(1, sum(lens), L + rot, dtype=BF, device="cuda")
    kv.attention(q, out, ints(table), ints(lens), ints([0, 1, 2, 3]), max_q=1, scale=0.07)
    kv.gather(rows, ints(table), ints(lens), ints(ref.offsets(lens)))
    torch.cuda.synchronize()
    fine(kv)
    for b, n in enumerate(lens):
        held = ref.held_rows(cache[0], table[b], n, P)
        assert torch.equal(rows[0, ref.offsets(lens)[b]:][:n], held)
        ref.check(out[0, b], *ref.rows(q[0, b], held, held[:, :L], torch.ones(H, n, dtype=torch.bool, device="cuda"), 0.07), f"request {b}")
    kv.close()


def test_captured_prompts_replay_with_new_lengths():
    """A prompt's step captured once: row tiles that are cut, whole ones, none at all, and rows of padding."""
    H, D, rot, T, S, B = 5, 128, 64, 700, 2200, 3
    g = gen(3)
    q, k, v, kr = [torch.randn(s, generator=g, device="cuda").to(BF) for s in ((1, T, H, D + rot), (1, S, H, D), (1, S, H, D), (1, S, rot))]
    out, starts, ks = torch.empty(1, T, H, D, dtype=BF, device="cuda"), ints([0] * (B + 1)), ints([0] * (B + 1))
    kv = sfar.SfarLatent(torch.zeros(1, 1, 16, 256 + rot, dtype=BF, device="cuda"), q_heads=H, rope_dim=rot)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.prompt(q, k, v, kr, out, starts, ks, max_q=T, scale=0.09)
    for lens, count in (([2000, 0, 1], [3, 0, 1]), ([700, 700, 700], [400, 100, 200]), ([0, 0, 0], [0, 0, 0]), ([5, 9, 2100], [5, 0, 300]), ([2200, 0, 0], [1, 0, 0])):
        starts.copy_(ints(ref.offsets(count)))
        ks.copy_(ints(ref.offsets(lens)))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        fine(kv)
        first = out.clone()
        for b, n in enumerate(lens):
            a, z, s = ref.offsets(count)[b], ref.offsets(count)[b + 1], slice(ref.offsets(lens)[b], ref.offsets(lens)[b + 1])
            for h in range(H if z > a else 0):
                want, off = ref.rows(q[0, a:z, h], torch.cat([k[0, s, h], kr[0, s]], -1), v[0, s, h], ref.causal(z - a, n, "cuda"), 0.09)
                ref.check(out[0, a:z, h], want, off, f"{lens} {count} request {b} head {h}")
        assert (out[:, sum(count):] == 0).all()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    kv.close()
