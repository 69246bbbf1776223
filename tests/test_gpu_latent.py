"""Rotary positions and the latent-attention operators on the GPU against their 64-bit forms."""
import pytest
import torch

import latent_ref as ref
from barrier_free_message_gb300 import _build, sfar

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def fine(h):
    code, f = h.status()
    assert code == sfar.SFAR_OK, (code, sfar.WAIT_NAMES.get(f.where, f.where), f.cta)


# ------------------------------------------------------------------------ rope
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("R,T,H,K,rot,D,far", [(2, 1, 1, 0, 16, 16, 10), (3, 7, 5, 2, 64, 192, 1 << 20), (2, 65, 3, 1, 96, 96, 2 ** 31 - 1),
                                               (8, 400, 8, 1, 128, 128, 9000), (2, 3, 2, 3, 1024, 1040, 131072)])
def test_rope(dtype, layout, R, T, H, K, rot, D, far):
    t = {"bf16": BF, "fp32": torch.float32}[dtype]
    g = gen(R * T + rot)
    q, k = [torch.randn(R, T, n, D, generator=g, device="cuda").to(t) for n in (H, K)]
    pos = torch.randint(0, far, (T,), generator=g, device="cuda").to(torch.int32)
    pos[T // 2] = -1
    pos[-1] = far
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda") / rot)
    qo, ko = [torch.full((R, T, n, rot + 8), 7.0, dtype=t, device="cuda") for n in (H, K)]
    h = sfar.Sfar(R, 1 << 16, dtype)
    keys = dict(k=k[..., D - rot:], k_out=ko[..., :rot]) if K else {}
    h.rope(q[..., D - rot:], qo[..., :rot], pos, freq, layout=layout, scale=1.25, **keys)
    torch.cuda.synchronize()
    for x, o in ((q, qo), (k, ko)):
        assert (o[..., rot:] == 7).all()
        for r in range(R if x.shape[2] else 0):
            want, off = ref.rope(x[r, ..., D - rot:], pos, freq, layout, 1.25)
            live = pos >= 0
            ref.check(o[r, live][..., :rot], want[live], off[live] * 1.01 + want[live].abs() * ref.HALF[t], f"{dtype} {layout} rank {r}")
            assert (o[r, ~live][..., :rot] == 7).all()
    # in place, queries and keys side by side in one tensor
    both = torch.cat([q, k], 2).contiguous()
    a, b = both[:, :, :H, D - rot:], both[:, :, H:, D - rot:]
    h.rope(a, a, pos, freq, layout=layout, scale=1.25, **(dict(k=b, k_out=b) if K else {}))
    torch.cuda.synchronize()
    live = pos >= 0
    assert torch.equal(both[:, live][:, :, :H, D - rot:], qo[:, live][..., :rot])
    assert torch.equal(both[:, live][:, :, H:, D - rot:], ko[:, live][..., :rot])
    assert torch.equal(both[..., :D - rot], torch.cat([q, k], 2)[..., :D - rot])
    assert torch.equal(both[:, ~live], torch.cat([q, k], 2)[:, ~live])
    h.close()


def test_rope_no_position_turns_nothing():
    x = torch.randn(2, 5, 3, 32, generator=gen(1), device="cuda").to(BF)
    out = torch.empty_like(x)
    h = sfar.Sfar(2, 1 << 16, "bf16")
    freq, scale = sfar.rope_frequencies(32)
    h.rope(x, out, ints([0] * 5), freq, scale=scale)
    torch.cuda.synchronize()
    assert scale == 1.0 and torch.equal(out, x)
    h.close()


@pytest.mark.parametrize("dtype", [sfar.SFAR_BF16, sfar.SFAR_FP32])
def test_rope_of_a_handle_with_the_c_type(dtype):
    mine, other = (BF, torch.float32) if dtype == sfar.SFAR_BF16 else (torch.float32, BF)
    h = sfar.Sfar(2, 1 << 16, dtype)
    x, freq = torch.randn(2, 3, 2, 32, generator=gen(2), device="cuda").to(mine), torch.ones(16, device="cuda")
    out = torch.empty_like(x)
    h.rope(x, out, ints([0, 0, 0]), freq)
    torch.cuda.synchronize()
    assert torch.equal(out, x)
    with pytest.raises(ValueError):
        h.rope(x.to(other), out.to(other), ints([0, 0, 0]), freq)
    h.close()


def test_rope_refuses():
    h = sfar.Sfar(2, 1 << 16, "bf16")
    x, pos, freq = torch.zeros(2, 4, 3, 64, dtype=BF, device="cuda"), ints([0] * 4), torch.ones(32, device="cuda")
    out = torch.empty_like(x)
    h.rope(x, out, pos, freq)
    for bad in (dict(layout="both"), dict(k=x), dict(pos=pos[:3]), dict(freq=freq[:31]), dict(freq=freq.double()),
                dict(q=x.float()), dict(q_out=out[:, :, :2]), dict(k=x[..., :32], k_out=out[..., :32])):
        with pytest.raises(ValueError):
            h.rope(**{**dict(q=x, q_out=out, pos=pos, freq=freq), **bad})
    wide = torch.zeros(2, 4, 3, 68, dtype=BF, device="cuda")
    for bad in (dict(q=wide[..., :64]), dict(q_out=wide[..., :64]), dict(scale=float("inf")),     # strides of 68
                dict(q_out=out.flatten()[:64].view(1, 1, 1, 64).expand(2, 4, 3, 64)),             # rows in one place
                dict(q=x[..., :24], q_out=out[..., :24], freq=freq[:12])):
        with pytest.raises(sfar.SfarError):
            h.rope(**{**dict(q=x, q_out=out, pos=pos, freq=freq), **bad})
    # an output that is its input moved by a token, or that another tensor lies in
    line = torch.zeros(2 * 5 * 3 * 64, dtype=BF, device="cuda")
    a = line[:2 * 4 * 3 * 64].view(2, 4, 3, 64)
    with pytest.raises(sfar.SfarError):
        h.rope(a, line[192:192 + 2 * 4 * 3 * 64].view(2, 4, 3, 64), pos, freq)
    with pytest.raises(sfar.SfarError):
        h.rope(a, out, pos, freq, k=a, k_out=out)
    h.close()


# ---------------------------------------------------------------------- append
def step(P, before, add, spare=3, seed=0):
    """(table, slots, positions, pages of the pool) of a step that adds `add` tokens to requests of `before`."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-(n + a) // P) for n, a in zip(before, add)]
    order = torch.randperm(sum(need) + spare, generator=g).tolist()
    width, table, at = max(max(need), 1) + 1, [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    pos = [n + i for n, a in zip(before, add) for i in range(a)]
    slots = [table[b][(n + i) // P] * P + (n + i) % P for b, (n, a) in enumerate(zip(before, add)) for i in range(a)]
    return table, slots, pos, sum(need) + spare


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("R,L,rot,P,before,add", [(1, 256, 32, 16, [0], [1]), (2, 512, 64, 64, [5, 63, 0, 200], [1, 1, 1, 1]),
                                                  (3, 256, 64, 128, [0, 130], [129, 40]), (8, 512, 32, 32, [31, 0, 7], [2, 0, 100])])
def test_append_and_gather(layout, R, L, rot, P, before, add):
    table, slots, pos, pages = step(P, before, add)
    T = len(slots)
    g = gen(T + L)
    wide = torch.randn(R, T, L + rot + 24, generator=g, device="cuda").to(BF)
    x = wide[..., 8:8 + L + rot]
    weight = torch.randn(L, generator=g, device="cuda").to(BF)
    freq, scale = sfar.rope_frequencies(rot, scaling="ramp", factor=8.0)
    cache = torch.full((R, pages, P, L + rot), float("nan"), dtype=BF, device="cuda")
    kv = sfar.SfarLatent(cache, q_heads=4, rope_dim=rot)
    out_of, no_pos = list(slots), list(pos)
    if T > 3:
        out_of[1], no_pos[2] = -1, -1                       # left out
    kv.append(x, weight, ints(no_pos), freq, ints(out_of), eps=1e-5, layout=layout, scale=scale)
    torch.cuda.synchronize()
    fine(kv)
    live = [i for i in range(T) if out_of[i] >= 0 and no_pos[i] >= 0]
    flat = cache.view(R, -1, L + rot)
    for r in range(R):
        want, off = ref.append(x[r], weight, ints(pos), freq, layout, scale, 1e-5, L)
        at = torch.tensor([slots[i] for i in live], device="cuda")
        ref.check(flat[r, at], want[live], off[live] * 1.01 + want[live].abs() * ref.HALF[BF], f"rank {r}")
    rest = torch.ones(pages * P, dtype=torch.bool, device="cuda")
    rest[torch.tensor([slots[i] for i in live], device="cuda")] = False
    assert torch.isnan(flat[:, rest]).all()                 # nothing else was written
    # read back: every request whole, the last one a token short, padding rows left
    cache.copy_(torch.randn(cache.shape, generator=g, device="cuda"))
    lens = [n + a for n, a in zip(before, add)]
    take = lens[:-1] + [max(lens[-1] - 1, 0)]
    starts = ref.offsets(take)
    out = torch.full((R, starts[-1] + 3, L + rot + 8), 5.0, dtype=BF, device="cuda")
    kv.gather(out[..., :L + rot], ints(table), ints(lens), ints(starts))
    torch.cuda.synchronize()
    fine(kv)
    for r in range(R):
        for b, n in enumerate(take):
            assert torch.equal(out[r, starts[b]:starts[b + 1], :L + rot], ref.held_rows(cache[r], table[b], n, P))
    assert (out[..., L + rot:] == 5).all() and (out[:, starts[-1]:] == 5).all()
    kv.close()


def test_append_records_bad_slots():
    cache = torch.zeros(2, 4, 16, 288, dtype=BF, device="cuda")
    kv = sfar.SfarLatent(cache, q_heads=1, rope_dim=32)
    x, w, f = torch.ones(2, 3, 288, dtype=BF, device="cuda"), torch.ones(256, dtype=BF, device="cuda"), torch.ones(16, device="cuda")
    kv.append(x, w, ints([0, 0, 0]), f, ints([3, 64, -1]))
    torch.cuda.synchronize()
    code, fault = kv.status()
    assert code == sfar.SFAR_ERR_INVALID and sfar.WAIT_NAMES[fault.where] == "slot" and fault.cta == 1
    assert (cache.view(2, -1, 288)[:, 3] != 0).any() and (cache.view(2, -1, 288)[:, 4:] == 0).all()
    kv.reset()
    torch.cuda.synchronize()
    fine(kv)
    kv.close()


def test_append_rows_that_are_not_finite_or_zero():
    cache = torch.zeros(1, 1, 16, 576, dtype=BF, device="cuda")
    kv = sfar.SfarLatent(cache, q_heads=1)
    x = torch.ones(1, 4, 576, dtype=BF, device="cuda")
    x[0, 0, 5] = float("nan")
    x[0, 1, 7] = float("inf")
    x[0, 2] = 0
    freq, _ = sfar.rope_frequencies(64)
    kv.append(x, torch.ones(512, dtype=BF, device="cuda"), ints([1, 2, 3, 4]), freq, ints([0, 1, 2, 3]))
    torch.cuda.synchronize()
    assert torch.isnan(cache[0, 0, 0, :512]).all() and torch.isnan(cache[0, 0, 1, 7]) and (cache[0, 0, 2] == 0).all()
    assert torch.isfinite(cache[0, 0, 3]).all() and torch.isfinite(cache[0, 0, :2, 512:]).all()
    kv.close()


def test_gather_leaves_out_what_is_not_there():
    P, W = 16, 288
    cache = torch.randn(2, 6, P, W, generator=gen(3), device="cuda").to(BF)
    kv = sfar.SfarLatent(cache, q_heads=1, rope_dim=32)
    table, lens, starts = [[0, 1], [2, 9], [3, 4], [5, 0]], [20, 32, 5, 0], [0, 20, 52, 60, 60]
    out = torch.full((2, 64, W), 5.0, dtype=BF, device="cuda")
    for rows, where in (([0], None), ([1], "page"), ([2], "tokens")):
        out.fill_(5.0)
        s = [0] + [starts[r + 1] - starts[r] for r in rows]
        kv.gather(out, ints([table[r] for r in rows]), ints([lens[r] for r in rows]), ints(s))
        torch.cuda.synchronize()
        code, fault = kv.status()
        assert (sfar.WAIT_NAMES[fault.where] if code else None) == where, rows
        kv.reset()
    kv.gather(out.fill_(5.0), ints(table), ints(lens), ints(starts))
    torch.cuda.synchronize()
    for r in range(2):
        assert torch.equal(out[r, :20], ref.held_rows(cache[r], table[0], 20, P))
        assert torch.equal(out[r, 20:36], cache[r, 2]) and (out[r, 36:52] == 5).all()
        assert torch.equal(out[r, 52:57], cache[r, 3, :5]) and (out[r, 57:] == 5).all()
    kv.reset()
    kv.gather(out.fill_(5.0), ints(table), ints(lens), ints([0, 30, 20, 10, 70]))      # offsets in no order
    torch.cuda.synchronize()
    assert kv.status()[0] == sfar.SFAR_ERR_INVALID
    kv.close()


# ------------------------------------------------------------------- attention
def cached(R, L, rot, P, lens, seed):
    """(cache, table): rows of a normal distribution, NaN where no request holds a token."""
    table, _, _, pages = step(P, [0] * len(lens), lens, seed=seed)
    cache = torch.randn(R, pages, P, L + rot, generator=gen(seed), device="cuda").to(BF)
    live = torch.zeros(pages, P, dtype=torch.bool, device="cuda")
    for row, n in zip(table, lens):
        for i in range(-(-n // P)):
            live[row[i], :min(P, n - i * P)] = True
    cache[:, ~live] = float("nan")
    return cache, table


def attend(cache, table, lens, count, H, rot, max_q=None, sigma=1.0, seed=5, pad=0, q=None, kv=None):
    """(out, q, starts) of a call."""
    R, W = cache.shape[0], cache.shape[-1]
    starts = ref.offsets(count)
    T = starts[-1] + pad
    if q is None:
        q = (sigma * torch.randn(R, T, H, W, generator=gen(seed), device="cuda")).to(BF)
    out = torch.full((R, T, H, W - rot), float("nan"), dtype=BF, device="cuda")
    own = kv or sfar.SfarLatent(cache, q_heads=H, rope_dim=rot)
    own.attention(q, out, ints(table), ints(lens), ints(starts), max_q=max(count) if max_q is None else max_q, scale=0.07)
    torch.cuda.synchronize()
    fine(own)
    if kv is None:
        own.close()
    return out, q, starts


def check_attention(out, q, cache, table, lens, starts, rot):
    R, T, H, W = q.shape
    P = cache.shape[2]
    for r in range(R):
        for b, n in enumerate(lens):
            a, z = starts[b], starts[b + 1]
            if a == z:
                continue
            rows = ref.held_rows(cache[r], table[b], n, P)
            seen = ref.causal(z - a, n, "cuda").repeat_interleave(H, 0)
            want, off = ref.rows(q[r, a:z].flatten(0, 1), rows, rows[:, :W - rot], seen, 0.07)
            ref.check(out[r, a:z].flatten(0, 1), want, off, f"rank {r} request {b}")
    assert (out[:, starts[-1]:] == 0).all()


@pytest.mark.parametrize("R,H,L,rot,P,lens,count", [
    (1, 1, 512, 64, 16, [1], [1]),
    (2, 16, 512, 64, 64, [128, 129, 1, 77], [1, 1, 1, 1]),
    (2, 12, 256, 32, 16, [99, 0, 300], [1, 0, 1]),
    (1, 20, 512, 64, 32, [700], [2]),
    (3, 5, 256, 64, 128, [200, 33], [3, 5]),
    (1, 40, 512, 32, 64, [513, 16], [1, 4]),
    (1, 16, 512, 64, 128, [2600], [1]),                    # ten parts and more, joined in groups
    (1, 7, 256, 64, 16, [5000, 3], [4, 3]),
    (8, 16, 512, 64, 64, [1025, 4000, 64], [1, 1, 1]),
    (2, 3, 512, 64, 32, [150], [150]),                      # a whole prompt
    (1, 130, 256, 32, 64, [260], [9])])
def test_attention(R, H, L, rot, P, lens, count):
    cache, table = cached(R, L, rot, P, lens, seed=len(lens) + H)
    out, q, starts = attend(cache, table, lens, count, H, rot, pad=2)
    check_attention(out, q, cache, table, lens, starts, rot)


LAYOUTS = ["slices of wider rows", "padded tokens", "heads outside", "one row for all tokens"]


def laid_out(layout, R, T, H, W, g):
    """A random [R, T, H, W] with the strides of a layout, on memory that holds NaN elsewhere."""
    shape = {"slices of wider rows": (R, T, H, W + 24), "padded tokens": (R, T, H * W + 8), "heads outside": (R, H, T + 1, W),
             "one row for all tokens": (R, 1, H, W)}[layout]
    wide = torch.full(shape, float("nan"), dtype=BF, device="cuda")
    x = {"slices of wider rows": lambda: wide[..., 16:16 + W], "padded tokens": lambda: wide[..., :H * W].unflatten(-1, (H, W)),
         "heads outside": lambda: wide[:, :, :T].transpose(1, 2), "one row for all tokens": lambda: wide.expand(R, T, H, W)}[layout]()
    if layout == "one row for all tokens":
        wide.copy_(torch.randn(shape, generator=g, device="cuda"))
    else:
        x.copy_(torch.randn(R, T, H, W, generator=g, device="cuda"))
    return x, wide


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("H,L,rot,lens,count", [(1, 256, 32, [70, 9], [1, 1]), (5, 512, 64, [300, 1000], [1, 3]), (30, 512, 32, [130], [2]),
                                                (70, 256, 64, [65, 500], [1, 2])])
def test_attention_strides(layout, H, L, rot, lens, count):
    cache, table = cached(2, L, rot, 32, lens, seed=H)
    g, T, starts = gen(H), sum(count) + 2, ref.offsets(count)
    q, _ = laid_out(layout, 2, T, H, L + rot, g)
    out, wide = laid_out(layout if layout != LAYOUTS[3] else LAYOUTS[0], 2, T, H, L, g)
    out.fill_(0)
    rest = torch.isnan(wide)
    kv = sfar.SfarLatent(cache, q_heads=H, rope_dim=rot)
    kv.attention(q, out, ints(table), ints(lens), ints(starts), max_q=max(count), scale=0.07)
    torch.cuda.synchronize()
    fine(kv)
    check_attention(out, q, cache, table, lens, starts, rot)
    assert torch.equal(torch.isnan(wide), rest)
    kv.close()


@pytest.mark.parametrize("max_q", [0, 1, 100])
def test_attention_any_hint(max_q):
    cache, table = cached(2, 512, 64, 32, [400, 90], seed=2)
    out, q, starts = attend(cache, table, [400, 90], [3, 1], 9, 64, max_q=max_q)
    check_attention(out, q, cache, table, [400, 90], starts, 64)


def test_attention_rows_of_nothing():
    cache, table = cached(2, 256, 32, 16, [3, 0, 20], seed=8)
    out, q, starts = attend(cache, table, [3, 0, 20], [6, 2, 1], 4, 32)
    assert (out[:, :3] == 0).all() and (out[:, 6:8] == 0).all()
    for r in range(2):
        rows = ref.held_rows(cache[r], table[0], 3, 16)
        for i in range(3):
            want, off = ref.rows(q[r, 3 + i], rows, rows[:, :256], torch.arange(3, device="cuda")[None] <= i, 0.07)
            ref.check(out[r, 3 + i], want, off)


def test_attention_many_requests():
    lens = [1 + (37 * i) % 290 for i in range(300)]
    cache, table = cached(1, 256, 32, 16, lens, seed=4)
    out, q, starts = attend(cache, table, lens, [1] * 300, 8, 32)
    check_attention(out, q, cache, table, lens, starts, 32)


def test_attention_steep_scores_move_the_references():
    """Scores that climb along the context by far more than a reference may be passed by."""
    lens = [1500, 260]
    cache, table = cached(1, 512, 64, 64, lens, seed=6)
    for b, n in enumerate(lens):
        for i, p in enumerate(table[b][:-(-n // 64)]):
            cache[0, p, :, 575] = torch.arange(64, device="cuda") + 64 * i
    q = torch.randn(1, 4, 16, 576, generator=gen(9), device="cuda").to(BF)
    q[0, :, :8, 575] = 10.0                                 # up, and down for the others
    q[0, :, 8:, 575] = -10.0
    out, q, starts = attend(cache, table, lens, [2, 2], 16, 64, q=q)
    check_attention(out, q, cache, table, lens, starts, 64)


def test_attention_row_depends_on_itself_alone():
    """The same bits whatever the other rows, and the tokens that a row does not see, hold."""
    lens, count = [300, 140], [4, 2]
    cache, table = cached(2, 512, 64, 64, lens, seed=7)
    kv = sfar.SfarLatent(cache, q_heads=6, rope_dim=64)
    out, q, starts = attend(cache, table, lens, count, 6, 64, kv=kv)
    other = q.clone()
    other[:, 1:] = float("nan")
    other[:, 0, 1:] *= 50
    again, _, _ = attend(cache, table, lens, count, 6, 64, q=other, kv=kv)
    assert torch.equal(again[:, 0, 0], out[:, 0, 0]) and torch.isnan(again[:, 1:]).all()
    # the last two tokens of the first request hold infinities and NaN: its rows 2 and 3 see the first of them
    for i, (at, v) in enumerate(((298, float("inf")), (299, float("nan")))):
        cache[:, table[0][at // 64], at % 64, 3 + i] = v
    again, _, _ = attend(cache, table, lens, count, 6, 64, q=q, kv=kv)
    assert torch.equal(again[:, :2], out[:, :2]) and torch.equal(again[:, 4:], out[:, 4:])
    assert torch.isnan(again[:, 2:4]).all()
    kv.close()


def test_attention_bad_pages_and_lengths_are_left_out():
    lens = [200, 100]
    cache, table = cached(1, 256, 32, 32, lens, seed=11)
    kv = sfar.SfarLatent(cache, q_heads=2, rope_dim=32)
    q = torch.randn(1, 2, 2, 288, generator=gen(1), device="cuda").to(BF)
    out = torch.empty(1, 2, 2, 256, dtype=BF, device="cuda")
    bad = [list(t) for t in table]
    bad[0][2], bad[1][0] = 1 << 20, -5
    kv.attention(q, out, ints(bad), ints(lens), ints([0, 1, 2]), max_q=1, scale=0.07)
    torch.cuda.synchronize()
    code, fault = kv.status()
    assert code == sfar.SFAR_ERR_INVALID and sfar.WAIT_NAMES[fault.where] == "page"
    for b, gone in ((0, range(64, 96)), (1, range(0, 32))):
        rows = ref.held_rows(cache[0], table[b], lens[b], 32)
        seen = torch.tensor([[j not in gone for j in range(lens[b])]] * 2, device="cuda")
        want, off = ref.rows(q[0, b], rows, rows[:, :256], seen, 0.07)
        ref.check(out[0, b], want, off)
    for lens2, starts, where in (([200, 100000], [0, 1, 2], "length"), ([200, -3], [0, 1, 2], "length"), ([200, 100], [0, 5, 2], "tokens"),
                                 ([200, 100], [0, 1, 7], "tokens")):
        kv.reset()
        kv.attention(q, out, ints(table), ints(lens2), ints(starts), max_q=1, scale=0.07)
        torch.cuda.synchronize()
        code, fault = kv.status()
        assert code == sfar.SFAR_ERR_INVALID and sfar.WAIT_NAMES[fault.where] in (where, "page"), (lens2, starts)
    kv.reset()
    out2, _, _ = attend(cache, table, lens, [1, 1], 2, 32, q=q, kv=kv)
    check_attention(out2, q, cache, table, lens, [0, 1, 2], 32)
    kv.close()


# ---------------------------------------------------------------------- prompt
def expanded(R, H, D, rot, lens, count, seed, pad=0, sigma=1.0):
    """q, k, v, kr as views of wider tensors, out."""
    g = gen(seed)
    S, T = sum(lens), sum(count) + pad
    new = lambda *s: (sigma * torch.randn(s, generator=g, device="cuda")).to(BF)          # noqa: E731
    kv, rows = new(R, S + 1, H, 2 * D + 8), new(R, S + 1, 2 * D + rot)
    return (new(R, T, H, D + rot), kv[:, :S, :, :D], kv[:, :S, :, D + 8:], rows[:, :S, 2 * D:],
            torch.full((R, T, H, D), float("nan"), dtype=BF, device="cuda"))


def prompt(kv, x, lens, count, max_q=None):
    q, k, v, kr, out = x
    kv.prompt(q, k, v, kr, out, ints(ref.offsets(count)), ints(ref.offsets(lens)), max_q=max(count) if max_q is None else max_q, scale=0.09)
    torch.cuda.synchronize()
    fine(kv)


def check_prompt(x, lens, count):
    q, k, v, kr, out = x
    starts, ks, H = ref.offsets(count), ref.offsets(lens), q.shape[2]
    for r in range(q.shape[0]):
        for b, n in enumerate(lens):
            a, z, s = starts[b], starts[b + 1], slice(ks[b], ks[b + 1])
            for h in range(H if z > a else 0):
                want, off = ref.rows(q[r, a:z, h], torch.cat([k[r, s, h], kr[r, s]], -1), v[r, s, h], ref.causal(z - a, n, "cuda"), 0.09)
                ref.check(out[r, a:z, h], want, off, f"rank {r} request {b} head {h}")
    assert (out[:, starts[-1]:] == 0).all()


def plain_handle(R, H, rot):
    return sfar.SfarLatent(torch.zeros(R, 1, 16, 256 + rot, dtype=BF, device="cuda"), q_heads=H, rope_dim=rot)


@pytest.mark.parametrize("R,H,D,rot,lens,count", [
    (1, 1, 128, 64, [1], [1]),
    (2, 3, 64, 32, [77], [77]),
    (1, 2, 128, 64, [128, 129, 300], [128, 129, 5]),
    (2, 5, 128, 32, [700, 0, 10], [260, 0, 10]),
    (1, 4, 64, 64, [1000, 513], [512, 513]),
    (3, 1, 128, 64, [385, 2], [385, 1]),
    (8, 4, 128, 64, [640, 300, 1], [130, 257, 1]),
    (2, 150, 64, 64, [130], [129]),
    (1, 6, 128, 64, [3000], [3])])
def test_prompt(R, H, D, rot, lens, count):
    x = expanded(R, H, D, rot, lens, count, seed=H + D, pad=3)
    kv = plain_handle(R, H, rot)
    prompt(kv, x, lens, count)
    check_prompt(x, lens, count)
    first = x[4].clone()
    for hint in (0, 1000):                                  # any hint is right
        x[4].fill_(float("nan"))
        prompt(kv, x, lens, count, max_q=hint)
        check_prompt(x, lens, count)
    x[4].fill_(float("nan"))
    prompt(kv, x, lens, count)
    assert torch.equal(x[4], first)                         # the same bits again
    kv.close()


@pytest.mark.parametrize("layout", LAYOUTS[:3])
@pytest.mark.parametrize("H,D,rot,lens,count", [(1, 64, 32, [130, 9], [129, 9]), (5, 128, 64, [300, 500], [290, 3]), (9, 128, 32, [700], [40])])
def test_prompt_strides(layout, H, D, rot, lens, count):
    g, S, T = gen(H), sum(lens), sum(count) + 2
    (q, _), (k, _), (v, _) = [laid_out(layout, 2, n, H, w, g) for n, w in ((T, D + rot), (S, D), (S, D))]
    kr = laid_out("slices of wider rows", 2, S, 1, rot, g)[0][:, :, 0]
    out, wide = laid_out(layout, 2, T, H, D, g)
    out.fill_(0)
    rest = torch.isnan(wide)
    kv = plain_handle(2, H, rot)
    prompt(kv, (q, k, v, kr, out), lens, count)
    check_prompt((q, k, v, kr, out), lens, count)
    assert torch.equal(torch.isnan(wide), rest)
    kv.close()


@pytest.mark.parametrize("B", [64, 65, 100])
def test_prompt_many_requests(B):
    count = [(7 * i) % 5 for i in range(B)]
    count[B // 2] = 150
    lens = [n + (11 * i) % 40 for i, n in enumerate(count)]
    x = expanded(1, 2, 64, 32, lens, count, seed=B, pad=1)
    kv = plain_handle(1, 2, 32)
    prompt(kv, x, lens, count)
    check_prompt(x, lens, count)
    kv.close()


def test_prompt_rows_of_nothing():
    lens, count = [3, 0, 140], [6, 2, 1]
    x = expanded(2, 2, 128, 64, lens, count, seed=8)
    kv = plain_handle(2, 2, 64)
    prompt(kv, x, lens, count)
    q, k, v, kr, out = x
    assert (out[:, :3] == 0).all() and (out[:, 6:8] == 0).all()
    for i in range(3):
        for h in range(2):
            want, off = ref.rows(q[0, 3 + i:4 + i, h], torch.cat([k[0, :3, h], kr[0, :3]], -1), v[0, :3, h],
                                 torch.arange(3, device="cuda")[None] <= i, 0.09)
            ref.check(out[0, 3 + i:4 + i, h], want, off)
    kv.close()


def test_prompt_without_a_context():
    q, out = torch.randn(1, 4, 2, 192, device="cuda").to(BF), torch.full((1, 4, 2, 128), 3.0, dtype=BF, device="cuda")
    k, kr = torch.zeros(1, 0, 2, 128, dtype=BF, device="cuda"), torch.zeros(1, 0, 64, dtype=BF, device="cuda")
    kv = plain_handle(1, 2, 64)
    kv.prompt(q, k, k, kr, out, ints([0, 4]), ints([0, 0]), max_q=4)
    torch.cuda.synchronize()
    fine(kv)
    assert (out == 0).all()
    kv.close()


def test_prompt_steep_scores_move_the_references():
    lens, count = [900], [600]
    q, k, v, kr, out = expanded(1, 4, 128, 64, lens, count, seed=6)
    kr[0, :, 63] = torch.arange(900, device="cuda") / 2
    q[0, :, :2, 191] = 20.0
    q[0, :, 2:, 191] = -20.0
    kv = plain_handle(1, 4, 64)
    prompt(kv, (q, k, v, kr, out), lens, count)
    check_prompt((q, k, v, kr, out), lens, count)
    kv.close()


@pytest.mark.parametrize("count", [[100, 60], [300, 60]])
def test_prompt_row_depends_on_itself_alone(count):
    lens = [420, 140]
    q, k, v, kr, out = expanded(2, 3, 128, 64, lens, count, seed=7)
    kv = plain_handle(2, 3, 64)
    run = lambda: (prompt(kv, (q, k, v, kr, out), lens, count), out.clone())[1]           # noqa: E731
    want, n = run(), count[0]
    # values and keys of a token in the middle of the new ones, and of the next request's first token
    at = 420 - n // 2
    kept = [t.clone() for t in (k, v, kr)]
    v[:, at, :, 5] = float("nan")
    v[:, at + 3, 1, 7] = float("inf")
    v[:, 420, :, 0] = float("-inf")
    got = run()
    first = n - n // 2                                      # the row at that token's position
    assert torch.equal(got[:, :first], want[:, :first])
    assert torch.isnan(got[:, first:n]).flatten(2).any(-1).all()
    assert torch.isnan(got[:, first:n, :, 5]).all()
    for t, x in zip((k, v, kr), kept):
        t.copy_(x)
    k[:, at] = float("inf")
    kr[:, 421] = float("nan")
    got = run()
    assert torch.equal(got[:, :first], want[:, :first]) and torch.isnan(got[:, first:n]).all()
    for t, x in zip((k, v, kr), kept):
        t.copy_(x)
    other = q.clone()
    q[:, 1:] = float("nan")
    got = run()
    assert torch.equal(got[:, 0], want[:, 0]) and torch.isnan(got[:, 1:]).all()
    q.copy_(other)
    assert torch.equal(run(), want)
    kv.close()


def test_prompt_offsets_out_of_order_are_left_out():
    lens, count = [200, 100], [50, 30]
    q, k, v, kr, out = expanded(1, 2, 128, 64, lens, count, seed=3)
    kv = plain_handle(1, 2, 64)
    for starts, ks in (([0, 50, 90], [0, 200, 300]), ([0, 50, 80], [0, 200, 301]), ([50, 0, 30], [0, 200, 300]), ([0, 50, 80], [-1, 200, 300])):
        kv.prompt(q, k, v, kr, out, ints(starts), ints(ks), max_q=50, scale=0.09)
        torch.cuda.synchronize()
        code, fault = kv.status()
        assert code == sfar.SFAR_ERR_INVALID and sfar.WAIT_NAMES[fault.where] == "tokens", (starts, ks)
        kv.reset()
    prompt(kv, (q, k, v, kr, out), lens, count)
    check_prompt((q, k, v, kr, out), lens, count)
    kv.close()
