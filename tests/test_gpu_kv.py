"""The paged 8-bit cache's operators on the GPU against the plain 64-bit
references of kv_ref: plans and quantised caches bit for bit, attention and
projection within bounds counted from their roundings."""
import ctypes
import random

import pytest
import torch

import kv_ref
from barrier_free_message_gb300 import sfar
from gpu_helpers import ensure_built
from kv_ref import F8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def cuda_int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def fresh(R=2, H=2, D=64, P=16, pages=8, q_heads=4, seed=0, sigma=60.0):
    """Random caches on the CPU and a handle on their copies on the GPU."""
    g = torch.Generator().manual_seed(seed)
    shape = (R, pages, H, P, D)
    k, v = [(torch.randn(shape, generator=g) * sigma).clamp(-448, 448).to(F8) for _ in range(2)]
    ks, vs = [0.01 * (0.5 + torch.rand(shape[:3], generator=g)) for _ in range(2)]
    dev = [t.cuda() for t in (k, v, ks, vs)]
    return (k, v, ks, vs), dev, sfar.SfarKv(*dev, q_heads=q_heads)


def ok(kv, where=None):
    torch.cuda.synchronize()
    code, f = kv.status()
    if where is None:
        assert code == sfar.SFAR_OK, (code, f.where, f.cta)
    else:
        assert code == sfar.SFAR_ERR_INVALID and f.where == where, (code, f.where)
        kv.reset()
        torch.cuda.synchronize()
        assert kv.status()[0] == sfar.SFAR_OK


# ---------------------------------------------------------------------- plan
def draw_plan(seed, B, P, W, most_add, spare):
    """A consistent state: distinct pages in tables and ring, the ring's free pages anywhere."""
    rng = random.Random(seed)
    lens = [rng.choice([0, rng.randint(0, W * P), rng.randint(0, W) * P]) for _ in range(B)]
    delta = [rng.choice([0, 1, 1, rng.randint(1, most_add), -rng.randint(1, W * P + 3)]) for _ in range(B)]
    held = [-(-n // P) for n in lens]
    pool = max(sum(held) + spare, 1)
    pages = list(range(pool))
    rng.shuffle(pages)
    table, at = [], 0
    for h in held:
        table.append(pages[at:at + h] + [-1] * (W - h))
        at += h
    ring, head = [-1] * pool, rng.randrange(pool)
    for i, p in enumerate(pages[at:]):
        ring[(head + i) % pool] = p
    return lens, delta, table, ring, [head, pool - at]


def run_plan(kv, lens, delta, table, ring, state, tokens, in_place=False):
    t = {"lens": cuda_int(lens), "delta": cuda_int(delta), "table": cuda_int(table), "ring": cuda_int(ring), "state": cuda_int(state)}
    B = len(lens)
    t["lens_out"] = t["lens"] if in_place else cuda_int([-7] * B)
    t["state_out"] = t["state"] if in_place else cuda_int([-7, -7])
    t |= {"starts": cuda_int([-7] * (B + 1)), "slots": cuda_int([-7] * tokens), "taken": cuda_int([-7] * B)}
    kv.plan(*t.values())
    torch.cuda.synchronize()
    return {k: v.tolist() for k, v in t.items() if k not in ("lens", "delta", "state")}


@pytest.mark.parametrize("B,P,W,most_add,spare,extra", [
    (1, 16, 1, 3, 0, 0), (1, 128, 40, 5000, 60, 3), (2, 16, 3, 40, 2, 1), (7, 32, 5, 9, 3, 0), (33, 64, 9, 300, 40, 5),
    (513, 16, 4, 20, 300, 2), (1500, 32, 11, 5, 900, 0), (2048, 16, 3, 60, 5, 7)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(B, P, W, most_add, spare, extra, in_place):
    lens, delta, table, ring, state = draw_plan(B * 7 + P, B, P, W, most_add, spare)
    tokens = sum(max(d, 0) for d in delta) + extra
    _, _, kv = fresh(P=P, pages=len(ring))
    got = run_plan(kv, lens, delta, table, ring, state, tokens, in_place)
    want = kv_ref.plan(P, lens, delta, table, ring, state, tokens)
    for name in want:
        assert got[name] == want[name], name
    ok(kv)


def test_plan_over_many_steps_keeps_every_page_once():
    """In place over 40 steps of growth, drops and refusals: pages are never shared or lost."""
    P, W, B, pool = 16, 6, 24, 70
    rng = random.Random(5)
    _, _, kv = fresh(P=P, pages=pool)
    lens, table, ring, state = [0] * B, [[-1] * W for _ in range(B)], list(range(pool)), [0, pool]
    for _ in range(40):
        delta = [rng.choice([0, 1, 5, rng.randint(1, 40), -rng.randint(1, 60)]) for _ in range(B)]
        tokens = sum(max(d, 0) for d in delta)
        got = run_plan(kv, lens, delta, table, ring, state, tokens, in_place=True)
        assert {k: got[k] for k in got} == kv_ref.plan(P, lens, delta, table, ring, state, tokens)
        lens, table, ring, state = got["lens_out"], got["table"], got["ring"], got["state_out"]
        held = [p for n, row in zip(lens, table) for p in row[:-(-n // P)]]
        free = [ring[(state[0] + i) % pool] for i in range(state[1])]
        assert sorted(held + free) == list(range(pool))
    ok(kv)


def test_plan_reports_what_is_out_of_range():
    P = 16
    base = dict(lens=[3, 20], delta=[1, 13], table=[[0, -1, -1], [1, 2, -1]], ring=[-1, -1, -1, 3], state=[3, 1])
    for change, where in ((dict(lens=[-1, 20]), sfar_where("length")), (dict(lens=[3, 49]), sfar_where("length")),
                          (dict(state=[4, 1]), sfar_where("ring")), (dict(state=[0, 5]), sfar_where("ring")),
                          (dict(state=[-1, 1]), sfar_where("ring")), (dict(ring=[-1, -1, -1, 4]), sfar_where("page")),
                          (dict(table=[[-1, -1, -1], [1, 2, -1]]), sfar_where("page")),
                          (dict(table=[[9, -1, -1], [1, 2, -1]]), sfar_where("page"))):
        c = {**base, **change}
        _, _, kv = fresh(P=P, pages=4)
        got = run_plan(kv, c["lens"], c["delta"], c["table"], c["ring"], c["state"], 14)
        assert all(-1 <= s < 4 * P for s in got["slots"])
        ok(kv, where)
    _, _, kv = fresh(P=P, pages=4)
    got = run_plan(kv, *base.values(), 9)                      # fewer rows than new tokens
    assert got["slots"] == kv_ref.plan(P, *base.values(), 14)["slots"][:9] and got["starts"] == [0, 1, 9]
    ok(kv, sfar_where("tokens"))
    # more pages given back than the pool has room for
    got = run_plan(kv, [32, 16], [-32, 0], [[0, 1], [2, -1]], [3, 0, 1, 2], [0, 4], 0)
    assert got["ring"] == [3, 0, 1, 2] and got["state_out"] == [0, 4]
    ok(kv, sfar_where("ring"))


def sfar_where(name):
    return {v: k for k, v in sfar.WAIT_NAMES.items()}[name]


# -------------------------------------------------------------------- append
def check_append(cpu, dev, x, slots, ctx=""):
    for i, name in enumerate(("k", "v")):
        for r in range(cpu[0].shape[0]):
            values, scales = kv_ref.append(cpu[i][r], cpu[i + 2][r], x[i][r], slots)
            got, got_s = dev[i][r].cpu().double(), dev[i + 2][r].cpu().double()
            assert torch.equal(got_s, scales), f"{ctx} scale of {name} of rank {r}"
            assert torch.equal(got.nan_to_num(1e9), values.nan_to_num(1e9)), f"{ctx} {name} of rank {r}"


def token_rows(g, R, T, H, D, wide):
    """k and v as slices of one wider tensor (wide), or contiguous."""
    loud = torch.exp(1.5 * torch.randn(R, T, 1, 1, generator=g))
    if not wide:
        return [(torch.randn(R, T, H, D, generator=g) * loud).to(torch.bfloat16) for _ in range(2)]
    qkv = (torch.randn(R, T, 3 * H + 1, D, generator=g) * loud).to(torch.bfloat16)
    return [qkv[:, :, H:2 * H], qkv[:, :, 2 * H:3 * H]]


@pytest.mark.parametrize("R,H,D,P,runs,wide", [
    (1, 1, 64, 16, [(0, 1)], False), (2, 1, 128, 16, [(15, 1), (0, 16), (3, 5)], True), (3, 2, 64, 32, [(0, 31), (31, 1), (1, 31)], True),
    (2, 3, 128, 64, [(0, 64), (0, 63), (40, 24), (63, 1)], False), (8, 1, 128, 128, [(0, 128), (1, 127), (100, 3), (0, 1)], True),
    (2, 8, 64, 128, [(0, 128), (7, 100)], False), (4, 2, 128, 32, [(i % 32, 1) for i in range(70)], True),
    (1, 1, 128, 16, [(0, 16)] * 150 + [(2, 14)], True)])
def test_append(R, H, D, P, runs, wide):
    """runs: (first offset, tokens) of one page each."""
    g = torch.Generator().manual_seed(R * 100 + P)
    cpu, dev, kv = fresh(R=R, H=H, D=D, P=P, pages=len(runs) + 2, q_heads=H, seed=P)
    pages = torch.randperm(len(runs) + 2, generator=g).tolist()
    slots = []
    for p, (first, n) in zip(pages, runs):
        slots += [p * P + first + i for i in range(n)] + ([-1] if n % 3 == 1 else [])
    x = token_rows(g, R, len(slots), H, D, wide)
    kv.append(x[0].cuda() if not wide else x[0].cuda(), x[1].cuda(), cuda_int(slots))
    ok(kv)
    check_append(cpu, dev, x, slots)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_append_many_tokens(D, P):
    """Whole pages, their parts and single tokens, enough of them that windows of many tokens are taken; zeros, infinities
    and NaN among them, growth of held pages, slots outside the pool."""
    R, H = 4, 3
    g = torch.Generator().manual_seed(D + P)
    runs = [(0, P), (0, P), (P - 1, 1), (1, P - 1), (0, P // 2 + 1), (P // 2, P // 2), (0, 1)]
    while sum(n for _, n in runs) < 650:
        first = int(torch.randint(0, P, (1,), generator=g))
        runs.append((first, int(torch.randint(1, P - first + 1, (1,), generator=g))))
    cpu, dev, kv = fresh(R=R, H=H, D=D, P=P, pages=len(runs) + 2, q_heads=H, seed=P)
    pages = torch.randperm(len(runs) + 2, generator=g).tolist()
    slots = []
    for i, (p, (first, n)) in enumerate(zip(pages, runs)):
        slots += [p * P + first + j for j in range(n)] + ([-1] * (i % 4) if i % 3 == 1 else [])
    x = token_rows(g, R, len(slots), H, D, True)
    for t in x:
        t[:, P + 3] = 0.0
        t[1, 2 * P - 1, 0, 5] = float("nan")
        t[2, 5, 1] = float("inf")
        t[0, :P, 2] = 0.0
        t[3, -1, 0, 0] = -3.3e38
    kv.append(x[0].cuda(), x[1].cuda(), cuda_int(slots))
    ok(kv)
    check_append(cpu, dev, x, slots)
    before, bad = [t.cpu() for t in dev], [-1 if i % 5 else len(cpu[0][0]) * P + i for i in range(len(slots))]
    kv.append(x[0].cuda(), x[1].cuda(), cuda_int(bad))
    ok(kv, sfar_where("slot"))
    check_append(before, dev, x, [-1] * len(slots))


def test_append_strided_slices_and_lists():
    """k and v as views into one tensor on the device; ranks as a list of tensors."""
    g = torch.Generator().manual_seed(3)
    cpu, dev, kv = fresh(R=3, H=2, D=64, P=16, pages=4, q_heads=2)
    qkv = torch.randn(3, 21, 7, 64, generator=g).to(torch.bfloat16).cuda()
    k, v = qkv[:, :, 2:4], qkv[:, :, 5:7]
    slots = list(range(16 + 9, 32)) + list(range(0, 14))
    kv.append([k[r] for r in range(3)], v, cuda_int(slots))
    ok(kv)
    check_append(cpu, dev, [k.cpu(), v.cpu()], slots)


def test_append_special_values():
    """Zeros, subnormals, the largest values, infinities and NaN; growth over many steps; a scale that is no power of two."""
    P, D = 16, 64
    for name, first, fill in (("zeros", 0, 0.0), ("tiny", 0, 1e-39), ("largest", 0, 3.3e38), ("largest held", 5, 3.3e38),
                              ("inf", 0, float("inf")), ("nan held", 7, float("nan")), ("edge", 0, 448.0), ("past edge", 0, 450.0)):
        cpu, dev, kv = fresh(R=1, H=1, D=D, P=P, pages=2, q_heads=1)
        x = [torch.randn(1, 3, 1, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16) for _ in range(2)]
        for t in x:
            t[0, 1] = fill
            t[0, 2, 0, ::2] = fill
        slots = [P + first + i for i in range(3)]
        kv.append(x[0].cuda(), x[1].cuda(), cuda_int(slots))
        ok(kv)
        check_append(cpu, dev, x, slots, name)
    cpu, dev, kv = fresh(R=1, H=2, D=D, P=P, pages=1, q_heads=2)
    for i in range(P):
        x = [(torch.randn(1, 1, 2, D, generator=torch.Generator().manual_seed(i)) * 2.0 ** (i - 3)).to(torch.bfloat16) for _ in range(2)]
        before = [t.cpu() for t in dev]
        kv.append(x[0].cuda(), x[1].cuda(), cuda_int([i]))
        ok(kv)
        check_append(before, dev, x, [i], f"step {i}")


def test_append_reports_bad_slots():
    cpu, dev, kv = fresh(R=2, H=2, D=64, P=16, pages=4)
    x = token_rows(torch.Generator().manual_seed(0), 2, 4, 2, 64, False)
    kv.append(x[0].cuda(), x[1].cuda(), cuda_int([64, 5, -2, 1 << 30]))
    ok(kv, sfar_where("slot"))
    check_append(cpu, dev, x, [-1, 5, -1, -1])


# ----------------------------------------------------------------- attention
def poison(cpu, P, table, lens):
    """NaN in every cached place that no request holds."""
    k, v = cpu[0], cpu[1]
    live = torch.zeros(k.shape[1], P, dtype=torch.bool)
    for row, n in zip(table, lens):
        for i in range(-(-n // P)):
            live[row[i], :min(P, n - i * P)] = True
    for c in (k, v):
        c.view(torch.uint8)[:, ~live[:, None, :].expand(-1, k.shape[2], -1)] = 0x7f
    dead = ~live.any(1)
    for s in cpu[2:]:
        s[:, dead] = float("nan")


def setup_attention(R, H, G, D, P, lens, counts, seed, pad_rows=0, sigma=60.0, q_sigma=1.5, wide=False):
    g = torch.Generator().manual_seed(seed)
    held = [-(-n // P) for n in lens]
    pages = sum(held) + 3
    perm = torch.randperm(pages, generator=g).tolist()
    W = max(max(held), 1) + 1
    table, at = [], 0
    for h in held:
        table.append(perm[at:at + h] + [-1] * (W - h))
        at += h
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + c)
    T = starts[-1] + pad_rows
    cpu, _, _ = fresh(R=R, H=H, D=D, P=P, pages=pages, q_heads=H * G, seed=seed, sigma=sigma)
    poison(cpu, P, table, lens)
    q = (torch.randn(R, T, H * G + (2 if wide else 0), D, generator=g) * q_sigma).to(torch.bfloat16)
    return cpu, table, starts, q


def run_attention(cpu, table, lens, starts, q, Hq, scale, window=0, max_q=None, wide=False, stream=None):
    dev = [t.cuda() for t in cpu]
    kv = sfar.SfarKv(*dev, q_heads=Hq)
    qd = q.cuda()[:, :, 1:1 + Hq] if wide else q.cuda()
    buf = torch.full_like(q.cuda(), 7.0)
    out = buf[:, :, :Hq] if wide else buf
    counts = [b - a for a, b in zip(starts, starts[1:])]
    kv.attention(qd, out, cuda_int(table), cuda_int(lens), cuda_int(starts), max_q=max(counts) if max_q is None else max_q,
                 scale=scale, window=window)
    ok(kv)
    if wide:
        assert (buf[:, :, Hq:] == 7.0).all()
    return out.cpu().double()


def check_attention(got, cpu, table, lens, starts, q, scale, window=0, ctx=""):
    """|out - o| <= 2^-8 |o| + 2^-10 m + n 2^-24 max|v|: one rounding to bf16; with m the weighted mean of |v|, the
    weights' rounding to 11 bits (2^-11) and as much again for the exponentials and binary32 sums; weights far
    below the largest may lose their last bits (2^-25 each, of n, twice).  A row of nothing is exactly zero."""
    n = max(lens + [1])
    for r in range(q.shape[0]):
        want, mag = kv_ref.attention(q[r], *[c[r] for c in cpu], table, lens, starts, scale, window)
        vmax = float((cpu[1][r].double() * cpu[3][r].double()[..., None, None]).nan_to_num(0.0).abs().max())
        bound = 2.0 ** -8 * want.abs() + 2.0 ** -10 * mag + n * 2.0 ** -24 * vmax
        bound[mag == 0] = 0
        off = (got[r] - want).abs()
        assert torch.isfinite(got[r]).all(), f"{ctx} rank {r}: not finite"
        worst = (off - bound).max()
        assert (off <= bound).all(), f"{ctx} rank {r}: {float(worst):.3g} over the bound at {int((off - bound).argmax())}"


CASES = [
    # R, H, G, D, P, lens, counts, window
    (1, 1, 1, 64, 16, [1], [1], 0),
    (2, 1, 8, 128, 16, [1, 2, 15, 16, 17, 63, 64, 65], [1] * 8, 0),
    (2, 2, 4, 64, 32, [100, 0, 33, 31, 32], [1, 1, 1, 1, 1], 0),
    (3, 2, 5, 128, 64, [129, 1000, 64], [1, 1, 1], 0),
    (2, 1, 16, 128, 128, [300, 128, 127], [1, 1, 1], 0),
    (1, 3, 7, 64, 128, [700, 5], [1, 1], 0),
    (1, 2, 32, 128, 32, [77, 400], [1, 1], 0),
    (2, 1, 3, 64, 16, [40, 41, 700], [1, 1, 1], 33),
    (2, 1, 8, 128, 64, [200, 70], [1, 1], 1),
    # several tokens at once, some requests without any, some with more tokens than context
    (2, 2, 2, 64, 16, [7, 50, 33, 16], [7, 4, 0, 2], 0),
    (1, 1, 8, 128, 64, [9, 130, 64], [2, 2, 2], 0),
    (1, 2, 3, 128, 32, [5, 90, 0, 3], [5, 7, 2, 6], 0),
    (2, 1, 4, 64, 16, [60, 128], [20, 9], 17),
    # chunks of prompts
    (2, 1, 8, 128, 64, [300, 129], [300, 40], 0),
    (1, 2, 4, 64, 32, [200, 333, 64], [64, 129, 1], 0),
    (1, 1, 5, 128, 16, [257], [191], 0),
    (1, 1, 1, 128, 128, [513, 140], [400, 140], 100),
    (2, 2, 16, 64, 64, [150, 31], [33, 31], 0),
    (1, 1, 24, 128, 32, [90], [50], 0),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attention(case):
    R, H, G, D, P, lens, counts, window = case
    cpu, table, starts, q = setup_attention(R, H, G, D, P, lens, counts, 11 + P)
    scale = D ** -0.5
    got = run_attention(cpu, table, lens, starts, q, H * G, scale, window)
    check_attention(got, cpu, table, lens, starts, q, scale, window)


def test_attention_long_context():
    """One request whose context is shared out over the whole GPU, and a batch of very unequal ones."""
    for lens, counts, P in (([20011], [1], 32), ([9001, 3, 700, 1, 4096, 64], [1] * 6, 64), ([6000, 6000], [2, 3], 16)):
        cpu, table, starts, q = setup_attention(2, 1, 8, 128, P, lens, counts, 5)
        got = run_attention(cpu, table, lens, starts, q, 8, 0.09)
        check_attention(got, cpu, table, lens, starts, q, 0.09, ctx=str(lens))


@pytest.mark.parametrize("R,H,G,D,P,lens,counts", [
    (1, 1, 16, 128, 32, [60007], [1]), (1, 1, 3, 64, 16, [40000, 17], [1, 1]), (1, 2, 8, 64, 64, [9000], [40]),
    (1, 1, 8, 128, 128, [20000, 300], [17, 2])])
def test_attention_of_few_rows_joined_from_many_parts(R, H, G, D, P, lens, counts):
    """One long context for a few rows: its parts are joined in groups, then the groups."""
    cpu, table, starts, q = setup_attention(R, H, G, D, P, lens, counts, 71)
    for _ in range(2):                                           # the counters of parts are clear again
        got = run_attention(cpu, table, lens, starts, q, H * G, 0.1)
        check_attention(got, cpu, table, lens, starts, q, 0.1, ctx=str(lens))


def test_attention_strided_rows_and_padding():
    """q and out as slices of wider tensors; rows past the last request are zeros; a hint that is too small."""
    for counts, lens in (([1, 1, 1], [40, 7, 90]), ([30, 2, 41], [64, 2, 200])):
        cpu, table, starts, q = setup_attention(2, 2, 4, 64, 16, lens, counts, 23, pad_rows=5, wide=True)
        for max_q in (None, 1):
            got = run_attention(cpu, table, lens, starts, q, 8, 0.125, max_q=max_q, wide=True)
            assert (got[:, starts[-1]:] == 0).all()
            check_attention(got, cpu, table, lens, starts, q[:, :, 1:9], 0.125)


def test_attention_extreme_scores():
    """Scores far apart (one key takes all the weight), equal scores (scale 0), and large and small queries."""
    lens, counts = [200, 65, 130], [1, 1, 64]
    for scale, q_sigma in ((0.0, 1.0), (0.125, 300.0), (0.125, 1e-30), (1.0, 1e-3), (1e-4, 1e5)):
        cpu, table, starts, q = setup_attention(1, 1, 4, 64, 16, lens, counts, 31, q_sigma=q_sigma)
        got = run_attention(cpu, table, lens, starts, q, 4, scale)
        if q_sigma < 200:
            check_attention(got, cpu, table, lens, starts, q, scale, ctx=f"{scale} {q_sigma}")
        else:
            # the scores' own binary32 sums are off by up to D 2^-24 sum|q k|, about 2^-6 here: the weights follow
            want = torch.stack([kv_ref.attention(q[r], *[c[r] for c in cpu], table, lens, starts, scale)[0] for r in range(1)])
            assert torch.allclose(got, want, rtol=2 ** -5, atol=2 ** -4)


def test_attention_nan_reaches_only_rows_that_see_it():
    """A NaN among the new tokens' keys or values makes the rows that attend to it NaN and leaves the others alone."""
    for counts, lens, G in (([4], [30], 2), ([40], [90], 4), ([300], [300], 8)):
        for which in (0, 1):
            cpu, table, starts, q = setup_attention(1, 1, G, 64, 16, lens, counts, 41)
            at = lens[0] - counts[0] // 2                        # a new token in the middle
            clean = [c.clone() for c in cpu]
            cpu[which].view(torch.uint8)[0, table[0][at // 16], 0, at % 16, 5] = 0x7f
            got = run_attention(cpu, table, lens, starts, q, G, 0.125)
            row = at - (lens[0] - counts[0])
            check_attention(got[:, :row], clean, table, [at], [0, row], q[:, :row], 0.125, ctx=f"{counts} {which}")
            if which == 0:
                assert torch.isnan(got[:, row:]).all()
            else:
                assert torch.isnan(got[:, row:, :, 5]).all()


def test_attention_reports_bad_pages_and_lengths():
    lens, counts = [40, 33], [1, 1]
    cpu, table, starts, q = setup_attention(1, 1, 2, 64, 16, lens, counts, 51)
    dev = [t.cuda() for t in cpu]
    kv = sfar.SfarKv(*dev, q_heads=2)
    qd = q.cuda()
    for page in (-1, cpu[0].shape[1], 1 << 30):
        bad = [list(r) for r in table]
        bad[0][1] = page
        out = torch.empty_like(qd)
        kv.attention(qd, out, cuda_int(bad), cuda_int(lens), cuda_int(starts), max_q=1, scale=0.125)
        ok(kv, sfar_where("page"))
        check_attention(out.cpu().double()[:, 1:], cpu, table[1:], lens[1:], [0, 1], q[:, 1:], 0.125)
    for n in (-5, len(table[0]) * 16 + 1, 1 << 30):
        out = torch.empty_like(qd)
        bad = [list(r) for r in table]
        bad[0] = [table[0][0]] * len(table[0])
        kv.attention(qd, out, cuda_int(bad), cuda_int([n, 33]), cuda_int(starts), max_q=1, scale=0.125)
        ok(kv, sfar_where("length"))
        check_attention(out.cpu().double()[:, 1:], cpu, table[1:], lens[1:], [0, 1], q[:, 1:], 0.125)


@pytest.mark.parametrize("max_q", [1, 512])
def test_attention_refuses_offsets_in_no_order(max_q):
    """Offsets that run back and forth give the requests more rows together than the step has: recorded, nothing written."""
    T, B = 512, 9
    cpu, table, _, q = setup_attention(1, 1, 8, 64, 64, [600] * B, [57] * 8 + [56], 53)
    assert q.shape[1] == T
    kv = sfar.SfarKv(*[t.cuda() for t in cpu], q_heads=8)
    out = torch.full_like(q, 7.0).cuda()
    args = [cuda_int(table), cuda_int([600] * B), cuda_int([0, T] * 5)]
    kv.attention(q.cuda(), out, *args, max_q=max_q, scale=0.125)
    ok(kv, sfar_where("tokens"))
    assert (out == 7.0).all()


def test_attention_side_stream_and_graph():
    """On a stream of its own, captured; replays follow lengths and caches that change between them."""
    R, H, G, D, P = 2, 1, 8, 128, 64
    lens, counts = [500, 90, 1], [1, 1, 1]
    cpu, table, starts, q = setup_attention(R, H, G, D, P, lens, counts, 61)
    dev = [t.cuda() for t in cpu]
    kv = sfar.SfarKv(*dev, q_heads=G)
    qd, td, ld, sd = q.cuda(), cuda_int(table), cuda_int(lens), cuda_int(starts)
    out = torch.empty_like(qd)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        kv.attention(qd, out, td, ld, sd, max_q=1)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=st):
            for _ in range(3):
                kv.attention(qd, out, td, ld, sd, max_q=1)
    for now in ([500, 90, 1], [257, 0, 1], [64, 63, 1]):
        ld.copy_(cuda_int(now))
        out.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        ok(kv)
        check_attention(out.cpu().double(), cpu, table, now, starts, q, D ** -0.5, ctx=str(now))


# ---------------------------------------------------------------- projection
def check_gemm(y, x8, sx, w8, sw, ctx=""):
    """|y - exact| <= 2^-8 |exact| + (k + 2 kb) 2^-23 sum|terms|: one rounding to bf16, and a sum of k products and
    kb scaled blocks in binary32 in any order, each step off by at most one unit (matrix units may truncate)."""
    for r in range(y.shape[0]):
        want, mag = kv_ref.gemm(x8[r], sx[r], w8[r], sw[r])
        k = x8.shape[2]
        bound = 2.0 ** -8 * want.abs() + (k + 2 * sw.shape[2]) * 2.0 ** -23 * mag
        off = (y[r].double() - want).abs()
        assert (off <= bound).all(), f"{ctx} rank {r}: {float((off - bound).max()):.3g} over the bound, at {int((off - bound).argmax())}"


@pytest.mark.parametrize("R,m,k,n", [
    (2, 1, 128, 128), (2, 1, 16, 8), (3, 3, 1000, 264), (2, 5, 7, 1), (4, 16, 256, 520), (2, 17, 300, 129), (2, 33, 128, 2056),
    (2, 64, 1024, 384), (16, 2, 130, 40), (2, 100, 384, 256), (2, 127, 200, 130), (2, 128, 512, 255), (2, 129, 640, 512),
    (3, 200, 1111, 391), (2, 300, 256, 1000), (8, 8, 3584, 256)])
def test_quantize_and_gemm(R, m, k, n):
    g = torch.Generator().manual_seed(m * 1000 + k + n)
    up = -(-k // 16) * 16
    x = (torch.randn(R, m, k, generator=g) * torch.exp(torch.randn(R, m, 1, generator=g))).to(torch.bfloat16)
    w = (torch.randn(R, n, up, generator=g) * 100).clamp(-448, 448).to(F8)
    w.view(torch.uint8)[:, :, k:] = 0x7f                       # past a row's end: NaN that must not be read
    sw = 1e-3 * (0.5 + torch.rand(R, -(-n // 128), -(-k // 128), generator=g))
    x8 = torch.full((R, m, up), 0x7f, dtype=torch.uint8, device="cuda").view(F8)[:, :, :k]
    sx = torch.empty(R, -(-k // 128), m, device="cuda")
    y = torch.full((R, m, n), 5.0, dtype=torch.bfloat16, device="cuda")
    h = sfar.Sfar(R, 1 << 16, "bf16")
    try:
        h.quantize_fp8(x.cuda(), x8, sx)
        h.rowpar_gemm_fp8(x8, sx, w.cuda()[:, :, :k], sw.cuda(), y)
        torch.cuda.synchronize()
        assert h.status()[0] == sfar.SFAR_OK
    finally:
        h.close()
    for r in range(R):
        q, s = kv_ref.quantize(x[r])
        assert torch.equal(sx[r].cpu().double(), s)
        assert torch.equal(x8[r].cpu().double(), q)
    check_gemm(y.cpu(), x8.cpu(), sx.cpu(), w[:, :, :k], sw, f"{R} {m} {k} {n}")


@pytest.mark.parametrize("R,m,k,n", [(8, 300, 200, 1000), (4, 513, 130, 1030), (2, 257, 72, 4832), (8, 260, 384, 1001),
                                     (3, 1100, 1027, 776), (8, 256, 1536, 2048)])
def test_quantize_and_gemm_of_many_tiles(R, m, k, n):
    """More tiles of 128 x 128 than there are SMs; last outputs that are no multiple of 128, 16 or 8."""
    test_quantize_and_gemm(R, m, k, n)


def test_quantize_rows_of_every_alignment():
    """Rows that begin on any even address, in a tensor that others' values surround; an infinity at one place."""
    R, m, k = 2, 17, 2200
    g = torch.Generator().manual_seed(12)
    h = sfar.Sfar(R, 1 << 16, "bf16")
    try:
        for at, wide in ((0, 2200), (1, 2203), (3, 2208), (4, 2204), (6, 2207), (7, 2209)):
            whole = torch.full((R, m + 2, wide + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
            xd = whole[:, 1:-1, at:at + k]
            x = (torch.randn(R, m, k, generator=g) * torch.exp(2 * torch.randn(R, m, 1, generator=g))).to(torch.bfloat16)
            x[1, m - 1, k - 1] = float("inf")
            xd.copy_(x)
            x8 = torch.zeros(R, m, 2208, dtype=torch.uint8, device="cuda").view(F8)[:, :, :k]
            sx = torch.empty(R, -(-k // 128), m, device="cuda")
            for given in (xd, [t.contiguous() for t in xd]):
                h.quantize_fp8(given, x8, sx)
                torch.cuda.synchronize()
                for r in range(R):
                    q, s = kv_ref.quantize(x[r])
                    assert torch.equal(sx[r].cpu().double(), s), (at, r)
                    assert torch.equal(x8[r].cpu().double().nan_to_num(1e9), q.nan_to_num(1e9)), (at, r)
    finally:
        h.close()


def test_quantize_special_values_and_strides():
    x = torch.randn(2, 6, 300, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    x[0, 0] = 0
    x[0, 1, 5], x[0, 1, 200] = float("inf"), float("nan")
    x[0, 2] = float("nan")
    x[0, 3] = 3.3e38
    x[1, 0] = 1e-39
    x[1, 1, ::7] = -448.0
    x[1, 2, 299] = 1e30
    h = sfar.Sfar(2, 1 << 16, "bf16")
    try:
        for wide_in, at, wide_out in ((300, 0, 304), (305, 1, 303), (320, 8, 304)):
            xd = torch.zeros(2, 6, wide_in + 8, dtype=torch.bfloat16, device="cuda")[:, :, at:at + 300]
            xd.copy_(x)
            x8 = torch.zeros(2, 6, wide_out, dtype=torch.uint8, device="cuda").view(F8)
            sx = torch.empty(2, 3, 6, device="cuda")
            h.quantize_fp8(xd, x8[:, :, :300], sx)
            torch.cuda.synchronize()
            assert (x8.view(torch.uint8)[:, :, 300:] == 0).all()
            for r in range(2):
                q, s = kv_ref.quantize(x[r])
                assert torch.equal(sx[r].cpu().double(), s)
                assert torch.equal(x8[r, :, :300].cpu().double().nan_to_num(1e9), q.nan_to_num(1e9))
    finally:
        h.close()


def test_gemm_nan_stays_in_its_row_and_column():
    R, m, k, n = 2, 40, 256, 300
    g = torch.Generator().manual_seed(9)
    x8 = torch.randn(R, m, k, generator=g).to(F8)
    w8 = torch.randn(R, n, k, generator=g).to(F8)
    sx, sw = torch.rand(R, 2, m, generator=g) + 0.5, torch.rand(R, 3, 2, generator=g) + 0.5
    x8.view(torch.uint8)[0, 7, 130] = 0x7f
    w8.view(torch.uint8)[1, 200, 3] = 0xff
    y = torch.empty(R, m, n, dtype=torch.bfloat16, device="cuda")
    h = sfar.Sfar(R, 1 << 16, "bf16")
    try:
        h.rowpar_gemm_fp8(x8.cuda(), sx.cuda(), w8.cuda(), sw.cuda(), y)
        torch.cuda.synchronize()
    finally:
        h.close()
    nan = torch.zeros(R, m, n, dtype=torch.bool)
    nan[0, 7], nan[1, :, 200] = True, True
    y = y.cpu()
    assert torch.equal(torch.isnan(y), nan)
    x8.view(torch.uint8)[0, 7] = 0
    w8.view(torch.uint8)[1, 200] = 0
    check_gemm(torch.where(nan, 0, y), x8, sx, w8, sw)


# ----------------------------------------------------------------- refusals
def rank_ptrs(tensors):
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def test_calls_refuse_bad_arguments():
    cpu, dev, kv = fresh(R=2, H=2, D=64, P=16, pages=4, q_heads=4)
    L, z = sfar.lib(), torch.zeros(4096, dtype=torch.int32, device="cuda")
    a = z.data_ptr()
    bf = torch.zeros(2, 4, 4, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(bf)
    x, o = [(rank_ptrs(t)) for t in (bf, out)]
    odd = rank_ptrs([bf[0].flatten()[1:], bf[1]])
    bad = sfar.SFAR_ERR_INVALID
    at = [a + 256 * i for i in range(10)]
    assert L.sfar_kv_plan(kv.h, *at, 4, 2, 8, None) == 0
    for args in ((0, 2, 8), (8193, 2, 8), (4, 0, 8), (4, 1 << 31, 8), (4, 2, 1 << 31), (4, 64, 8)):
        assert L.sfar_kv_plan(kv.h, *at, *args, None) == bad, args
    for i in range(10):
        assert L.sfar_kv_plan(kv.h, *[v if j != i else None for j, v in enumerate(at)], 4, 2, 8, None) == bad, i
        assert L.sfar_kv_plan(kv.h, *[v if j != i else v + 2 for j, v in enumerate(at)], 4, 2, 8, None) == bad, i
    for i, j in ((5, 1), (2, 3), (8, 9), (6, 0), (7, 2)):
        assert L.sfar_kv_plan(kv.h, *[v if n != i else at[j] + 4 for n, v in enumerate(at)], 4, 2, 8, None) == bad, (i, j)
    for p in (None, odd):
        assert L.sfar_kv_append(kv.h, p, x, a, 4, 256, 64, 256, 64, None) == bad
        assert L.sfar_kv_append(kv.h, x, p, a, 4, 256, 64, 256, 64, None) == bad
        assert L.sfar_kv_attention(kv.h, p, o, a, a, a, 1, 1, 4, 256, 64, 256, 64, 1, 1.0, 0, None) == bad
        assert L.sfar_kv_attention(kv.h, x, p, a, a, a, 1, 1, 4, 256, 64, 256, 64, 1, 1.0, 0, None) == bad
    assert L.sfar_kv_append(kv.h, x, x, None, 4, 256, 64, 256, 64, None) == bad
    assert L.sfar_kv_append(kv.h, x, x, a, 4, 252, 64, 256, 64, None) == bad
    assert L.sfar_kv_append(kv.h, x, x, None, 0, 256, 64, 256, 64, None) == 0          # nothing to do
    for args in ((0, 1, 4), (8193, 1, 4), (1, 0, 4), (1, 1, 1 << 31)):
        assert L.sfar_kv_attention(kv.h, x, o, a, a, a, *args, 256, 64, 256, 64, 1, 1.0, 0, None) == bad
    for scale in (-1.0, float("inf"), float("nan")):
        assert L.sfar_kv_attention(kv.h, x, o, a, a, a, 1, 1, 4, 256, 64, 256, 64, 1, scale, 0, None) == bad
    for width, tokens, strides, max_q in ((1, 1 << 28, 0, 1), (1, 1 << 28, 0, 64), (1 << 30, 1 << 20, 0, 1), (1 << 30, 1 << 27, 0, 64),
                                          (1, 4, 1 << 40, 1)):           # more than the kernels' sums hold
        assert L.sfar_kv_attention(kv.h, x, o, a, a, a, 1, width, tokens, *[strides] * 4, max_q, 1.0, 0, None) == bad, (width, tokens)
    assert L.sfar_kv_append(kv.h, x, x, a, 4, 1 << 40, 64, 256, 64, None) == bad
    assert L.sfar_kv_attention(kv.h, x, x, a, a, a, 1, 1, 4, 256, 64, 256, 64, 1, 1.0, 0, None) == bad
    assert L.sfar_kv_attention(kv.h, x, o, a, a, a, 1, 1, 4, 256, 60, 256, 64, 1, 1.0, 0, None) == bad
    assert L.sfar_kv_attention(kv.h, x, o, a, a, a, 1, 1, 0, 256, 64, 256, 64, 1, 1.0, 0, None) == 0
    ok(kv)
    fp32 = sfar.Sfar(2, 1 << 16, "fp32")
    h = sfar.Sfar(2, 1 << 16, "bf16")
    try:
        f = torch.zeros(2, 8192, device="cuda")
        b1, b2, s1, s2 = [rank_ptrs(f[:, 2048 * i:2048 * i + 2048]) for i in range(4)]
        assert L.sfar_quantize_fp8(fp32.h, b1, b2, s1, 2, 64, 64, 64, None) == bad
        assert L.sfar_rowpar_gemm_fp8(fp32.h, b1, s1, b2, s2, o, 2, 64, 8, 64, 64, None) == bad
        assert L.sfar_quantize_fp8(h.h, b1, b2, s1, 2, 64, 64, 64, None) == 0
        assert L.sfar_rowpar_gemm_fp8(h.h, b1, s1, b2, s2, o, 2, 64, 8, 64, 64, None) == 0
        for args in ((0, 64, 64, 64), (2, 0, 64, 64), (2, 64, 63, 64), (2, 64, 64, 63)):
            assert L.sfar_quantize_fp8(h.h, b1, b2, s1, *args, None) == bad
        assert L.sfar_quantize_fp8(h.h, b1, b1, s1, 2, 64, 64, 64, None) == bad
        assert L.sfar_quantize_fp8(h.h, b1, b2, b2, 2, 64, 64, 64, None) == bad
        for args in ((0, 64, 8, 64, 64), (2, 0, 8, 64, 64), (2, 64, 0, 64, 64), (2, 64, 8, 48, 64), (2, 64, 8, 64, 72)):
            assert L.sfar_rowpar_gemm_fp8(h.h, b1, s1, b2, s2, o, *args, None) == bad
        assert L.sfar_rowpar_gemm_fp8(h.h, b1, s1, b2, s2, b2, 2, 64, 8, 64, 64, None) == bad
        assert L.sfar_rowpar_gemm_fp8(h.h, b1, None, b2, s2, o, 2, 64, 8, 64, 64, None) == bad
        torch.cuda.synchronize()
    finally:
        h.close()
        fp32.close()
