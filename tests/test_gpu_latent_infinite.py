"""Infinities among the queries, keys and values of latent attention: scores of -inf are no masked ones, and what a row
holds does not depend on the kind of tile in which a token lies."""
import math

import pytest
import torch

import latent_ref as ref
from barrier_free_message_gb300 import _build, sfar
from test_gpu_latent import attend, cached, ints

pytestmark = pytest.mark.gpu
BF, INF = torch.bfloat16, float("inf")
LENGTHS = [1, 5, 63, 64, 200, 700, 5000]                    # whole tiles and cut ones, row tiles in one part and in many


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def without(q, k, v, gone, scale):
    """Rows [n, W] that attend to all tokens but those of `gone`."""
    seen = torch.ones(len(q), len(k), dtype=torch.bool, device="cuda")
    seen[:, gone] = False
    return ref.rows(q, torch.where(seen[0, :, None], k, 0), v, seen, scale)


def place(table, P, at):
    return table[at // P], at % P


# -------------------------------------------------------------- absorbed form
@pytest.mark.parametrize("L,rot,H", [(512, 64, 3), (256, 32, 40)])
@pytest.mark.parametrize("n", LENGTHS)
def test_absorbed_infinite_query(n, L, rot, H):
    """Such a row is NaN whatever the sign of its scores; the others are as they were."""
    cache, table = cached(1, L, rot, 32, [n], seed=n)
    cache[..., 3] = -cache[..., 3].abs().clamp_min(0.01)
    cache[..., L + 5] = cache[..., L + 5].abs().clamp_min(0.01)
    count = min(n, 2)
    q = torch.randn(1, count, H, L + rot, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(BF)
    clean, _, _ = attend(cache, table, [n], [count], H, rot, q=q)
    for value in (INF, -INF, float("nan")):
        bad = q.clone()
        bad[0, 0, 1, 3] = value
        bad[0, -1, 2, L + 5] = value
        got, _, _ = attend(cache, table, [n], [count], H, rot, q=bad)
        assert torch.isnan(got[0, 0, 1]).all() and torch.isnan(got[0, -1, 2]).all(), value
        got[0, 0, 1], got[0, -1, 2] = clean[0, 0, 1], clean[0, -1, 2]
        assert torch.equal(got, clean)


@pytest.mark.parametrize("value", [INF, -INF, torch.finfo(BF).min])
@pytest.mark.parametrize("n", LENGTHS)
def test_absorbed_infinite_keys(n, value):
    """A rotated key with an infinity, or so large that its products pass binary32: rows for which that is +inf are NaN,
    the others leave the token out, wherever it lies."""
    L, rot, H, P = 512, 64, 4, 64
    clean, table = cached(1, L, rot, P, [n], seed=n + 1)
    q = torch.randn(1, 1, H, L + rot, generator=torch.Generator("cuda").manual_seed(2), device="cuda").to(BF)
    q[0, 0, :2, L + 9], q[0, 0, 2:, L + 9] = 40.0, -40.0
    for gone in {(0,), (n - 1,), (n // 2,), tuple(range(min(n, 64))), tuple(range(max(0, n - 70), n)), tuple(range(n))}:
        cache = clean.clone()
        for at in gone:
            cache[0, place(table[0], P, at)[0], place(table[0], P, at)[1], L + 9] = value
        got, _, _ = attend(cache, table, [n], [1], H, rot, q=q)
        up, down = (got[0, 0, :2], got[0, 0, 2:]) if value > 0 else (got[0, 0, 2:], got[0, 0, :2])
        if math.isinf(value):
            assert torch.isnan(up).all(), gone
        if len(gone) == n:
            assert math.isfinite(value) or torch.isnan(down).all(), gone
            continue
        heads = q[0, 0, 2:] if value > 0 else q[0, 0, :2]
        rows = ref.held_rows(clean[0], table[0], n, P)
        want, off = without(heads, rows, rows[:, :L], list(gone), 0.07)
        ref.check(down, want, off, f"without {gone[:3]}..")


@pytest.mark.parametrize("H,L", [(2, 512), (12, 256), (33, 512)])
@pytest.mark.parametrize("n", LENGTHS)
def test_absorbed_infinite_latents(n, H, L):
    """A row that attends to a latent with an infinity is NaN, though that token's weight is 0 and whatever tile it is in."""
    rot, P, count = 64, 16, min(n, 3)
    clean, table = cached(1, L, rot, P, [n], seed=n + 2)
    q = torch.randn(1, count, H, L + rot, generator=torch.Generator("cuda").manual_seed(3), device="cuda").to(BF)
    q[..., 7] = -q[..., 7].abs().clamp_min(0.1)             # times +inf: a score of -inf
    want, _, _ = attend(clean, table, [n], [count], H, rot, q=q)
    assert torch.isfinite(want).all()
    for at in {0, n // 2, n - 1, max(0, n - 2), max(0, n - 70)}:
        cache = clean.clone()
        cache[0, place(table[0], P, at)[0], place(table[0], P, at)[1], 7] = INF
        got, _, _ = attend(cache, table, [n], [count], H, rot, q=q)
        first = max(0, at - (n - count))                    # the first row at or past that token
        assert torch.isnan(got[:, first:]).all(), at
        assert torch.equal(got[:, :first], want[:, :first]), at


# -------------------------------------------------------------- expanded form
def prompt_of(H, D, rot, lens, count, seed):
    """q, k, v, kr of contexts `lens` whose last `count` are new, and a call that gives the results."""
    g = torch.Generator("cuda").manual_seed(seed)
    S, T = sum(lens), sum(count)
    q, k, v, kr = [torch.randn(s, generator=g, device="cuda").to(BF) for s in ((1, T, H, D + rot), (1, S, H, D), (1, S, H, D), (1, S, rot))]

    def run(q, k, v, kr, max_q):
        out = torch.full((1, T, H, D), 7.0, dtype=BF, device="cuda")
        kv = sfar.SfarLatent(torch.zeros(1, 1, 16, 256 + rot, dtype=BF, device="cuda"), q_heads=H, rope_dim=rot)
        kv.prompt(q, k, v, kr, out, ints(ref.offsets(count)), ints(ref.offsets(lens)), max_q=max_q, scale=0.09)
        torch.cuda.synchronize()
        assert kv.status()[0] == sfar.SFAR_OK
        kv.close()
        return out
    return q, k, v, kr, run


# contexts and new tokens: one step and less, whole steps ahead, row tiles in one part and in many, two tiles at a time
PROMPTS = [([1], [1], 2), ([5], [3], 2), ([63], [63], 2), ([64], [2], 2), ([200], [131], 3), ([300], [300], 2), ([1500], [20], 2), ([2200], [300], 9),
           ([9000], [1], 2), ([700, 400], [400, 300], 40)]


@pytest.mark.parametrize("D,rot", [(128, 64), (64, 32)])
@pytest.mark.parametrize("lens,count,H", PROMPTS)
def test_expanded_infinite_query(lens, count, H, D, rot):
    """Such a row is NaN whatever the sign of its scores; the others are as they were."""
    q, k, v, kr, run = prompt_of(H, D, rot, lens, count, seed=sum(lens))
    k[..., 3] = -k[..., 3].abs().clamp_min(0.01)
    kr[..., 5] = kr[..., 5].abs().clamp_min(0.01)
    for max_q in {max(count), 1000}:
        clean = run(q, k, v, kr, max_q)
        assert torch.isfinite(clean).all()
        for value in (INF, -INF, float("nan")):
            bad = q.clone()
            bad[0, 0, 1, 3] = value
            bad[0, -1, 0, D + 5] = value
            got = run(bad, k, v, kr, max_q)
            assert torch.isnan(got[0, 0, 1]).all() and torch.isnan(got[0, -1, 0]).all(), value
            got[0, 0, 1], got[0, -1, 0] = clean[0, 0, 1], clean[0, -1, 0]
            assert torch.equal(got, clean)


@pytest.mark.parametrize("value", [INF, -INF, torch.finfo(BF).min])
@pytest.mark.parametrize("n,count", [(1, 1), (5, 1), (63, 1), (64, 1), (200, 1), (200, 100), (1500, 1), (1500, 140), (9000, 3)])
def test_expanded_infinite_keys(n, count, value):
    """A key, or rotated key, with an infinity, or so large that its products pass binary32: rows for which that is +inf are
    NaN, the others leave the token out, wherever it lies."""
    D, rot, H = 128, 64, 2
    q, k, v, kr, run = prompt_of(H, D, rot, [n], [count], seed=n)
    q[:, :, 0, D + 9], q[:, :, 1, D + 9] = 40.0, -40.0
    q[:, :, 0, 9], q[:, :, 1, 9] = 40.0, -40.0
    for gone in {(0,), (n - 1,), (n // 2,), tuple(range(min(n, 64))), tuple(range(min(n, 130))), tuple(range(max(0, n - 140), n)), tuple(range(n))}:
        at = torch.tensor(gone, device="cuda")
        for rotated in (True, False):
            bad, bad_r = k.clone(), kr.clone()
            if rotated:
                bad_r[0, at, 9] = value
            else:
                bad[0, at, :, 9] = value
            got = run(q, bad, v, bad_r, count)
            seen = ref.causal(count, n, "cuda")
            kept = seen.clone()
            kept[:, at] = False
            up = 0 if value > 0 else 1
            if math.isinf(value):
                assert torch.isnan(got[0, seen[:, at].any(1), up]).all(), gone
                assert torch.isnan(got[0, ~kept.any(1), 1 - up]).all(), gone
            some = kept.any(1)
            keys = torch.cat([k[0, :, 1 - up], kr[0]], -1)
            if some.any():
                want, off = ref.rows(q[0, :, 1 - up], keys, v[0, :, 1 - up], kept, 0.09)
                ref.check(got[0, some, 1 - up], want[some], off[some], f"without {gone[:3]}..")


@pytest.mark.parametrize("D,rot", [(128, 64), (64, 32)])
@pytest.mark.parametrize("lens,count,H", PROMPTS)
def test_expanded_infinite_values(lens, count, H, D, rot):
    """An infinite value is one in its own element of the rows that attend to it, whatever tile it is in."""
    q, k, v, kr, run = prompt_of(H, D, rot, lens, count, seed=sum(lens) + 1)
    n, m, h = lens[0], count[0], H - 1
    clean = {max_q: run(q, k, v, kr, max_q) for max_q in {max(count), 1000}}
    for i, at in enumerate(sorted({0, n // 2, n - m, n - m // 2 - 1, n - 1, max(0, n - 129)})):
        bad, values = v.clone(), [(D - 1, INF), (3, -INF), (D // 2, float("nan"))]
        for d, value in values:
            bad[0, at, h, d] = value
        if at:
            bad[0, at - 1, h, 3] = INF                      # of both signs: NaN where a row attends to both
        for max_q, before in clean.items():
            got = run(q, k, bad, kr, max_q)
            first, lone = max(0, at - (n - m)), bool(at) and at - 1 >= n - m       # lone: a row that attends to at - 1 only
            for d, value in values:
                mine = got[0, first:m, h, d]
                want = float("nan") if math.isnan(value) or (d == 3 and at) else value
                assert (mine.isnan() if math.isnan(want) else mine == want).all(), (at, d, max_q)
            if lone:
                assert (got[0, first - 1, h, 3] == INF).all(), (at, max_q)
            rest = torch.ones_like(got, dtype=torch.bool)
            rest[0, first:m, h, [d for d, _ in values]] = False
            if at:
                rest[0, max(0, first - 1):m, h, 3] = False
            assert torch.equal(got[rest], before[rest]), (at, max_q)


# ------------------------------------------------------------- scores far from 0
def far_scores(n, power):
    """Multiples of 2^power, the largest at one place: numbers of 8 bits, exact in bf16, for keys; times the like for a query."""
    order = torch.randperm(n, generator=torch.Generator().manual_seed(n + power)).cuda() % 200
    order[n // 3] = 201
    return (order + 32).double() * 2.0 ** (power // 2), 2.0 ** (power - power // 2)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [20, 32, 40, 60, 100])
@pytest.mark.parametrize("n", [1, 5, 64, 200, 1500, 5000])
def test_scores_far_from_zero(n, power, sign):
    """Both forms, scores up to 2^108: weights stay in their range, and beyond 2^32 the largest score has them all."""
    H, D, L, rot, P = 2, 64, 256, 32, 32
    at, times = far_scores(n, power)
    if sign < 0:
        at, times = at.flip(0), -times
    clean, table = cached(1, L, rot, P, [n], seed=n)
    rows = ref.held_rows(clean[0], table[0], n, P).clone()
    rows[:, L + 1] = at.to(BF)
    cache = clean.clone()
    for i in range(n):
        cache[0, place(table[0], P, i)[0], place(table[0], P, i)[1], L + 1] = rows[i, L + 1]
    q = torch.randn(1, 1, H, L + rot, generator=torch.Generator("cuda").manual_seed(4), device="cuda").to(BF)
    q[..., L + 1] = times
    best = torch.nonzero(at == (at.max() if sign > 0 else at.min())).flatten()
    got, _, _ = attend(cache, table, [n], [1], H, rot, q=q)
    if len(best) == 1 and (power > 30 or n == 1):           # steps of 2^power * 0.07 in the exponent
        assert torch.equal(got[0, 0], rows[best[0], :L].expand(H, L))
    assert torch.isfinite(got).all()
    count = min(n, 3)
    x = prompt_of(H, D, rot, [n], [count], seed=n + 5)
    x[3][0, :, 1] = at.to(BF)
    x[0][..., D + 1] = times
    for max_q in (count, 1000):
        out = x[4](*x[:4], max_q)
        assert torch.isfinite(out).all()
        for i in range(count if power > 30 else 0):
            seen = at[:n - count + 1 + i]
            best = torch.nonzero(seen == (seen.max() if sign > 0 else seen.min())).flatten()
            if len(best) == 1:
                assert torch.equal(out[0, i], x[2][0, best[0]]), (i, max_q)


@pytest.mark.parametrize("n", [1, 100, 200, 1500])
def test_scores_past_binary32(n):
    """Products that are finite, scores that pass binary32 once scaled: +inf, so NaN, or -inf, weight 0; alike in both forms."""
    D, L, rot = 64, 256, 32
    clean, table = cached(1, L, rot, 32, [n], seed=n)
    q = torch.randn(1, 1, 2, L + rot, generator=torch.Generator("cuda").manual_seed(5), device="cuda").to(BF)
    q[0, 0, 0, L + 1], q[0, 0, 1, L + 1] = 2.0 ** 63, -(2.0 ** 63)
    for at in {0, n // 2, n - 1}:
        cache = clean.clone()
        cache[..., L + 1] = 0
        cache[0, place(table[0], 32, at)[0], place(table[0], 32, at)[1], L + 1] = 2.0 ** 63
        out = torch.empty(1, 1, 2, L, dtype=BF, device="cuda")
        kv = sfar.SfarLatent(cache, q_heads=2, rope_dim=rot)
        rows = ref.held_rows(cache[0], table[0], n, 32)
        kv.attention(q, out, ints(table), ints([n]), ints([0, 1]), max_q=1, scale=8.0)
        k, v = rows[:, None, :D].expand(n, 2, D).contiguous()[None], rows[:, None, D:2 * D].expand(n, 2, D).contiguous()[None]
        qp, op = torch.cat([q[..., :D], q[..., L:]], -1).contiguous(), torch.empty(1, 1, 2, D, dtype=BF, device="cuda")
        kv.prompt(qp, k, v, rows[None, :, L:].contiguous(), op, ints([0, 1]), ints([0, n]), max_q=1, scale=8.0)
        torch.cuda.synchronize()
        assert torch.isnan(out[0, 0, 0]).all() and torch.isnan(op[0, 0, 0]).all(), at
        if n == 1:
            assert torch.isnan(out[0, 0, 1]).all() and torch.isnan(op[0, 0, 1]).all()
        else:
            rows = rows.clone()
            rows[at, L + 1] = 0
            want, off = without(q[0, 0, 1:], rows, rows[:, :L], [at], 8.0)
            ref.check(out[0, 0, 1:], want, off, f"absorbed without {at}")
            want, off = without(qp[0, 0, 1:], torch.cat([rows[:, :D], rows[:, L:]], -1), rows[:, D:2 * D], [at], 8.0)
            ref.check(op[0, 0, 1:], want, off, f"expanded without {at}")
        kv.close()
