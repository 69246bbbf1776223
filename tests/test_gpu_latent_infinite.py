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
