"""The plan of the paged cache's steps: more pages given back than the pool holds, bad pages given
back, and thousands of requests."""
import pytest

import kv_ref
from test_gpu_kv import _built, draw_plan, fresh, ok, run_plan, sfar_where  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def test_more_pages_given_back_than_are_held():
    """Pages beyond the pool's are dropped and not counted, whether or not pages are taken in the same call."""
    _, _, kv = fresh(P=16, pages=4)
    # three of four pages free by the state, one held by that; request 1 gives back two and request 0 takes one
    got = run_plan(kv, [0, 32], [1, -32], [[-1, -1], [0, 1]], [3, 2, 1, 0], [1, 3], 1)
    assert got["table"] == [[2, -1], [0, 1]] and got["slots"] == [32]
    assert got["ring"] == [0, 2, 1, 0]                           # behind the free ones, ring[1..3]: the first of the two
    assert got["state_out"] == [2, 3]
    ok(kv, sfar_where("ring"))
    # exactly what is held: no fault
    got = run_plan(kv, [0, 16], [1, -16], [[-1, -1], [0, -1]], [3, 2, 1, 0], [1, 3], 1)
    assert got["ring"] == [0, 2, 1, 0] and got["state_out"] == [2, 3] and got["slots"] == [32]
    ok(kv)
    # none of four held, two given back, four taken
    got = run_plan(kv, [0, 32], [64, -32], [[-1] * 4, [0, 1, -1, -1]], [3, 2, 1, 0], [1, 4], 64)
    assert got["ring"] == [3, 2, 1, 0] and got["state_out"] == [1, 0] and got["table"][0] == [2, 1, 0, 3]
    ok(kv, sfar_where("ring"))


def test_bad_pages_given_back_leave_the_ring():
    """A page number outside the pool that a request gives back is recorded, and no page is free at its place."""
    for bad in (-1, 4, 1 << 30, -1 << 31):
        _, _, kv = fresh(P=16, pages=4)
        got = run_plan(kv, [40, 1], [-40, 0], [[0, bad, 1], [2, -1, -1]], [3, -1, -1, -1], [0, 1], 0)
        assert got["ring"] == [3, 0, -1, 1] and got["state_out"] == [0, 4]
        ok(kv, sfar_where("page"))
        # the place is found again when it is taken: recorded, no slot
        got = run_plan(kv, [0, 1], [48, 0], [[-1] * 3, [2, -1, -1]], got["ring"], [1, 3], 48)
        assert got["table"][0] == [0, -1, 1] and got["slots"] == list(range(16)) + [-1] * 16 + list(range(16, 32))
        ok(kv, sfar_where("page"))


@pytest.mark.parametrize("B,P,W,most_add,spare", [(257, 32, 5, 3, 60), (1024, 16, 4, 30, 400), (2049, 64, 3, 100, 900), (4097, 16, 5, 2, 100),
                                                  (8192, 16, 4, 40, 9000), (8192, 128, 2, 1, 3)])
def test_thousands_of_requests(B, P, W, most_add, spare):
    lens, delta, table, ring, state = draw_plan(B + P, B, P, W, most_add, spare)
    tokens = sum(max(d, 0) for d in delta) + 1
    _, _, kv = fresh(R=1, H=1, P=P, pages=len(ring), q_heads=1)
    got = run_plan(kv, lens, delta, table, ring, state, tokens, in_place=B % 2 == 0)
    want = kv_ref.plan(P, lens, delta, table, ring, state, tokens)
    for name in want:
        assert got[name] == want[name], name
    ok(kv)
