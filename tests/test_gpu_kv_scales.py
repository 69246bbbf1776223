"""Attention over pages whose scales are zero, negative, subnormal or far apart, by both of its kernels."""
import pytest
import torch

from kv_rows import cache, check, offsets, reference
from test_gpu_kv import _built, run_attention  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

FEW, MANY = 1, 512                   # what max_q picks
LENS, COUNTS = [1500, 700, 5, 130, 6000], [1, 3, 2, 1, 2]


def queries(R, T, Hq, D, seed):
    return (torch.randn(R, T, Hq, D, generator=torch.Generator().manual_seed(seed)) * 1.5).to(torch.bfloat16)


VALUE_SCALES = {
    "zero between": lambda b, i: 0.0 if i % 3 == 1 else 0.01,
    "zero first": lambda b, i: 0.0 if i < 20 else 0.01,
    "zero last": lambda b, i: 0.0 if i > 10 else -0.02,
    "all zero": lambda b, i: 0.0,
    "negative": lambda b, i: (-0.01, 0.013, -0.007)[(i + b) % 3],
    "far apart": lambda b, i: (1 - 2 * (i % 2)) * 2.0 ** (-60 + 7 * (i * 5 % 13)),
    "a zero among small": lambda b, i: 0.0 if i == 2 else 2.0 ** -30,
    "zeros among small": lambda b, i: 0.0 if i % 4 == 0 else -2.0 ** -40,
    "zeros among large": lambda b, i: 0.0 if i % 4 == 0 else 2.0 ** 40,
    "zeros as the append writes them": lambda b, i: 2.0 ** -100 if i % 3 == 0 else 2.0 ** 7,
    "the largest": lambda b, i: -2.0 ** 100 if i % 3 == 0 else 3.0,
    "the smallest": lambda b, i: 2.0 ** -99 if i % 3 == 0 else -0.9,
    "all smallest": lambda b, i: 1.1 * 2.0 ** -100,
}


def scales(form, name, D, P):
    H, G = 2, 4
    cpu, table = cache(1, H, D, P, LENS, lambda b, i: 0.01, VALUE_SCALES[name], 5 + D)
    starts = offsets(COUNTS)
    q = queries(1, starts[-1], H * G, D, P)
    got = run_attention(cpu, table, LENS, starts, q, H * G, D ** -0.5, max_q=form)
    check(got, cpu, table, LENS, starts, q, D ** -0.5, ctx=name)
    if name == "all zero":
        assert (got == 0).all()


@pytest.mark.parametrize("name", VALUE_SCALES)
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_value_scales_few_rows(name, D, P):
    scales(FEW, name, D, P)


@pytest.mark.parametrize("name", VALUE_SCALES)
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_value_scales_many_rows(name, D, P):
    scales(MANY, name, D, P)


def loud_zeros(form, nats, D, P):
    """Pages of value scale 0 whose scores lie `nats` above the others': the row's weight is theirs, its value the others'."""
    G, lens, counts = 4, [300, 2000, 6000], [1, 2, 1]
    big = nats / (1024.0 * D ** -0.5)
    cpu, table = cache(1, 1, D, P, lens, lambda b, i: big if i % 5 == 0 else 0.01, lambda b, i: 0.0 if i % 5 == 0 else 0.01, 9)
    k = cpu[0].view(torch.uint8)
    for row, n in zip(table, lens):
        for i, page in enumerate(row[:-(-n // P)]):
            k[0, page, 0, :, 0] = 0
            if i % 5 == 0:
                k[0, page] = 0
                k[0, page, 0, :, 0] = 0x78                       # 256: with the query's 4 exactly `nats`
    starts = offsets(counts)
    q = queries(1, starts[-1], G, D, 3)
    q[..., 0] = 4.0
    got = run_attention(cpu, table, lens, starts, q, G, D ** -0.5, max_q=form)
    check(got, cpu, table, lens, starts, q, D ** -0.5, ctx=f"{nats} nats")


@pytest.mark.parametrize("nats", [20, 60, 95, 150, 300])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 32)])
def test_loud_tokens_of_zero_scale_few_rows(nats, D, P):
    loud_zeros(FEW, nats, D, P)


@pytest.mark.parametrize("nats", [20, 60, 95, 150, 300])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 32)])
def test_loud_tokens_of_zero_scale_many_rows(nats, D, P):
    loud_zeros(MANY, nats, D, P)


@pytest.mark.parametrize("form", [FEW, MANY])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_key_scales(form, D, P):
    """Zero and negative key scales, with negative value scales beside them."""
    starts = offsets(COUNTS)
    q = queries(1, starts[-1], 8, D, 77)
    for ks in (lambda b, i: (0.01, -0.012, 0.0)[i % 3], lambda b, i: -0.01, lambda b, i: 0.0):
        cpu, table = cache(1, 2, D, P, LENS, ks, lambda b, i: (0.01, -0.02)[i // 2 % 2], 21)
        got = run_attention(cpu, table, LENS, starts, q, 8, D ** -0.5, max_q=form)
        check(got, cpu, table, LENS, starts, q, D ** -0.5)
        windowed = run_attention(cpu, table, LENS, starts, q, 8, D ** -0.5, window=333, max_q=form)
        check(windowed, cpu, table, LENS, starts, q, D ** -0.5, window=333)


@pytest.mark.parametrize("form", [FEW, MANY])
def test_the_least_value_scales_count_as_zero(form):
    """Up to 2^-100: they stand for values up to 448 * 2^-100."""
    starts = offsets(COUNTS)
    q = queries(1, starts[-1], 8, 64, 78)
    for vs in (lambda b, i: 1e-40, lambda b, i: -1.4e-45, lambda b, i: (0.01, 1e-39, -1e-41)[i % 3], lambda b, i: (0.01, 2.0 ** -100)[i % 2]):
        cpu, table = cache(1, 2, 64, 16, LENS, lambda b, i: 0.01, vs, 22)
        got = run_attention(cpu, table, LENS, starts, q, 8, 0.125, max_q=form)
        check(got, cpu, table, LENS, starts, q, 0.125, floor=448 * 2.0 ** -100)


@pytest.mark.parametrize("form", [FEW, MANY])
def test_nan_under_a_zero_scale_stays_nan(form):
    """A NaN value times a scale of zero is a NaN, for the rows and the element that see it."""
    cpu, table = cache(1, 1, 64, 16, [400], lambda b, i: 0.01, lambda b, i: 0.0 if i % 2 else 0.01, 23)
    for at in (20, 397):                                         # in a tile that every row sees whole, and among the new tokens
        one = [t.clone() for t in cpu]
        one[1].view(torch.uint8)[0, table[0][at // 16], 0, at % 16, 7] = 0xff
        one[3][0, table[0][at // 16]] = 0.0
        clean = [t.clone() for t in one]
        clean[1].view(torch.uint8)[0, table[0][at // 16], 0, at % 16, 7] = 0
        q = queries(1, 6, 4, 64, 79)
        got = run_attention(one, table, [400], [0, 6], q, 4, 0.125, max_q=form)
        sees = max(0, at - 394)
        assert torch.isnan(got[:, sees:, :, 7]).all() and torch.isfinite(got[:, :sees]).all()
        check(torch.where(torch.isnan(got), reference(clean, 0, table, [400], [0, 6], q, 0.125)[0], got), clean, table, [400], [0, 6], q, 0.125)
