"""Plain 64-bit forms of the rotary positions and the latent-attention operators, for the tests, with what their
tolerances are counted from.  Written from the definitions in include/sfar_rope.h and include/sfar_latent.h."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}     # half a step, relative


def rope(x, pos, freq, layout, scale):
    """x [tokens, heads, rot] -> (turned, bound of its error before the rounding), both binary64."""
    x, rot = x.double(), x.shape[-1]
    theta = pos.double()[:, None] * freq.double()[None, :]
    pairs = [(i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1) for i in range(rot // 2)]
    out, off = torch.empty_like(x), torch.empty_like(x)
    for i, (m, n) in enumerate(pairs):
        a, b, c, s = x[..., m], x[..., n], theta[:, i, None].cos(), theta[:, i, None].sin()
        out[..., m], out[..., n] = scale * (a * c - b * s), scale * (b * c + a * s)
        # the angle, then cosine or sine (2 units), scale and two products and a sum in binary32
        off[..., m] = off[..., n] = scale * (a.abs() + b.abs()) * (2.0 ** -20 + 2.0 ** -46 * theta[:, i, None].abs() + 8 * 2.0 ** -24)
    return out, off


def append(x, weight, pos, freq, layout, scale, eps, L):
    """x [tokens, L + rot] -> (rows, bound of their error before the rounding)."""
    x = x.double()
    c = x[:, :L] * weight.double() / (x[:, :L].square().mean(-1, keepdim=True) + eps).sqrt()
    k, off = rope(x[:, None, L:], pos, freq, layout, scale)
    # 16 squares a lane and 5 sums of lanes (half of it after the root), root, reciprocal and two products
    return torch.cat([c, k[:, 0]], -1), torch.cat([c.abs() * 2.0 ** -24 * (21 / 2 + 8), off[:, 0]], -1)


def rows(q, k, v, seen, scale):
    """One head: q [n, W], k [m, W], v [m, V], seen [n, m] -> (out, bound of its error), binary64.

    Score: W products and sums in binary32, each sum off by at most 2^-23 of the terms' magnitudes (the tensor core
    need not round to nearest), and exp2's argument and result; weight: a rounding to bf16 (2^-8); sums of m weights and
    products; the reciprocal and the last product."""
    q, k, v = q.double(), k.double(), v.double()
    m, W = k.shape
    s = (q @ k.T * scale).masked_fill(~seen, -math.inf)
    p = torch.nan_to_num(torch.softmax(s, -1))
    out, mag = p @ v, p @ v.abs()
    size = ((q.abs() @ k.abs().T) * scale * seen).amax(-1, keepdim=True)
    score = size * W * 2.0 ** -23 + 4 * 2.0 ** -23 * (size + 8)
    rel = 2 * score + 2.0 ** -8 + m * 2.0 ** -23 + 2.0 ** -20
    return out, out.abs() * 2.0 ** -8 + mag * rel * 1.01


def causal(count, n, device):
    """[count, n]: the new tokens are the last of n."""
    return torch.arange(n, device=device)[None, :] <= (n - count + torch.arange(count, device=device))[:, None]


def offsets(counts):
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + c)
    return starts


def held_rows(cache, table, n, P):
    """The n cached rows of a request whose pages are `table`."""
    pages = torch.tensor(table[:-(-n // P)], dtype=torch.long, device=cache.device)
    return cache[pages].flatten(0, 1)[:n]


def check(got, want, off, ctx=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{ctx}: not finite at {torch.nonzero(~torch.isfinite(got))[0].tolist()}"
    over = (got - want).abs() - off
    assert (over <= 0).all(), f"{ctx}: {float(over.max()):.3g} over the bound at {torch.unravel_index(over.argmax(), over.shape)}"
