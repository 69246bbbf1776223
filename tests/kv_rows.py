"""Rows of attention over the paged 8-bit cache in binary64, with what their tolerance is counted from, and caches of
given page scales."""
import torch

from kv_ref import F8


def reference(cpu, r, table, lens, starts, q, scale, window=0, lost=None):
    """Rank r.  Returns (out, weighted mean of |v|) [T, Hq, D] and the largest weight times |value scale| [T, Hq, 1].
    lost: (first, last) tokens of every context that are left out (a mistake, for tests of the tolerance)."""
    k_cache, v_cache, k_scale, v_scale = [t[r] for t in cpu]
    T, Hq, D = q[r].shape
    H, P = k_cache.shape[1:3]
    G = Hq // H
    out, mag, top = [torch.zeros(T, Hq, d, dtype=torch.float64) for d in (D, D, 1)]
    for b, n in enumerate(lens):
        a, z = starts[b], starts[b + 1]
        if n <= 0 or a == z:
            continue
        pages = torch.tensor(table[b][:-(-n // P)], dtype=torch.long)
        for h in range(H):
            ks, vs = [s[pages, h].double().repeat_interleave(P)[:n] for s in (k_scale, v_scale)]
            k, v = [c.view(torch.uint8)[pages, h].view(F8).double().reshape(-1, D)[:n] for c in (k_cache, v_cache)]
            x = q[r, a:z, h * G:(h + 1) * G].double().reshape(-1, D)
            s = (x @ k.T) * ks * scale
            pos = (n - (z - torch.arange(a, z))).repeat_interleave(G)[:, None]
            j = torch.arange(n)
            seen = j <= pos
            if window:
                seen &= j > pos - window
            if lost:
                seen &= (j < lost[0]) | (j >= lost[1])
            p = torch.nan_to_num(torch.softmax(s.masked_fill(~seen, float("-inf")), -1))
            for to, w in ((out, p @ (v * vs[:, None])), (mag, p @ (v * vs[:, None]).abs()), (top, (p * vs.abs()).amax(-1, keepdim=True))):
                to[a:z, h * G:(h + 1) * G] = w.reshape(z - a, G, -1)
    return out, mag, top


def bound(out, mag, top, n, vmax):
    """2^-8 |o| (one rounding to bf16) + 2^-10 of the weighted mean of |v| (the weights' rounding to 11 bits, and as much
    again for the exponentials and the binary32 sums) + n times 2^-33 of the row's largest weighted value (weights below
    2^-22 of it lie below binary16's normal range) + 2^-100 of the largest value (weights that small count as none)."""
    return 2.0 ** -8 * out.abs() + 2.0 ** -10 * mag + n * 2.0 ** -33 * 448.0 * top + 2.0 ** -100 * 448.0 * vmax


def check(got, cpu, table, lens, starts, q, scale, window=0, floor=0.0, ctx=""):
    for r in range(q.shape[0]):
        out, mag, top = reference(cpu, r, table, lens, starts, q, scale, window)
        limit = bound(out, mag, top, max(lens), float(cpu[3][r].nan_to_num(0.0).abs().max())) + floor
        off = (got[r] - out).abs()
        assert torch.isfinite(got[r]).all(), f"{ctx} rank {r}: not finite"
        assert (off <= limit).all(), f"{ctx} rank {r}: {float((off - limit).max()):.3g} over the bound at {int((off - limit).argmax())}"


def cache(R, H, D, P, lens, k_scale, v_scale, seed, sigma=60.0):
    """(caches and scales on the CPU, table): page i of request b has k_scale(b, i) and v_scale(b, i); what no request
    holds is NaN."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-n // P) for n in lens]
    pages = sum(held) + 3
    perm = torch.randperm(pages, generator=g).tolist()
    k, v = [(torch.randn(R, pages, H, P, D, generator=g) * sigma).clamp(-448, 448).to(F8) for _ in range(2)]
    ks, vs = [torch.full((R, pages, H), float("nan")) for _ in range(2)]
    table, at = [], 0
    live = torch.zeros(pages, P, dtype=torch.bool)
    for b, (n, h) in enumerate(zip(lens, held)):
        row = perm[at:at + h]
        at += h
        table.append(row + [-1] * (max(held) + 1 - h))
        for i, p in enumerate(row):
            live[p, :min(P, n - i * P)] = True
            ks[:, p], vs[:, p] = k_scale(b, i), v_scale(b, i)
    for c in (k, v):
        c.view(torch.uint8)[:, ~live[:, None, :].expand(-1, H, -1)] = 0x7f
    return (k, v, ks, vs), table


def offsets(counts):
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + c)
    return starts
