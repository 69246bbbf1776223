"""Plain 64-bit implementations of the paged 8-bit operators, for the tests.

Written from the definitions in include/sfar_kv.h and include/sfar_fp8.h; they
share no code with the library.  Everything runs on the CPU in binary64 (the
plan in Python integers).
"""
import math

import torch

F8 = torch.float8_e4m3fn


def e4m3_round(x):
    """binary64 -> nearest e4m3 value (ties to even); |x| <= 448; NaN stays."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def scale_exponent(amax: float) -> int:
    """The least e >= -100 with amax <= 448 * 2^e."""
    e = -100
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def plan(P, lens, delta, table, ring, state, tokens):
    """Lists in, dict of lists out; table and ring are copied."""
    table, ring = [list(r) for r in table], list(ring)
    pool, W = len(ring), len(table[0])
    head, free = state
    need_sum, used, back = 0, 0, 0
    lens_out, taken, starts, slots = [], [], [0], []
    for b, (n, d) in enumerate(zip(lens, delta)):
        after = max(0, n + d)
        have, want = -(-n // P), -(-after // P)
        ok = True
        if d > 0:
            if want > W:
                ok = False
            else:
                need = want - have
                if need:
                    need_sum += need
                    ok = need_sum <= free
                if ok and need:
                    for j in range(need):
                        table[b][have + j] = ring[(head + need_sum - need + j) % pool]
                    used = need_sum
        elif d < 0:
            for j in range(want, have):
                ring[(head + free + back) % pool] = table[b][j]
                back += 1
        lens_out.append(after if ok else n)
        taken.append(int(ok))
        starts.append(starts[-1] + max(d, 0))
        for i in range(max(d, 0)):
            slots.append(table[b][(n + i) // P] * P + (n + i) % P if ok else -1)
    slots += [-1] * (tokens - len(slots))
    return {"lens_out": lens_out, "taken": taken, "starts": starts, "slots": slots, "table": table, "ring": ring,
            "state_out": [(head + used) % pool, free - used + back]}


def append(cache, scale, x, slots):
    """One rank's keys or values.  cache [pages, H, P, D] e4m3, scale [pages, H] fp32, x [T, H, D] bf16, slots a
    list; returns the new (cache as binary64 e4m3 values, scale as binary64)."""
    P = cache.shape[2]
    values, scales, x = cache.double(), scale.double(), x.double()
    runs = {}
    for t, s in enumerate(slots):
        if s >= 0:
            runs.setdefault(s // P, []).append((s % P, t))
    for page, tokens in runs.items():
        first = min(o for o, _ in tokens)
        for h in range(x.shape[1]):
            new = torch.stack([x[t, h] for _, t in tokens])
            finite = new[torch.isfinite(new)].abs()
            s = 2.0 ** scale_exponent(float(finite.max()) if finite.numel() else 0.0)
            old = float(scales[page, h])
            if first:
                s = max(s, old)
                if s > old:
                    values[page, h, :first] = e4m3_round(values[page, h, :first] * (old / s))
            scales[page, h] = s
            new = torch.where(torch.isfinite(new), new, torch.full_like(new, math.nan))
            for (o, _), row in zip(tokens, new):
                values[page, h, o] = e4m3_round(row / s)
    return values, scales


def attention(q, k_cache, v_cache, k_scale, v_scale, table, lens, starts, scale, window=0):
    """One rank.  q [T, Hq, D]; returns (out, weighted mean of |v|) [T, Hq, D] in binary64."""
    T, Hq, D = q.shape
    H, P = k_cache.shape[1:3]
    G = Hq // H
    out, mag = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    for b, n in enumerate(lens):
        a, z = starts[b], starts[b + 1]
        if n <= 0 or a == z:
            continue
        pages = torch.tensor(table[b][:-(-n // P)], dtype=torch.long)
        k = (k_cache.view(torch.uint8)[pages].view(F8).double() * k_scale[pages].double()[..., None, None]).transpose(0, 1).reshape(H, -1, D)[:, :n]
        v = (v_cache.view(torch.uint8)[pages].view(F8).double() * v_scale[pages].double()[..., None, None]).transpose(0, 1).reshape(H, -1, D)[:, :n]
        for t in range(a, z):
            pos = n - (z - t)
            lo = max(0, pos - window + 1) if window else 0
            if pos < lo:
                continue
            for h in range(H):
                s = (q[t, h * G:(h + 1) * G].double() @ k[h, lo:pos + 1].T) * scale
                p = torch.softmax(s, -1)
                out[t, h * G:(h + 1) * G] = p @ v[h, lo:pos + 1]
                mag[t, h * G:(h + 1) * G] = p @ v[h, lo:pos + 1].abs()
    return out, mag


def quantize(x):
    """x [m, k] bf16 -> (e4m3 values as binary64 [m, k], scales [kb, m])."""
    m, k = x.shape
    kb = -(-k // 128)
    x = x.double()
    q, s = torch.zeros_like(x), torch.zeros(kb, m, dtype=torch.float64)
    for i in range(m):
        for b in range(kb):
            part = x[i, 128 * b:128 * b + 128]
            finite = part[torch.isfinite(part)].abs()
            s[b, i] = 2.0 ** scale_exponent(float(finite.max()) if finite.numel() else 0.0)
            part = torch.where(torch.isfinite(part), part, torch.full_like(part, math.nan))
            q[i, 128 * b:128 * b + 128] = e4m3_round(part / s[b, i])
    return q, s


def gemm(x8, sx, w8, sw):
    """Binary64 product and the sum of its terms' magnitudes: [m, n] each."""
    k, n = x8.shape[1], w8.shape[0]
    x = x8.double() * sx.double().T.repeat_interleave(128, 1)[:, :k]
    w = w8.double() * sw.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return x @ w.T, x.abs() @ w.abs().T
