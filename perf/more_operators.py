"""What the latent-attention operators of libsfar cost: cases, inputs, plain forms.

Five operators of a tensor-parallel layer whose keys and values come from one
latent vector a token (shared by all heads) and one rotated key (shared too),
held in a paged bf16 cache by each of R simulated ranks:

  rope       rotary positions of queries and keys, half or interleaved pairs,
             with any table of frequencies (Sfar.rope);
  append     a step's latents, normalised, and keys, rotated, into their
             places of the cache (SfarLatent.append);
  gather     cached rows of every request read back in order, for the keys and
             values that are expanded from them (SfarLatent.gather);
  attention  absorbed form: queries already multiplied into the latent's space
             over the cached rows, causal (SfarLatent.attention);
  prompt     expanded form: queries over keys and values of every head, the
             rotated part of the keys shared by the heads (SfarLatent.prompt).

``run`` computes them in plain binary32 torch operations (angles in 64 bits),
or, where ``own`` is true, by the library.  ``exact`` computes them in
binary64.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# --------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's queries and keys: 64 requests, 8 heads and one key head of 128, whole heads rotated
        {"name": "rope decode 64", "op": "rope", "R": 8, "T": 64, "H": 8, "K": 1, "rot": 128, "D": 128, "layout": "half",
         "type": "bf16", "far": 9000, "factor": 1.0},
        # prompts: the rotated 64 of each 192-element head, interleaved, positions far beyond the trained ones
        {"name": "rope prompt 5k", "op": "rope", "R": 8, "T": 5003, "H": 20, "K": 1, "rot": 64, "D": 192, "layout": "interleaved",
         "type": "bf16", "far": 163000, "factor": 40.0},
        # binary32 activations, 96 of 160 elements, two key heads
        {"name": "rope fp32", "op": "rope", "R": 4, "T": 1777, "H": 6, "K": 2, "rot": 96, "D": 160, "layout": "half",
         "type": "fp32", "far": 131072, "factor": 1.0},
        # decode step: one token of each of 48 requests
        {"name": "append decode 48", "op": "append", "R": 8, "L": 512, "rot": 64, "P": 64, "B": 48, "lo": 1, "hi": 4000, "add_lo": 1,
         "add_hi": 1, "layout": "interleaved"},
        # prompts of several requests at once
        {"name": "append prompt 16k", "op": "append", "R": 4, "L": 512, "rot": 64, "P": 32, "B": 9, "lo": 0, "hi": 3000, "add_lo": 1501,
         "add_hi": 2139, "layout": "half"},
        # a short context read back
        {"name": "gather 3 short", "op": "gather", "R": 2, "L": 256, "rot": 32, "P": 16, "B": 3, "lo": 41, "hi": 290},
        # the contexts of a batch of prompt chunks read back
        {"name": "gather 30k", "op": "gather", "R": 8, "L": 512, "rot": 64, "P": 64, "B": 5, "lo": 3001, "hi": 8999},
        # the smallest call: one request, short context (latency)
        {"name": "latent decode 1 short", "op": "attention", "R": 2, "H": 12, "L": 256, "rot": 32, "P": 16, "B": 1, "lo": 99, "hi": 99,
         "q_lo": 1, "q_hi": 1},
        # a decode batch, ragged contexts, 20 heads a rank
        {"name": "latent decode 32", "op": "attention", "R": 8, "H": 20, "L": 512, "rot": 64, "P": 64, "B": 32, "lo": 301, "hi": 6100,
         "q_lo": 1, "q_hi": 1},
        # one request with a very long context, a guessed token beside the sampled one
        {"name": "latent decode 131k", "op": "attention", "R": 4, "H": 10, "L": 512, "rot": 64, "P": 32, "B": 1, "lo": 131071,
         "hi": 131071, "q_lo": 2, "q_hi": 2},
        # a short prompt (latency)
        {"name": "prompt 1 short", "op": "prompt", "R": 2, "H": 5, "nope": 64, "rot": 32, "V": 64, "B": 1, "lo": 77, "hi": 77, "q_lo": 77,
         "q_hi": 77},
        # chunks of prompts over what came before them
        {"name": "prompt chunks", "op": "prompt", "R": 8, "H": 12, "nope": 128, "rot": 64, "V": 128, "B": 3, "lo": 1100, "hi": 4099,
         "q_lo": 700, "q_hi": 1024},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "gather", "attention", "attention", "prompt"])
    R, P = rng.choice([1, 2, 3, 4, 8]), rng.choice([16, 32, 64, 128])
    L, rot = rng.choice([(512, 64), (512, 64), (256, 32), (256, 64)])
    layout = rng.choice(["half", "interleaved"])
    if op == "rope":
        R, H, K, rot = max(R, 2), rng.randint(1, 24), rng.randint(0, 3), 16 * rng.randint(1, 8)
        most = max(1, (8 * 5003 * 21 * 64) // (R * (H + K) * rot))
        return {"op": op, "R": R, "T": _log(rng, 1, min(most, 16384)), "H": H, "K": K, "rot": rot, "D": rot + 16 * rng.choice([0, 0, 1, 4, 8]),
                "layout": layout, "type": rng.choice(["bf16", "bf16", "fp32"]), "far": _log(rng, 100, 1 << 20),
                "factor": rng.choice([1.0, 1.0, 4.0, 32.0])}
    if op in ("append", "gather"):
        B = _log(rng, 1, 128)
        most = max(1, (8 * 30000 * 576 if op == "gather" else 4 * 16384 * 576) // (R * (L + rot) * B))
        n = _log(rng, 1, min(most, 30000))
        if op == "gather":
            return {"op": op, "R": R, "L": L, "rot": rot, "P": P, "B": B, "lo": max(1, n // rng.choice([1, 2, 7])), "hi": n}
        return {"op": op, "R": R, "L": L, "rot": rot, "P": P, "B": B, "lo": 0, "hi": rng.randint(1, 3000), "add_lo": (n + 1) // 2, "add_hi": n,
                "layout": layout}
    if op == "attention":
        H, B, q = rng.randint(1, 40), _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 4, 9])
        most = min(131072, (800 << 20) // (R * 2 * (L + rot) * B), (1 << 28) // (R * H * B * q))
        hi = _log(rng, min(q + 1, max(q, most)), max(q + 1, most))
        return {"op": op, "R": R, "H": H, "L": L, "rot": rot, "P": P, "B": B, "lo": max(1, hi // rng.choice([1, 2, 7])), "hi": hi,
                "q_lo": rng.choice([1, q]), "q_hi": q}
    H, B, q = rng.randint(1, 20), rng.randint(1, 6), _log(rng, 1, 1500)
    most = max(q, min(16384, (1 << 29) // (R * H * B * q), (600 << 20) // (R * H * L * B)))
    q = min(q, most)
    hi = rng.choice([q, rng.randint(q, most)])
    return {"op": op, "R": R, "H": H, "nope": 2 * L // 8, "rot": rot, "V": 2 * L // 8, "B": B, "lo": max(1, hi // rng.choice([1, 2, 7])),
            "hi": hi, "q_lo": rng.choice([1, q]), "q_hi": q}


# ------------------------------------------------------- lengths and generators
def _spread(n, lo, hi, phase=0.37):
    """n whole numbers spread evenly over [lo, hi] in a mixed order; the same for every seed."""
    return [lo + int((hi - lo + 1) * ((phase + (b + 1) * 0.6180339887498949) % 1.0)) for b in range(n)]


def _lengths(c):
    """(context with the new tokens, new tokens) of every request."""
    q = _spread(c["B"], c["q_lo"], c["q_hi"], 0.11)
    return [max(n, a) for n, a in zip(_spread(c["B"], c["lo"], c["hi"]), q)], q


def _added(c):
    """(tokens held before, tokens added) of every request."""
    return _spread(c["B"], c["lo"], c["hi"]), _spread(c["B"], c["add_lo"], c["add_hi"], 0.11)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _shuffled(seed, *lists):
    """The lists, reordered together by the seed."""
    order = torch.randperm(len(lists[0]), generator=torch.Generator().manual_seed(seed)).tolist()
    return [[v[i] for i in order] for v in lists]


def _normal(g, shape, sigma=1.0, dtype=torch.bfloat16):
    """Values of a normal distribution, made a part at a time."""
    t = torch.empty(shape, dtype=dtype, device=DEV)
    flat = t.view(-1)
    for part in flat.split(1 << 27):
        part.copy_(torch.randn(part.numel(), generator=g, device=DEV).mul_(sigma))
    return t


def _tables(g, pages, W, pool):
    """A random block table [B, W], -1 past a request's pages."""
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    n = _int(pages)
    j = torch.arange(W, device=DEV)
    at = (torch.cumsum(n, 0) - n)[:, None] + j[None, :]
    return torch.where(j[None, :] < n[:, None], order[at.clamp(max=pool - 1)], -1).to(torch.int32).contiguous()


def _starts(counts):
    return _int([0] + torch.tensor(counts).cumsum(0).tolist())


def _frequencies(rot, factor):
    """theta_i = 10000^(-2 i / rot), stretched by `factor` where a turn is longer than the trained context of 4096."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    return torch.where(f * 4096 < 2 * math.pi, f / factor, f).float()


def _up(n, p):
    return -(-n // p)


# ------------------------------------------------------------------- prepare
def prepare(case, seed):
    return {"rope": _prepare_rope, "append": _prepare_append, "gather": _prepare_gather, "attention": _prepare_attention,
            "prompt": _prepare_prompt}[case["op"]](case, seed)


def _prepare_rope(c, seed):
    g = _gen(seed)
    R, T, rot, D = c["R"], c["T"], c["rot"], c["D"]
    dtype = torch.bfloat16 if c["type"] == "bf16" else torch.float32
    q, k = _normal(g, (R, T, c["H"], D), dtype=dtype), _normal(g, (R, T, c["K"], D), dtype=dtype)
    s = {"op": "rope", "layout": c["layout"], "scale": 1.0 + 0.1 * math.log(c["factor"]), "freq": _frequencies(rot, c["factor"]),
         "pos": torch.randint(0, c["far"], (T,), generator=g, device=DEV).to(torch.int32),
         "q": q[..., D - rot:], "k": k[..., D - rot:], "q_out": torch.empty((R, T, c["H"], rot), dtype=dtype, device=DEV),
         "k_out": torch.empty((R, T, c["K"], rot), dtype=dtype, device=DEV)}
    if own:
        from barrier_free_message_gb300 import sfar
        s["h"] = sfar.Sfar(R, 1 << 16, c["type"])
    return s


def _cache(c, g, pages):
    """A block table, and the cache of every rank: normalised latents and rotated keys."""
    pool = sum(pages) + 5
    return _tables(g, pages, max(1, max(pages)), pool), _normal(g, (c["R"], pool, c["P"], c["L"] + c["rot"]))


def _handle(s, c):
    s["L"] = c["L"]
    if own:
        from barrier_free_message_gb300 import sfar
        s["kv"] = sfar.SfarLatent(s["cache"], q_heads=c.get("H", 1), rope_dim=c["rot"])
    return s


def _prepare_append(c, seed):
    g = _gen(seed)
    before, add = _shuffled(seed, *_added(c))
    P, T = c["P"], sum(add)
    table, cache = _cache(c, g, [_up(n + a, P) for n, a in zip(before, add)])
    start = _starts(add)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    pos = (_int(before)[b] + t - start[b]).to(torch.int32)
    slots = table[b, pos.long() // P] * P + pos % P
    # a token's latent and key as a projection gives them, one row wider than both
    x = _normal(g, (c["R"], T, c["L"] + c["rot"] + 64), 0.6)[..., :c["L"] + c["rot"]]
    return _handle({"op": "append", "cache": cache, "x": x, "weight": (1.0 + 0.2 * torch.randn(c["L"], generator=g, device=DEV)).to(torch.bfloat16),
                    "pos": pos, "slots": slots.to(torch.int32), "freq": _frequencies(c["rot"], 1.0), "layout": c["layout"], "scale": 1.0}, c)


def _prepare_gather(c, seed):
    g = _gen(seed)
    lens, = _shuffled(seed, _spread(c["B"], c["lo"], c["hi"]))
    table, cache = _cache(c, g, [_up(n, c["P"]) for n in lens])
    return _handle({"op": "gather", "cache": cache, "table": table, "lens": _int(lens), "starts": _starts(lens),
                    "out": torch.empty((c["R"], sum(lens), c["L"] + c["rot"]), dtype=torch.bfloat16, device=DEV)}, c)


def _prepare_attention(c, seed):
    g = _gen(seed)
    lens, q = _shuffled(seed, *_lengths(c))
    table, cache = _cache(c, g, [_up(n, c["P"]) for n in lens])
    return _handle({"op": "attention", "cache": cache, "table": table, "lens": _int(lens), "starts": _starts(q),
                    "q": _normal(g, (c["R"], sum(q), c["H"], c["L"] + c["rot"])),
                    "out": torch.empty((c["R"], sum(q), c["H"], c["L"]), dtype=torch.bfloat16, device=DEV), "max_q": max(q),
                    "scale": (c["L"] // 4 + c["rot"]) ** -0.5}, c)


def _prepare_prompt(c, seed):
    g = _gen(seed)
    lens, q = _shuffled(seed, *_lengths(c))
    R, H, N, V, rot, S, T = c["R"], c["H"], c["nope"], c["V"], c["rot"], sum(lens), sum(q)
    # keys and values as one projection of the latents gives them; the rotated keys behind the latents they came with
    kv, rows = _normal(g, (R, S, H, N + V)), _normal(g, (R, S, 4 * N + rot))
    s = {"op": "prompt", "q": _normal(g, (R, T, H, N + rot), 1.2), "k": kv[..., :N], "v": kv[..., N:], "kr": rows[..., 4 * N:],
         "out": torch.empty((R, T, H, V), dtype=torch.bfloat16, device=DEV), "starts": _starts(q), "k_starts": _starts(lens),
         "max_q": max(q), "max_k": max(lens), "scale": (N + rot) ** -0.5}
    if own:
        from barrier_free_message_gb300 import sfar
        s["kv"] = sfar.SfarLatent(torch.zeros((R, 1, 16, 4 * N + rot), dtype=torch.bfloat16, device=DEV), q_heads=H, rope_dim=rot)
    return s


# ----------------------------------------------------------------------- run
def run(state):
    return {"rope": _run_rope, "append": _run_append, "gather": _run_gather, "attention": _run_attention, "prompt": _run_prompt}[state["op"]](state)


def _rotated(x, pos, freq, layout, scale):
    """x [..., tokens, heads, rot], pos [tokens], freq [rot / 2]; angles in 64 bits."""
    angle = pos.double()[:, None] * freq.double()
    cos, sin = [(f(angle) * scale).float()[:, None, :] for f in (torch.cos, torch.sin)]
    x = x.float()
    if layout == "half":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _run_rope(s):
    if own:
        s["h"].rope(s["q"], s["q_out"], s["pos"], s["freq"], k=s["k"], k_out=s["k_out"], layout=s["layout"], scale=s["scale"])
        return {"q": s["q_out"], "k": s["k_out"]}
    return {n: _rotated(s[n], s["pos"], s["freq"], s["layout"], s["scale"]).to(s[n].dtype) for n in ("q", "k")}


def _run_append(s):
    if own:
        s["kv"].append(s["x"], s["weight"], s["pos"], s["freq"], s["slots"], eps=EPS, layout=s["layout"], scale=s["scale"])
        return s["cache"]
    L, x, cache = s["L"], s["x"].float(), s["cache"]
    c = x[..., :L]
    c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    k = _rotated(x[..., None, L:], s["pos"], s["freq"], s["layout"], s["scale"])[..., 0, :]
    rows = torch.cat([c, k], -1).to(torch.bfloat16)
    live = s["slots"] >= 0
    cache.view(cache.shape[0], -1, cache.shape[-1])[:, s["slots"][live].long()] = rows[:, live]
    return cache


def _places(table, starts, P, T):
    """The slot of each of T rows: row starts[b] + i is token i of request b."""
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    i = t - starts[b]
    return table[b, i // P].long() * P + i % P


def _run_gather(s):
    if own:
        s["kv"].gather(s["out"], s["table"], s["lens"], s["starts"])
        return s["out"]
    cache = s["cache"]
    R, _, P, W = cache.shape
    return cache.view(R, -1, W)[:, _places(s["table"], s["starts"], P, s["out"].shape[1])]


def _softmax(a, seen):
    a = a.masked_fill(~seen, -math.inf)
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _padded(x, starts, n):
    """Rows of every request, [..., B, n, ...], from [R, T, ...]; the last one repeated past a request's end."""
    return x[:, (starts[:-1, None] + torch.arange(n, device=x.device)).clamp(max=x.shape[1] - 1).long()]


def _seen(lens, count, n, L):
    """[B, n, L]: which of the context each new token sees."""
    at = (lens - count)[:, None] + torch.arange(n, device=lens.device)
    j = torch.arange(L, device=lens.device)
    return (j <= at[..., None]) & (j < lens[:, None, None])


def _packed(o, starts, T):
    """[R, B, n, ...] back to [R, T, ...]."""
    t = torch.arange(T, device=o.device)
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    return o[:, b, t - starts[b]]


def _run_attention(s):
    if own:
        s["kv"].attention(s["q"], s["out"], s["table"], s["lens"], s["starts"], max_q=s["max_q"], scale=s["scale"])
        return s["out"]
    q, cache, table, lens, starts, n, L = s["q"], s["cache"], s["table"].clamp(min=0).long(), s["lens"], s["starts"], s["max_q"], s["L"]
    R, T, H, _ = q.shape
    B = table.shape[0]
    rows = cache[:, table].float().flatten(2, 3)                                    # [R, B, context, latent and key]
    x = _padded(q, starts, n).float().reshape(R, B, n * H, -1)
    seen = _seen(lens, starts[1:] - starts[:-1], n, rows.shape[2]).repeat_interleave(H, 1)
    p = _softmax(torch.matmul(x, rows.transpose(-1, -2)) * s["scale"], seen)
    return _packed(torch.matmul(p, rows[..., :L]).view(R, B, n, H, L), starts, T).to(torch.bfloat16)


def _run_prompt(s):
    if own:
        s["kv"].prompt(s["q"], s["k"], s["v"], s["kr"], s["out"], s["starts"], s["k_starts"], max_q=s["max_q"], scale=s["scale"])
        return s["out"]
    starts, ks, n, m = s["starts"], s["k_starts"], s["max_q"], s["max_k"]
    T, H, N = s["q"].shape[1], s["q"].shape[2], s["k"].shape[3]
    q = _padded(s["q"], starts, n).float().transpose(2, 3)                         # [R, B, H, n, nope and rot]
    k, v = [_padded(s[i], ks, m).float().transpose(2, 3) for i in ("k", "v")]
    kr = _padded(s["kr"], ks, m).float()
    a = torch.matmul(q[..., :N], k.transpose(-1, -2)) + torch.matmul(q[..., N:], kr.transpose(-1, -2)[:, :, None])
    p = _softmax(a * s["scale"], _seen(ks[1:] - ks[:-1], starts[1:] - starts[:-1], n, m)[:, None])
    return _packed(torch.matmul(p, v).transpose(2, 3), starts, T).to(torch.bfloat16)


# ---------------------------------------------------------------------- work
def work(case):
    c = case
    R = c["R"]
    if c["op"] == "rope":
        each = 2 if c["type"] == "bf16" else 4
        n = R * c["T"] * (c["H"] + c["K"]) * c["rot"]
        return {"bytes": 2 * n * each + 4 * c["T"] + 2 * c["rot"], "flops": 3 * n}
    if c["op"] == "append":
        T, W = sum(_added(c)[1]), c["L"] + c["rot"]
        return {"bytes": 8 * T + 4 * R * T * W, "flops": R * T * (4 * c["L"] + 3 * c["rot"])}
    if c["op"] == "gather":
        lens = _spread(c["B"], c["lo"], c["hi"])
        return {"bytes": 4 * R * sum(lens) * (c["L"] + c["rot"]) + 4 * sum(_up(n, c["P"]) for n in lens), "flops": 0}
    lens, q = _lengths(c)
    pairs = sum(a * n - a * (a - 1) // 2 for n, a in zip(lens, q))
    if c["op"] == "attention":
        W = c["L"] + c["rot"]
        return {"bytes": 2 * R * (sum(lens) * W + sum(q) * c["H"] * (W + c["L"])) + 4 * sum(_up(n, c["P"]) for n in lens),
                "flops": 2 * R * c["H"] * pairs * (W + c["L"])}
    N, V, rot, H = c["nope"], c["V"], c["rot"], c["H"]
    return {"bytes": 2 * R * (sum(lens) * (H * (N + V) + rot) + sum(q) * H * (N + rot + V)), "flops": 2 * R * H * pairs * (N + rot + V)}


# --------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "gather": _exact_gather, "attention": _exact_attention,
            "prompt": _exact_prompt}[case["op"]](s)


def _turned(x, pos, freq, layout, scale):
    """The pairs of x [..., tokens, heads, rot] as complex numbers, turned by their angles."""
    x = x.double()
    half = x.shape[-1] // 2
    z = torch.complex(x[..., :half], x[..., half:]) if layout == "half" else torch.view_as_complex(x.unflatten(-1, (half, 2)).contiguous())
    z = z * torch.polar(torch.full((), scale, dtype=torch.float64, device=x.device).expand(len(pos), half), torch.outer(pos.double(), freq.double()))[:, None]
    return torch.cat([z.real, z.imag], -1) if layout == "half" else torch.view_as_real(z).flatten(-2)


def _exact_rope(s):
    return {n: _turned(s[n], s["pos"], s["freq"], s["layout"], s["scale"]) for n in ("q", "k")}


def _exact_append(s):
    L, x = s["L"], s["x"].double()
    cache = s["cache"].double()
    R, pages, P, W = cache.shape
    norm = torch.linalg.vector_norm(x[..., :L], dim=-1, keepdim=True)
    row = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    row[..., :L] = x[..., :L] / (norm * norm / L + EPS).sqrt() * s["weight"].double()
    row[..., L:] = _turned(x[:, :, None, L:], s["pos"], s["freq"], s["layout"], s["scale"])[:, :, 0]
    flat = cache.view(R, pages * P, W)
    for t in range(0, x.shape[1], 4096):
        to = s["slots"][t:t + 4096].long()
        flat.index_copy_(1, to, row[:, t:t + 4096])
    return cache


def _exact_gather(s):
    lens, P = s["lens"].tolist(), s["cache"].shape[2]
    return torch.cat([s["cache"][:, s["table"][b, :_up(n, P)].long()].flatten(1, 2)[:, :n] for b, n in enumerate(lens)], 1).double()


def _rows_of(q, k, v, n, scale, at, seen_from):
    """Softmax rows in 64 bits: q [.., tokens, W], k [.., n, W], v [.., n, V]; token i sees up to position seen_from + i."""
    a = (q @ k.transpose(-1, -2)) * scale
    j = torch.arange(n, device=q.device)
    i = torch.arange(q.shape[-2], device=q.device) + at
    a = torch.where(j[None] <= seen_from + i[:, None], a, -math.inf)
    return torch.nan_to_num(torch.softmax(a, -1)) @ v


def _exact_attention(s):
    q, cache, starts, L = s["q"], s["cache"], s["starts"].tolist(), s["L"]
    R, T, H, _ = q.shape
    P = cache.shape[2]
    out = torch.zeros((R, T, H, L), dtype=torch.float64, device=q.device)
    for b, n in enumerate(s["lens"].tolist()):
        pages = s["table"][b, :_up(n, P)].long()
        t0, t1 = starts[b], starts[b + 1]
        for r in range(R):
            rows = cache[r, pages].flatten(0, 1)[:n].double()
            out[r, t0:t1] = _rows_of(q[r, t0:t1].double().transpose(0, 1), rows, rows[:, :L], n, s["scale"], 0, n - (t1 - t0)).transpose(0, 1)
    return out


def _exact_prompt(s):
    q, starts, ks = s["q"], s["starts"].tolist(), s["k_starts"].tolist()
    R, T, H, _ = q.shape
    out = torch.zeros((R, T, H, s["v"].shape[3]), dtype=torch.float64, device=q.device)
    for b in range(len(ks) - 1):
        n, t0, t1 = ks[b + 1] - ks[b], starts[b], starts[b + 1]
        for r in range(R):
            kr = s["kr"][r, ks[b]:ks[b + 1]].double().expand(H, -1, -1)
            k, v = [s[i][r, ks[b]:ks[b + 1]].double().transpose(0, 1) for i in ("k", "v")]
            k = torch.cat([k, kr], -1)
            for at in range(t0, t1, 512):
                to = min(at + 512, t1)
                out[r, at:to] = _rows_of(q[r, at:to].double().transpose(0, 1), k, v, n, s["scale"], at - t0, n - (t1 - t0)).transpose(0, 1)
    return out
