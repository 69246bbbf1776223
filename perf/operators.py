"""What the paged-decode operators of libsfar cost: cases, inputs, plain forms.

Four operators of a tensor-parallel layer whose R simulated ranks hold their
heads' keys and values in a paged cache of 8-bit floating point (e4m3) and
their projection weights in e4m3 with a scale for each 128 x 128 block:

  plan       block tables, slot maps and token offsets from the requests'
             lengths (SfarKv.plan);
  append     new keys and values into the cache, one power-of-two scale for
             each page and head, grown (and the page requantised) when a new
             token needs it (SfarKv.append);
  attention  the new tokens of every request over its cached context, causal,
             optionally within a sliding window (SfarKv.attention);
  project    row-parallel matrix product in e4m3: the bf16 input quantised
             with a scale for each 128 values of a row, times the 8-bit
             weights (Sfar.quantize_fp8, Sfar.rowpar_gemm_fp8).

``run`` computes them in plain binary32 torch operations, or, where ``own`` is
true, by the library.  ``exact`` computes them in binary64.  The sizes follow
the repository's decode shape (8 ranks, hidden 8192, projections with 1024
and 3584 rows per rank) and smaller ones.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
EXP_MIN = -100                      # smallest exponent of a quantisation scale


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a full batch: every request adds a token, a few open a page
        {"name": "plan decode 256", "op": "plan", "B": 256, "W": 128, "P": 64, "lo": 1, "hi": 8000, "add_lo": 1, "add_hi": 1,
         "drop_every": 0, "pool": 1.0},
        # prompts and decodes mixed over many requests, finished ones leave, the pool runs out near the end
        {"name": "plan mixed 2039", "op": "plan", "B": 2039, "W": 96, "P": 32, "lo": 0, "hi": 2500, "add_lo": 0, "add_hi": 61,
         "drop_every": 7, "pool": 0.97},
        # decode step: one token of each of 64 requests
        {"name": "append decode 64", "op": "append", "R": 8, "H": 1, "D": 128, "P": 64, "B": 64, "lo": 1, "hi": 4000, "add_lo": 1,
         "add_hi": 1},
        # prompts of several requests at once, their first tokens in half-filled pages
        {"name": "append prompt 16k", "op": "append", "R": 4, "H": 2, "D": 128, "P": 32, "B": 9, "lo": 0, "hi": 3000, "add_lo": 1501,
         "add_hi": 2139},
        # the smallest call: one request, short context (latency)
        {"name": "attn decode 1 short", "op": "attention", "R": 2, "H": 2, "G": 4, "D": 64, "P": 16, "B": 1, "lo": 99, "hi": 99,
         "q_lo": 1, "q_hi": 1, "window": 0},
        # an ordinary decode batch, ragged contexts
        {"name": "attn decode 16", "op": "attention", "R": 8, "H": 1, "G": 8, "D": 128, "P": 64, "B": 16, "lo": 301, "hi": 4096,
         "q_lo": 1, "q_hi": 1, "window": 0},
        # the largest decode batch: a gigabyte of cache
        {"name": "attn decode 64 long", "op": "attention", "R": 8, "H": 1, "G": 8, "D": 128, "P": 64, "B": 64, "lo": 6003, "hi": 10400,
         "q_lo": 1, "q_hi": 1, "window": 0},
        # one request with a very long context: few rows, the axis of tokens is all there is to share out
        {"name": "attn decode 131k", "op": "attention", "R": 4, "H": 2, "G": 5, "D": 128, "P": 32, "B": 1, "lo": 131071, "hi": 131071,
         "q_lo": 1, "q_hi": 1, "window": 0},
        # chunks of prompts over what is cached already
        {"name": "attn prompt chunks", "op": "attention", "R": 8, "H": 1, "G": 8, "D": 128, "P": 64, "B": 3, "lo": 1100, "hi": 4099,
         "q_lo": 700, "q_hi": 1024, "window": 0},
        # few tokens, odd sizes (latency)
        {"name": "project 3", "op": "project", "R": 4, "M": 3, "K": 1000, "N": 2056},
        # a decode batch through the widest projection: the weights' bytes bound it
        {"name": "project 64", "op": "project", "R": 8, "M": 64, "K": 3584, "N": 8192},
        # prompts through the same projection: the tensor cores bound it
        {"name": "project 2048", "op": "project", "R": 8, "M": 2048, "K": 3584, "N": 8192},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention", "project", "project"])
    P = rng.choice([16, 32, 64, 128])
    if op == "plan":
        hi = rng.randint(1, 6000)
        add = _log(rng, 1, 60)
        return {"op": op, "B": _log(rng, 1, 2039), "W": -(-(hi + add) // P) + rng.randint(0, 5), "P": P, "lo": 0, "hi": hi,
                "add_lo": rng.choice([0, 1]), "add_hi": add, "drop_every": rng.choice([0, 3, 7]), "pool": rng.choice([1.0, 1.0, 0.9])}
    R, D = rng.choice([2, 3, 4, 8]), rng.choice([64, 128])
    if op == "append":
        H, B = rng.choice([1, 2, 3, 4, 8]), _log(rng, 1, 128)
        most = max(1, (16384 * 4 * 2 * 128) // (R * H * D * B))
        add = _log(rng, 1, most)
        return {"op": op, "R": R, "H": H, "D": D, "P": P, "B": B, "lo": 0, "hi": rng.randint(1, 3000), "add_lo": (add + 1) // 2, "add_hi": add}
    if op == "attention":
        H, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        if rng.random() < 0.6:                                   # decode, or a few guessed tokens at once
            B, q = _log(rng, 1, 96), rng.choice([1, 1, 1, 2, 4, 7])
            most = min(131072, (900 << 20) // (R * H * D * 2 * B), (3 << 29) // (R * H * G * B * q))
        else:                                                    # chunks of prompts
            B, q = rng.randint(1, 6), _log(rng, 16, 1000)
            most = min(32768, (200 << 20) // (R * H * G * B * q), (1 << 30) // (R * H * D * 2 * B))
        hi = _log(rng, min(q + 1, max(q, most)), max(q + 1, most))
        return {"op": op, "R": R, "H": H, "G": G, "D": D, "P": P, "B": B, "lo": max(1, rng.choice([hi, hi // 2, hi // 7])), "hi": hi,
                "q_lo": rng.choice([1, q]), "q_hi": q, "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)])}
    N, K = 8 * rng.randint(16, 1024), rng.choice([_log(rng, 64, 3584), 128 * rng.randint(1, 28)])
    return {"op": op, "R": R, "M": _log(rng, 1, 2048), "K": K, "N": N}


# ------------------------------------------------------- lengths and generators
def _spread(n, lo, hi, phase=0.37):
    """n whole numbers spread evenly over [lo, hi] in a mixed order; the same for every seed."""
    return [lo + int((hi - lo + 1) * ((phase + (b + 1) * 0.6180339887498949) % 1.0)) for b in range(n)]


def _lengths(c):
    """(tokens held before, tokens added) of every request, in the order of no seed."""
    before = _spread(c["B"], c["lo"], c["hi"])
    add = _spread(c["B"], c["add_lo"], c["add_hi"], 0.11)
    if c.get("drop_every"):
        add = [-(before[b] if b % 2 else before[b] // 3) if b % c["drop_every"] == 3 else a for b, a in enumerate(add)]
    return before, add


def _attn_lengths(c):
    """(context with the new tokens, new tokens) of every request."""
    q = _spread(c["B"], c["q_lo"], c["q_hi"], 0.11)
    return [max(n, a) for n, a in zip(_spread(c["B"], c["lo"], c["hi"]), q)], q


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _shuffled(seed, *lists):
    """The lists, reordered together by the seed."""
    order = torch.randperm(len(lists[0]), generator=torch.Generator().manual_seed(seed)).tolist()
    return [[v[i] for i in order] for v in lists]


def _f8(g, shape, sigma):
    """e4m3 values of a normal distribution."""
    t = torch.empty(shape, dtype=F8, device=DEV)
    flat = t.view(-1)
    step = 1 << 27
    for at in range(0, flat.numel(), step):
        part = flat[at:at + step]
        part.copy_(torch.randn(part.numel(), generator=g, device=DEV, dtype=torch.float16).mul_(sigma).clamp_(-F8_MAX, F8_MAX))
    return t


def _tables(g, pages, W, pool):
    """A random block table [B, W] (-1 past a request's pages) and the pool's other pages in a random order."""
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    n = _int(pages)
    j = torch.arange(W, device=DEV)
    at = (torch.cumsum(n, 0) - n)[:, None] + j[None, :]
    used = j[None, :] < n[:, None]
    return torch.where(used, order[at.clamp(max=max(pool - 1, 0))], -1).to(torch.int32).contiguous(), order[int(sum(pages)):]


def _starts(add):
    return _int([0] + torch.tensor(add).clamp(min=0).cumsum(0).tolist())


# ------------------------------------------------------------------- prepare
def prepare(case, seed):
    return {"plan": _prepare_plan, "append": _prepare_append, "attention": _prepare_attention, "project": _prepare_project}[case["op"]](case, seed)


def _up(n, p):
    return -(-n // p)


def _prepare_plan(c, seed):
    g = _gen(seed)
    before, add = _shuffled(seed, *_lengths(c))
    P = c["P"]
    pages = [_up(n, P) for n in before]
    need = sum(max(0, _up(n + a, P) - _up(n, P)) for n, a in zip(before, add))
    free = max(1, int(need * c["pool"]) + (64 if c["pool"] >= 1.0 else 0))
    pool = sum(pages) + free
    table, rest = _tables(g, pages, c["W"], pool)
    head = seed % pool                                           # the ring's first free page is anywhere in it
    ring = torch.full((pool,), -1, dtype=torch.int32, device=DEV)
    ring[(head + torch.arange(free, device=DEV)) % pool] = rest
    T = sum(max(a, 0) for a in add)
    s = {"op": "plan", "P": P, "T": T, "lens": _int(before), "delta": _int(add), "table": table, "ring": ring, "state": _int([head, free]),
         "lens_out": _int(before), "state_out": _int([0, 0]), "starts": torch.zeros(c["B"] + 1, dtype=torch.int32, device=DEV),
         "slots": torch.zeros(T, dtype=torch.int32, device=DEV), "taken": torch.zeros(c["B"], dtype=torch.int32, device=DEV)}
    if own:
        from barrier_free_message_gb300 import sfar
        caches = [torch.zeros((2, pool, 1, P, 64), dtype=F8, device=DEV) for _ in range(2)]
        s["kv"] = sfar.SfarKv(*caches, *[torch.ones((2, pool, 1), device=DEV) for _ in range(2)], q_heads=1)
    return s


def _cache(c, g, pool):
    """Caches and scales of every rank: [R, pages, heads, tokens of a page, head dim], [R, pages, heads]."""
    shape = (c["R"], pool, c["H"], c["P"], c["D"])
    k, v = _f8(g, shape, 100.0), _f8(g, shape, 100.0)
    ks, vs = [0.005 * (1.0 + 2.0 * torch.rand(shape[:3], generator=g, device=DEV)) for _ in range(2)]
    return k, v, ks, vs


def _handle(s, q_heads):
    if own:
        from barrier_free_message_gb300 import sfar
        s["kv"] = sfar.SfarKv(s["kc"], s["vc"], s["ks"], s["vs"], q_heads=q_heads)
    return s


def _prepare_append(c, seed):
    g = _gen(seed)
    before, add = _shuffled(seed, *_lengths(c))
    P, T = c["P"], sum(add)
    pages = [_up(n + a, P) for n, a in zip(before, add)]
    pool = sum(pages) + 3
    table, _ = _tables(g, pages, max(pages), pool)
    kc, vc, ks, vs = _cache(c, g, pool)
    ks, vs = torch.exp2(torch.floor(torch.log2(ks))), torch.exp2(torch.floor(torch.log2(vs)))
    start = _starts(add)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    pos = (_int(before)[b] + t - start[b]).long()
    slots = table[b, pos // P] * P + pos % P
    # keys and values as slices of one projection's output, so a token's row is wider than its heads;
    # a token's loudness varies, so that pages meet values beyond their scale
    loud = torch.exp(0.7 * torch.randn((c["R"], T, 1, 1), generator=g, device=DEV))
    qkv = (torch.randn((c["R"], T, 2 * c["H"], c["D"]), generator=g, device=DEV) * loud).to(torch.bfloat16)
    return _handle({"op": "append", "P": P, "kc": kc, "vc": vc, "ks": ks, "vs": vs, "slots": slots.to(torch.int32),
                    "k": qkv[:, :, :c["H"]], "v": qkv[:, :, c["H"]:]}, c["H"])


def _prepare_attention(c, seed):
    g = _gen(seed)
    lens, q = _shuffled(seed, *_attn_lengths(c))
    pages = [_up(n, c["P"]) for n in lens]
    pool = sum(pages) + 5
    table, _ = _tables(g, pages, max(pages), pool)
    kc, vc, ks, vs = _cache(c, g, pool)
    qs = (1.5 * torch.randn((c["R"], sum(q), c["H"] * c["G"], c["D"]), generator=g, device=DEV)).to(torch.bfloat16)
    return _handle({"op": "attention", "kc": kc, "vc": vc, "ks": ks, "vs": vs, "table": table, "lens": _int(lens), "starts": _starts(q),
                    "q": qs, "out": torch.empty_like(qs), "max_q": max(q), "window": c["window"], "scale": 1.0 / math.sqrt(c["D"])},
                   c["H"] * c["G"])


def _prepare_project(c, seed):
    g = _gen(seed)
    R, M, K, N = c["R"], c["M"], c["K"], c["N"]
    nb, kb, Kp = _up(N, 128), _up(K, 128), _up(K, 16) * 16
    # activations with a few loud channels, as a layer's are
    x = torch.randn((R, M, K), generator=g, device=DEV) * torch.exp(0.8 * torch.randn((R, 1, K), generator=g, device=DEV))
    s = {"op": "project", "x": x.to(torch.bfloat16), "w": _f8(g, (R, N, Kp), 110.0)[:, :, :K],
         "sw": 2e-4 * (0.5 + torch.rand((R, nb, kb), generator=g, device=DEV)), "y": torch.empty((R, M, N), dtype=torch.bfloat16, device=DEV)}
    if own:
        from barrier_free_message_gb300 import sfar
        s["x8"] = torch.empty((R, M, Kp), dtype=F8, device=DEV)[:, :, :K]
        s["sx"] = torch.empty((R, kb, M), dtype=torch.float32, device=DEV)
        s["h"] = sfar.Sfar(R, 1 << 16, "bf16")
    return s


# ----------------------------------------------------------------------- run
def run(state):
    return {"plan": _run_plan, "append": _run_append, "attention": _run_attention, "project": _run_project}[state["op"]](state)


def _run_plan(s):
    if own:
        s["kv"].plan(s["lens"], s["delta"], s["table"], s["ring"], s["state"], s["lens_out"], s["state_out"], s["starts"], s["slots"], s["taken"])
        return {k: s[k] for k in ("lens_out", "state_out", "starts", "slots", "taken", "table", "ring")}
    P, table, ring = s["P"], s["table"], s["ring"]
    B, W = table.shape
    pool = ring.shape[0]
    before, add = s["lens"].long(), s["delta"].long()
    after = (before + add).clamp(min=0)
    have, want = (before + P - 1) // P, (after + P - 1) // P
    grow = add > 0
    fits = want <= W
    need = torch.where(grow & fits, want - have, 0)
    upto = torch.cumsum(need, 0)
    head, free = s["state"][0].long(), s["state"][1].long()
    taken = ~grow | (fits & ((need == 0) | (upto <= free)))
    back = torch.where(add < 0, have - want, 0)
    backto = torch.cumsum(back, 0)
    j = torch.arange(W, device=table.device)[None, :]
    new = (grow & taken)[:, None] & (j >= have[:, None]) & (j < want[:, None])
    at = (head + (upto - need)[:, None] + j - have[:, None]) % pool
    old = (add < 0)[:, None] & (j >= want[:, None]) & (j < have[:, None])
    to = (head + free + (backto - back)[:, None] + j - want[:, None]) % pool
    table.copy_(torch.where(new, ring[at], table))
    ring[to[old]] = table[old]
    used = torch.where(taken, upto * (need > 0), 0).amax()
    lens = torch.where(taken, after, before)
    count = add.clamp(min=0)
    starts = torch.cat([torch.zeros_like(count[:1]), torch.cumsum(count, 0)])
    t = torch.arange(s["T"], device=table.device)
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    pos = before[b] + t - starts[b]
    slots = torch.where(taken[b], table[b, (pos // P).clamp(max=W - 1)].long() * P + pos % P, -1)
    state = torch.stack([(head + used) % pool, free - used + backto[-1]])
    whole = {"lens_out": lens, "state_out": state, "starts": starts, "slots": slots, "taken": taken, "table": table, "ring": ring}
    return {k: v.to(torch.int32) for k, v in whole.items()}


def _scale_exponent(amax):
    """The least e with amax <= 448 * 2^e, at least EXP_MIN."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), EXP_MIN).clamp(min=EXP_MIN)


def _append_one(cache, scale, x, slots):
    """One of keys and values: cache [R, pages, H, P, D], scale [R, pages, H], x [R, T, H, D]."""
    R, pool, H, P, D = cache.shape
    raw = cache.view(torch.uint8)
    live = slots >= 0
    at = slots[live].long()
    x = x[:, live].float()
    page, off = at // P, at % P
    amax = x.abs().amax(-1)                                                        # [R, tokens, H]
    most = torch.zeros((R, pool, H), device=x.device).index_reduce_(1, page, amax, "amax")
    first = torch.full((pool,), P, dtype=torch.long, device=x.device).index_reduce_(0, page, off, "amin")
    hit = (first < P).nonzero().flatten()
    old = torch.where((first[hit] > 0)[None, :, None], scale[:, hit], 0.0)
    new = torch.maximum(old, torch.ldexp(torch.ones_like(old), _scale_exponent(most[:, hit])))
    held = torch.arange(P, device=x.device)[None, :] < first[hit][:, None]
    ratio = torch.where(old > 0, old / new, torch.ones_like(old))[..., None, None]
    again = (raw[:, hit].view(F8).float() * ratio).to(F8).view(torch.uint8)
    raw[:, hit] = torch.where(held[None, :, None, :, None], again, raw[:, hit])
    scale[:, hit] = new
    raw[:, page, :, off] = (x / scale[:, page][..., None]).to(F8).view(torch.uint8).movedim(1, 0)


def _run_append(s):
    if own:
        s["kv"].append(s["k"], s["v"], s["slots"])
    else:
        _append_one(s["kc"], s["ks"], s["k"], s["slots"])
        _append_one(s["vc"], s["vs"], s["v"], s["slots"])
    return {"k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}


def _run_attention(s):
    if own:
        s["kv"].attention(s["q"], s["out"], s["table"], s["lens"], s["starts"], max_q=s["max_q"], scale=s["scale"], window=s["window"])
        return s["out"]
    q, table, lens, starts, n = s["q"], s["table"].clamp(min=0).long(), s["lens"].long(), s["starts"].long(), s["max_q"]
    R, T, Hq, D = q.shape
    _, _, H, P, _ = s["kc"].shape
    B, W = table.shape
    G, L = Hq // H, W * P
    count = starts[1:] - starts[:-1]
    i = torch.arange(n, device=q.device)
    rows = q[:, (starts[:-1, None] + i).clamp(max=T - 1)].float()                   # [R, B, n, Hq, D]
    rows = rows.view(R, B, n, H, G, D).permute(0, 1, 3, 2, 4, 5).reshape(R, B, H, n * G, D)

    def gathered(cache, scale):
        x = cache.view(torch.uint8)[:, table].view(F8).float() * scale[:, table][..., None, None]
        return x.transpose(2, 3).reshape(R, B, H, L, D)

    a = torch.matmul(rows, gathered(s["kc"], s["ks"]).transpose(-1, -2)) * s["scale"]
    at = (lens - count)[:, None] + i                                                # position of each new token
    j = torch.arange(L, device=q.device)
    seen = (j <= at[..., None]) & (j < lens[:, None, None])
    if s["window"]:
        seen &= j > at[..., None] - s["window"]
    seen = seen.repeat_interleave(G, 1)[None, :, None]
    a = a.masked_fill(~seen, -math.inf)
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    o = torch.matmul(p, gathered(s["vc"], s["vs"])) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(R, B, H, n, G, D).permute(0, 1, 3, 2, 4, 5).reshape(R, B, n, Hq, D)
    t = torch.arange(T, device=q.device)
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    return o[:, b, t - starts[b]].to(torch.bfloat16)


def _run_project(s):
    if own:
        s["h"].quantize_fp8(s["x"], s["x8"], s["sx"])
        s["h"].rowpar_gemm_fp8(s["x8"], s["sx"], s["w"], s["sw"], s["y"])
        return {"y": s["y"], "x8": s["x8"], "sx": s["sx"]}
    x, w, sw = s["x"].float(), s["w"], s["sw"]
    R, M, K = x.shape
    N, kb = w.shape[1], sw.shape[2]
    blocks = torch.nn.functional.pad(x, (0, kb * 128 - K)).view(R, M, kb, 128)
    sx = torch.ldexp(torch.ones((), device=x.device), _scale_exponent(blocks.abs().amax(-1)))
    x8 = (blocks / sx[..., None]).to(F8)
    xq = (x8.float() * sx[..., None]).view(R, M, kb * 128)[:, :, :K]
    wq = w.float() * sw.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    y = torch.matmul(xq, wq.transpose(1, 2)).to(torch.bfloat16)
    return {"y": y, "x8": x8.view(R, M, kb * 128)[:, :, :K], "sx": sx.transpose(1, 2)}


# ---------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "plan":
        before, add = _lengths(c)
        T, B = sum(max(a, 0) for a in add), c["B"]
        moved = sum(abs(_up(max(n + a, 0), c["P"]) - _up(n, c["P"])) for n, a in zip(before, add))
        # lengths, changes, starts, answers; pages taken or given back; a table entry for each page that tokens go to; slots
        return {"bytes": 4 * (5 * B + 1) + 8 * moved + 4 * B + 4 * T, "flops": T}
    if c["op"] == "append":
        before, add = _lengths(c)
        T, heads = sum(add), 2 * c["R"] * c["H"]
        touched = sum(_up(n + a, c["P"]) - n // c["P"] for n, a in zip(before, add))
        return {"bytes": 4 * T + heads * (T * c["D"] * 3 + 8 * touched), "flops": 3 * heads * T * c["D"]}
    if c["op"] == "attention":
        pairs = keys = pages = tokens = 0
        for n, q in zip(*_attn_lengths(c)):
            w = c["window"] or n
            pairs += sum(min(n - q + i + 1, w) for i in range(q))
            k = min(n, q - 1 + w)
            keys, pages, tokens = keys + k, pages + _up(k, c["P"]), tokens + q
        heads = c["R"] * c["H"]
        return {"bytes": heads * (2 * keys * c["D"] + 8 * pages + 4 * tokens * c["G"] * c["D"]) + 4 * pages,
                "flops": 4 * heads * c["G"] * c["D"] * pairs}
    R, M, K, N = c["R"], c["M"], c["K"], c["N"]
    kb = _up(K, 128)
    return {"bytes": R * (N * K + 4 * _up(N, 128) * kb + 3 * M * K + 4 * M * kb + 2 * M * N), "flops": 2 * R * M * K * N}


# --------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "project": _exact_project}.get(case["op"], lambda s: None)(s)


def _e4m3(x):
    """binary64 values rounded to the nearest e4m3 value (ties to even), |x| <= 448; by the format's definition."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def _scale64(amax):
    k = torch.full_like(amax, EXP_MIN)
    for e in range(EXP_MIN + 1, 121):
        k = torch.where(amax > F8_MAX * 2.0 ** (e - 1), float(e), k)
    return torch.exp2(k)


def _exact_append(s):
    P, slots = s["P"], s["slots"].tolist()
    out = {}
    for name, x, cache, scale in (("k", s["k"], s["kc"], s["ks"]), ("v", s["v"], s["vc"], s["vs"])):
        values, scales, x = cache.float(), scale.double(), x.double()
        t = 0
        while t < len(slots):
            page, first = divmod(slots[t], P)
            n = 1
            while t + n < len(slots) and slots[t + n] == slots[t] + n and (first + n) < P:
                n += 1
            part = x[:, t:t + n].transpose(1, 2)                                    # [R, H, n, D]
            need = _scale64(part.abs().amax((-1, -2)))
            new = torch.maximum(scales[:, page], need) if first else need
            if first:
                values[:, page, :, :first] = _e4m3(values[:, page, :, :first].double() * (scales[:, page] / new)[..., None, None]).float()
            scales[:, page] = new
            values[:, page, :, first:first + n] = _e4m3(part / new[..., None, None]).float()
            t += n
        out[name], out[name + "_scale"] = values.to(F8), scales.float()
    return out


def _exact_attention(s):
    q, starts, lens, table, w = s["q"], s["starts"].tolist(), s["lens"].tolist(), s["table"].long(), s["window"]
    R, T, Hq, D = q.shape
    H, P = s["kc"].shape[2:4]
    G = Hq // H
    out = torch.zeros((R, T, Hq, D), dtype=torch.float64, device=q.device)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pages = table[b, :_up(n, P)]
        for r in range(R):
            k, v = [(c[r].view(torch.uint8)[pages].view(F8).double() * sc[r][pages].double()[..., None, None]).transpose(0, 1).reshape(H, -1, D)[:, :n]
                    for c, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"]))]
            for at in range(starts[b], starts[b + 1], 256):
                to = min(at + 256, starts[b + 1])
                pos = n - (starts[b + 1] - torch.arange(at, to, device=q.device))
                j = torch.arange(n, device=q.device)
                seen = j[None] <= pos[:, None]
                if w:
                    seen &= j[None] > pos[:, None] - w
                x = q[r, at:to].double().view(to - at, H, G, D).permute(1, 2, 0, 3)   # [H, G, tokens, D]
                a = (x @ k[:, None].transpose(-1, -2)) * s["scale"]
                a = torch.where(seen, a, -math.inf)
                o = torch.nan_to_num(torch.softmax(a, -1)) @ v[:, None]
                out[r, at:to] = o.permute(2, 0, 1, 3).reshape(to - at, Hq, D)
    return out


def _exact_project(s):
    x, sw = s["x"].double(), s["sw"].double()
    R, M, K = x.shape
    N = s["w"].shape[1]
    y = torch.zeros((R, M, N), dtype=torch.float64, device=x.device)
    x8, sx = torch.zeros_like(x), torch.zeros((R, sw.shape[2], M), dtype=torch.float64, device=x.device)
    for b in range(sw.shape[2]):
        part = slice(128 * b, min(128 * b + 128, K))
        sx[:, b] = _scale64(x[:, :, part].abs().amax(-1))
        x8[:, :, part] = _e4m3(x[:, :, part] / sx[:, b, :, None])
        product = x8[:, :, part] @ s["w"][:, :, part].double().transpose(1, 2)
        y += product * sx[:, b, :, None] * sw[:, :, b].repeat_interleave(128, 1)[:, None, :N]
    return {"y": y, "x8": x8.float().to(F8), "sx": sx.float()}
