"""The attention set over an 8-bit paged key/value cache, as cases that can be measured: block tables and slot maps
from request lengths, storing and reading back cache rows, and attention over the cache.

`run` computes each in plain torch operations (fp32, rounded once at the end), or, with `own` true, through the
library's entry points. `exact` computes the same from the definitions in 64 bits.

The cache: int8 pages [pages, kv heads, page tokens, head size], one fp32 scale per (page, kv head), for keys and for
values. A request's token i lives in page block_table[r, i // page] at row i % page.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
DEV = "cuda"
MIN_SCALE = 2.0 ** -126      # a block whose scale would be below the smallest normal number holds zeros
SPARE = 5                    # padding tokens of the slot map, as a batch padded to a graph's size has them


# ------------------------------------------------------------------------------------------------------ cases
def listed():
    attend = {"kind": "attend"}
    return [
        # one decoding step of 64 running requests: a handful of pages change hands
        {"name": "plan_step", "kind": "plan", "page": 16, "requests": 64, "past_min": 30, "past_max": 8191,
         "new_min": 1, "new_max": 1},
        # a large batch of prompts and continuations, scheduled at once
        {"name": "plan_prompts", "kind": "plan", "page": 32, "requests": 2048, "past_min": 1, "past_max": 2000,
         "new_min": 1, "new_max": 300},
        # the same step's cache rows of one layer: 64 tokens, most of them into pages that already hold some
        {"name": "store_step", "kind": "store", "dtype": "bf16", "kv_heads": 8, "dim": 128, "page": 16,
         "requests": 64, "past_min": 30, "past_max": 2000, "new_min": 1, "new_max": 1},
        # ragged prompts of eight requests, fp32 activations as the library's projections write them
        {"name": "store_prompts", "kind": "store", "dtype": "f32", "kv_heads": 8, "dim": 128, "page": 64,
         "requests": 8, "past_min": 1, "past_max": 700, "new_min": 500, "new_max": 4001},
        # one user, a short context: the latency of a decoding step at 32 heads of 64 (fp32)
        {"name": "decode_one", **attend, "dtype": "f32", "q_heads": 32, "kv_heads": 8, "dim": 64, "page": 16,
         "requests": 1, "past_min": 999, "past_max": 999, "new_min": 1, "new_max": 1, "window": 0},
        # a serving batch at 32 query and 8 key/value heads of 128, ragged contexts
        {"name": "decode_batch", **attend, "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "requests": 64, "past_min": 200, "past_max": 8190, "new_min": 1, "new_max": 1, "window": 0},
        # few requests with very long contexts: few rows, a long axis to split
        {"name": "decode_long", **attend, "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 128,
         "requests": 4, "past_min": 100000, "past_max": 131071, "new_min": 1, "new_max": 1, "window": 0},
        # every query head with its own keys (fp16)
        {"name": "decode_mha", **attend, "dtype": "f16", "q_heads": 16, "kv_heads": 16, "dim": 128, "page": 32,
         "requests": 24, "past_min": 77, "past_max": 4000, "new_min": 1, "new_max": 1, "window": 0},
        # speculative decoding: a few draft tokens of each request verified at once (fp32)
        {"name": "verify", **attend, "dtype": "f32", "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 32,
         "requests": 16, "past_min": 100, "past_max": 4000, "new_min": 2, "new_max": 8, "window": 0},
        # one long prompt
        {"name": "prefill", **attend, "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64,
         "requests": 1, "past_min": 0, "past_max": 0, "new_min": 8192, "new_max": 8192, "window": 0},
        # ragged prompts in fp32 at heads of 64
        {"name": "prefill_f32", **attend, "dtype": "f32", "q_heads": 32, "kv_heads": 8, "dim": 64, "page": 16,
         "requests": 6, "past_min": 0, "past_max": 0, "new_min": 37, "new_max": 1500, "window": 0},
        # chunks of prompts next to decoding requests, a sliding window, seven query heads a key head (fp16)
        {"name": "chunks_window", **attend, "dtype": "f16", "q_heads": 14, "kv_heads": 2, "dim": 64, "page": 16,
         "requests": 16, "past_min": 3, "past_max": 4000, "new_min": 1, "new_max": 512, "window": 1000},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["plan", "store", "attend", "attend", "attend", "attend"])
    page = rng.choice([16, 16, 32, 64, 128])
    if kind == "plan":
        n = _log_int(rng, 1, 4096)
        new = _log_int(rng, 1, max(2, 300000 // n))
        past = _log_int(rng, 1, 8000)
        return {"kind": kind, "page": page, "requests": n, "past_min": rng.randint(0, past), "past_max": past,
                "new_min": rng.randint(0, min(3, new)), "new_max": min(new, 20000)}
    dtype, dim = rng.choice(["f32", "f16", "bf16"]), rng.choice([64, 128])
    heads = rng.choice([1, 2, 3, 4, 8, 8, 16])
    if kind == "store":
        n = _log_int(rng, 1, 128)
        new = _log_int(rng, 1, max(2, 16000 * 8 // (n * heads)))
        past = _log_int(rng, 1, 500)
        return {"kind": kind, "dtype": dtype, "kv_heads": heads, "dim": dim, "page": page, "requests": n,
                "past_min": rng.randint(0, past), "past_max": past, "new_min": rng.randint(1, new),
                "new_max": min(new, 8000)}
    group = rng.choice([1, 2, 4, 4, 5, 7, 8, 16])
    form = rng.choice(["decode", "decode", "verify", "prefill", "chunk"])
    window = rng.choice([0, 0, 0, _log_int(rng, 20, 3000)])
    if form in ("decode", "verify"):
        n = _log_int(rng, 1, 128)
        kv = _log_int(rng, 8, min(100000, 500000 * 8 // (n * heads)))
        new = 1 if form == "decode" else rng.randint(2, 12)
        past = (kv // 7 if rng.random() < 0.7 else kv, kv)
    else:
        rows = rng.choice([500, 2000, 6000])
        n = 1 if rng.random() < 0.4 else rng.randint(2, 12)
        new = _log_int(rng, 20, max(21, rows // (1 + n // 4)))
        kv = 0 if form == "prefill" else _log_int(rng, 8, 6000)
        past = (kv // 7, kv)
        # the plain form holds a padded score matrix: keep it under about 6 GB
        while n * heads * group * new * (new + kv) * 4 > 6e9:
            new = max(13, new // 2)
            n = max(1, n // 2)
    new_min = new if rng.random() < 0.5 else rng.randint(1, new)
    return {"kind": kind, "dtype": dtype, "q_heads": heads * group, "kv_heads": heads, "dim": dim, "page": page,
            "requests": n, "past_min": past[0], "past_max": past[1], "new_min": new_min, "new_max": new,
            "window": window}


def _spread(lo, hi, n, phase):
    """n whole numbers from lo to hi, spread evenly over their logarithm in a scrambled order; the first is hi."""
    out = []
    for i in range(n):
        f = (i * 0.6180339887498949 + phase) % 1.0
        a, b = math.log(lo + 1.0), math.log(hi + 1.0)
        out.append(hi if i == 0 else min(hi, max(lo, int(round(math.exp(b - f * (b - a)) - 1.0)))))
    return out


def lengths(case):
    """(tokens already in the cache, new tokens) of each request: by the case alone."""
    n = case["requests"]
    return _spread(case["past_min"], case["past_max"], n, 0.0), _spread(case["new_min"], case["new_max"], n, 0.37)


def _ceil(a, b):
    return -(-a // b)


def _visible(past, new, window):
    """Visible (query, key) pairs of one request under the causal mask, and the first key that any row sees."""
    if new == 0:
        return 0, 0
    if window <= 0:
        return new * past + new * (new + 1) // 2, 0
    full = max(0, min(new, past + new - window))         # rows whose window is cut on the left: pos + 1 > window
    pairs = sum(min(past + t + 1, window) for t in range(new)) if full else new * past + new * (new + 1) // 2
    return pairs, max(0, past + 1 - window)


def work(case):
    past, new = lengths(case)
    P, T = case["page"], sum(new)
    if case["kind"] == "plan":
        pages = sum(_ceil(a + b, P) - _ceil(a, P) for a, b in zip(past, new))
        partly = sum(1 for a, b in zip(past, new) if a % P and b)
        return {"bytes": 16 * len(past) + 8 * pages + 4 * partly + 12 * (T + SPARE), "flops": 0}
    row = case["kv_heads"] * case["dim"] * 2             # a token's keys and values, one byte each
    if case["kind"] == "store":
        back = sum(b + a % P for a, b in zip(past, new))
        wide = BYTES[case["dtype"]]
        return {"bytes": T * (row * wide + row + 8) + back * (row + row * wide + 8), "flops": 2 * row * (T + back)}
    read = pairs = 0
    for a, b in zip(past, new):
        p, first = _visible(a, b, case["window"])
        pairs += p
        read += (a + b - first) * row + _ceil(a + b - first, P) * case["kv_heads"] * 8 if b else 0
    rows = T * case["q_heads"]
    return {"bytes": read + rows * (2 * case["dim"] * BYTES[case["dtype"]] + 4),
            "flops": 4 * case["dim"] * case["q_heads"] * pairs}


# ----------------------------------------------------------------------------------------------------- inputs
def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _tables(case, gen):
    """Lengths, a pool of pages in random order, and the table of the pages that hold the past tokens."""
    past, new = lengths(case)
    P, n = case["page"], len(past)
    have = [_ceil(a, P) for a in past]
    total = [_ceil(a + b, P) for a, b in zip(past, new)]
    wide = max(max(total), 1) + 1
    pages = sum(total) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    col = torch.arange(wide, device=DEV)[None, :]
    h = _ints(have, torch.int64)
    at = (h.cumsum(0) - h)[:, None] + col
    table = torch.where(col < h[:, None], order[at.clamp(max=pages - 1)], -1).to(torch.int32)
    return past, new, pages, table, order[sum(have):].contiguous()


def _pages(case, pages, gen):
    """Cache contents: normal values at about 36 steps a standard deviation, scales that differ by block."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    out = []
    for _ in range(2):
        x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float16)
        out.append((x * 36.0).round_().clamp_(-127, 127).to(torch.int8))
        out.append(0.022 + 0.012 * torch.rand(shape[:2], generator=gen, device=DEV))
    return out[0], out[2], out[1], out[3]                # keys, values, key scales, value scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    past, new, pages, table, free = _tables(case, gen)
    s = {"case": case, "past": _ints(past), "new": _ints(new), "pages": pages, "tokens": sum(new) + SPARE}
    if case["kind"] == "plan":
        s.update(table=table, free=free)
        return s
    dt, H, D, P = DTYPES[case["dtype"]], case["kv_heads"], case["dim"], case["page"]
    past_t, new_t = _ints(past, torch.int64), _ints(new, torch.int64)
    table, kv_len, q_start, slots, _ = _plan(past_t, new_t, table, free, P, sum(new))
    s["k"], s["v"], s["k_scale"], s["v_scale"] = _pages(case, pages, gen)
    if case["kind"] == "store":
        # keys and values as slices of one projection's rows, the query part of them in front
        rows = torch.randn((sum(new), 3 * H * D), generator=gen, device=DEV).to(dt)
        s["rows_k"], s["rows_v"] = rows[:, H * D:2 * H * D], rows[:, 2 * H * D:]
        # what is read back: every token of the pages that were written to
        first = torch.div(past_t, P, rounding_mode="floor") * P
        _, there, _ = _slots(first, past_t + new_t - first, table, P, sum(b + a % P for a, b in zip(past, new)))
        s.update(slots=slots, back=there)
        return s
    s["q"] = (2.0 * torch.randn((sum(new), case["q_heads"], D), generator=gen, device=DEV)).to(dt)
    s.update(table=table, kv_len=kv_len, q_start=q_start, max_new=max(new), max_kv=max(a + b for a, b in zip(past, new)))
    s["ws"] = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)   # scratch that a program keeps, zeroed once
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _plan(past, new, table, free, P, tokens):
    kv = past + new
    have = torch.div(past + P - 1, P, rounding_mode="floor")
    need = torch.div(kv + P - 1, P, rounding_mode="floor") - have
    start = need.cumsum(0) - need
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    at = (start[:, None] + col - have[:, None]).clamp(0, free.shape[0] - 1)
    table = torch.where(fresh, free[at], table)
    q_start, slots, positions = _slots(past, new, table, P, tokens)
    return table, kv.to(torch.int32), q_start, slots, positions


def _slots(past, new, table, P, tokens):
    """First token of each request, and each token's place in the cache and position in its request."""
    q_end = new.cumsum(0)
    t = torch.arange(tokens, device=table.device)
    r = torch.searchsorted(q_end, t, right=True).clamp(max=past.shape[0] - 1)
    pos = past[r] + t - (q_end - new)[r]
    on = t < q_end[-1]
    page = table[r, torch.div(pos, P, rounding_mode="floor").clamp(max=table.shape[1] - 1)].to(torch.int64)
    slots = torch.where(on, page * P + pos % P, -1)
    q_start = torch.cat([torch.zeros_like(q_end[:1]), q_end]).to(torch.int32)
    return q_start, slots, torch.where(on, pos, -1).to(torch.int32)


def _run_plan(s):
    past, new = s["past"].to(torch.int64), s["new"].to(torch.int64)
    P = s["case"]["page"]
    table, kv, q_start, slots, pos = _plan(past, new, s["table"], s["free"], P, s["tokens"])
    s["table"].copy_(table)
    used = (torch.div(past + new + P - 1, P, rounding_mode="floor") - torch.div(past + P - 1, P, rounding_mode="floor")).sum()
    return {"table": s["table"], "kv_len": kv, "q_start": q_start, "slots": slots, "positions": pos,
            "pages": used.to(torch.int32)}


def _round_away(x):
    t = x.trunc()
    return t + torch.sign(x) * ((x - t).abs() >= 0.5)


def _store(x, slots, q, scale):
    """New rows x [tokens, heads, size] into q (pages, in place) and scale [pages, heads] (in place)."""
    P = q.shape[2]
    page, off = torch.div(slots, P, rounding_mode="floor"), slots % P
    x = x.float()
    far = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
    first = torch.full((q.shape[0],), P, device=q.device).index_reduce_(0, page, off, "amin")     # first new row
    old = torch.where((first == 0)[:, None], 0.0, scale)
    want = far / torch.full_like(far, 127.0)
    want = torch.where(want < MIN_SCALE, 0.0, want)
    now = torch.where((first == P)[:, None], scale, torch.maximum(old, want))
    hit = torch.nonzero(first < P).squeeze(1)            # the pages that get new rows
    ratio = torch.where(now > 0, old / torch.where(now > 0, now, 1.0), 0.0)[hit]
    row = torch.arange(P, device=q.device)[None, None, :, None]
    held = q[hit].float()
    q[hit] = torch.where(row < first[hit][:, None, None, None], _round_away(held * ratio[:, :, None, None]), held).to(torch.int8)
    inv = torch.where(now > 0, 1.0 / torch.where(now > 0, now, 1.0), 0.0)[page]
    q[page, :, off] = _round_away(x * inv[:, :, None]).clamp(-127, 127).to(torch.int8)
    scale.copy_(now)


def _read(q, scale, slots, dt):
    P = q.shape[2]
    page, off = torch.div(slots, P, rounding_mode="floor"), slots % P
    return (q[page, :, off].float() * scale[page][:, :, None]).to(dt)


def _run_store(s):
    c = s["case"]
    dt, shape = DTYPES[c["dtype"]], (-1, c["kv_heads"], c["dim"])
    _store(s["rows_k"].reshape(shape), s["slots"], s["k"], s["k_scale"])
    _store(s["rows_v"].reshape(shape), s["slots"], s["v"], s["v_scale"])
    return {"k": _read(s["k"], s["k_scale"], s["back"], dt), "v": _read(s["v"], s["v_scale"], s["back"], dt),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _run_attend(s):
    c = s["case"]
    P, H, D = c["page"], c["kv_heads"], c["dim"]
    G, R, N = c["q_heads"] // H, c["requests"], s["max_new"]
    pages = s["table"][:, :_ceil(s["max_kv"], P)].clamp(min=0).to(torch.int64)
    L = pages.shape[1] * P

    def rows(q, scale):                                  # [R, H, L, D]
        x = q[pages].float() * scale[pages][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(R, H, L, D)

    kv, start = s["kv_len"].to(torch.int64), s["q_start"].to(torch.int64)
    n = start[1:] - start[:-1]
    t = torch.arange(N, device=DEV)
    at = (start[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float().view(-1, H, G, D)[at].permute(0, 2, 1, 3, 4).reshape(R, H, N * G, D)
    score = torch.matmul(q, rows(s["k"], s["k_scale"]).transpose(-1, -2)) * (1.0 / math.sqrt(D))
    i = ((kv - n)[:, None] + t)[:, :, None]              # the rows' positions
    j = torch.arange(L, device=DEV)
    see = (j <= i) & (j < kv[:, None, None])
    if c["window"] > 0:
        see &= j > i - c["window"]
    see = see[:, None, :, None, :].expand(R, 1, N, G, L).reshape(R, 1, N * G, L)
    score.masked_fill_(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score, rows(s["v"], s["v_scale"])) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log()).squeeze(-1)
    out = out.view(R, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(R, N, H * G, D)
    lse = lse.view(R, H, N, G).permute(0, 2, 1, 3).reshape(R, N, H * G)
    tok = torch.arange(s["q"].shape[0], device=DEV)
    r = torch.searchsorted(start[1:], tok, right=True)
    return {"out": out[r, tok - start[r]].to(s["q"].dtype), "lse": lse[r, tok - start[r]]}


# ------------------------------------------------------------------------------------------------------- runs
def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(state, kind)
    return {"plan": _run_plan, "store": _run_store, "attend": _run_attend}[kind](state)


def _own(s, kind):
    from gemm_gguf_block_gb300 import cq
    if kind == "plan":
        kv, q_start, slots, pos, used = cq.kv_plan_t(s["past"], s["new"], s["table"], s["free"], s["case"]["page"],
                                                     s["pages"], s["tokens"])
        return {"table": s["table"], "kv_len": kv, "q_start": q_start, "slots": slots, "positions": pos,
                "pages": used[0]}
    cache = s.get("cache")
    if cache is None:                                    # the object that a program makes when it allocates the pages
        cache = s["cache"] = cq.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if kind == "store":
        cq.kv_append_t(cache, s["rows_k"], s["rows_v"], s["slots"])
        k, v = cq.kv_read_t(cache, s["back"], DTYPES[s["case"]["dtype"]])
        return {"k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    out, lse = cq.attn_paged_t(s["q"], cache, s["table"], s["kv_len"], s["q_start"], s["max_new"], s["max_kv"],
                               window=s["case"]["window"], ws=s["ws"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    P = case["page"]
    past, new = lengths(case)
    if case["kind"] == "plan":
        return None                                      # whole numbers only
    if case["kind"] == "store":
        return _exact_store(case, s, past, new)
    if sum(_visible(a, b, case["window"])[0] for a, b in zip(past, new)) * case["q_heads"] * case["dim"] > 8e12:
        return None
    H, D = case["kv_heads"], case["dim"]
    G = case["q_heads"] // H
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    first = 0
    for r, (a, b) in enumerate(zip(past, new)):
        if b == 0:
            continue
        kv = a + b
        ids = s["table"][r, :_ceil(kv, P)].long()
        pos = torch.arange(a, kv, device=DEV)
        step = max(1, int(2e8 // (kv * G)))
        for h in range(H):
            k = (s["k"][ids, h].double() * s["k_scale"][ids, h].double()[:, None, None]).reshape(-1, D)[:kv]
            v = (s["v"][ids, h].double() * s["v_scale"][ids, h].double()[:, None, None]).reshape(-1, D)[:kv]
            for t in range(0, b, step):
                i = pos[t:t + step]
                q = s["q"][first + t:first + t + i.numel(), h * G:(h + 1) * G].double()
                z = (q.reshape(-1, D) @ k.t()).view(i.numel(), G, kv) / math.sqrt(D)
                j = torch.arange(kv, device=DEV)[None, :]
                hide = j > i[:, None]
                if case["window"] > 0:
                    hide |= j <= i[:, None] - case["window"]
                z.masked_fill_(hide[:, None, :], -math.inf)
                lse[first + t:first + t + i.numel(), h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                out[first + t:first + t + i.numel(), h * G:(h + 1) * G] = torch.softmax(z, -1) @ v
        first += b
    return {"out": out, "lse": lse}


def _exact_store(case, s, past, new):
    P, H, D = case["page"], case["kv_heads"], case["dim"]
    got = {}
    for name in ("k", "v"):
        x = s["rows_" + name].reshape(-1, H, D).double().cpu()
        q, scale, slots = s[name].cpu(), s[name + "_scale"].double().cpu(), s["slots"].cpu()
        pieces, first = [], 0
        for a, b in zip(past, new):
            lo = a // P * P
            while lo < a + b and b:                      # one page after another, as the tokens arrive in it
                begin, end = max(lo, a), min(lo + P, a + b)
                rows = x[first + begin - a:first + end - a].permute(1, 0, 2)            # [H, rows, D]
                page = int(slots[first + begin - a]) // P
                old = scale[page] if begin > lo else torch.zeros(H, dtype=torch.float64)
                now = torch.maximum(old, rows.abs().amax((1, 2)) / 127.0)
                safe = torch.where(now > 0, now, 1.0)[:, None, None]
                held = q[page, :, :begin - lo].double() * old[:, None, None]
                all_rows = torch.cat([held, rows], 1) / safe
                whole = torch.sign(all_rows) * torch.floor(all_rows.abs() + 0.5)
                pieces.append((whole.clamp(-127, 127) * now[:, None, None]).permute(1, 0, 2))
                scale[page] = now
                lo += P
            first += b
        got[name], got[name + "_scale"] = torch.cat(pieces), scale
    return got
