"""A step of tree speculative decoding over the 8-bit paged key/value cache, as cases that can be measured: masks and
positions of a tree of drafted tokens, per-head norms and rotation of queries and keys, attention of the tree over the
cache, its verification against the target's probabilities, and the cache put in order afterwards.

`run` computes each in plain torch operations, or, with `own` true, through the library's entry points. `exact`
computes the same from the definitions in 64 bits.

The cache: int8 pages [pages, kv heads, page tokens, head size], one fp32 scale per (page, kv head), for keys and for
values. A request's token i lives in page block_table[r, i // page] at row i % page.

A tree: a request's new tokens in order, each with its parent's index among them (-1: it follows the cache alone).
Token 0 is the last one that was sampled, the others are drafts.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
DEV = "cuda"
EPS = 1e-6
MOST = 64                    # tokens of a tree


# ------------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of 64 requests: fp32 rows of the fused projection, 32 query and 8 key heads of 128
        {"name": "rope_step", "kind": "rope", "from": "f32", "to": "f32", "tokens": 64, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "rot": 128, "adjacent": False, "norm": True, "far": 8191},
        # prompts of 16k tokens: the projections' fp32 rows become bfloat16 queries and keys
        {"name": "rope_prompts", "kind": "rope", "from": "f32", "to": "bf16", "tokens": 16003, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "rot": 128, "adjacent": False, "norm": True, "far": 131071},
        # a chunk in fp16, seven query heads a key head, half of each head turned in adjacent pairs, no norm
        {"name": "rope_partial", "kind": "rope", "from": "f16", "to": "f16", "tokens": 1023, "q_heads": 14,
         "kv_heads": 2, "dim": 64, "rot": 32, "adjacent": True, "norm": False, "far": 4000},
        # one request's tree of 64 tokens
        {"name": "plan_one", "kind": "plan", "requests": 1, "past_min": 999, "past_max": 999, "new_min": 64, "new_max": 64},
        # trees of a large batch
        {"name": "plan_batch", "kind": "plan", "requests": 1024, "past_min": 30, "past_max": 8191, "new_min": 1, "new_max": 64},
        # one user, a wide tree over a short context (fp32)
        {"name": "tree_one", "kind": "attend", "dtype": "f32", "q_heads": 32, "kv_heads": 8, "dim": 64, "page": 16,
         "requests": 1, "past_min": 999, "past_max": 999, "new_min": 60, "new_max": 60},
        # a serving batch: 64 ragged contexts, trees of a few tokens each
        {"name": "tree_batch", "kind": "attend", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "requests": 64, "past_min": 200, "past_max": 8190, "new_min": 3, "new_max": 9},
        # few requests with long contexts and trees of up to 48 tokens (fp16)
        {"name": "tree_long", "kind": "attend", "dtype": "f16", "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64,
         "requests": 4, "past_min": 30000, "past_max": 60000, "new_min": 24, "new_max": 48},
        # five drafts in a row for each of 64 requests, drawn by a draft model whose probabilities are known
        {"name": "verify_chain", "kind": "verify", "vocab": 128256, "requests": 64, "new_min": 6, "new_max": 6,
         "chain": True, "draft": True, "temp": 0.8},
        # one request's tree of the likeliest tokens, no draft probabilities, an odd vocabulary
        {"name": "verify_tree", "kind": "verify", "vocab": 32003, "requests": 1, "new_min": 25, "new_max": 25,
         "chain": False, "draft": False, "temp": 1.0},
        # the accepted paths of 64 trees put in order in one layer's cache, and the pages behind them given back
        {"name": "keep_batch", "kind": "keep", "kv_heads": 8, "dim": 128, "page": 16, "requests": 64, "past_min": 30,
         "past_max": 2000, "new_min": 16, "new_max": 48},
        # the same of many requests, a key head for each of 16 query heads
        {"name": "keep_many", "kind": "keep", "kv_heads": 16, "dim": 128, "page": 32, "requests": 512, "past_min": 3,
         "past_max": 700, "new_min": 32, "new_max": 64},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope", "plan", "attend", "attend", "attend", "verify", "verify", "verify", "keep"])
    heads, dim = rng.choice([1, 2, 3, 4, 8, 8, 16]), rng.choice([64, 128])
    group = rng.choice([1, 2, 4, 4, 5, 7, 8])
    page = rng.choice([16, 16, 32, 64, 128])
    new = _log_int(rng, 2, MOST)
    new_min = rng.randint(1, new)
    if kind == "rope":
        a, b = rng.choice([("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")])
        most = min(16000 * 40 * 128 // (heads * (group + 1) * dim), 60000)
        return {"kind": kind, "from": a, "to": b, "tokens": _log_int(rng, 1, most), "q_heads": heads * group,
                "kv_heads": heads, "dim": dim, "rot": rng.choice([dim, dim, dim // 2, 24]),
                "adjacent": rng.random() < 0.4, "norm": rng.random() < 0.6, "far": _log_int(rng, 10, 1000000)}
    if kind == "verify":
        vocab, draft = _log_int(rng, 300, 200000), rng.random() < 0.5
        chain = draft or rng.random() < 0.3
        new = min(new, 12) if chain else new
        n = _log_int(rng, 1, max(2, min(256, 49000000 // (vocab * new))))
        return {"kind": kind, "vocab": vocab, "requests": n, "new_min": rng.randint(1, new), "new_max": new,
                "chain": chain, "draft": draft, "temp": rng.choice([0.0, 0.5, 0.8, 1.0, 1.3])}
    if kind == "plan":
        past = _log_int(rng, 1, 8000)
        return {"kind": kind, "requests": _log_int(rng, 1, 2048), "past_min": rng.randint(0, past), "past_max": past,
                "new_min": new_min, "new_max": new}
    if kind == "keep":
        past = _log_int(rng, 1, 1500)
        n = _log_int(rng, 1, max(2, min(512, 512 * 16 * 128 * 700 // (heads * dim * (past + 64)))))
        return {"kind": kind, "kv_heads": heads, "dim": dim, "page": page, "requests": n,
                "past_min": rng.randint(0, past), "past_max": past, "new_min": new_min, "new_max": new}
    n = _log_int(rng, 1, 96)
    # the plain form holds a padded score matrix and the cache in fp32
    past = _log_int(rng, 8, max(9, min(60000, 300000 * 8 // (n * heads))))
    while n * heads * group * new * (past + new) * 4 > 4e9:
        past = max(8, past // 2)
    return {"kind": "attend", "dtype": rng.choice(["f32", "f16", "bf16"]), "q_heads": heads * group, "kv_heads": heads,
            "dim": dim, "page": page, "requests": n, "past_min": past // 7 if rng.random() < 0.7 else past,
            "past_max": past, "new_min": new_min, "new_max": new}


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
    past = _spread(case["past_min"], case["past_max"], n, 0.0) if "past_max" in case else [0] * n
    return past, _spread(case["new_min"], case["new_max"], n, 0.37)


def _ceil(a, b):
    return -(-a // b)


def work(case):
    if case["kind"] == "rope":
        values = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": values * (BYTES[case["from"]] + BYTES[case["to"]]) + 4 * case["tokens"], "flops": 10 * values}
    past, new = lengths(case)
    T = sum(new)
    if case["kind"] == "plan":
        return {"bytes": 8 * len(new) + 16 * T, "flops": 0}
    if case["kind"] == "attend":
        row = case["kv_heads"] * case["dim"] * 2
        P = case["page"]
        read = sum((a + b) * row + _ceil(a + b, P) * case["kv_heads"] * 8 for a, b in zip(past, new))
        pairs = sum(b * a + 2 * b for a, b in zip(past, new))          # the past, itself, its parent at least
        return {"bytes": read + T * case["q_heads"] * (2 * case["dim"] * BYTES[case["dtype"]] + 4),
                "flops": 4 * case["dim"] * case["q_heads"] * pairs}
    if case["kind"] == "verify":
        # each request's first row at least; where drafts are taken over, about one more
        rows = len(new) * 2 if case["new_max"] > 1 else len(new)
        values = rows * case["vocab"] * (2 if case["draft"] else 1)
        return {"bytes": 4 * values + 12 * T, "flops": 10 * values}
    row = case["kv_heads"] * (case["dim"] * 2 + 8)
    moved = sum(max(0, _kept(b) - 2) for b in new)
    back = sum(a % case["page"] + _kept(b) for a, b in zip(past, new))
    return {"bytes": 2 * moved * row + back * (5 * row + 8) + 8 * T, "flops": 4 * moved * row + 2 * back * row}


# ----------------------------------------------------------------------------------------------------- inputs
def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _kept(n):
    """Tokens that a verification keeps of n, in the cache's cases."""
    return max(1, min(n // 4, 6))


def _parents(new, chain, gen):
    """int64 [R, most new]: parents of random trees (or chains), breadth first as drafting makes them; -1 for token 0."""
    most = max(new)
    i = torch.arange(most, device=DEV)
    if chain:
        return (i - 1).expand(len(new), most).contiguous()
    # between i / 3 and i - 1, never falling: a tree that widens first
    lo, hi = torch.div(i, 3, rounding_mode="floor"), (i - 1).clamp(min=0)
    u = torch.rand((len(new), most), generator=gen, device=DEV)
    p = lo + (u * (hi - lo + 1)).long().clamp(max=MOST)
    p = torch.minimum(p, hi).cummax(1).values.minimum(hi)
    p[:, 0] = -1
    return p


def _flat(x, new):
    """Rows of a padded [R, most, ...] array one after the other."""
    return torch.cat([x[r, :n] for r, n in enumerate(new)]) if len(new) < 8 else \
        x[torch.arange(x.shape[1], device=DEV)[None, :] < _ints(new)[:, None]]


def _cache(case, pages, gen):
    """Cache contents: normal values at about 36 steps a standard deviation, scales that differ by block."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    out = []
    for _ in range(2):
        x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float16)
        out.append((x * 36.0).round_().clamp_(-127, 127).to(torch.int8))
        out.append(0.022 + 0.012 * torch.rand(shape[:2], generator=gen, device=DEV))
    return {"k": out[0], "v": out[2], "k_scale": out[1], "v_scale": out[3]}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": case}
    if case["kind"] == "rope":
        T, Hq, Hk, D = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        dt = DTYPES[case["from"]]
        rows = torch.randn((T, (Hq + 2 * Hk) * D), generator=gen, device=DEV).mul_(3.0).to(dt)      # q, k, v
        s["q"] = rows[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = rows[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
        s["positions"] = torch.randint(0, case["far"] + 1, (T,), generator=gen, device=DEV, dtype=torch.int32)
        i = torch.arange(case["rot"] // 2, dtype=torch.float64)
        s["freqs"] = (500000.0 ** (-2.0 * i / case["rot"])).to(DEV)
        for name in ("q_norm", "k_norm"):
            s[name] = 1.0 + 0.2 * torch.randn(D, generator=gen, device=DEV) if case["norm"] else None
        return s
    past, new = lengths(case)
    n_t, past_t = _ints(new, torch.int64), _ints(past, torch.int64)
    s["new"] = n_t
    q_start = torch.cat([torch.zeros_like(n_t[:1]), n_t.cumsum(0)])
    s["q_start"], s["kv_len"] = q_start.to(torch.int32), (past_t + n_t).to(torch.int32)
    if case["kind"] != "keep":
        parent = _parents(new, case.get("chain", False), gen)
        s["parent"] = _flat(parent, new).to(torch.int32)
    if case["kind"] == "plan":
        return s
    if case["kind"] == "verify":
        return _prepare_verify(case, s, new, gen)
    P = case["page"]
    blocks = [_ceil(a + b, P) for a, b in zip(past, new)]
    pages, wide = sum(blocks) + 3, max(blocks) + 1
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    b_t = _ints(blocks, torch.int64)
    col = torch.arange(wide, device=DEV)[None, :]
    s["table"] = torch.where(col < b_t[:, None], order[((b_t.cumsum(0) - b_t)[:, None] + col).clamp(max=pages - 1)], -1)
    s["pages"], s["old_len"] = pages, s["kv_len"]
    s.update(_cache(case, pages, gen))
    if case["kind"] == "keep":
        # accepted paths: token 0, perhaps its first child, then tokens from behind the places they go to (behind the
        # pages, where those are two: a pass then leaves what the next one reads as it was)
        path, count = torch.full((len(new), 8), -1, dtype=torch.int32), []
        u = torch.rand((len(new), MOST), generator=gen, device=DEV).cpu()
        for r, n in enumerate(new):
            c = _kept(n)
            ids = [0] + ([1] if c > 1 else [])
            last = (past[r] + c - 1) // P
            begin = c if past[r] // P == last else max(c, (last + 1) * P - past[r])
            left = u[r, :max(n - begin, 0)].argsort()[:c - len(ids)]
            ids += sorted((left + begin).tolist())
            path[r, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
            count.append(len(ids))
        s["path"], s["count"] = path.to(DEV), _ints(count)
        # what is read back: the rows that are kept, from the beginning of the first page that may change
        back = [s["table"][r, t // P].long() * P + t % P for r, (a, c) in enumerate(zip(past, count))
                for t in [torch.arange(a // P * P, a + c, device=DEV)]]
        s["back"] = torch.cat(back)
        return s
    s["dense"] = parent                                     # padded, for the plain form's masks
    s["q"] = (2.0 * torch.randn((sum(new), case["q_heads"], case["dim"]), generator=gen, device=DEV)).to(DTYPES[case["dtype"]])
    s["max_new"], s["max_kv"] = max(new), max(a + b for a, b in zip(past, new))
    s["mask"], _ = _plan(s)
    s["ws"] = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)   # scratch that a program keeps, zeroed once
    return s


def _prepare_verify(case, s, new, gen):
    T, V, t = sum(new), case["vocab"], case["temp"]
    # a few likely tokens above a long tail, as a language model's logits lie
    z = torch.randn((T, V), generator=gen, device=DEV).mul_(4.0)
    s["logits"] = z
    s["temperature"] = torch.full((len(new),), t, device=DEV)
    s["u_accept"] = torch.rand(T, generator=gen, device=DEV)
    s["u_sample"] = torch.rand(len(new), generator=gen, device=DEV)
    s["max_path"] = max(new)
    parent, first = s["parent"].long(), s["q_start"].long()[:-1].repeat_interleave(s["new"])
    at = first + parent.clamp(min=0)                         # the parent's row
    tokens = torch.randint(0, V, (T,), generator=gen, device=DEV)
    if case["draft"]:
        # a draft model that is right about most of it; each draft is drawn from its parent's row
        y = torch.randn((T, V), generator=gen, device=DEV).mul_(0.7).add_(z)
        y = torch.softmax(y.div_(t if t > 0 else 1.0), -1)
        s["draft"] = y
        for c0 in range(0, T, 64):
            rows = y[at[c0:c0 + 64]].cumsum_(-1)
            u = torch.rand((rows.shape[0], 1), generator=gen, device=DEV) * rows[:, -1:]
            tokens[c0:c0 + 64] = torch.searchsorted(rows, u).squeeze(1).clamp(max=V - 1)
    else:
        s["draft"] = None
        # the k-th child of a node is its k-th likeliest token
        i = torch.arange(T, device=DEV)
        nth = ((at[None, :] == at[:, None]) & (i[None, :] < i[:, None]) & (parent >= 0)[None, :]).sum(1)
        best = torch.topk(z, min(MOST, V), dim=-1).indices
        tokens = best[at, nth.clamp(max=best.shape[1] - 1)]
    s["tokens"] = tokens.to(torch.int32)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _run_rope(s):
    c = s["case"]
    half, rot = c["rot"] // 2, c["rot"]
    turn = s["positions"].double()[:, None] * s["freqs"]                                   # angles in 64 bits
    cos, sin = turn.cos().float()[:, None, :], turn.sin().float()[:, None, :]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["adjacent"] else (x[..., :half], x[..., half:rot])
        a2, b2 = a * cos - b * sin, b * cos + a * sin
        y = torch.stack((a2, b2), -1).flatten(-2) if c["adjacent"] else torch.cat((a2, b2), -1)
        return torch.cat((y, x[..., rot:]), -1).to(DTYPES[c["to"]])

    return {"q": one(s["q"], s["q_norm"]), "k": one(s["k"], s["k_norm"])}


def _plan(s):
    """Masks (bit j: token j of the request is the token itself or an ancestor) and positions."""
    parent, start = s["parent"].long(), s["q_start"].long()
    n = start[1:] - start[:-1]
    first = start[:-1].repeat_interleave(n)
    t = torch.arange(parent.shape[0], device=DEV)
    mask, depth = torch.zeros_like(parent), torch.zeros_like(parent) - 1
    here = t - first
    for _ in range(MOST):                                    # up one generation at a time
        on = here >= 0
        mask = mask | torch.where(on, torch.ones_like(mask) << here.clamp(min=0), 0)
        depth = depth + on
        here = torch.where(on, parent[first + here.clamp(min=0)], -1)
    base = (s["kv_len"].long() - n).repeat_interleave(n)
    return mask, (base + depth).to(torch.int32)


def _run_plan(s):
    mask, positions = _plan(s)
    return {"mask": mask, "positions": positions}


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
    j = torch.arange(L, device=DEV) - (kv - n)[:, None]  # [R, L]: place among the new tokens
    bit = (s["mask"][at][:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1
    see = (j < 0)[:, None, :] | ((j < n[:, None])[:, None, :] & (bit != 0))
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


def _run_verify(s):
    """All requests side by side, one drafted token after the other; probabilities in 64 bits."""
    start, parent, tokens = s["q_start"].long()[:-1], s["parent"].long(), s["tokens"].long()
    R, V, T = start.shape[0], s["logits"].shape[1], parent.shape[0]
    r_ = torch.arange(R, device=DEV)
    temp = s["temperature"].double()
    greedy = temp <= 0

    def target(rows):
        z = s["logits"][rows].double()
        best = torch.zeros_like(z).scatter_(1, z.argmax(1, keepdim=True), 1.0)
        p = ((z - z.amax(1, keepdim=True)) / torch.where(greedy, 1.0, temp)[:, None]).exp()
        return torch.where(greedy[:, None], best, p / p.sum(1, keepdim=True))

    node = torch.zeros_like(start)
    count = torch.ones_like(start)
    path = torch.full((R, s["max_path"]), -1, dtype=torch.int64, device=DEV)
    path[:, 0] = 0
    p = target(start)
    for i in range(1, s["max_path"]):                    # a parent comes before its children
        at = (start + i).clamp(max=T - 1)
        child = (i < s["new"]) & (parent[at] == node)
        x = tokens[at]
        if s["draft"] is None:
            q = torch.zeros_like(p).scatter_(1, x[:, None], 1.0)
        else:
            q = s["draft"][start + node].double()
            q = torch.where(greedy[:, None], torch.zeros_like(q).scatter_(1, x[:, None], 1.0), q)
        take = child & (s["u_accept"][at].double() * q[r_, x] < p[r_, x])
        rest = (p - q).clamp_(min=0.0)
        total = rest.sum(1, keepdim=True)
        rest = torch.where(total > 0, rest / torch.where(total > 0, total, 1.0), p)
        p = torch.where((child & ~take)[:, None], rest, p)
        node = torch.where(take, i, node)
        p = torch.where(take[:, None], target(start + node), p)
        path[r_, torch.where(take, count, 0)] = torch.where(take, i, path[:, 0])
        count = count + take
    c = p.cumsum(1)
    token = (c <= s["u_sample"].double()[:, None] * c[:, -1:]).sum(1).clamp(max=V - 1)
    return {"count": count.to(torch.int32), "path": path.to(torch.int32), "next": token.to(torch.int32)}


def _round_away(x):
    t = x.trunc()
    return t + torch.sign(x) * ((x - t).abs() >= 0.5)


def _move(q, scale, table, past, count, path):
    """Rows past + path[i] of each request to past + i. q: pages, scale: [pages, heads], both in place."""
    P = q.shape[2]
    i = torch.arange(path.shape[1], device=DEV)[None, :].expand_as(path)
    on = (i < count[:, None]) & (path != i)
    r = torch.arange(path.shape[0], device=DEV)[:, None].expand_as(path)[on]
    src, dst = (past[:, None] + path)[on], (past[:, None] + i)[on]
    ps, os_ = table[r, torch.div(src, P, rounding_mode="floor")], src % P
    pd, od = table[r, torch.div(dst, P, rounding_mode="floor")], dst % P
    rows, s_src = q[ps, :, os_].float(), scale[ps]
    now = scale.clone().index_reduce_(0, pd, s_src, "amax")
    hit = torch.unique(pd)
    held = q[hit].float()
    ratio = torch.where(now[hit] > 0, scale[hit] / now[hit], 0.0)
    q[hit] = _round_away(held * ratio[:, :, None, None]).to(torch.int8)
    ratio = torch.where(now[pd] > 0, s_src / now[pd], 0.0)
    q[pd, :, od] = _round_away(rows * ratio[:, :, None]).to(torch.int8)
    scale.copy_(now)


def _read(q, scale, slots):
    P = q.shape[2]
    page, off = torch.div(slots, P, rounding_mode="floor"), slots % P
    return q[page, :, off].float() * scale[page][:, :, None]


def _run_keep(s):
    P = s["case"]["page"]
    table, count, path = s["table"].long(), s["count"].long(), s["path"].long()
    old = s["kv_len"].long()
    past = old - s["new"]
    _move(s["k"], s["k_scale"], table, past, count, path)
    _move(s["v"], s["v_scale"], table, past, count, path)
    now = past + count
    have, left = torch.div(old + P - 1, P, rounding_mode="floor"), torch.div(now + P - 1, P, rounding_mode="floor")
    col = torch.arange(table.shape[1], device=DEV)[None, :]
    gone = (col >= left[:, None]) & (col < have[:, None])
    freed = torch.full((s["new"].shape[0] * (_ceil(MOST, P) + 1),), -1, dtype=torch.int32, device=DEV)
    at = gone.flatten().cumsum(0) - 1
    freed[torch.where(gone.flatten(), at, freed.shape[0] - 1)] = torch.where(gone, s["table"], -1).flatten()
    return {"k": _read(s["k"], s["k_scale"], s["back"]), "v": _read(s["v"], s["v_scale"], s["back"]),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"], "len": now.to(torch.int32),
            "freed": torch.where(torch.arange(freed.shape[0], device=DEV) < gone.sum(), freed, -1),
            "pages": gone.sum().to(torch.int32)}


# ------------------------------------------------------------------------------------------------------- runs
def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(state, kind)
    return {"rope": _run_rope, "plan": _run_plan, "attend": _run_attend, "verify": _run_verify, "keep": _run_keep}[kind](state)


def _own(s, kind):
    from gemm_gguf_block_gb300 import cq
    c = s["case"]
    if kind == "rope":
        q, k = cq.qk_rope_t(s["q"], s["k"], s["positions"], s["freqs"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS,
                            adjacent=c["adjacent"], dtype=DTYPES[c["to"]])
        return {"q": q, "k": k}
    if kind == "plan":
        mask, positions = cq.tree_plan_t(s["kv_len"], s["q_start"], s["parent"])
        return {"mask": mask, "positions": positions}
    if kind == "verify":
        count, path, token = cq.tree_verify_t(s["logits"], s["tokens"], s["parent"], s["q_start"], s["temperature"],
                                              s["u_accept"], s["u_sample"], s["max_path"], draft=s["draft"])
        return {"count": count, "path": path, "next": token}
    cache = s.get("cache")
    if cache is None:                                    # the object that a program makes when it allocates the pages
        cache = s["cache"] = cq.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if kind == "attend":
        out, lse = cq.attn_tree_t(s["q"], cache, s["table"], s["kv_len"], s["q_start"], s["mask"], s["max_new"], ws=s["ws"])
        return {"out": out, "lse": lse}
    now = cq.kv_move_t(cache, s["table"], s["kv_len"], s["q_start"], s["count"], s["path"])
    most = s["new"].shape[0] * (_ceil(MOST, c["page"]) + 1)
    freed, used = cq.kv_release_t(s["table"], s["kv_len"], now, c["page"], s["pages"], most)
    k, v = cq.kv_read_t(cache, s["back"])
    return {"k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"], "len": now, "freed": freed, "pages": used[0]}


# ------------------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    if case["kind"] in ("plan", "verify"):
        return None                                      # whole numbers only
    s = prepare(case, seed)
    if case["kind"] == "rope":
        return _exact_rope(case, s)
    past, new = lengths(case)
    if case["kind"] == "keep":
        return _exact_keep(case, s, past)
    if sum(b * (a + b) for a, b in zip(past, new)) * case["q_heads"] * case["dim"] > 4e12:
        return None
    P, H, D = case["page"], case["kv_heads"], case["dim"]
    G = case["q_heads"] // H
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    parents = s["dense"].tolist()
    first = 0
    for r, (a, b) in enumerate(zip(past, new)):
        see = torch.zeros((b, a + b), dtype=torch.bool)
        see[:, :a] = True
        for t in range(b):
            up = t
            while up >= 0:
                see[t, a + up] = True
                up = parents[r][up]
        hide = ~see.to(DEV)
        ids = s["table"][r, :_ceil(a + b, P)].long()
        for h in range(H):
            k = (s["k"][ids, h].double() * s["k_scale"][ids, h].double()[:, None, None]).reshape(-1, D)[:a + b]
            v = (s["v"][ids, h].double() * s["v_scale"][ids, h].double()[:, None, None]).reshape(-1, D)[:a + b]
            q = s["q"][first:first + b, h * G:(h + 1) * G].double()
            z = (q.reshape(-1, D) @ k.t()).view(b, G, a + b) / math.sqrt(D)
            z.masked_fill_(hide[:, None, :], -math.inf)
            lse[first:first + b, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
            out[first:first + b, h * G:(h + 1) * G] = torch.softmax(z, -1) @ v
        first += b
    return {"out": out, "lse": lse}


def _exact_rope(case, s):
    rot, D = case["rot"], case["dim"]
    d = torch.arange(rot, device=DEV)
    pair = d // 2 if case["adjacent"] else d % (rot // 2)
    other = d ^ 1 if case["adjacent"] else (d + rot // 2) % rot
    lead = d % 2 == 0 if case["adjacent"] else d < rot // 2
    sign = torch.where(lead, -1.0, 1.0).double()
    got = {}
    for name in ("q", "k"):
        x, w = s[name].double(), s[name + "_norm"]
        if w is not None:
            x = x / ((x ** 2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
        y = x.clone()
        for t0 in range(0, x.shape[0], 2048):
            phi = (s["positions"][t0:t0 + 2048].double()[:, None] * s["freqs"][pair])[:, None, :]
            part = x[t0:t0 + 2048]
            y[t0:t0 + 2048, :, :rot] = part[..., :rot] * phi.cos() + sign * part[..., other] * phi.sin()
        got[name] = y
    return got


def _exact_keep(case, s, past):
    P, D = case["page"], case["dim"]
    count, path, table = s["count"].tolist(), s["path"].tolist(), s["table"].tolist()
    got, back = {"len": None, "freed": None, "pages": None}, s["back"].cpu()
    for name in ("k", "v"):
        q, scale = s[name].cpu(), s[name + "_scale"].double().cpu()
        now, moves = scale.clone(), []
        for r, a in enumerate(past):
            for i in range(count[r]):
                if path[r][i] != i:
                    src, dst = a + path[r][i], a + i
                    ps, pd = table[r][src // P], table[r][dst // P]
                    moves.append((q[ps, :, src % P].double() * scale[ps][:, None], pd, dst % P))
                    now[pd] = torch.maximum(now[pd], scale[ps])
        new_q = q.clone()
        for pd in {m[1] for m in moves}:
            x = q[pd].double() * (scale[pd] / now[pd])[:, None, None]
            new_q[pd] = (torch.sign(x) * torch.floor(x.abs() + 0.5)).to(torch.int8)
        for row, pd, od in moves:
            x = row / now[pd][:, None]
            new_q[pd, :, od] = (torch.sign(x) * torch.floor(x.abs() + 0.5)).to(torch.int8)
        page, off = torch.div(back, P, rounding_mode="floor"), back % P
        got[name], got[name + "_scale"] = new_q[page, :, off].double() * now[page][:, :, None], now
    return got
