"""Plain implementations of the cache and attention calls in 64 bits (numpy), and the error bounds of the results.

The stored integers and scales follow the fp32 rule of include/cq_kv.h and are compared exactly; attention is compared
with its formula in 64 bits.
"""
import numpy as np


def plan(past, new, table, free, P, num_pages, T):
    """cq_kv_plan by loops. Returns table, kv_len, q_start, slots, positions, used."""
    R, wide = table.shape
    table = table.copy()
    bits = taken = 0
    q_start, slots, pos_out, kv_len = [0], [], [], []
    for r in range(R):
        a, b = int(past[r]), int(new[r])
        if a < 0 or b < 0:
            bits |= 0x08
        a, b = max(a, 0), max(b, 0)
        have, total = -(-a // P), -(-(a + b) // P)
        if total > wide:
            bits |= 0x10
        kv_len.append(min(a + b, wide * P))
        pages = {}
        for c in range(min(have, wide), min(total, wide)):
            if taken < len(free):
                page = int(free[taken])
                taken += 1
                if not 0 <= page < num_pages:
                    bits |= 0x80
                    page = -1
            else:
                bits |= 0x20
                page = -1
            table[r, c] = pages[c] = page
        for t in range(b):
            if len(slots) == T:
                bits |= 0x40
                break
            p, c = a + t, (a + t) // P
            page = -1
            if c < wide:
                page = pages[c] if c in pages else int(table[r, c])
                if not 0 <= page < num_pages:
                    if c not in pages:
                        bits |= 0x80
                    page = -1
            slots.append(page * P + p % P if page >= 0 else -1)
            pos_out.append(p)
        q_start.append(len(slots))
    pad = T - len(slots)
    return (table, np.array(kv_len, np.int32), np.array(q_start, np.int32), np.array(slots + [-1] * pad, np.int64),
            np.array(pos_out + [-1] * pad, np.int32), np.array([taken, bits], np.int32))


def round_away(x):
    t = np.trunc(x)
    return t + np.sign(x) * (np.abs(x - t) >= 0.5)


def append(q, scale, x, slots):
    """cq_kv_append for keys or values: q int8 [pages, H, P, D], scale fp32 [pages, H] in place; x fp32 [T, H, D]."""
    P = q.shape[2]
    f = np.float32
    t = 0
    while t < len(slots):
        if slots[t] < 0 or slots[t] // P >= q.shape[0]:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == slots[t] + n and slots[t + n] // P == slots[t] // P:
            n += 1
        page, off = slots[t] // P, slots[t] % P
        for h in range(q.shape[1]):
            rows = x[t:t + n, h].astype(f)
            old = f(0) if off == 0 else scale[page, h]
            if not np.isfinite(rows).all() or np.isnan(old):
                q[page, h, :off + n] = 0
                scale[page, h] = np.nan
                continue
            want = f(np.abs(rows).max() / f(127))
            s = max(old, want if want >= f(2.0 ** -126) else f(0))
            if s != old and off:
                q[page, h, :off] = round_away(q[page, h, :off].astype(f) * (f(old) / s if s > 0 else f(0)))
            inv = f(1) / s if s > 0 else f(0)
            q[page, h, off:off + n] = np.clip(round_away(rows * inv), -127, 127)
            scale[page, h] = s
        t += n


def attend(q, k, v, ks, vs, table, kv_len, q_start, scale, causal, window, dtype):
    """Attention in 64 bits. q [T, Hq, D] (the values that the call gets), k, v int8 pages, ks, vs scales.
    Returns out, lse, and bounds on the errors of both for results of `dtype` ("f32", "f16", "bf16").

    The bounds, per output: with A = max_j scale * sum_d |q_d k_jd|, n keys, p the probabilities,
      a score is off by at most e_s = 2^-18 A: fp32 queries are taken to 22 bits, products are summed in fp32 in
        at most D/16 steps of 16 truncating additions, and the scale and logarithm factors round a few times;
      so the sum of p |v| moves by 2 e_s of itself, by (n / 16 + 64) 2^-23 through exponentials and fp32 sums, and
        by 2^-11 through probabilities rounded to binary16 (16-bit types);
      the result is rounded to its type.
    """
    T, Hq, D = q.shape
    pages, H, P, _ = k.shape
    G = Hq // H
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    e_out, e_lse = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    q = q.astype(np.float64)
    for r in range(len(kv_len)):
        first, last = int(q_start[r]), int(q_start[r + 1])
        n, kv = last - first, int(kv_len[r])
        if n <= 0 or kv <= 0:
            continue
        ids = table[r, :-(-kv // P)]
        good = (ids >= 0) & (ids < pages)
        at = np.where(good, ids, 0)
        j = np.arange(kv)
        i = kv - n + np.arange(n)
        see = np.repeat(good, P)[:kv][None, :] & (j[None, :] >= 0)
        see = np.broadcast_to(see, (n, kv)).copy()
        if causal:
            see &= j[None, :] <= i[:, None]
        if window > 0:
            see &= j[None, :] > i[:, None] - window
        for h in range(H):
            kk = (k[at, h].astype(np.float64) * ks[at, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:kv]
            vv = (v[at, h].astype(np.float64) * vs[at, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:kv]
            kept = see.any(0)
            for g in range(G):
                qq = q[first:last, h * G + g]
                z = np.full((n, kv), -np.inf)
                z[:, kept] = scale * (qq @ kk[kept].T)
                z = np.where(see, z, -np.inf)
                top = z.max(1)
                ok = top > -np.inf
                e = np.where(see, np.exp(z - np.where(ok, top, 0.0)[:, None]), 0.0)
                tot = e.sum(1)
                p = e / np.where(ok, tot, 1.0)[:, None]
                o = p[:, kept] @ vv[kept]
                av = p[:, kept] @ np.abs(vv[kept])
                A = (abs(scale) * (np.abs(qq) @ np.abs(kk[kept]).T) * see[:, kept]).max(1, initial=0.0)
                with np.errstate(divide="ignore"):
                    ll = np.where(ok, np.where(ok, top, 0.0) + np.log(np.where(ok, tot, 1.0)), -np.inf)
                es = 2.0 ** -18 * A + (kv / 16 + 64) * 2.0 ** -23
                rel = 2.0 * es + (0.0 if dtype == "f32" else 2.0 ** -11)
                half = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
                out[first:last, h * G + g] = o
                lse[first:last, h * G + g] = ll
                e_out[first:last, h * G + g] = rel[:, None] * av + half * np.abs(o) + 2.0 ** -24 * (dtype == "f16") + 1e-37
                e_lse[first:last, h * G + g] = es + 2.0 ** -22 * np.abs(np.where(ok, ll, 0.0))
    return out, lse, e_out, e_lse
