"""Plain implementations of a tree decoding step's calls (include/cq_tree.h) by loops in 64 bits and more (numpy).

Whole numbers -- masks, positions, kept paths, next tokens, moved rows and their scales, pages -- are compared exactly;
norm and rotation within the bound that rope() gives.
"""
import numpy as np

from kv_ref import round_away

DEV_TREE, DEV_LOGITS, DEV_KV_PAGE = 0x100, 0x200, 0x80


def tree_plan(kv_len, q_start, parent, T):
    """Masks (uint64), positions and status bits of cq_tree_plan."""
    mask, pos, bits = np.zeros(T, np.uint64), np.full(T, -1, np.int32), 0
    for r in range(len(kv_len)):
        first, n = int(q_start[r]), int(q_start[r + 1]) - int(q_start[r])
        for i in range(n):
            m, depth, j = 0, 0, i
            if n <= 64:
                while True:
                    m |= 1 << j
                    p = int(parent[first + j])
                    if p < -1 or p >= j:
                        bits |= DEV_TREE
                        p = -1
                    if p < 0:
                        break
                    j, depth = p, depth + 1
            else:
                depth = i
            mask[first + i] = m
            at = int(kv_len[r]) - n + depth
            pos[first + i] = at if 0 <= at < 2 ** 31 else -1
    return mask, pos, bits


def rope(x, w, eps, positions, freqs, adjacent, half_step):
    """Norm and rotation of x [T, heads, D] (what the call gets) in long doubles, and a bound on the error of results
    whose type rounds by half_step (relative). With u = 2^-24, per output a cos phi - b sin phi:
      the norm: squares and sums of positive numbers 8 u, halved by the root; mean and eps 0.5 u, the root 2 ulp = 4 u,
        two products 2 u: 10.5 u of the value;
      sine and cosine: the angle in half turns rounds by u of at most pi, each function by 1 ulp = 2 u: 5.2 u;
      the products and their sum: 2 u;
    18 u (|a| + |b|) in all, and the rounding to the result's type (with its smallest subnormal step).
    """
    L = np.longdouble
    x = x.astype(L)
    D, half = x.shape[-1], len(freqs)
    if w is not None:
        x = x * w.astype(L) / np.sqrt((x * x).mean(-1, keepdims=True) + L(np.float32(eps)))
    y, size = x.copy(), np.abs(x)
    phi = positions.astype(L)[:, None] * freqs.astype(L)
    c, s = np.cos(phi)[:, None, :], np.sin(phi)[:, None, :]
    ia = np.arange(0, 2 * half, 2) if adjacent else np.arange(half)
    ib = ia + 1 if adjacent else ia + half
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    bound = 18 * 2.0 ** -24 * size
    return y, bound + half_step * (np.abs(y) + bound) + (2.0 ** -25 if half_step == 2.0 ** -11 else 2.0 ** -149)


def verify(logits, tokens, parent, q_start, temperature, u_accept, u_sample, max_path, draft=None):
    """cq_tree_verify by its definition. Returns count, path, next and status bits."""
    R, V = len(temperature), logits.shape[1]
    count, path, nxt, bits = np.zeros(R, np.int32), np.full((R, max_path), -1, np.int32), np.full(R, -1, np.int32), 0

    def unit(u):
        u = np.float64(u)
        return 0.0 if not u > 0 else min(u, 1 - 2.0 ** -24)

    for r in range(R):
        first, n = int(q_start[r]), int(q_start[r + 1]) - int(q_start[r])
        if n <= 0 or n > 64:
            bits |= DEV_TREE if n > 64 else 0
            continue
        up = []
        for i in range(n):
            p = int(parent[first + i])
            if p < -1 or p >= i:
                bits |= DEV_TREE
                p = -1
            up.append(p)
        t = np.float64(temperature[r])
        greedy = not t >= 2.0 ** -64
        t = min(t, 2.0 ** 64)
        c, kept = 0, [0]
        while True:
            z = logits[first + c].astype(np.float64)
            top = z.max()
            if not np.isfinite(top):                     # NaN among them too: max gives it
                bits |= DEV_LOGITS
                break
            if greedy:
                p = np.zeros(V)
                p[int(z.argmax())] = 1.0
            else:
                p = np.exp((z - top) / t)
                p[p < 2.0 ** -46] = 0.0                  # less than half a unit of 2^-45
                p /= p.sum()
            taken = None
            for j in range(1, n):
                if up[j] != c or len(kept) == max_path:
                    continue
                x = int(tokens[first + j])
                if not 0 <= x < V:
                    continue
                if draft is None or greedy:
                    q = np.zeros(V)
                    q[x] = 1.0
                else:
                    q = np.clip(np.nan_to_num(draft[first + c].astype(np.float64), nan=0.0), 0.0, 1.0)
                if unit(u_accept[first + j]) * q[x] < p[x]:
                    taken = j
                    break
                rest = np.maximum(p - q, 0.0)
                if rest.sum() > 0:
                    p = rest / rest.sum()
            if taken is None:
                cum = np.cumsum(p)
                nxt[r] = min(int((cum <= unit(u_sample[r]) * cum[-1]).sum()), V - 1)
                break
            kept.append(taken)
            c = taken
        count[r] = len(kept)
        path[r, :len(kept)] = kept
    return count, path, nxt, bits


def move(q, scale, table, kv_len, q_start, count, path):
    """cq_kv_move for keys or values: q int8 [pages, H, P, D], scale fp32 [pages, H], both in place. Returns the new
    lengths and status bits."""
    f, P, pages = np.float32, q.shape[2], q.shape[0]
    new_len, bits = [], 0
    for r in range(len(kv_len)):
        n = max(int(q_start[r + 1]) - int(q_start[r]), 0)
        base = int(kv_len[r]) - n
        if n > 64:                                       # no tree: it keeps its tokens
            new_len.append(max(int(kv_len[r]), 0))
            continue
        c = min(max(int(count[r]), 0), n, path.shape[1])
        bits |= DEV_TREE if c != int(count[r]) else 0
        new_len.append(max(base + c, 0))

        def place(i):
            at = base + i
            b = at // P
            page = int(table[r, b]) if at >= 0 and b < table.shape[1] else -1
            return (page, at % P) if 0 <= page < pages else None
        moves = []
        for i in range(c):
            s = int(path[r, i])
            if not 0 <= s < n:
                bits |= DEV_TREE
            elif s != i:
                a, b = place(s), place(i)
                if a is None or b is None:
                    bits |= DEV_KV_PAGE
                else:
                    moves.append((a, b))
        for h in range(q.shape[1]):
            rows = [q[a[0], h, a[1]].copy() for a, _ in moves]
            old = {p: scale[p, h] for m in moves for p in (m[0][0], m[1][0])}
            now = dict(old)
            for (a, _), (b, _) in moves:
                s = old[a]
                now[b] = f(np.nan) if np.isnan(now[b]) or np.isnan(s) else max(now[b], s)

            def ratio(x, s):
                return f(x) / s if s > 0 else f(0)
            for p in {b[0] for _, b in moves}:
                if now[p] != old[p]:
                    q[p, h] = round_away(q[p, h].astype(f) * ratio(old[p], now[p]))
                    scale[p, h] = now[p]
            for row, ((a, _), (b, at)) in zip(rows, moves):
                q[b, h, at] = row if old[a] == now[b] and now[b] > 0 else round_away(row.astype(f) * ratio(old[a], now[b]))
    return np.array(new_len, np.int32), bits


def release(table, old_len, new_len, P, num_pages, capacity):
    """Freed pages and used of cq_kv_release."""
    out, bits, wide = [], 0, table.shape[1]
    for r in range(len(old_len)):
        o, w = int(old_len[r]), int(new_len[r])
        bits |= 0x08 if o < 0 or w < 0 else 0
        a, b = -(-max(w, 0) // P), -(-max(o, 0) // P)
        bits |= 0x10 if b > wide else 0
        for c in range(min(a, wide), min(b, wide)):
            out.append(int(table[r, c]))
    if len(out) > capacity:
        bits |= 0x20
        out = out[:capacity]
    for i, page in enumerate(out):
        if not 0 <= page < num_pages:
            bits |= 0x80
            out[i] = -1
    return np.array(out + [-1] * (capacity - len(out)), np.int32), [len(out), bits]


def random_parents(rng, n, chain=False):
    if chain:
        return list(range(-1, n - 1))
    return [-1] + [int(rng.integers(max(0, i // 3 - 1), i)) for i in range(1, n)]
