"""One attention layer on the library's calls: quantised projections, the 8-bit paged cache and attention over it.

``AttentionBlock`` keeps the weights (any format that cq_gemm takes), the cache, the block table and the workspace of
a layer; ``step`` takes the new tokens of a set of requests -- prompts, chunks of them, drafts or single tokens, in
one call -- through

    cq_quantize_act -> cq_gemv / cq_gemm (q, k, v in one matrix) -> cq_kv_plan -> [cq_qk_rope] -> cq_kv_append
    -> cq_attn_paged -> cq_quantize_act -> cq_gemv / cq_gemm (output projection).

With ``freqs`` (or norms) queries and keys are normed by head and turned by their positions; without them they are used
as they are projected. Where the new tokens are trees of drafts (``parents``), cq_tree_plan gives their masks and
positions and cq_attn_tree attends; ``keep`` moves the rows of the accepted ones together (cq_kv_move) and gives the
pages behind them back (cq_kv_release), ``end`` a whole request's. It shows the calls together and is no scheduler:
the lengths are the host's and go to the device with every step.

    python -m gemm_gguf_block_gb300.attn_block      two prompts, then single tokens, checked against 64 bits; then
                                                    trees of drafts through an LM head and their verification
"""
from __future__ import annotations

from . import cq


class AttentionBlock:
    """wqkv: [(q_heads + 2 kv_heads) * head_dim] rows of weight blocks, wo: [hidden] rows of q_heads * head_dim.
    freqs (fp64 [rot / 2]), q_norm, k_norm (fp32 [head_dim]), eps, adjacent: as cq.qk_rope_t takes them; without any of the
    first three the projections are used as they are."""

    def __init__(self, wqkv, wo, fmt: int, hidden: int, q_heads: int, kv_heads: int, head_dim: int, *, requests: int,
                 num_pages: int, page_size: int = 16, freqs=None, q_norm=None, k_norm=None, eps: float = 1e-6,
                 adjacent: bool = False):
        import torch
        self.wqkv, self.wo, self.fmt, self.hidden = wqkv, wo, fmt, hidden
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        dev = wqkv.device
        self.cache = cq.KVCache.empty(num_pages, kv_heads, page_size, head_dim, dev)
        self.table = torch.full((requests, num_pages), -1, dtype=torch.int32, device=dev)
        self.free = torch.arange(num_pages, dtype=torch.int32, device=dev)     # pages are taken from the front
        self.taken = 0
        self.past = [0] * requests                                             # the host's copy of the lengths
        self.open = False                                                      # whether the last step may still be kept
        self.ended = set()                                                     # requests that ended since
        self.ws = cq.attn_workspace_t(q_heads, kv_heads, head_dim, dev)
        self.mask = None
        self.rope = None if freqs is None and q_norm is None and k_norm is None else \
            dict(freqs=freqs, q_norm=q_norm, k_norm=k_norm, eps=eps, adjacent=adjacent)

    def _product(self, w, x, rows_in: int):
        xq = cq.quantize_act_t(x, cq.ACT_FOR[self.fmt])
        return (cq.gemv_t if x.shape[0] <= 16 else cq.gemm_t)(w, xq, self.fmt, rows_in)

    def step(self, x, new, parents=None):
        """x: fp32 [T, hidden], the new tokens of all requests in order; new: their number for each request (0 for a
        request that takes no part; T in all, at least 1). parents: int32 [T] on the device where the new tokens are trees
        (requests of more than cq.TREE_MAX are prompts all the same). Returns fp32 [T, hidden]."""
        import torch
        new = [int(n) for n in new]
        if len(new) != len(self.past) or min(new, default=0) < 0 or sum(new) < 1 or x.shape != (sum(new), self.hidden):
            raise cq.CqError("AttentionBlock.step", cq.ERR_SHAPE)
        P, dev = self.cache.page_size, x.device
        need = sum(-(-(a + b) // P) - -(-a // P) for a, b in zip(self.past, new))
        if self.taken + need > self.free.shape[0]:
            raise cq.CqError("AttentionBlock.step", cq.ERR_WORKSPACE)
        past_t = torch.tensor(self.past, dtype=torch.int32, device=dev)
        new_t = torch.tensor(new, dtype=torch.int32, device=dev)
        kv_len, q_start, slots, self.positions, self.used = cq.kv_plan_t(
            past_t, new_t, self.table, self.free[self.taken:], P, self.cache.num_pages, x.shape[0])
        self.mask = None
        if parents is not None:
            self.mask, self.positions = cq.tree_plan_t(kv_len, q_start, parents)
        width, kv_width = self.q_heads * self.head_dim, self.kv_heads * self.head_dim
        qkv = self._product(self.wqkv, x, self.hidden)
        q = qkv[:, :width].unflatten(1, (self.q_heads, self.head_dim))
        k = qkv[:, width:width + kv_width].unflatten(1, (self.kv_heads, self.head_dim))
        if self.rope is not None:
            cq.qk_rope_t(q, k, self.positions, q_out=q, k_out=k, **self.rope)              # in place
        cq.kv_append_t(self.cache, k, qkv[:, width + kv_width:], slots)
        after = [a + b for a, b in zip(self.past, new)]
        if parents is None:
            self.attended, _ = cq.attn_paged_t(q, self.cache, self.table, kv_len, q_start, max(new), max(after), ws=self.ws,
                                               lse=None)
        else:
            self.attended, _ = cq.attn_tree_t(q, self.cache, self.table, kv_len, q_start, self.mask, max(new), ws=self.ws,
                                              lse=None)
        y = self._product(self.wo, self.attended.view(x.shape[0], width), width)
        self.taken += need
        self.past, self.q, self.slots = after, q, slots
        self.kv_len, self.q_start, self.open, self.ended = kv_len, q_start, True, set()
        return y

    def keep(self, count, path):
        """After a step: the tokens path[r][0 .. count[r]) of each request's new ones stay (int32 [R], [R, most] on the
        device, as cq.tree_verify_t gives them; count 0 for a request that had none new), the others go, with the pages
        that nothing is left in. A request of more than cq.TREE_MAX new tokens keeps them all, whatever its count.
        Once a step: what it has moved is not where the path says any more. A request that ended since the step keeps
        nothing, whatever its count: its pages may be another's by now."""
        import torch
        if not self.open:
            raise cq.CqError("AttentionBlock.keep", cq.ERR_INVALID_ARG)
        here = None
        if self.ended:
            if count.dtype != torch.int32 or count.shape != (len(self.past),) or count.device != self.table.device:
                raise cq.CqError("AttentionBlock.keep", cq.ERR_SHAPE)
            here = torch.tensor([int(r not in self.ended) for r in range(len(self.past))], dtype=torch.int32,
                                device=self.table.device)
            count = count * here                         # 0: none of its rows is read or written
        new_len = cq.kv_move_t(self.cache, self.table, self.kv_len, self.q_start, count, path)
        self.open = False
        if here is not None:
            new_len = new_len * here
        self._give_back(new_len, new_len.tolist())       # the one read of the step: the host's lengths

    def end(self, r: int):
        """Request r ends: its pages are given back, its place is free for another one. Between a step and its keep() too
        (its accepted tokens hold the text's end, say): the others' tokens are kept as if it were not there."""
        import torch
        if not 0 <= r < len(self.past):
            raise cq.CqError("AttentionBlock.end", cq.ERR_SHAPE)
        left = [0 if i == r else n for i, n in enumerate(self.past)]
        self.ended.add(r)
        self._give_back(torch.tensor(left, dtype=torch.int32, device=self.table.device), left)

    def _give_back(self, new_len, left):
        import torch
        P = self.cache.page_size
        n = sum(-(-a // P) - -(-b // P) for a, b in zip(self.past, left))
        if n > 0:
            old = torch.tensor(self.past, dtype=torch.int32, device=self.table.device)
            freed, _ = cq.kv_release_t(self.table, old, new_len, P, self.cache.num_pages, n)
            self.taken -= n
            self.free[self.taken:self.taken + n] = freed  # in front of the pages that were never taken
        self.past = left

    def dense(self, r: int, first: int, n: int):
        """What the last step's attention of request r's n tokens (from row `first` of x) is in 64 bits, from the
        cache read back: [n, q_heads, head_dim]."""
        import torch
        P, kv = self.cache.page_size, self.past[r]
        pos = torch.arange(kv, device=self.table.device)
        slots = self.table[r, pos // P].long() * P + pos % P
        k, v = (t.double().repeat_interleave(self.q_heads // self.kv_heads, 1) for t in cq.kv_read_t(self.cache, slots))
        q = self.q[first:first + n].double()
        z = torch.einsum("nhd,khd->hnk", q, k) * self.head_dim ** -0.5
        hide = pos[None, :] > pos[kv - n:, None]
        if self.mask is not None and n <= cq.TREE_MAX:
            hide[:, kv - n:] = (self.mask[first:first + n, None] >> torch.arange(n, device=pos.device)) & 1 == 0
        return torch.einsum("hnk,khd->nhd", z.masked_fill(hide, -float("inf")).softmax(-1), v)


def demo(hidden=2048, q_heads=32, kv_heads=8, head_dim=64, prompts=(700, 45), steps=20, fmt="q8_0", seed=0):
    """Two prompts in one call, then single tokens. Returns the block and the largest relative error (2-norm) of its
    attention against 64 bits over all calls."""
    import numpy as np
    import torch

    from . import synth
    rng = np.random.default_rng(seed)
    weights = [torch.from_numpy(np.ascontiguousarray(synth.GEN[fmt](rng, n, k))).cuda()
               for n, k in (((q_heads + 2 * kv_heads) * head_dim, hidden), (hidden, q_heads * head_dim))]
    pages = sum(-(-(n + steps) // 16) for n in prompts)
    block = AttentionBlock(*weights, cq.FMT[fmt], hidden, q_heads, kv_heads, head_dim, requests=len(prompts), num_pages=pages)
    probe = torch.from_numpy(rng.standard_normal((16, hidden)).astype(np.float32)).cuda()
    size = 2.0 / block._product(block.wqkv, probe, hidden).std().item()        # queries and keys of about 2
    worst = 0.0
    for new in [list(prompts)] + [[1] * len(prompts)] * steps:
        x = torch.from_numpy(rng.standard_normal((sum(new), hidden)).astype(np.float32)).cuda() * size
        y = block.step(x, new)
        assert torch.isfinite(y).all()
        first = 0
        for r, n in enumerate(new):
            want = block.dense(r, first, n)
            worst = max(worst, ((block.attended[first:first + n].double() - want).norm() / want.norm()).item())
            first += n
    return block, worst


def tree_demo(hidden=1024, q_heads=16, kv_heads=4, head_dim=64, vocab=32000, prompts=(300, 45), steps=12, drafts=15,
              temperature=0.7, fmt="q8_0", seed=0):
    """Prompts, then steps of tree decoding: each request's last token and a tree of drafts through the layer (norms and
    rotation among it) and an LM head, verified, the accepted ones kept, the last request ended. Embeddings and drafts are
    random, the drafts among the head's likely tokens for the parent, so that some are kept. Returns the block, the largest
    relative error (2-norm) of its attention against 64 bits, and the kept tokens a step and request."""
    import numpy as np
    import torch

    from . import synth
    rng = np.random.default_rng(seed)
    R, dev = len(prompts), "cuda"
    weights = [torch.from_numpy(np.ascontiguousarray(synth.GEN[fmt](rng, n, k))).cuda()
               for n, k in (((q_heads + 2 * kv_heads) * head_dim, hidden), (hidden, q_heads * head_dim), (vocab, hidden))]
    pages = sum(-(-(n + (steps + 1) * (drafts + 1)) // 16) for n in prompts)
    freqs = 10000.0 ** (-torch.arange(head_dim // 2, dtype=torch.float64, device=dev) * 2.0 / head_dim)
    norms = [torch.from_numpy((1.0 + 0.2 * rng.standard_normal(head_dim)).astype(np.float32)).cuda() for _ in range(2)]
    block = AttentionBlock(*weights[:2], cq.FMT[fmt], hidden, q_heads, kv_heads, head_dim, requests=R, num_pages=pages,
                           freqs=freqs, q_norm=norms[0], k_norm=norms[1])
    table = torch.from_numpy(rng.standard_normal((vocab, hidden)).astype(np.float32)).cuda()          # embeddings

    def checked(x, new, parents=None):
        y = block.step(x, new, parents)
        first, worst = 0, 0.0
        for r, n in enumerate(new):
            want = block.dense(r, first, n)
            worst = max(worst, ((block.attended[first:first + n].double() - want).norm() / want.norm()).item())
            first += n
        logits = block._product(weights[2], x + y * (x.norm() / y.norm()), hidden)       # around the layer, and the head
        return logits * (5.0 / logits.std()), worst

    ids = torch.from_numpy(rng.integers(0, vocab, sum(prompts))).cuda()
    logits, worst = checked(table[ids], list(prompts))
    last = logits[torch.tensor(prompts).cumsum(0) - 1].argmax(1)
    kept = []
    for _ in range(steps):
        n = drafts + 1
        parent = torch.tensor(([-1] + [(i - 1) // 2 for i in range(1, n)]) * R, dtype=torch.int32, device=dev)
        # the drafts: likely continuations of each parent's embedding alone
        tokens = torch.zeros((R, n), dtype=torch.long, device=dev)
        tokens[:, 0] = last
        for i in range(1, n):
            guess = block._product(weights[2], table[tokens[:, (i - 1) // 2]], hidden)
            tokens[:, i] = guess.topk(2, 1).indices[:, (i - 1) % 2]
        flat = tokens.flatten()
        logits, err = checked(table[flat], [n] * R, parent)
        worst = max(worst, err)
        u = torch.from_numpy(rng.random(R * n + R).astype(np.float32)).cuda()
        temps = torch.full((R,), temperature, device=dev)
        args = (logits, flat.int(), parent, block.q_start, temps, u[:R * n], u[R * n:])
        count, path, token = cq.tree_verify_t(*args, n)
        kept.append((args, count, path, token))
        block.keep(count, path)
        last = token.long()
    return block, worst, kept


if __name__ == "__main__":
    b, err, kept = tree_demo()
    print(f"{len(b.past)} requests, {len(kept)} steps of tree decoding, tokens a step and request: "
          f"{sum(c.sum().item() for _, c, _, _ in kept) / len(kept) / len(b.past):.2f}, lengths {b.past}, {b.taken} pages: "
          f"attention within {err:.1e} of 64 bits (2-norm)")
    b, err = demo()
    print(f"{len(b.past)} requests, lengths {b.past}, {b.taken} pages: attention within {err:.1e} of 64 bits (2-norm)")
