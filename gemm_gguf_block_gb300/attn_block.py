"""One attention layer on the library's calls: quantised projections, the 8-bit paged cache and attention over it.

``AttentionBlock`` keeps the weights (any format that cq_gemm takes), the cache, the block table and the workspace of
a layer; ``step`` takes the new tokens of a set of requests -- prompts, chunks of them, drafts or single tokens, in
one call -- through

    cq_quantize_act -> cq_gemv / cq_gemm (q, k, v in one matrix) -> cq_kv_plan -> cq_kv_append -> cq_attn_paged
    -> cq_quantize_act -> cq_gemv / cq_gemm (output projection).

The plan's positions are what a rotary embedding would take; the library has none, so queries and keys are used as
they are projected. It shows the calls together and is no scheduler: requests do not end, pages are not given back, and
the lengths go to the device with every step.

    python -m gemm_gguf_block_gb300.attn_block      two prompts, then single tokens, checked against 64 bits
"""
from __future__ import annotations

from . import cq


class AttentionBlock:
    """wqkv: [(q_heads + 2 kv_heads) * head_dim] rows of weight blocks, wo: [hidden] rows of q_heads * head_dim."""

    def __init__(self, wqkv, wo, fmt: int, hidden: int, q_heads: int, kv_heads: int, head_dim: int, *, requests: int,
                 num_pages: int, page_size: int = 16):
        import torch
        self.wqkv, self.wo, self.fmt, self.hidden = wqkv, wo, fmt, hidden
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        dev = wqkv.device
        self.cache = cq.KVCache.empty(num_pages, kv_heads, page_size, head_dim, dev)
        self.table = torch.full((requests, num_pages), -1, dtype=torch.int32, device=dev)
        self.free = torch.arange(num_pages, dtype=torch.int32, device=dev)     # pages are taken from the front
        self.taken = 0
        self.past = [0] * requests                                             # the host's copy of the lengths
        self.ws = cq.attn_workspace_t(q_heads, kv_heads, head_dim, dev)

    def _product(self, w, x, rows_in: int):
        xq = cq.quantize_act_t(x, cq.ACT_FOR[self.fmt])
        return (cq.gemv_t if x.shape[0] <= 16 else cq.gemm_t)(w, xq, self.fmt, rows_in)

    def step(self, x, new):
        """x: fp32 [T, hidden], the new tokens of all requests in order; new: their number for each request (0 for a
        request that takes no part; T in all, at least 1). Returns fp32 [T, hidden]."""
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
        width, kv_width = self.q_heads * self.head_dim, self.kv_heads * self.head_dim
        qkv = self._product(self.wqkv, x, self.hidden)
        cq.kv_append_t(self.cache, qkv[:, width:width + kv_width], qkv[:, width + kv_width:], slots)
        q = qkv[:, :width].unflatten(1, (self.q_heads, self.head_dim))
        after = [a + b for a, b in zip(self.past, new)]
        self.attended, _ = cq.attn_paged_t(q, self.cache, self.table, kv_len, q_start, max(new), max(after), ws=self.ws,
                                           lse=None)
        y = self._product(self.wo, self.attended.view(x.shape[0], width), width)
        self.taken += need
        self.past, self.q, self.slots = after, q, slots
        return y

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


if __name__ == "__main__":
    b, err = demo()
    print(f"{len(b.past)} requests, lengths {b.past}, {b.taken} pages: attention within {err:.1e} of 64 bits (2-norm)")
