"""The calls of a tree decoding step where offsets pass 32 bits, and at their smallest and largest sizes."""
import numpy as np
import pytest

import kv_ref
import tree_ref
from helpers import cq_built, dev, torch_cuda

pytestmark = pytest.mark.gpu


def test_rope_rows_far_apart():
    """Rows 2^31 values apart, in and out."""
    torch, cq = torch_cuda(), cq_built()
    big = torch.empty((2, 2 ** 31 + 256), dtype=torch.bfloat16, device="cuda")
    q, k = big[:, :256].unflatten(1, (2, 128)), big[:, 2 ** 31 - 128:2 ** 31].unflatten(1, (1, 128))
    x = torch.randn(2, 3, 128, device="cuda").bfloat16()
    q.copy_(x[:, :2])
    k.copy_(x[:, 2:])
    pos = torch.tensor([7, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    freqs = torch.rand(64, dtype=torch.float64, device="cuda")
    want = cq.qk_rope_t(x[:, :2].contiguous(), x[:, 2:].contiguous(), pos, freqs)
    got = cq.qk_rope_t(q, k, pos, freqs, q_out=q, k_out=k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_verify_rows_far_apart():
    torch, cq = torch_cuda(), cq_built()
    V = 5000
    big = torch.empty((4, 2 ** 30), device="cuda")
    z = torch.randn(4, V, device="cuda") * 3
    big[:, :V] = z
    i32 = dict(dtype=torch.int32, device="cuda")
    args = (torch.tensor([0, int(z[0].argmax()), int(z[1].argmax()), int(z[2].argmax())], **i32), torch.tensor([-1, 0, 1, 2], **i32),
            torch.tensor([0, 4], **i32), torch.ones(1, device="cuda"), torch.full((4,), 1e-6, device="cuda"),
            torch.full((1,), 0.5, device="cuda"), 4)
    got, want = cq.tree_verify_t(big[:, :V], *args), cq.tree_verify_t(z, *args)
    assert got[0].item() == 4 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_pages_far_apart():
    """Pages 2^30 bytes apart, five of them: rows moved, and attention under masks in both kernels."""
    torch, cq = torch_cuda(), cq_built()
    P, H, D, stride = 16, 2, 128, 2 ** 30
    pool = torch.empty(5 * stride, dtype=torch.int8, device="cuda")
    view = lambda off: torch.as_strided(pool, (5, H, P, D), (stride, P * D, D, 1), off)
    rng = np.random.default_rng(0)
    n, past = 40, 24
    k, v = (rng.integers(-127, 128, (5, H, P, D)).astype(np.int8) for _ in range(2))
    sc = (0.01 + 0.02 * rng.random((2, 5, H))).astype(np.float32)
    kt, vt = view(0), view(H * P * D)
    kt.copy_(dev(torch, k))
    vt.copy_(dev(torch, v))
    cache = cq.KVCache(kt, vt, dev(torch, sc[0]), dev(torch, sc[1]))
    table, kv, q_start = np.array([[4, 2, 0, 3]], np.int32), np.array([past + n], np.int32), np.array([0, n], np.int32)
    mask = tree_ref.tree_plan(kv, q_start, tree_ref.random_parents(rng, n), n)[0]
    for Hq, m in ((2, 6), (16, n)):                      # 6 rows of a kv head, 320
        q = torch.randn(m, Hq, D, device="cuda")
        start, length = np.array([0, m], np.int32), np.array([past + m], np.int32)
        out, lse = cq.attn_tree_t(q, cache, dev(torch, table), dev(torch, length), dev(torch, start),
                                  dev(torch, mask[:m].view(np.int64)), m)
        for t in (0, m // 2, m - 1):
            seen = np.array(list(range(past)) + [past + j for j in range(m) if int(mask[t]) >> j & 1])
            page, row = table[0][seen // P], seen % P
            want, _, eo, _ = kv_ref.attend(q[t:t + 1].cpu().numpy(), k[page, :, row][:, :, None], v[page, :, row][:, :, None],
                                           sc[0][page], sc[1][page], np.arange(len(seen))[None], [len(seen)], [0, 1],
                                           float(np.float32(D ** -0.5)), False, 0, "f32")
            assert (np.abs(out[t].cpu().numpy() - want[0]) <= eo[0]).all()
    path, count = np.array([[0, 3, 17, 30, 39]], np.int32), np.array([5], np.int32)
    new_len = cq.kv_move_t(cache, dev(torch, table), dev(torch, kv), dev(torch, q_start), dev(torch, count), dev(torch, path))
    for x, s, t, st in ((k, sc[0], kt, cache.k_scale), (v, sc[1], vt, cache.v_scale)):
        tree_ref.move(x, s, table, kv, q_start, count, path)
        assert np.array_equal(t.cpu().numpy(), x) and np.array_equal(st.cpu().numpy(), s)
    assert new_len.tolist() == [past + 5]


def test_nothing_to_do():
    """No requests, no tokens, requests without tokens."""
    torch, cq = torch_cuda(), cq_built()
    i32 = dict(dtype=torch.int32, device="cuda")
    none, zero = torch.empty(0, **i32), torch.zeros(1, **i32)
    f = lambda *s: torch.zeros(*s, device="cuda")
    cache = cq.KVCache.empty(4, 2, 16, 64)
    mask, pos = cq.tree_plan_t(none, zero, torch.zeros(3, **i32))
    assert mask.tolist() == [0, 0, 0] and pos.tolist() == [-1, -1, -1]
    assert cq.tree_plan_t(zero, torch.zeros(2, **i32), none)[0].numel() == 0
    q, k = cq.qk_rope_t(f(0, 4, 64), f(0, 2, 64), none, None)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    out, lse = cq.attn_tree_t(f(0, 4, 64), cache, torch.zeros((1, 2), **i32), zero, torch.zeros(2, **i32), torch.empty(0, dtype=torch.int64, device="cuda"), 0)
    assert out.numel() == 0
    count, path, token = cq.tree_verify_t(f(0, 100), none, none, torch.zeros(3, **i32), f(2), f(0), f(2), 3)
    assert count.tolist() == [0, 0] and token.tolist() == [-1, -1] and path.tolist() == [[-1] * 3] * 2
    assert cq.kv_move_t(cache, torch.zeros((0, 2), **i32), none, zero, none, torch.zeros((0, 3), **i32)).numel() == 0
    assert cq.kv_move_t(cache, torch.zeros((1, 2), **i32), torch.tensor([9], **i32), torch.zeros(2, **i32), zero,
                        torch.zeros((1, 3), **i32)).tolist() == [9]
    freed, used = cq.kv_release_t(torch.zeros((0, 2), **i32), none, none, 16, 4, 3)
    assert freed.tolist() == [-1] * 3 and used.tolist() == [0, 0]
    assert cq.cq_read_global_status() == (cq.OK, 0)


def test_most_requests():
    """16384 requests: plans and lists whole, a token each through verification."""
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(1)
    R = 16384
    lens = rng.integers(0, 3, R)
    q_start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(q_start[-1])
    kv = (lens + rng.integers(0, 100, R)).astype(np.int32)
    parent = np.concatenate([[-1, 0][:n] for n in lens] + [[]]).astype(np.int32)
    mask, pos = cq.tree_plan_t(dev(torch, kv), dev(torch, q_start), dev(torch, parent))
    want, wp, _ = tree_ref.tree_plan(kv, q_start, parent, T)
    assert np.array_equal(mask.cpu().numpy().view(np.uint64), want) and np.array_equal(pos.cpu().numpy(), wp)
    z = (rng.standard_normal((T, 40)) * 3).astype(np.float32)
    tokens = rng.integers(0, 40, T).astype(np.int32)
    temp, ua, us = np.ones(R, np.float32), rng.random(T).astype(np.float32), rng.random(R).astype(np.float32)
    got = cq.tree_verify_t(*(dev(torch, x) for x in (z, tokens, parent, q_start, temp, ua, us)), 2)
    ref = tree_ref.verify(z, tokens, parent, q_start, temp, ua, us, 2)
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, ref))
    table = rng.integers(0, 9000, (R, 7)).astype(np.int32)
    new = np.maximum(kv - rng.integers(0, 60, R), 0).astype(np.int32)
    freed, used = cq.kv_release_t(dev(torch, table), dev(torch, kv), dev(torch, new), 16, 9000, 30000)
    wf, wu = tree_ref.release(table, kv, new, 16, 9000, 30000)
    assert used.tolist() == wu and np.array_equal(freed.cpu().numpy(), wf)


@pytest.mark.parametrize("first", [0, 1000])
def test_plan_of_as_many_tokens_as_it_takes(first):
    """The largest T: a request of all but a few tokens, padding, the last entries as the first (34 GB)."""
    torch, cq = torch_cuda(), cq_built()
    T = 2 ** 31 - 1
    parent = torch.empty(T, dtype=torch.int32, device="cuda")
    parent[first + T - first - 70:] = -1
    q_start = np.array([first, T - 70, T - 67], np.int32)
    kv = np.array([T - 70 - first + 5, 9], np.int32)
    mask, pos = cq.tree_plan_t(dev(torch, kv), dev(torch, q_start), parent)
    n = T - 70 - first
    assert pos[:first].eq(-1).all() and pos[T - 67:].eq(-1).all() and mask[T - 67:].eq(0).all()
    assert pos[first:first + 3].tolist() == [5, 6, 7] and pos[T - 73:T - 67].tolist() == [n + 2, n + 3, n + 4, 6, 6, 6]
    assert mask[T - 70:T - 67].tolist() == [1, 2, 4] and mask[first:T - 70].count_nonzero().item() == 0
    step = pos[first + 1:T - 70:1000003] - pos[first:T - 71:1000003]
    assert step.eq(1).all()
    assert cq.cq_read_global_status() == (cq.OK, 0)
