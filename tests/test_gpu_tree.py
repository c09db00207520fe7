"""Masks and positions, norm and rotation, attention under masks, rows moved and pages given back, against plain
implementations in 64 bits and more."""
import numpy as np
import pytest

import kv_ref
import tree_ref
from helpers import cq_built, dev, torch_cuda
from test_gpu_attn import _case

pytestmark = pytest.mark.gpu
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _dt(torch, name):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


# ------------------------------------------------------------------------------------------------------- plan
@pytest.mark.parametrize("lens", [[1], [64], [5, 0, 64, 1, 65, 2, 33], [3] * 700, [0], [200, 7, 0, 0, 63]])
@pytest.mark.parametrize("pad", [0, 9])
def test_plan(lens, pad):
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(len(lens))
    q_start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(q_start[-1]) + pad
    kv = (np.array(lens) + rng.integers(0, 5000, len(lens))).astype(np.int32)
    parent = np.full(T, 7, np.int32)
    for r, n in enumerate(lens):
        parent[q_start[r]:q_start[r + 1]] = tree_ref.random_parents(rng, n) if n else []
    mask, pos = cq.tree_plan_t(dev(torch, kv), dev(torch, q_start), dev(torch, parent))
    want, wp, bits = tree_ref.tree_plan(kv, q_start, parent, T)
    assert bits == 0 and np.array_equal(mask.cpu().numpy().view(np.uint64), want) and np.array_equal(pos.cpu().numpy(), wp)
    assert cq.cq_read_global_status() == (cq.OK, 0)


def test_plan_bad_parents():
    """Parents that do not come before their children count as -1 and are flagged; lengths shorter than the tokens."""
    torch, cq = torch_cuda(), cq_built()
    parent = np.array([0, 0, -2, 5, 2, -1, 2 ** 31 - 1], np.int32)
    kv, q_start = np.array([3], np.int32), np.array([0, 7], np.int32)
    mask, pos = cq.tree_plan_t(dev(torch, kv), dev(torch, q_start), dev(torch, parent))
    want, wp, bits = tree_ref.tree_plan(kv, q_start, parent, 7)
    assert np.array_equal(mask.cpu().numpy().view(np.uint64), want) and np.array_equal(pos.cpu().numpy(), wp)
    assert bits == cq.DEV_TREE and cq.cq_read_global_status() == (cq.ERR_DEVICE_STATUS, cq.DEV_TREE)


# ------------------------------------------------------------------------------------------------------- rope
def _rope(torch, cq, seed, a, b, T, Hq, Hk, D, rot, adjacent, norm, far=131071, extra=0, pad=0, scale=3.0):
    rng = np.random.default_rng(seed)
    rows = rng.standard_normal((T, (Hq + Hk) * D + extra)) * scale
    t = dev(torch, rows.astype(np.float32)).to(_dt(torch, a))
    q, k = t[:, :Hq * D].unflatten(1, (Hq, D)), t[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    pos = rng.integers(0, far + 1, T).astype(np.int32)
    if pad:
        pos[rng.permutation(T)[:pad]] = -1
    freqs = 10000.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
    w = [(1 + 0.3 * rng.standard_normal(D)).astype(np.float32) if norm else None for _ in range(2)]
    wt = [None if x is None else dev(torch, x) for x in w]
    outs = [torch.full((T, h, D), 7.0, dtype=_dt(torch, b), device="cuda") for h in (Hq, Hk)]
    got = cq.qk_rope_t(q, k, dev(torch, pos), dev(torch, freqs) if rot else None, q_norm=wt[0], k_norm=wt[1], eps=1e-5,
                       adjacent=adjacent, q_out=outs[0], k_out=outs[1])
    for x, y, wn in ((q, got[0], w[0]), (k, got[1], w[1])):
        x = x.float().cpu().numpy()
        want, bound = tree_ref.rope(x, wn, 1e-5, pos, freqs, adjacent, HALF[b])
        y = y.float().cpu().numpy().astype(np.longdouble)
        on = pos >= 0
        off = np.abs(y - want)[on]
        assert (off <= bound[on]).all(), f"worst {(off / bound[on]).max():.2f} of its bound"
        assert (y[~on] == 7.0).all()
    return q, k, got


@pytest.mark.parametrize("a,b", [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 32), (64, 8), (64, 24), (128, 128), (128, 64), (128, 40), (128, 0)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rope(a, b, D, rot, adjacent, norm):
    torch, cq = torch_cuda(), cq_built()
    _rope(torch, cq, [D, rot], a, b, 37, 6, 2, D, rot, adjacent, norm, extra=64, pad=3)


@pytest.mark.parametrize("T", [1, 2, 7, 1000, 5003])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (1, 0), (0, 3), (32, 8), (14, 2), (71, 1)])
def test_rope_shapes(T, Hq, Hk):
    torch, cq = torch_cuda(), cq_built()
    if T * (Hq + Hk) > 100000:
        T = 100000 // (Hq + Hk)
    _rope(torch, cq, [T, Hq, Hk], "f32", "bf16", T, Hq, Hk, 128 if Hq % 2 else 64, 64, False, True)


@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_far_positions(adjacent):
    """Positions up to 2^31 - 1: the angle is reduced without loss."""
    torch, cq = torch_cuda(), cq_built()
    _rope(torch, cq, 3, "f32", "f32", 64, 2, 1, 128, 128, adjacent, False, far=2 ** 31 - 1)


@pytest.mark.parametrize("scale", [1e-20, 1e-4, 1e15])
def test_rope_sizes_of_values(scale):
    torch, cq = torch_cuda(), cq_built()
    _rope(torch, cq, 4, "f32", "f32", 9, 2, 2, 64, 64, False, True, scale=scale)


def test_rope_odd_frequencies():
    """Negative, zero, tiny and large frequencies."""
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(5)
    x = rng.standard_normal((50, 2, 64)).astype(np.float32)
    pos = rng.integers(0, 10000, 50).astype(np.int32)
    freqs = np.concatenate([[0.0, -0.5, 1e-30, -1e-18, 3.0, 1e6, -1e9, 2.0 ** -40], rng.standard_normal(24) * 10])
    q, _ = cq.qk_rope_t(dev(torch, x), dev(torch, x[:, :1]), dev(torch, pos), dev(torch, freqs))
    # a frequency is taken to 2^-62 of a turn; fp64 holds the large ones to 2^-53 of themselves, as the reference does
    want, bound = tree_ref.rope(x, None, 0.0, pos, freqs, False, HALF["f32"])
    assert (np.abs(q.cpu().numpy().astype(np.longdouble) - want) <= bound).all()


@pytest.mark.parametrize("a", ["f32", "f16", "bf16"])
def test_rope_in_place(a):
    torch, cq = torch_cuda(), cq_built()
    x = torch.randn(33, 5 * 128, device="cuda").to(_dt(torch, a))
    pos = torch.arange(33, dtype=torch.int32, device="cuda") * 91
    freqs = torch.rand(64, dtype=torch.float64, device="cuda")
    q, k = x[:, :3 * 128].unflatten(1, (3, 128)), x[:, 3 * 128:].unflatten(1, (2, 128))
    want = [t.clone() for t in cq.qk_rope_t(q, k, pos, freqs)]
    got = cq.qk_rope_t(q, k, pos, freqs, q_out=q, k_out=k)
    assert got[0].data_ptr() == q.data_ptr() and all(torch.equal(g, w) for g, w in zip(got, want))


# -------------------------------------------------------------------------------------------------- attention
def _tree_attend(torch, cq, c, masks, **kw):
    return cq.attn_tree_t(c["q"], c["cache"], dev(torch, c["table"]), dev(torch, c["kv"]), dev(torch, c["q_start"]),
                          dev(torch, masks.view(np.int64)), kw.pop("max_new", int(c["new"].max(initial=0))), **kw)


def _tree_check(c, out, lse, masks, scale=None):
    """Row by row: what a row sees is put together as a cache of its own, for kv_ref.attend's formula and bounds."""
    scale = float(np.float32(c["D"] ** -0.5 if scale is None else scale))
    q, got, gl = c["q"].float().cpu().numpy(), out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    P = c["k"].shape[2]
    for r in range(len(c["kv"])):
        n, kv, first = int(c["new"][r]), int(c["kv"][r]), int(c["q_start"][r])
        for t in range(n):
            if n > 64:
                seen = list(range(0, max(kv - n + t + 1, 0)))
            else:
                m = int(masks[first + t])
                seen = list(range(0, max(kv - n, 0))) + [kv - n + j for j in range(n) if m >> j & 1 and kv - n + j >= 0]
            seen = np.array(seen, int)
            page, row = c["table"][r][seen // P], seen % P
            # one key a page of one row: the same numbers
            k1, v1 = c["k"][page, :, row][:, :, None], c["v"][page, :, row][:, :, None]
            if len(seen) == 0:
                assert (got[first + t] == 0).all() and np.isneginf(gl[first + t]).all()
                continue
            want, wl, eo, el = kv_ref.attend(q[first + t:first + t + 1], k1, v1, c["ks"][page], c["vs"][page],
                                             np.arange(len(seen))[None], [len(seen)], [0, 1], scale, False, 0, c["dtype"])
            off = np.abs(got[first + t] - want[0])
            assert (off <= eo[0]).all(), f"out {r},{t}: worst {(off / eo[0]).max():.2f} of its bound"
            assert (np.abs(gl[first + t] - wl[0]) <= el[0]).all(), f"lse {r},{t}"


def _masks(rng, c, tree=True):
    T = c["T"]
    out = np.zeros(T, np.uint64)
    for r, n in enumerate(c["new"]):
        first = int(c["q_start"][r])
        if n == 0 or n > 64:
            out[first:first + n] = 0xdeadbeef            # not read
        elif tree:
            out[first:first + n] = tree_ref.tree_plan([n], [0, n], tree_ref.random_parents(rng, n), n)[0]
        else:                                            # any pattern, with bits past the request's tokens
            out[first:first + n] = rng.integers(0, 2 ** 63, n).astype(np.uint64) << np.uint64(1)
            out[first] = 0
    return out


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,P,Hq,H", [(64, 16, 8, 2), (128, 32, 4, 4), (128, 128, 14, 2), (64, 64, 32, 1)])
@pytest.mark.parametrize("tree", [True, False])
def test_attn_ragged(dtype, D, P, Hq, H, tree):
    """Trees of all widths, single tokens, a prompt and requests without tokens, in one call."""
    torch, cq = torch_cuda(), cq_built()
    new = [1, 0, 5, 70, 1, 33, 16, 3, 0, 64, 12]
    kv = [300, 50, 5, 90, 1, 500, 400, 129, 0, 1000, 12]
    rng = np.random.default_rng([D, P, Hq])
    c = _case(torch, cq, [D, P, Hq], dtype, Hq, H, D, P, kv, new, stride_extra=64, joint=True)
    masks = _masks(rng, c, tree)
    _tree_check(c, *_tree_attend(torch, cq, c, masks), masks)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Hq,H", [(4, 4), (8, 1)])
@pytest.mark.parametrize("n,past", [(1, 0), (2, 0), (64, 0), (64, 1), (63, 65), (17, 2000), (64, 2047), (8, 127), (40, 120)])
def test_attn_one_tree(dtype, Hq, H, n, past):
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng([n, past])
    c = _case(torch, cq, [n, past], dtype, Hq, H, 128, 16, [past + n], [n])
    masks = _masks(rng, c)
    _tree_check(c, *_tree_attend(torch, cq, c, masks), masks)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("max_new", [0, 1, 12, 64, 65, 10 ** 6])
def test_attn_bound_of_new_tokens_is_a_hint(dtype, max_new):
    """max_new chooses kernels and their tiles; whatever it says, the results are right."""
    torch, cq = torch_cuda(), cq_built()
    new, kv = [9, 64, 1, 70, 30], [400, 300, 50, 170, 30]
    c = _case(torch, cq, 8, dtype, 8, 2, 64, 16, kv, new)
    masks = _masks(np.random.default_rng(4), c)
    _tree_check(c, *_tree_attend(torch, cq, c, masks, max_new=max_new), masks)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R", [40, 128, 129, 300])
def test_attn_many_requests(dtype, R):
    """More requests than are put in order, ragged lengths among them."""
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(R)
    new = rng.integers(0, 8, R)
    new[R // 2] = 7
    c = _case(torch, cq, R, dtype, 4, 1, 64, 16, new + rng.integers(0, 200, R), new)
    masks = _masks(rng, c)
    _tree_check(c, *_tree_attend(torch, cq, c, masks), masks)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,Hq,H", [(48, 8, 2), (16, 8, 2), (64, 2, 2)])
def test_attn_long_contexts_in_parts(dtype, n, Hq, H):
    """Few items over long contexts: split over their keys, joined by the other kernel."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, n, dtype, Hq, H, 128, 64, [9000, 20011], [n, n - 5])
    masks = _masks(np.random.default_rng(n), c)
    masks[2:n - 8] = masks[1]                            # most rows alike: the check goes row by row
    keep = [0, 1, n - 8, n - 1, n, n + 2, 2 * n - 6]
    out, lse = _tree_attend(torch, cq, c, masks)
    q_start = c["q_start"]
    for t in keep:
        r = int(t >= q_start[1])
        one = dict(c, q=c["q"][t:t + 1], table=c["table"][r:r + 1])
        first, m, kv = int(q_start[r]), int(c["new"][r]), int(c["kv"][r])
        seen = list(range(kv - m)) + [kv - m + j for j in range(m) if int(masks[t]) >> j & 1]
        page, row = c["table"][r][np.array(seen) // 64], np.array(seen) % 64
        want, wl, eo, el = kv_ref.attend(one["q"].float().cpu().numpy(), c["k"][page, :, row][:, :, None], c["v"][page, :, row][:, :, None],
                                         c["ks"][page], c["vs"][page], np.arange(len(seen))[None], [len(seen)], [0, 1],
                                         float(np.float32(128 ** -0.5)), False, 0, dtype)
        assert (np.abs(out[t].float().cpu().numpy() - want[0]) <= eo[0]).all() and (np.abs(lse[t].cpu().numpy() - wl[0]) <= el[0]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attn_chain_is_causal(dtype):
    """A chain's masks see what the causal call sees: the same results within both calls' rounding."""
    torch, cq = torch_cuda(), cq_built()
    new, kv = [5, 64, 1, 20], [700, 1500, 33, 20]
    c = _case(torch, cq, 5, dtype, 8, 2, 128, 16, kv, new)
    masks = np.concatenate([tree_ref.tree_plan([n], [0, n], tree_ref.random_parents(None, n, True), n)[0] for n in new])
    out, lse = _tree_attend(torch, cq, c, masks)
    want = cq.attn_paged_t(c["q"], c["cache"], dev(torch, c["table"]), dev(torch, c["kv"]), dev(torch, c["q_start"]), 64, 1500)
    _tree_check(c, out, lse, masks)
    e = {"f32": 2e-5, "bf16": 2e-2}[dtype]
    assert ((out - want[0]).float().norm() <= e * want[0].float().norm()).item()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_attn_rows_that_see_nothing(dtype):
    """Masks of nothing over an empty past, and lengths shorter than the new tokens."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, 4, dtype, 4, 2, 64, 16, [3, 0, 40, 5], [5, 2, 40, 50])
    masks = _masks(np.random.default_rng(1), c)
    masks[c["q_start"][2]:c["q_start"][2] + 20] = 0
    out, lse = _tree_attend(torch, cq, c, masks)
    _tree_check(c, out, lse, masks)


@pytest.mark.parametrize("n", [3, 40])
def test_attn_hidden_keys_never_count(n):
    """NaN scales of pages that only hidden tokens lie in leave the rows as they were."""
    torch, cq = torch_cuda(), cq_built()
    P, past = 16, 320
    c = _case(torch, cq, n, "f32", 8, 2, 64, P, [past + n], [n])
    # the tokens of the request's last page are leaves
    last = max((past + n - 1) // P * P - past, 1)
    masks = np.array([1 << i | 1 if i < last else (1 << i) | 1 for i in range(n)], np.uint64)
    want = [x.clone() for x in _tree_attend(torch, cq, c, masks)]
    page = int(c["table"][0, (past + n - 1) // P])
    if (past + n - 1) // P > past // P:
        c["cache"].k_scale[page] = float("nan")
        c["cache"].v_scale[page] = float("inf")
        out, lse = _tree_attend(torch, cq, c, masks)
        assert torch.equal(out[:last], want[0][:last]) and torch.equal(lse[:last], want[1][:last])
        assert not torch.isfinite(out[last:]).all()


def test_attn_padding_rows_and_other_streams():
    """Rows of no request stay as they are; the call runs on the current stream, and in a captured graph."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, 9, "bf16", 8, 2, 128, 16, [200, 90], [7, 50], T_extra=5)
    masks = _masks(np.random.default_rng(2), c)
    args = [dev(torch, x) for x in (c["table"], c["kv"], c["q_start"], masks.view(np.int64))]
    ws = cq.attn_workspace_t(8, 2, 128)
    out = torch.full_like(c["q"], 3.0)
    want, wl = cq.attn_tree_t(c["q"], c["cache"], *args, 50, ws=ws, out=out)
    _tree_check(c, want, wl, masks)
    assert (out[57:] == 3.0).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again, al = cq.attn_tree_t(c["q"], c["cache"], *args, 50, ws=ws)
        g = torch.cuda.CUDAGraph()
        held = torch.zeros_like(c["q"])
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            cq.attn_tree_t(c["q"], c["cache"], *args, 50, ws=ws, out=held, lse=wl)
    torch.cuda.synchronize()
    for _ in range(2):
        held.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(held[:57], want[:57]) and torch.equal(again[:57], want[:57])


# --------------------------------------------------------------------------------------------- move and release
def _cache_case(rng, R, P, H, D, past, new, pages_extra=3, alike=False):
    past, new = np.asarray(past), np.asarray(new)
    kv = (past + new).astype(np.int32)
    need = -(-kv // P)
    pages = int(need.sum()) + pages_extra
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((R, int(need.max(initial=0)) + 1), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    q = rng.integers(-127, 128, (2, pages, H, P, D)).astype(np.int8)
    sc = np.full((2, pages, H), 0.5, np.float32) if alike else (0.01 + rng.random((2, pages, H))).astype(np.float32)
    return kv, np.concatenate([[0], np.cumsum(new)]).astype(np.int32), table, q, sc


def _move_check(torch, cq, q, sc, table, kv, q_start, count, path):
    cache = cq.KVCache(dev(torch, q[0]), dev(torch, q[1]), dev(torch, sc[0]), dev(torch, sc[1]))
    got = cq.kv_move_t(cache, dev(torch, table), dev(torch, kv), dev(torch, q_start), dev(torch, count), dev(torch, path))
    bits = 0
    for i, (t, s) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        want, b = tree_ref.move(q[i], sc[i], table, kv, q_start, count, path)
        bits |= b
        assert np.array_equal(s.cpu().numpy(), sc[i], equal_nan=True), "scales"
        assert np.array_equal(t.cpu().numpy(), q[i]), "values"
    assert np.array_equal(got.cpu().numpy(), want)
    assert cq.cq_read_global_status() == ((cq.ERR_DEVICE_STATUS, bits) if bits else (cq.OK, 0))
    return cache


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("D,H", [(64, 1), (128, 3), (64, 8)])
@pytest.mark.parametrize("alike", [False, True])
def test_move(P, D, H, alike):
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng([P, D, H])
    new = [1, 64, 0, 20, 64, 33, 5, 2, 64, 17, 65]
    past = [0, 0, 7, 127, 63, 1000, 15, 16, 250, 3, 40]
    kv, q_start, table, q, sc = _cache_case(rng, len(new), P, H, D, past, new, alike=alike)
    path = np.full((len(new), 64), -1, np.int32)
    count = np.zeros(len(new), np.int32)
    for r, n in enumerate(new):
        if n:
            count[r] = int(rng.integers(1, n + 1)) if r != 4 else 64
            path[r, :count[r]] = np.sort(rng.permutation(n)[:count[r]]) if r != 6 else rng.permutation(n)[:count[r]]
            path[r, 0] = 0 if r % 2 else path[r, 0]
    _move_check(torch, cq, q, sc, table, kv, q_start, count, path)


def test_move_unusual_scales():
    """Scales of 0 and NaN, and rows from several pages into one."""
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(1)
    kv, q_start, table, q, sc = _cache_case(rng, 3, 16, 2, 64, [14, 0, 33], [60, 40, 64])
    sc[0, table[0, 1]], sc[0, table[0, 2], 0], sc[1, table[2, 3]] = 0.0, 0.0, np.nan
    sc[1, table[1, 0]] = np.nan
    q[0, table[0, 1]], q[0, table[0, 2], 0] = 0, 0
    path = np.array([[0, 3, 17, 20, 50, 59], [0, 1, 2, 3, 30, 31], [5, 4, 40, 3, 50, 0]], np.int32)
    _move_check(torch, cq, q, sc, table, kv, q_start, np.array([6, 6, 6], np.int32), path)


def test_move_refuses_what_is_outside():
    """Counts, paths and pages outside the request and the cache: flagged, nothing else is touched."""
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(2)
    kv, q_start, table, q, sc = _cache_case(rng, 5, 16, 2, 64, [10, 0, 33, 20, 5], [30, 40, 64, 30, 8])
    table[1, 2], table[2, 3] = 10 ** 6, -1
    kv[4] = 3                                            # shorter than its new tokens
    path = np.array([[0, 30, -1, 5], [0, 39, 1, 12], [0, 20, 21, 63], [0, 3, 9, 29], [7, 6, 5, 4]], np.int32)
    _move_check(torch, cq, q, sc, table, kv, q_start, np.array([4, 9, 4, -3, 4], np.int32), path)


def test_move_twice():
    """Where no source is overwritten and no page that gets rows gives any on, the second call changes nothing."""
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(3)
    kv, q_start, table, q, sc = _cache_case(rng, 2, 16, 4, 128, [14, 16], [50, 40])
    path, count = np.array([[0, 1, 30, 40], [0, 20, 25, 39]], np.int32), np.array([4, 4], np.int32)
    cache = _move_check(torch, cq, q, sc, table, kv, q_start, count, path)
    was = [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    cq.kv_move_t(cache, dev(torch, table), dev(torch, kv), dev(torch, q_start), dev(torch, count), dev(torch, path))
    assert all(torch.equal(a, b) for a, b in zip(was, (cache.k, cache.v, cache.k_scale, cache.v_scale)))


@pytest.mark.parametrize("R", [1, 3, 700, 2000])
@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("short", [False, True])
def test_release(R, P, short):
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng([R, P])
    old = rng.integers(0, 900, R).astype(np.int32)
    new = np.maximum(old - rng.integers(-40, 300, R), 0).astype(np.int32)
    new[0] = 0
    table = rng.integers(0, 5000, (R, -(-900 // P))).astype(np.int32)
    cap = 40 if short else R * (-(-900 // P))
    want, used = tree_ref.release(table, old, new, P, 5000, cap)
    freed, u = cq.kv_release_t(dev(torch, table), dev(torch, old), dev(torch, new), P, 5000, cap)
    assert u.tolist() == used and np.array_equal(freed.cpu().numpy(), want)


def test_release_refuses_what_is_outside():
    torch, cq = torch_cuda(), cq_built()
    table = np.array([[0, 9, 2], [-1, 4, 10], [5, 6, 7]], np.int32)
    old, new = np.array([48, 500, -3], np.int32), np.array([1, 0, -1], np.int32)
    want, used = tree_ref.release(table, old, new, 16, 10, 8)
    freed, u = cq.kv_release_t(dev(torch, table), dev(torch, old), dev(torch, new), 16, 10, 8)
    assert u.tolist() == used and np.array_equal(freed.cpu().numpy(), want) and used[1] == 0x98
    freed, u = cq.kv_release_t(dev(torch, table), dev(torch, old), dev(torch, new), 16, 10, 0)
    assert u.tolist() == [0, 0x38]
