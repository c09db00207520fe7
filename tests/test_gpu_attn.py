"""Attention over the 8-bit paged cache against its formula in 64 bits."""
import numpy as np
import pytest

import kv_ref
from helpers import cq_built, dev, torch_cuda

pytestmark = pytest.mark.gpu


def _case(torch, cq, seed, dtype, Hq, H, D, P, kv, new, T_extra=0, stride_extra=0, spread=2.0, joint=False):
    rng = np.random.default_rng(seed)
    kv, new = np.asarray(kv, np.int32), np.asarray(new, np.int32)
    need = -(-np.maximum(kv, 0) // P)
    pages = int(need.sum()) + 2
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(kv), int(need.max(initial=0)) + 1), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    k = np.clip(np.round(rng.standard_normal((pages, H, P, D)) * 36), -127, 127).astype(np.int8)
    v = np.clip(np.round(rng.standard_normal((pages, H, P, D)) * 36), -127, 127).astype(np.int8)
    ks = (0.02 + 0.015 * rng.random((pages, H))).astype(np.float32)
    vs = (0.03 * np.exp(rng.uniform(-2, 2, (pages, H)))).astype(np.float32)
    q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(q_start[-1]) + T_extra
    rows = rng.standard_normal((T, Hq * D + stride_extra)) * spread
    tq = dev(torch, rows.astype(np.float32)).to({"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype])
    tq = tq[:, :Hq * D].view(T, Hq, D) if stride_extra == 0 else tq[:, :Hq * D].unflatten(1, (Hq, D))
    if joint:
        kv_t = dev(torch, np.stack([k, v], 1))
        sc_t = dev(torch, np.stack([ks, vs], 1))
        cache = cq.KVCache(kv_t[:, 0], kv_t[:, 1], sc_t[:, 0], sc_t[:, 1])
    else:
        cache = cq.KVCache(dev(torch, k), dev(torch, v), dev(torch, ks), dev(torch, vs))
    return dict(q=tq, cache=cache, k=k, v=v, ks=ks, vs=vs, table=table, kv=kv, q_start=q_start, dtype=dtype, T=T,
                new=new, D=D)


def _run(torch, cq, c, causal=True, window=0, scale=None, **kw):
    max_new = kw.pop("max_new", int(c["new"].max(initial=0)))
    max_kv = kw.pop("max_kv", int(c["kv"].max(initial=0)))
    return cq.attn_paged_t(c["q"], c["cache"], dev(torch, c["table"]), dev(torch, c["kv"]), dev(torch, c["q_start"]),
                           max_new, max_kv, causal=causal, window=window, scale=scale, **kw)


def _check(c, out, lse, causal=True, window=0, scale=None, rows=None):
    scale = np.float32(c["D"] ** -0.5 if scale is None else scale)
    want, wl, eo, el = kv_ref.attend(c["q"].float().cpu().numpy(), c["k"], c["v"], c["ks"], c["vs"], c["table"],
                                     c["kv"], c["q_start"], float(scale), causal, window, c["dtype"])
    n = int(c["q_start"][-1]) if rows is None else rows
    got = out.float().cpu().numpy().astype(np.float64)[:n]
    assert np.isfinite(got).all()
    off = np.abs(got - want[:n])
    assert (off <= eo[:n]).all(), f"out: worst {(off / eo[:n]).max():.2f} of its bound"
    if lse is not None:
        gl = lse.cpu().numpy().astype(np.float64)[:n]
        empty = np.isinf(wl[:n])
        assert np.array_equal(np.isneginf(gl), empty)
        off = np.abs(gl[~empty] - wl[:n][~empty])
        assert (off <= el[:n][~empty]).all(), f"lse: worst {(off / el[:n][~empty]).max():.2f} of its bound"


HEADS = [(1, 1), (4, 1), (8, 2), (14, 2), (6, 6), (32, 2), (20, 1)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 16), (128, 64), (64, 128), (128, 128), (64, 32)])
@pytest.mark.parametrize("Hq,H", HEADS)
def test_decode(dtype, D, P, Hq, H):
    """One token a request, lengths from one to some thousands."""
    torch, cq = torch_cuda(), cq_built()
    kv = [1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 500, 1000, 2049]
    c = _case(torch, cq, [D, P, Hq], dtype, Hq, H, D, P, kv, [1] * len(kv))
    _check(c, *_run(torch, cq, c))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv", [1, 16, 40, 700, 5000, 40001])
def test_decode_one_request(dtype, D, kv):
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, kv, dtype, 8, 2, D, 16, [kv], [1])
    _check(c, *_run(torch, cq, c))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,P,Hq,H", [(64, 16, 8, 2), (128, 32, 4, 4), (128, 128, 14, 2), (64, 64, 32, 1)])
@pytest.mark.parametrize("window", [0, 1, 13, 100])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_mixed(dtype, D, P, Hq, H, window, causal):
    """Prompts, chunks, drafts and single tokens in one call, requests without tokens between them."""
    torch, cq = torch_cuda(), cq_built()
    new = [1, 0, 5, 130, 1, 33, 16, 3, 0]
    kv = [300, 50, 5, 130, 1, 500, 400, 129, 0]
    c = _case(torch, cq, [D, P, Hq, window], dtype, Hq, H, D, P, kv, new, stride_extra=64, joint=True)
    _check(c, *_run(torch, cq, c, causal=causal, window=window), causal=causal, window=window)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,Hq,H", [(64, 8, 2), (128, 4, 1), (128, 5, 5), (64, 3, 1)])
@pytest.mark.parametrize("n,past", [(1, 0), (127, 0), (128, 0), (129, 0), (257, 0), (600, 0), (64, 1000), (300, 777)])
def test_prefill(dtype, D, Hq, H, n, past):
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, [n, past], dtype, Hq, H, D, 16, [past + n], [n])
    _check(c, *_run(torch, cq, c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [2, 4, 7, 8, 16])
def test_verify(dtype, n):
    torch, cq = torch_cuda(), cq_built()
    kv = [n, 100, 1000, 4000]
    c = _case(torch, cq, n, dtype, 32, 8, 128, 32, kv, [n, 1, n, n])
    _check(c, *_run(torch, cq, c))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rows_that_see_nothing(dtype):
    """More new tokens than the cache holds, and empty caches: out 0 and lse -inf there."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, 4, dtype, 4, 2, 64, 16, [3, 0, 40, 0, 5], [5, 2, 50, 140, 200])
    out, lse = _run(torch, cq, c)
    _check(c, out, lse)
    assert (out[:2].float() == 0).all() and torch.isneginf(lse[:2]).all()
    out, lse = _run(torch, cq, c, causal=False)
    _check(c, out, lse, causal=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 40, 200])
def test_hidden_keys_never_count(dtype, n):
    """NaN and infinite scales of blocks that a row does not see, and rows past the length, leave it unchanged."""
    torch, cq = torch_cuda(), cq_built()
    P, kv = 16, 333
    c = _case(torch, cq, n, dtype, 8, 2, 64, P, [kv, 90], [n, 90])
    want = [x.clone() for x in _run(torch, cq, c, window=50)]
    first = max(0, kv - n + 1 - 50)                      # first key that any row of request 0 sees
    for page in c["table"][0, :first // P]:
        c["cache"].k_scale[int(page)] = float("nan")
        c["cache"].v_scale[int(page)] = float("inf")
    c["cache"].v_scale[int(c["table"][1, 5])] = float("nan")   # keys 80..89 of request 1: seen from position 80 on
    out, lse = _run(torch, cq, c, window=50)
    keep = list(range(n + 80))
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])
    assert torch.isnan(out[n + 80:].float()).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 150])
def test_bad_pages_are_hidden_and_flagged(dtype, n):
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, 9, dtype, 4, 2, 128, 32, [600, 200], [n, 1])
    c["table"][0, 3], c["table"][0, 7], c["table"][1, :] = -1, 1 << 30, -5
    cq.cq_read_global_status()
    out, lse = _run(torch, cq, c)
    assert cq.cq_read_global_status() == (cq.ERR_DEVICE_STATUS, cq.DEV_KV_PAGE)
    _check(c, out, lse)
    assert (out[n].float() == 0).all()


@pytest.mark.parametrize("n", [1, 200])
def test_zero_and_uneven_value_scales(n):
    """Blocks whose values are all zero count in the sum; blocks of very unequal scale keep their weight."""
    torch, cq = torch_cuda(), cq_built()
    for dtype in ("f32", "bf16"):
        c = _case(torch, cq, 2, dtype, 4, 2, 64, 16, [400], [n])
        pages = [int(p) for p in c["table"][0, :25]]
        for i, page in enumerate(pages):
            c["vs"][page] = 0.0 if i % 3 == 0 else 1e-6 if i % 3 == 1 else 50.0
            if i % 3 == 0:
                c["v"][page] = 0
            if i % 5 == 0:
                c["ks"][page], c["k"][page] = 0.0, 0
        for name, a in (("k", c["k"]), ("v", c["v"]), ("k_scale", c["ks"]), ("v_scale", c["vs"])):
            getattr(c["cache"], name).copy_(dev(torch, a))
        _check(c, *_run(torch, cq, c))


@pytest.mark.parametrize("n", [1, 130])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales_of_the_scores(n, scale):
    """A flat softmax, a negative scale, and scores of some hundreds."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, 8, "f32", 4, 2, 64, 16, [700], [n], spread=4.0 if scale == 3.0 else 1.0)
    _check(c, *_run(torch, cq, c, scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("size", [1e-6, 1e4])
def test_small_and_large_queries(dtype, size):
    """Queries near the ends of binary16's range: scores stay right (the scale makes up for them)."""
    torch, cq = torch_cuda(), cq_built()
    for n in (1, 140):
        c = _case(torch, cq, 8, dtype, 4, 2, 64, 16, [300], [n], spread=size)
        _check(c, *_run(torch, cq, c, scale=0.1 / size), scale=0.1 / size)


def test_queries_that_are_not_finite_spoil_their_row_alone():
    torch, cq = torch_cuda(), cq_built()
    for n, dtype in ((1, "f32"), (1, "bf16"), (150, "f32"), (150, "bf16")):
        c = _case(torch, cq, 8, dtype, 4, 2, 64, 16, [300], [n])
        want, wl = _run(torch, cq, c)
        c["q"][n // 2, 2, 7] = float("nan")
        out, lse = _run(torch, cq, c)
        assert torch.isnan(out[n // 2, 2].float()).all() and torch.isnan(lse[n // 2, 2])
        out[n // 2, 2], lse[n // 2, 2] = want[n // 2, 2], wl[n // 2, 2]
        assert torch.equal(out, want) and torch.equal(lse, wl)


def test_same_bits_each_time_and_workspace_left_clean():
    """Results do not depend on timing, the workspace is left zeroed where it has to be, padding rows stay."""
    torch, cq = torch_cuda(), cq_built()
    kv, new = [5000, 70, 9000, 1, 333], [1, 1, 1, 1, 1]
    c = _case(torch, cq, 3, "bf16", 8, 2, 128, 16, kv, new, T_extra=3)
    ws = cq.attn_workspace_t(8, 2, 128)
    out = torch.full((c["T"], 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    _, first = _run(torch, cq, c, ws=ws, out=out)
    a = out.clone()
    assert (out[5:] == 7.0).all()
    for _ in range(5):
        out.zero_()
        _run(torch, cq, c, ws=ws, out=out, lse=None)
        assert torch.equal(out[:5], a[:5])
    d = _case(torch, cq, 5, "f32", 16, 2, 64, 32, [3000, 2000], [1, 3])
    _check(d, *_run(torch, cq, d, ws=cq.attn_workspace_t(16, 2, 64)))
    _check(d, *_run(torch, cq, d, ws=ws if ws.numel() >= cq.cq_attn_workspace_size(16, 2, 64) else None))
    _check(c, out, None)


@pytest.mark.parametrize("max_new,max_kv", [(1, 1), (0, 0), (10 ** 6, 10 ** 7)])
def test_hints_do_not_change_what_is_right(max_new, max_kv):
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, 3, "bf16", 8, 2, 64, 16, [900, 60, 200], [1, 60, 150])
    _check(c, *_run(torch, cq, c, max_new=max_new, max_kv=max_kv))


def test_many_requests():
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(0)
    kv = rng.integers(1, 60, 1500)
    c = _case(torch, cq, 1, "f16", 4, 2, 64, 16, kv, np.ones(1500, np.int32))
    _check(c, *_run(torch, cq, c))


def test_side_stream_and_graph():
    """A large pool, a side stream, and a captured graph replayed with other lengths."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, 3, "f32", 4, 2, 128, 128, [500, 260], [1, 140])
    n, H, P, D = c["k"].shape
    far = [20000 - 1 - i for i in range(n)]
    pool = torch.zeros((2, 20000, H, P, D), dtype=torch.int8, device="cuda")
    scales = torch.zeros((2, 20000, H), device="cuda")
    pool[0, far], pool[1, far] = dev(torch, c["k"]), dev(torch, c["v"])
    scales[0, far], scales[1, far] = dev(torch, c["ks"]), dev(torch, c["vs"])
    far_cache = cq.KVCache(pool[0], pool[1], scales[0], scales[1])
    table = c["table"].copy()
    want = _run(torch, cq, c)
    far_table = np.where(table >= 0, np.array(far)[np.maximum(table, 0)], -1).astype(np.int32)
    ws = cq.attn_workspace_t(4, 2, 128)
    t_table, t_kv, t_qs = dev(torch, far_table), dev(torch, c["kv"]), dev(torch, c["q_start"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = cq.attn_paged_t(c["q"], far_cache, t_table, t_kv, t_qs, 140, 500, ws=ws)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    out = torch.zeros_like(want[0])
    with torch.cuda.graph(graph):
        cq.attn_paged_t(c["q"], far_cache, t_table, t_kv, t_qs, 140, 500, ws=ws, out=out, lse=None)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])
    c["kv"] = np.array([333, 200], np.int32)
    t_kv.copy_(dev(torch, c["kv"]))
    graph.replay()
    torch.cuda.synchronize()
    _check(c, out, None)


def test_offsets_past_32_bits():
    """A cache of more than 4 GB a side: pages at both ends of it."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, 3, "bf16", 128, 64, 64, 128, [300, 200], [1, 100])
    n, H, P, D = c["k"].shape
    pages = (1 << 32) // (H * P * D) + 8
    pool = torch.zeros((pages, H, P, D), dtype=torch.int8, device="cuda")
    vals = torch.zeros((pages, H, P, D), dtype=torch.int8, device="cuda")
    ids = [pages - 1 - i if i % 2 else i for i in range(n)]
    ks, vs = torch.zeros((pages, H), device="cuda"), torch.zeros((pages, H), device="cuda")
    pool[ids], vals[ids] = dev(torch, c["k"]), dev(torch, c["v"])
    ks[ids], vs[ids] = dev(torch, c["ks"]), dev(torch, c["vs"])
    want = _run(torch, cq, c)
    c["cache"] = cq.KVCache(pool, vals, ks, vs)
    c["table"] = np.where(c["table"] >= 0, np.array(ids)[np.maximum(c["table"], 0)], -1).astype(np.int32)
    got = _run(torch, cq, c)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,Hq,H,P", [(64, 8, 2, 16), (128, 4, 1, 64), (128, 7, 1, 16), (64, 4, 4, 128)])
@pytest.mark.parametrize("kv,n", [([3000], [40]), ([5000, 2111], [100, 64]), ([1500, 90, 4100], [70, 90, 1])])
def test_few_rows_over_long_contexts(dtype, D, Hq, H, P, kv, n):
    """Chunks of some tens of tokens: work split over the keys and joined."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, [D, Hq, kv[0]], dtype, Hq, H, D, P, kv, n)
    for causal, window in ((True, 0), (True, 700), (False, 0), (False, 2000)):
        _check(c, *_run(torch, cq, c, causal=causal, window=window), causal=causal, window=window)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_chunk_among_many_tokens(dtype):
    """More requests than a warp looks over at once, one of them a chunk; a workspace used again by another shape."""
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(7)
    ws = None
    for R, at, n in ((70, 66, 150), (500, 3, 60), (2, 0, 50)):
        kv = rng.integers(1, 400, R)
        new = np.ones(R, np.int32)
        kv[at], new[at] = 2500, n
        c = _case(torch, cq, R, dtype, 8, 2, 64, 16, kv, new)
        ws = cq.attn_workspace_t(8, 2, 64) if ws is None else ws
        out, lse = _run(torch, cq, c, ws=ws)
        _check(c, out, lse)
        again = _run(torch, cq, c, ws=ws)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
