"""The 8-bit paged cache on the GPU: block tables and slot maps, rows written and read back."""
import numpy as np
import pytest

import kv_ref
from helpers import cq_built, dev, torch_cuda

pytestmark = pytest.mark.gpu


def _tdtype(torch, name):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _requests(rng, R, past_max, new_max, zeros=True):
    past = rng.integers(0, past_max + 1, R)
    new = rng.integers(0 if zeros else 1, new_max + 1, R)
    return past.astype(np.int32), new.astype(np.int32)


def _table(rng, past, new, P, extra=2):
    """A table with the past tokens' pages filled in, the free pages, and the size of the pool."""
    have, total = -(-past // P), -(-(past + new) // P)
    pages = int(total.sum()) + 3
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(past), int(total.max(initial=0)) + extra), -1, np.int32)
    at = 0
    for r, h in enumerate(have):
        table[r, :h] = order[at:at + h]
        at += h
    return table, order[at:].copy(), pages


def _run_plan(torch, cq, past, new, table, free, P, pages, T):
    t = dev(torch, table)
    got = cq.kv_plan_t(dev(torch, past), dev(torch, new), t, dev(torch, free), P, pages, T)
    return [x.cpu().numpy() for x in (t, *got)]


def _check_plan(torch, cq, past, new, table, free, P, pages, T):
    got = _run_plan(torch, cq, past, new, table, free, P, pages, T)
    want = kv_ref.plan(past, new, table, free, P, pages, T)
    for g, w, name in zip(got, want, ("table", "kv_len", "q_start", "slots", "positions", "used")):
        assert np.array_equal(g, w), name
    return got


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("R,past_max,new_max", [(1, 0, 1), (1, 500, 1), (3, 40, 70), (64, 900, 1), (511, 50, 9),
                                                (513, 300, 40), (1100, 20, 3)])
def test_plan(P, R, past_max, new_max):
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(R + P)
    past, new = _requests(rng, R, past_max, new_max)
    table, free, pages = _table(rng, past, new, P)
    got = _check_plan(torch, cq, past, new, table, free, P, pages, int(new.sum()) + 5)
    assert got[-1][1] == 0
    # the updated table gives the same again
    again = _run_plan(torch, cq, past, new, got[0], free, P, pages, int(new.sum()) + 5)
    assert all(np.array_equal(a, b) for a, b in zip(got, again))


def test_plan_exact_pages_and_zeros():
    """Lengths at page borders, requests without new tokens, all of them without any."""
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(1)
    past = np.array([0, 16, 15, 17, 32, 0, 31, 1], np.int32)
    for new in ([16, 16, 1, 15, 0, 0, 2, 47], [0] * 8):
        new = np.array(new, np.int32)
        table, free, pages = _table(rng, past, new, 16)
        _check_plan(torch, cq, past, new, table, free, 16, pages, int(new.sum()))
        _check_plan(torch, cq, past, new, table, free, 16, pages, int(new.sum()) + 700)


@pytest.mark.parametrize("R", [5, 700])
def test_plan_faults(R):
    """What does not fit is left out and flagged; the rest is as without it."""
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(R)
    past, new = _requests(rng, R, 100, 60)
    table, free, pages = _table(rng, past, new, 16)
    T = int(new.sum())
    assert _check_plan(torch, cq, past, new, table, free[:len(free) // 2], 16, pages, T)[-1][1] == cq.DEV_KV_PAGES
    assert _check_plan(torch, cq, past, new, table, free[:0], 16, pages, T)[-1][1] == cq.DEV_KV_PAGES
    assert _check_plan(torch, cq, past, new, table[:, :5], free, 16, pages, T)[-1][1] == cq.DEV_KV_BLOCKS
    assert _check_plan(torch, cq, past, new, table, free, 16, pages, T // 2)[-1][1] & cq.DEV_KV_TOKENS
    bad = free.copy()
    bad[[0, 2]] = [pages, -7]
    assert _check_plan(torch, cq, past, new, table, bad, 16, pages, T)[-1][1] == cq.DEV_KV_PAGE
    minus = new.copy()
    minus[1], new[2] = -5, 3
    assert _check_plan(torch, cq, past, minus, table, free, 16, pages, T)[-1][1] == cq.DEV_KV_LENGTH
    part = past.copy()
    part[2] = 17                                        # its second page is partly filled
    table[2, 1] = pages + 4
    assert _check_plan(torch, cq, part, new, table, free, 16, pages, T)[-1][1] & cq.DEV_KV_PAGE


def test_plan_no_requests():
    torch, cq = torch_cuda(), cq_built()
    z = np.zeros(0, np.int32)
    got = _run_plan(torch, cq, z, z, np.zeros((0, 4), np.int32), z, 16, 0, 9)
    assert got[2].tolist() == [0] and got[5].tolist() == [0, 0] and (got[3] == -1).all() and (got[4] == -1).all()


def _cache(torch, cq, rng, pages, H, P, D, joint=False):
    q = rng.integers(-127, 128, (2, pages, H, P, D)).astype(np.int8)
    s = (0.01 + 0.03 * rng.random((2, pages, H))).astype(np.float32)
    if joint:                                           # keys and values of a page side by side
        tq = dev(torch, np.ascontiguousarray(q.transpose(1, 0, 2, 3, 4)))
        ts = dev(torch, np.ascontiguousarray(s.transpose(1, 0, 2)))
        return cq.KVCache(tq[:, 0], tq[:, 1], ts[:, 0], ts[:, 1]), q, s
    tq, ts = dev(torch, q), dev(torch, s)
    return cq.KVCache(tq[0], tq[1], ts[0], ts[1]), q, s


def _same_cache(cache, q, s):
    for i, (tq, ts) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        assert np.array_equal(ts.cpu().numpy(), s[i], equal_nan=True)
        assert np.array_equal(tq.cpu().numpy(), q[i])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 16), (128, 32), (64, 128), (128, 128)])
@pytest.mark.parametrize("R,H,past_max,new_max", [(1, 1, 0, 1), (9, 2, 70, 1), (5, 3, 40, 150), (40, 8, 200, 2)])
def test_append(dtype, D, P, R, H, past_max, new_max):
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng([D, P, R, H])
    past, new = _requests(rng, R, past_max, new_max, zeros=R > 1)
    table, free, pages = _table(rng, past, new, P)
    T = int(new.sum()) + 3
    slots = kv_ref.plan(past, new, table, free, P, pages, T)[3]
    cache, q, s = _cache(torch, cq, rng, pages, H, P, D, joint=R == 5)
    x = rng.standard_normal((T, 3 * H * D)) * np.exp(rng.uniform(-3, 3, (T, 1)))    # rows of unequal size: scales grow
    rows = dev(torch, x.astype(np.float32)).to(_tdtype(torch, dtype))
    k, v = rows[:, H * D:2 * H * D], rows[:, 2 * H * D:]
    ts = dev(torch, slots)
    cq.kv_append_t(cache, k, v, ts)
    kv_ref.append(q[0], s[0], k.float().cpu().numpy().reshape(T, H, D), slots)
    kv_ref.append(q[1], s[1], v.float().cpu().numpy().reshape(T, H, D), slots)
    _same_cache(cache, q, s)
    cq.kv_append_t(cache, k, v, ts)                     # once more: nothing moves
    _same_cache(cache, q, s)
    # in 64 bits: every new value within half a step of what was given
    on = slots >= 0
    back = cq.kv_read_t(cache, ts)
    for i, given in enumerate((k, v)):
        step = s[i][slots[on] // P].astype(np.float64)[:, :, None]
        off = np.abs(back[i].cpu().numpy().astype(np.float64)[on] - given.double().cpu().numpy().reshape(T, H, D)[on])
        assert (off <= step * (0.5 + 1e-4)).all()
        assert (back[i].cpu().numpy()[~on] == 0).all()


def test_append_edge_values():
    """Zero blocks, subnormal and huge values, ties, infinities and NaN; a page begun anew forgets its scale."""
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(5)
    H, P, D, pages = 1, 16, 64, 12
    cache, q, s = _cache(torch, cq, rng, pages, H, P, D)
    x = rng.standard_normal((pages * 2, H, D)).astype(np.float32)
    x[0] = 0.0
    x[1] = 1e-40
    x[2] = 3e38
    x[3] = np.round(x[3] * 40) + 0.5                    # with 127 in the row: exact halves
    x[3, 0, 0] = 127.0
    x[4, 0, 3] = np.nan
    x[5, 0, 9] = -np.inf
    x[6] = 1e-36
    x[7] = 0.0
    slots = np.concatenate([np.arange(pages) * P + np.array([0, 0, 0, 0, 0, 7, 3, 5, 9, 0, 15, 1]), np.full(pages, -1)])
    for name in ("first", "second"):                    # the second meets NaN scales from the first
        cq.kv_append_t(cache, dev(torch, x), dev(torch, x[::-1].copy()), dev(torch, slots))
        kv_ref.append(q[0], s[0], x, slots)
        kv_ref.append(q[1], s[1], x[::-1], slots)
        _same_cache(cache, q, s)
        slots = slots.copy()
        slots[:pages] = (slots[:pages] // P) * P + (slots[:pages] % P + 1) % P
        x = rng.standard_normal(x.shape).astype(np.float32)


def test_append_and_read_skip_what_is_outside():
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(6)
    cache, q, s = _cache(torch, cq, rng, 3, 2, 16, 64)
    slots = np.array([-1, 3 * 16, 17, 1 << 40, 2, -(1 << 50)], np.int64)
    x = rng.standard_normal((6, 2, 64)).astype(np.float32)
    cq.cq_read_global_status()
    cq.kv_append_t(cache, dev(torch, x), dev(torch, x), dev(torch, slots))
    assert cq.cq_read_global_status() == (cq.ERR_DEVICE_STATUS, cq.DEV_KV_PAGE)
    for i in range(2):
        kv_ref.append(q[i], s[i], x, slots)
    _same_cache(cache, q, s)
    k, v = cq.kv_read_t(cache, dev(torch, slots))
    assert cq.cq_read_global_status() == (cq.ERR_DEVICE_STATUS, cq.DEV_KV_PAGE)
    for i, got in enumerate((k, v)):
        want = np.zeros((6, 2, 64), np.float32)
        for t in (2, 4):
            page, row = divmod(int(slots[t]), 16)
            want[t] = q[i][page, :, row].astype(np.float32) * s[i][page][:, None]
        assert np.array_equal(got.cpu().numpy(), want)
    assert cq.cq_read_global_status() == (cq.OK, 0)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,H,D,P", [(1, 1, 64, 16), (37, 3, 128, 64), (1000, 8, 64, 32)])
def test_read(dtype, T, H, D, P):
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(T)
    cache, q, s = _cache(torch, cq, rng, 20, H, P, D, joint=True)
    slots = rng.integers(0, 20 * P, T)
    k, v = cq.kv_read_t(cache, dev(torch, slots), _tdtype(torch, dtype))
    for i, got in enumerate((k, v)):
        exact = q[i][slots // P, :, slots % P].astype(np.float32) * s[i][slots // P][:, :, None]
        want = torch.from_numpy(exact).to(_tdtype(torch, dtype))
        assert torch.equal(got.cpu(), want)


def test_far_pages_and_another_stream():
    """Pages whose offsets pass 32 bits, on a side stream and in a captured graph."""
    torch, cq = torch_cuda(), cq_built()
    H, P, D = 64, 128, 128                              # 1 MB a page and side: 2^32 bytes at page 4096
    n = 4100
    kv = torch.zeros((2, n, H, P, D), dtype=torch.int8, device="cuda")
    sc = torch.zeros((2, n, H), dtype=torch.float32, device="cuda")
    cache = cq.KVCache(kv[0], kv[1], sc[0], sc[1])
    rng = np.random.default_rng(3)
    slots = np.array([4098 * P + 5, 4098 * P + 6, 2049 * P + 127, 4099 * P], np.int64)
    x = rng.standard_normal((2, 4, H, D)).astype(np.float32)
    q, s = np.zeros((2, 3, H, P, D), np.int8), np.zeros((2, 3, H), np.float32)
    small = np.array([5, 6, P + 127, 2 * P])
    for i in range(2):
        kv_ref.append(q[i], s[i], x[i], small)
    side = torch.cuda.Stream()
    tk, tv, ts = dev(torch, x[0]), dev(torch, x[1]), dev(torch, slots)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cq.kv_append_t(cache, tk, tv, ts)
        got = cq.kv_read_t(cache, ts)
    side.synchronize()
    ids = [4098, 2049, 4099]
    assert np.array_equal(kv[:, ids].cpu().numpy(), q) and np.array_equal(sc[:, ids].cpu().numpy(), s)
    for i in range(2):
        want = q[i][small // P, :, small % P].astype(np.float32) * s[i][small // P][:, :, None]
        assert np.array_equal(got[i].cpu().numpy(), want)
    kv[:, ids] = 0
    sc.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cq.kv_append_t(cache, tk, tv, ts)
    assert (kv[:, ids] == 0).all()
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(kv[:, ids].cpu().numpy(), q) and np.array_equal(sc[:, ids].cpu().numpy(), s)
