"""Attention over the 8-bit cache at the ends of its ranges: value scales, windows and lengths."""
import os

import numpy as np
import pytest

from helpers import cq_built, dev, torch_cuda
from test_gpu_attn import _case, _check, _run

pytestmark = pytest.mark.gpu


def _value_scales(torch, c, scales):
    """The cache's value scales, page by page of the table; blocks of scale 0 hold zeros."""
    pages = [int(p) for row in c["table"] for p in row if p >= 0]
    for i, page in enumerate(pages):
        c["vs"][page] = scales[i % len(scales)]
        if scales[i % len(scales)] == 0.0:
            c["v"][page] = 0
    c["cache"].v.copy_(dev(torch, c["v"]))
    c["cache"].v_scale.copy_(dev(torch, c["vs"]))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 3, 200])
@pytest.mark.parametrize("small", [1e-4, 1e-6, 1e-8, 1e-10, 1e-15])
def test_zero_blocks_beside_small_ones(dtype, n, small):
    """Blocks of zeros count in the sum alone: the others keep their bits however small their scale (fp16 results of
    the smallest are zero: of those, lse alone says something)."""
    torch, cq = torch_cuda(), cq_built()
    for zeros in ([0.0, small, small], [0.0, small], [small, 0.0, 0.0, 0.0]):
        c = _case(torch, cq, [n, len(zeros)], dtype, 4, 2, 64, 16, [400], [n])
        _value_scales(torch, c, zeros)
        _check(c, *_run(torch, cq, c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,D,kv,n", [(4, 64, [400], [1]), (4, 64, [400], [200]), (8, 128, [9000], [1]),
                                       (4, 64, [6000], [30]), (8, 128, [300, 5000], [100, 5])])
@pytest.mark.parametrize("scales", [[2.0 ** -126], [2.0 ** -120, 1.5 * 2.0 ** -118], [2.0 ** -116, 2.0 ** -60, 2.0 ** -30],
                                    [2.0 ** 60], [2.0 ** 60, 1.0, 2.0 ** -30]])
def test_value_scales_of_any_size(dtype, Hq, D, kv, n, scales):
    """The sum of the probabilities does not depend on the values' size."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, [D, kv[0]], dtype, Hq, 2, D, 16, kv, n)
    _value_scales(torch, c, scales)
    _check(c, *_run(torch, cq, c))


@pytest.mark.parametrize("n", [1, 200])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 63 - 1])
def test_windows_wider_than_any_length(n, causal, window):
    """... leave everything to be seen, by tokens in front of the cache's first key too (more new tokens than keys)."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, 5, "bf16", 4, 2, 64, 16, [300, 150, 3], [n, 190, 5])
    _check(c, *_run(torch, cq, c, causal=causal, window=window), causal=causal, window=2 ** 31 - 1)


def _longest(torch, cq, dtype, n, P=16, pages=4096):
    """A request of as many tokens as a table takes, 2^31 - P, whose pages are a few over and over."""
    rng = np.random.default_rng([n, pages])
    blocks = 2 ** 31 // P - 1
    k = np.clip(np.round(rng.standard_normal((pages, 1, P, 64)) * 36), -127, 127).astype(np.int8)
    v = np.clip(np.round(rng.standard_normal((pages, 1, P, 64)) * 36), -127, 127).astype(np.int8)
    s = (0.02 + 0.015 * rng.random((2, pages, 1))).astype(np.float32)
    cache = cq.KVCache(dev(torch, k), dev(torch, v), dev(torch, s[0]), dev(torch, s[1]))
    table = (torch.arange(blocks, device="cuda", dtype=torch.int32) % pages)[None]
    q = dev(torch, (2.0 * rng.standard_normal((n, 1, 64))).astype(np.float32)).to(dtype)
    lens = dev(torch, np.array([blocks * P], np.int32)), dev(torch, np.array([0, n], np.int32))
    return q, cache, table, lens, k, v, s, blocks


@pytest.mark.parametrize("n", [1, 50, 300])
@pytest.mark.parametrize("dtype,P", [("float32", 16), ("bfloat16", 16), ("bfloat16", 32)])
def test_window_at_the_end_of_the_longest_request(dtype, n, P):
    """The same as a request that holds the last pages alone. (The tiles begin at other keys there: other roundings,
    of some 1e-6 in fp32; in bfloat16 of 2^-12 in the probabilities, and of a place in the result.)"""
    torch, cq = torch_cuda(), cq_built()
    q, cache, table, (kv, start), *_, blocks = _longest(torch, cq, getattr(torch, dtype), n, P)
    out, lse = cq.attn_paged_t(q, cache, table, kv, start, n, blocks * P, window=100)
    tail = 1 + (n + 100) // P + 8
    short = table[:, -tail:].contiguous()
    want, wl = cq.attn_paged_t(q, cache, short, dev(torch, np.array([tail * P], np.int32)), start, n, tail * P, window=100)
    tol = dict(atol=1e-5, rtol=1e-5) if dtype == "float32" else dict(atol=2.0 ** -9, rtol=2.0 ** -7)
    torch.testing.assert_close(out, want, **tol)
    torch.testing.assert_close(lse, wl, atol=1e-5, rtol=1e-5)
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("n", [1, 64])
def test_every_key_of_the_longest_request_counts(n):
    """Queries of zero: lse is the logarithm of the number of keys. A CTA adds up to kv / 150 / 16 terms one after
    another in fp32, each addition off by 2^-24 of the sum at most: 5.4e-2 in all."""
    torch, cq = torch_cuda(), cq_built()
    q, cache, table, (kv, start), *_ = _longest(torch, cq, torch.bfloat16, n)
    _, lse = cq.attn_paged_t(torch.zeros_like(q), cache, table, kv, start, n, 2 ** 31 - 16, causal=False)
    assert (lse.double() - np.log(2.0 ** 31 - 16)).abs().max().item() <= 5.4e-2


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_both_kernels_take_the_same_factors_from_a_scale(dtype, D):
    """Zero queries that see one key each: nothing but the value scale's factors is left in lse, and both kernels (the
    hint of no new tokens sends wide requests to the one for few rows) have the same bits. (fp32 has another offset in
    each, which rounds.)"""
    torch, cq = torch_cuda(), cq_built()
    R, n = 60, 45
    c = _case(torch, cq, D, dtype, 4, 4, D, 16, [1] * R, [n] * R)
    c["q"].zero_()
    wide = _run(torch, cq, c, causal=False)
    few = _run(torch, cq, c, causal=False, max_new=0)
    assert torch.equal(wide[1], few[1])
    _check(c, *wide, causal=False)
    _check(c, *few, causal=False)


@pytest.mark.parametrize("max_new,max_kv", [(2 ** 62, 0), (2 ** 63 - 1, 2 ** 63 - 1)])
def test_hints_of_any_size(max_new, max_kv):
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, 3, "bf16", 8, 2, 64, 16, [900, 60, 200], [1, 60, 150])
    want = _run(torch, cq, c)
    out, lse = _run(torch, cq, c, max_new=max_new, max_kv=max_kv)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 128)])
def test_a_workspace_holds_anything_behind_its_zeros(dtype, D):
    """Work shared over the keys in both kernels, and joined: nothing is read that the call has not written. Every byte
    is 0xff, numbers that are not finite, but for the first ones, which the call leaves zero."""
    torch, cq = torch_cuda(), cq_built()
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "cq_kv.h")
    assert f"#define CQ_ATTN_WORKSPACE_ZERO {cq.ATTN_WORKSPACE_ZERO}\n" in open(header).read()
    for kv, new in (([40000], [1]), ([9000, 300, 20], [100, 1, 20]), ([3000] * 30, [1] * 30)):
        c = _case(torch, cq, kv[0], dtype, 8, 2, D, 16, kv, new)
        ws = cq.attn_workspace_t(8, 2, D)
        want = _run(torch, cq, c, ws=ws)
        assert not ws[:cq.ATTN_WORKSPACE_ZERO].any()
        ws[cq.ATTN_WORKSPACE_ZERO:] = 255
        for _ in range(2):
            out, lse = _run(torch, cq, c, ws=ws)
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
            assert not ws[:cq.ATTN_WORKSPACE_ZERO].any()
        _check(c, out, lse)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,D,kv,n", [(4, 64, [400], [1]), (4, 64, [400], [200]), (4, 64, [6000], [30])])
@pytest.mark.parametrize("scales", [[2.0 ** 96], [1.7 * 2.0 ** 90, 2.0 ** 60, 2.0 ** 20], [2.0 ** -126, 2.0 ** -90]])
def test_value_scales_at_the_ends_of_their_range(dtype, Hq, D, kv, n, scales):
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, [D, kv[0], 1], dtype, Hq, 2, D, 16, kv, n)
    _value_scales(torch, c, scales)
    _check(c, *_run(torch, cq, c))


@pytest.mark.parametrize("n", [1, 150])
@pytest.mark.parametrize("page", [-1, -2 ** 31, 2 ** 31 - 1])
def test_any_page_outside_the_cache_is_flagged(n, page):
    torch, cq = torch_cuda(), cq_built()
    c = _case(torch, cq, 9, "bf16", 4, 2, 128, 32, [600], [n])
    c["table"][0, 3] = page
    cq.cq_read_global_status()
    out, lse = _run(torch, cq, c)
    assert cq.cq_read_global_status() == (cq.ERR_DEVICE_STATUS, cq.DEV_KV_PAGE)
    _check(c, out, lse)
