"""The cache and attention calls without a GPU: arguments that they refuse before any launch."""
import ctypes as C
import os
import re

import pytest

from gemm_gguf_block_gb300 import build, cq

A = 1 << 20   # an aligned fake address: validation fails before it is ever used


@pytest.fixture(scope="module")
def L():
    build.build()
    return cq.lib()


def cache(**kw):
    a = dict(k=A, v=A, k_scale=A, v_scale=A, num_pages=10, page_stride=4 * 16 * 64, scale_stride=4, page_size=16,
             kv_heads=4, head_dim=64, reserved=0)
    a.update(kw)
    return cq.cq_kv_cache(*[a[n] for n, _ in cq.cq_kv_cache._fields_])


BAD_CACHES = [(dict(k=None), cq.ERR_INVALID_ARG), (dict(v_scale=None), cq.ERR_INVALID_ARG),
              (dict(num_pages=-1), cq.ERR_INVALID_ARG), (dict(num_pages=1 << 31), cq.ERR_SHAPE),
              (dict(page_size=8), cq.ERR_SHAPE), (dict(page_size=48), cq.ERR_SHAPE), (dict(head_dim=96), cq.ERR_SHAPE),
              (dict(kv_heads=0), cq.ERR_SHAPE), (dict(kv_heads=1025, page_stride=1 << 30, scale_stride=2000), cq.ERR_SHAPE),
              (dict(reserved=1), cq.ERR_SHAPE), (dict(page_stride=4 * 16 * 64 - 16), cq.ERR_SHAPE),
              (dict(scale_stride=3), cq.ERR_SHAPE), (dict(page_stride=4 * 16 * 64 + 8), cq.ERR_ALIGNMENT),
              (dict(k=A + 8), cq.ERR_ALIGNMENT), (dict(v=A + 4), cq.ERR_ALIGNMENT), (dict(k_scale=A + 2), cq.ERR_ALIGNMENT)]


def test_every_declared_symbol_is_exported(L):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "cq_kv.h")).read()
    names = set(re.findall(r"^(?:cq_status|size_t) (cq_[a-z_]+)\(", text, re.M))
    assert len(names) == 5
    for n in names:
        assert hasattr(L, n) and n in cq.SIGNATURES, n


def test_struct_layout(L):
    assert C.sizeof(cq.cq_kv_cache) == 4 * 8 + 3 * 8 + 4 * 4


def test_status_bits_are_distinct():
    bits = [cq.DEV_BAD_EXPERT_ID, cq.DEV_DUP_EXPERT_ID, cq.DEV_WAIT_TIMEOUT, cq.DEV_KV_LENGTH, cq.DEV_KV_BLOCKS,
            cq.DEV_KV_PAGES, cq.DEV_KV_TOKENS, cq.DEV_KV_PAGE]
    assert len({b for b in bits}) == len(bits) and all(b & (b - 1) == 0 for b in bits)


@pytest.mark.parametrize("bad,want", BAD_CACHES)
def test_bad_caches(L, bad, want):
    c = cache(**bad)
    p = C.addressof(c)
    assert cq.cq_kv_append(p, cq.F32, 1, A, 256, A, 256, A) == want
    assert cq.cq_kv_read(p, cq.F32, 1, A, A, A) == want
    assert cq.cq_attn_paged(p, cq.F32, 1, 1, 4, 1, 1, A, 256, A, 1, A, A, 1.0, 1, 0, A, 256, None, A, 1 << 30) == want


def test_plan_refusals(L):
    def call(R=2, P=16, mb=4, pages=10, past=A, new=A, free=A, n=3, table=A, T=5, kv=A, qs=A, slots=A, pos=A, used=A):
        return cq.cq_kv_plan(R, P, mb, pages, past, new, free, n, table, T, kv, qs, slots, pos, used)
    for kw in (dict(R=-1), dict(mb=-1), dict(pages=-1), dict(n=-1), dict(T=-1), dict(past=None), dict(new=None),
               dict(free=None), dict(table=None), dict(kv=None), dict(qs=None), dict(slots=None), dict(pos=None),
               dict(used=None)):
        assert call(**kw) == cq.ERR_INVALID_ARG, kw
    for kw in (dict(P=0), dict(P=24), dict(P=256), dict(R=16385), dict(T=1 << 31), dict(n=1 << 31), dict(pages=1 << 31),
               dict(mb=1 << 27)):
        assert call(**kw) == cq.ERR_SHAPE, kw
    for kw in (dict(past=A + 2), dict(table=A + 1), dict(slots=A + 4), dict(used=A + 2)):
        assert call(**kw) == cq.ERR_ALIGNMENT, kw


def test_append_refusals(L):
    c = cache()
    p = C.addressof(c)

    def call(cc=p, dt=cq.F32, T=2, k=A, ks=256, v=A, vs=256, slots=A):
        return cq.cq_kv_append(cc, dt, T, k, ks, v, vs, slots)
    assert call(dt=2) == cq.ERR_UNSUPPORTED_FORMAT and call(dt=-1) == cq.ERR_UNSUPPORTED_FORMAT
    for kw in (dict(cc=None), dict(T=-1), dict(k=None), dict(v=None), dict(slots=None)):
        assert call(**kw) == cq.ERR_INVALID_ARG, kw
    for kw in (dict(ks=255), dict(vs=0), dict(vs=-256), dict(T=1 << 31), dict(ks=1 << 41)):
        assert call(**kw) == cq.ERR_SHAPE, kw
    for kw in (dict(k=A + 4), dict(ks=257), dict(dt=cq.BF16, vs=260), dict(slots=A + 4)):
        assert call(**kw) == cq.ERR_ALIGNMENT, kw
    assert call(T=0, k=None, v=None, slots=None) == cq.OK


def test_read_refusals(L):
    c = cache()
    p = C.addressof(c)
    assert cq.cq_kv_read(p, 7, 1, A, A, A) == cq.ERR_UNSUPPORTED_FORMAT
    assert cq.cq_kv_read(None, cq.F32, 1, A, A, A) == cq.ERR_INVALID_ARG
    assert cq.cq_kv_read(p, cq.F32, -1, A, A, A) == cq.ERR_INVALID_ARG
    assert cq.cq_kv_read(p, cq.F32, 1, None, A, A) == cq.ERR_INVALID_ARG
    assert cq.cq_kv_read(p, cq.F32, 1 << 31, A, A, A) == cq.ERR_SHAPE
    assert cq.cq_kv_read(p, cq.F32, 1, A + 4, A, A) == cq.ERR_ALIGNMENT
    assert cq.cq_kv_read(p, cq.F32, 1, A, A + 8, A) == cq.ERR_ALIGNMENT
    assert cq.cq_kv_read(p, cq.F32, 0, None, None, None) == cq.OK
    assert cq.cq_kv_read(p, cq.F32, 5, A, None, None) == cq.OK


def test_attn_refusals(L):
    c = cache()
    p = C.addressof(c)
    need = cq.cq_attn_workspace_size(8, 4, 64)
    assert need > 0
    for a in ((0, 4, 64), (8, 0, 64), (9, 4, 64), (8, 4, 80), (2048, 4, 64), (-4, 4, 64)):
        assert cq.cq_attn_workspace_size(*a) == 0

    def call(cc=p, dt=cq.F32, R=2, T=3, hq=8, mn=1, mk=9, q=A, qs=512, table=A, mb=4, kv=A, start=A, scale=1.0, causal=1,
             window=0, out=A, os=512, lse=A, ws=A, wb=need):
        return cq.cq_attn_paged(cc, dt, R, T, hq, mn, mk, q, qs, table, mb, kv, start, scale, causal, window, out, os,
                                lse, ws, wb)
    assert call(dt=3) == cq.ERR_UNSUPPORTED_FORMAT
    for kw in (dict(cc=None), dict(R=-1), dict(T=-1), dict(hq=-8), dict(mn=-1), dict(mk=-1), dict(mb=-1), dict(window=-1),
               dict(causal=2), dict(q=None), dict(out=None), dict(table=None), dict(kv=None), dict(start=None)):
        assert call(**kw) == cq.ERR_INVALID_ARG, kw
    for kw in (dict(hq=0), dict(hq=9), dict(hq=1028), dict(R=16385), dict(T=1 << 31), dict(T=(1 << 29) + 1), dict(qs=511), dict(os=8),
               dict(mb=1 << 27)):
        assert call(**kw) == cq.ERR_SHAPE, kw
    for kw in (dict(q=A + 8), dict(out=A + 4), dict(qs=513), dict(dt=cq.F16, os=516), dict(kv=A + 1), dict(start=A + 2),
               dict(table=A + 2), dict(lse=A + 2), dict(ws=A + 16)):
        assert call(**kw) == cq.ERR_ALIGNMENT, kw
    for kw in (dict(ws=None), dict(wb=need - 1)):
        assert call(**kw) == cq.ERR_WORKSPACE, kw
    assert call(R=0, q=None, out=None, ws=None, wb=0) == cq.OK
    assert call(T=0, q=None, out=None, ws=None, wb=0) == cq.OK


def test_tensor_helpers_refuse(L):
    """The tensor helpers check types, shapes and layouts before they pass pointers on (host tensors: nothing runs)."""
    torch = pytest.importorskip("torch")
    k = torch.zeros(3, 2, 16, 64, dtype=torch.int8)
    s = torch.zeros(3, 2)
    c = cq.KVCache(k, k.clone(), s, s.clone())
    x, slots = torch.zeros(5, 128), torch.zeros(5, dtype=torch.int64)
    table, n = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q, qs, ws = torch.zeros(5, 4, 64), torch.zeros(3, dtype=torch.int32), torch.zeros(8, dtype=torch.uint8)
    for f in (lambda: cq.KVCache(k.float(), k.float(), s, s), lambda: cq.KVCache(k, k[:2], s, s),
              lambda: cq.KVCache(k, k, s[:, :1], s[:, :1]), lambda: cq.KVCache(k[..., :32], k[..., :32], s, s),
              lambda: cq.KVCache(k, k, s.double(), s.double()), lambda: cq.KVCache(k.transpose(1, 2), k.transpose(1, 2), s, s),
              lambda: cq.kv_append_t(c, x[:, :64], x, slots), lambda: cq.kv_append_t(c, x, x[:4], slots),
              lambda: cq.kv_append_t(c, x, x.half(), slots), lambda: cq.kv_append_t(c, x, x, slots.int()),
              lambda: cq.kv_append_t(c, x, x, slots[:4]), lambda: cq.kv_append_t(c, x.t().contiguous().t(), x, slots),
              lambda: cq.kv_append_t(c, x.double(), x.double(), slots), lambda: cq.kv_read_t(c, slots, torch.float64),
              lambda: cq.kv_read_t(c, slots.int()), lambda: cq.kv_plan_t(n.long(), n, table, n, 16, 3, 5),
              lambda: cq.kv_plan_t(n, n, table[:1], n, 16, 3, 5), lambda: cq.kv_plan_t(n, n, table[:, :2], n, 16, 3, 5),
              lambda: cq.attn_paged_t(q[..., :32], c, table, n, qs, 1, 1, ws=ws),
              lambda: cq.attn_paged_t(q, c, table, n, qs[:2], 1, 1, ws=ws),
              lambda: cq.attn_paged_t(q, c, table.long(), n, qs, 1, 1, ws=ws),
              lambda: cq.attn_paged_t(q, c, table, n, qs, 1, 1, ws=ws, out=q.half()),
              lambda: cq.attn_paged_t(q, c, table, n, qs, 1, 1, ws=ws, lse=torch.zeros(5, 3)),
              lambda: cq.attn_paged_t(q.transpose(0, 1), c, table, n, qs, 1, 1, ws=ws)):
        with pytest.raises((cq.CqError, AssertionError)):
            f()
