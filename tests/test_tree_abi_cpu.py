"""The calls of a tree decoding step without a GPU: arguments that they refuse before any launch, the reference's own
properties."""
import ctypes as C
import os
import re

import numpy as np
import pytest

import tree_ref
from gemm_gguf_block_gb300 import build, cq
from test_kv_abi_cpu import A, BAD_CACHES, cache


@pytest.fixture(scope="module")
def L():
    build.build()
    return cq.lib()


def test_every_declared_symbol_is_exported(L):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "cq_tree.h")).read()
    names = set(re.findall(r"^cq_status (cq_[a-z_]+)\(", text, re.M))
    assert len(names) == 6
    for n in names:
        assert hasattr(L, n) and n in cq.SIGNATURES, n
    for name, value in (("CQ_TREE_MAX", cq.TREE_MAX), ("CQ_DEV_TREE", cq.DEV_TREE), ("CQ_DEV_LOGITS", cq.DEV_LOGITS)):
        assert int(re.search(rf"#define {name}\s+(\w+)", text).group(1), 0) == value


def test_status_bits_are_distinct():
    bits = [getattr(cq, n) for n in dir(cq) if n.startswith("DEV_")]
    assert len(bits) == 10 and len(set(bits)) == 10 and all(b & (b - 1) == 0 for b in bits)


def test_rope_refusals(L):
    def call(i=cq.F32, o=cq.F32, T=2, hq=4, hk=2, D=64, rot=64, adj=0, q=A, qs=256, k=A, ks=128, pos=A, fr=A, qn=None,
             kn=None, eps=1e-6, qo=2 * A, qos=256, ko=2 * A, kos=128):
        return cq.cq_qk_rope(i, o, T, hq, hk, D, rot, adj, q, qs, k, ks, pos, fr, qn, kn, eps, qo, qos, ko, kos)
    for kw in (dict(i=2), dict(o=-1), dict(i=cq.F16), dict(i=cq.F16, o=cq.BF16), dict(i=cq.BF16, o=cq.F32)):
        assert call(**kw) == cq.ERR_UNSUPPORTED_FORMAT, kw
    for kw in (dict(T=-1), dict(hq=-1), dict(hk=-1), dict(rot=-8), dict(adj=2), dict(eps=-1e-9), dict(eps=float("nan")),
               dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(fr=None),
               dict(qo=A, qos=512), dict(ko=A, o=cq.BF16)):
        assert call(**kw) == cq.ERR_INVALID_ARG, kw
    for kw in (dict(D=96), dict(D=256), dict(D=0), dict(rot=60), dict(rot=72), dict(hq=1025, qs=1 << 20), dict(hk=1025),
               dict(T=1 << 31), dict(qs=255), dict(ks=127), dict(qos=0), dict(kos=-128), dict(qs=1 << 41)):
        assert call(**kw) == cq.ERR_SHAPE, kw
    for kw in (dict(q=A + 4), dict(k=A + 8), dict(qo=2 * A + 8), dict(qs=257), dict(o=cq.F16, kos=132), dict(pos=A + 2),
               dict(fr=A + 4), dict(qn=A + 4), dict(kn=A + 8)):
        assert call(**kw) == cq.ERR_ALIGNMENT, kw
    assert call(T=0, q=None, k=None, pos=None, fr=None) == cq.OK
    assert call(hq=0, hk=0, q=None, k=None) == cq.OK


def test_plan_refusals(L):
    def call(R=2, T=5, kv=A, qs=A, parent=A, mask=A, pos=A):
        return cq.cq_tree_plan(R, T, kv, qs, parent, mask, pos)
    for kw in (dict(R=-1), dict(T=-1), dict(kv=None), dict(qs=None), dict(parent=None)):
        assert call(**kw) == cq.ERR_INVALID_ARG, kw
    for kw in (dict(R=16385), dict(T=1 << 31)):
        assert call(**kw) == cq.ERR_SHAPE, kw
    for kw in (dict(kv=A + 2), dict(qs=A + 1), dict(parent=A + 2), dict(mask=A + 4), dict(pos=A + 2)):
        assert call(**kw) == cq.ERR_ALIGNMENT, kw
    assert call(T=0, parent=None) == cq.OK and call(mask=None, pos=None) == cq.OK


def test_attn_refusals(L):
    c = cache()
    p = C.addressof(c)

    def call(cc=p, dt=cq.F32, R=2, T=3, hq=8, mn=3, q=A, qs=512, table=A, mb=4, kv=A, start=A, mask=A, out=A, os_=512,
             lse=None, ws=A, wb=1 << 30):
        return cq.cq_attn_tree(cc, dt, R, T, hq, mn, q, qs, table, mb, kv, start, mask, 1.0, out, os_, lse, ws, wb)
    assert call(dt=2) == cq.ERR_UNSUPPORTED_FORMAT
    for kw in (dict(cc=None), dict(R=-1), dict(T=-1), dict(mn=-1), dict(mb=-1), dict(q=None), dict(out=None), dict(kv=None),
               dict(start=None), dict(table=None), dict(mask=None)):
        assert call(**kw) == cq.ERR_INVALID_ARG, kw
    for kw in (dict(hq=6), dict(hq=0), dict(R=16385), dict(T=1 << 31), dict(mb=1 << 27), dict(qs=511), dict(os_=0)):
        assert call(**kw) == cq.ERR_SHAPE, kw
    for kw in (dict(ws=None), dict(wb=16)):
        assert call(**kw) == cq.ERR_WORKSPACE, kw
    for kw in (dict(q=A + 4), dict(mask=A + 4), dict(lse=A + 2), dict(kv=A + 2), dict(ws=A + 16)):
        assert call(**kw) == cq.ERR_ALIGNMENT, kw
    assert call(T=0, mask=None) == cq.OK and call(R=0, mask=None) == cq.OK


def test_verify_refusals(L):
    def call(R=2, T=5, V=100, z=A, zs=100, d=None, ds=0, tok=A, par=A, qs=A, temp=A, ua=A, us=A, mp=4, cnt=A, path=A, nx=A):
        return cq.cq_tree_verify(R, T, V, z, zs, d, ds, tok, par, qs, temp, ua, us, mp, cnt, path, nx)
    for kw in (dict(R=-1), dict(T=-1), dict(V=0), dict(mp=0), dict(z=None), dict(tok=None), dict(par=None), dict(qs=None),
               dict(temp=None), dict(ua=None), dict(us=None), dict(cnt=None), dict(path=None), dict(nx=None)):
        assert call(**kw) == cq.ERR_INVALID_ARG, kw
    for kw in (dict(R=16385), dict(T=1 << 31), dict(V=262145, zs=1 << 20), dict(mp=65), dict(zs=99), dict(d=A, ds=99),
               dict(zs=1 << 41), dict(d=A, ds=1 << 41)):
        assert call(**kw) == cq.ERR_SHAPE, kw
    for kw in (dict(z=A + 2), dict(d=A + 1, ds=100), dict(tok=A + 2), dict(nx=A + 1), dict(path=A + 2)):
        assert call(**kw) == cq.ERR_ALIGNMENT, kw
    assert call(R=0, z=None) == cq.OK


def test_move_refusals(L):
    c = cache()
    p = C.addressof(c)

    def call(cc=p, R=2, table=A, mb=4, kv=A, qs=A, cnt=A, path=A, mp=4, new=A):
        return cq.cq_kv_move(cc, R, table, mb, kv, qs, cnt, path, mp, new)
    for bad, want in BAD_CACHES:
        b = cache(**bad)
        assert call(cc=C.addressof(b)) == want
    for kw in (dict(cc=None), dict(R=-1), dict(mb=-1), dict(mp=0), dict(table=None), dict(kv=None), dict(qs=None),
               dict(cnt=None), dict(path=None)):
        assert call(**kw) == cq.ERR_INVALID_ARG, kw
    for kw in (dict(R=16385), dict(mp=65), dict(mb=1 << 27)):
        assert call(**kw) == cq.ERR_SHAPE, kw
    for kw in (dict(table=A + 2), dict(path=A + 1), dict(new=A + 2)):
        assert call(**kw) == cq.ERR_ALIGNMENT, kw
    assert call(R=0, kv=None) == cq.OK


def test_release_refusals(L):
    def call(R=2, P=16, table=A, mb=4, pages=10, old=A, new=A, freed=A, cap=7, used=A):
        return cq.cq_kv_release(R, P, table, mb, pages, old, new, freed, cap, used)
    for kw in (dict(R=-1), dict(mb=-1), dict(pages=-1), dict(cap=-1), dict(table=None), dict(old=None), dict(new=None),
               dict(freed=None), dict(used=None)):
        assert call(**kw) == cq.ERR_INVALID_ARG, kw
    for kw in (dict(P=8), dict(P=48), dict(R=16385), dict(cap=1 << 31), dict(pages=1 << 31), dict(mb=1 << 27)):
        assert call(**kw) == cq.ERR_SHAPE, kw
    for kw in (dict(table=A + 2), dict(old=A + 1), dict(freed=A + 2), dict(used=A + 2)):
        assert call(**kw) == cq.ERR_ALIGNMENT, kw


def test_reference_verification_keeps_the_distribution():
    """One draft drawn from q, kept or replaced as the rule says, is distributed as p: exact over a grid of the numbers."""
    p, q = np.array([0.5, 0.25, 0.125, 0.125]), np.array([0.125, 0.5, 0.25, 0.125])
    logits = np.log(np.stack([p, p])).astype(np.float32)
    got, m = np.zeros(4), 64
    for x in range(4):
        for ua in (np.arange(m) + 0.5) / m:
            for us in (np.arange(m) + 0.5) / m:
                c, path, nxt, _ = tree_ref.verify(logits, [0, x], [-1, 0], [0, 2], [1.0], [0.0, ua], [us], 2,
                                                  np.stack([q, q]).astype(np.float32))
                got[x if c[0] == 2 else nxt[0]] += q[x] / m / m
                if c[0] == 2:
                    break                                # (the last token does not depend on what is kept)
            else:
                continue
            got[x] += q[x] / m / m * (m - 1)
    assert np.abs(got - p).max() < 2 / m


def test_reference_moves_rows_as_they_are_where_scales_are_alike():
    rng = np.random.default_rng(0)
    q = rng.integers(-127, 128, (4, 2, 16, 64)).astype(np.int8)
    scale = np.full((4, 2), 0.5, np.float32)
    was = q.copy()
    table = np.array([[2, 0]], np.int32)
    new, bits = tree_ref.move(q, scale, table, [14 + 10], [0, 10], [3], np.array([[0, 4, 9]], np.int32))
    assert new.tolist() == [17] and bits == 0
    assert (q[2, :, 15] == was[0, :, 2]).all() and (q[0, :, 0] == was[0, :, 7]).all() and (q[2, :, :15] == was[2, :, :15]).all()
