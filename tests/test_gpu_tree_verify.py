"""Verification of drafted tokens against its definition in 64 bits: the same tokens, paths and flags."""
import numpy as np
import pytest

import tree_ref
from helpers import cq_built, dev, torch_cuda

pytestmark = pytest.mark.gpu


def _case(seed, V, lens, temp=1.0, chain=False, draft=False, spread=3.0, pad=0, stride=0):
    rng = np.random.default_rng(seed)
    q_start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(q_start[-1]) + pad
    c = dict(logits=(rng.standard_normal((T, V + stride)) * spread).astype(np.float32), q_start=q_start, max_path=64,
             parent=np.full(T, -1, np.int32), tokens=rng.integers(0, V, T).astype(np.int32), draft=None, V=V,
             temperature=np.full(len(lens), temp, np.float32), u_accept=rng.random(T).astype(np.float32),
             u_sample=rng.random(len(lens)).astype(np.float32))
    if draft:
        c["draft"] = np.zeros((T, V + stride), np.float32)
        z = c["logits"][:, :V] + rng.standard_normal((T, V)) * 0.7
        e = np.exp((z - z.max(1, keepdims=True)) / max(temp, 0.1))
        c["draft"][:, :V] = e / e.sum(1, keepdims=True)
    for r, n in enumerate(lens):
        f = int(q_start[r])
        c["parent"][f:f + n] = tree_ref.random_parents(rng, n, chain) if n else []
        for i in range(1, min(n, 64)):
            p = f + int(c["parent"][f + i])
            if draft:
                c["tokens"][f + i] = min(np.searchsorted(np.cumsum(c["draft"][p, :V]), rng.random()), V - 1)
            else:                                        # one of the parent's likeliest tokens
                top = np.argsort(-c["logits"][p, :V])[:6]
                c["tokens"][f + i] = top[int(rng.integers(0, len(top)))]
    return c


def _run(torch, cq, c):
    V = c["V"]
    t = {k: dev(torch, v) for k, v in c.items() if isinstance(v, np.ndarray)}
    draft = t["draft"][:, :V] if c["draft"] is not None else None
    return cq.tree_verify_t(t["logits"][:, :V], t["tokens"], t["parent"], t["q_start"], t["temperature"], t["u_accept"],
                            t["u_sample"], c["max_path"], draft=draft)


def _check(torch, cq, c):
    V = c["V"]
    got = [x.cpu().numpy() for x in _run(torch, cq, c)]
    count, path, nxt, bits = tree_ref.verify(c["logits"][:, :V], c["tokens"], c["parent"], c["q_start"], c["temperature"],
                                             c["u_accept"], c["u_sample"], c["max_path"],
                                             None if c["draft"] is None else c["draft"][:, :V])
    assert np.array_equal(got[0], count) and np.array_equal(got[1], path)
    assert np.array_equal(got[2], nxt), np.argwhere(got[2] != nxt)[:5].tolist()
    assert cq.cq_read_global_status() == ((cq.ERR_DEVICE_STATUS, bits) if bits else (cq.OK, 0))
    return count, path, nxt


@pytest.mark.parametrize("V", [1, 2, 31, 257, 4096, 4097, 32003, 128256])
@pytest.mark.parametrize("temp", [0.0, 0.6, 1.0, 2.5])
@pytest.mark.parametrize("draft", [False, True])
def test_ragged(V, temp, draft):
    torch, cq = torch_cuda(), cq_built()
    lens = [6, 1, 0, 12, 3, 64, 2] if V < 100000 else [6, 1, 0, 12, 3]
    _check(torch, cq, _case([V, draft], V, lens, temp, draft=draft, pad=2))


@pytest.mark.parametrize("V", [300, 8191, 40001])
@pytest.mark.parametrize("draft", [False, True])
def test_chains_of_many_requests(V, draft):
    torch, cq = torch_cuda(), cq_built()
    count, _, _ = _check(torch, cq, _case(V, V, [5] * (200 if V < 10000 else 40), 0.9, chain=True, draft=draft))
    assert count.min() == 1 and count.max() > 1           # both outcomes are among them


@pytest.mark.parametrize("draft", [False, True])
def test_largest_vocabulary(draft):
    torch, cq = torch_cuda(), cq_built()
    _check(torch, cq, _case(7, 262144, [4, 7], 0.7, draft=draft))


@pytest.mark.parametrize("V,stride", [(1000, 1), (1000, 24), (5000, 3)])
def test_strided_rows(V, stride):
    torch, cq = torch_cuda(), cq_built()
    _check(torch, cq, _case(V + stride, V, [9, 5, 30], 1.0, draft=stride == 24, stride=stride))


@pytest.mark.parametrize("spread", [0.0, 0.01, 30.0, 1e4])
def test_flat_and_peaked(spread):
    """All logits alike: the distribution function has V equal steps; and one token above all others."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(11, 50000, [5] * 20, 1.0, spread=spread)
    _check(torch, cq, c)
    c["temperature"][:] = 0.0                            # ties go to the smallest index
    _check(torch, cq, c)


def test_several_rejections_at_one_node():
    """Twenty children of one token, drawn from the draft's probabilities: the residual of the residual, and so on."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(12, 3000, [21] * 30, 1.0, draft=True)
    rng = np.random.default_rng(0)
    for f in c["q_start"][:-1]:
        c["parent"][f + 1:f + 21] = 0
        c["tokens"][f + 1:f + 21] = np.minimum(np.searchsorted(np.cumsum(c["draft"][f, :3000]), rng.random(20)), 2999)
    c["u_accept"] = (1 - rng.random(len(c["u_accept"])) * 0.05).astype(np.float32)
    c["draft"] = c["draft"][rng.permutation(len(c["draft"]))]        # a draft that is wrong about everything
    _check(torch, cq, c)


def test_same_token_twice():
    """Siblings with one token: the second has nothing left. Tokens outside the vocabulary are never kept."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(13, 500, [6] * 50, 1.0)
    for f in c["q_start"][:-1]:
        c["parent"][f + 1:f + 6] = 0
        best = int(c["logits"][f].argmax())
        c["tokens"][f + 1:f + 6] = [best, best, -1, 500, best]
    _check(torch, cq, c)
    c["temperature"][:] = 0.0
    _check(torch, cq, c)


@pytest.mark.parametrize("u", [0.0, -1.0, float("nan"), 0.99999994, 1.0, 7.0])
def test_edges_of_the_random_numbers(u):
    torch, cq = torch_cuda(), cq_built()
    c = _case(14, 700, [5] * 10, 1.0)
    c["u_accept"][:] = u
    c["u_sample"][:] = u
    _check(torch, cq, c)


@pytest.mark.parametrize("t", [-1.0, float("nan"), 1e-30, 2.0 ** -64, 1e-6, 1e6, 2.0 ** 64, float("inf")])
def test_edges_of_the_temperature(t):
    torch, cq = torch_cuda(), cq_built()
    c = _case(15, 900, [5] * 10, 1.0)
    c["temperature"][:] = t
    _check(torch, cq, c)


def test_masked_logits():
    """-infinity and the type's lowest value among the logits, rows of the lowest value alone, and what has no
    distribution: NaN, +infinity, nothing finite -- flagged where it is reached."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(16, 1000, [3] * 8, 1.0, chain=True)
    z, low = c["logits"], np.finfo(np.float32).min
    z[0:3, ::2] = -np.inf
    z[3:6, 5:] = low
    z[6:9] = low
    c["u_accept"][:] = 0.5
    _check(torch, cq, c)
    z[9] = -np.inf
    z[12, 7] = np.nan
    z[15, 999] = np.inf
    z[18 + 2, 3] = np.nan                                # only if it is reached
    z[22] = -np.inf
    z[22, 500] = 1.0
    _check(torch, cq, c)


def test_bad_trees():
    torch, cq = torch_cuda(), cq_built()
    c = _case(17, 100, [5, 65, 4, 3], 0.0)
    c["parent"][1], c["parent"][3] = 1, -7
    f = int(c["q_start"][2])
    c["parent"][f + 1] = -1                              # hangs off the cache: never kept
    c["tokens"][:] = 3
    c["logits"][:, 3] = 50
    count, path, nxt = _check(torch, cq, c)
    assert count[1] == 0 and nxt[1] == -1


@pytest.mark.parametrize("most", [1, 2, 5])
def test_short_paths(most):
    torch, cq = torch_cuda(), cq_built()
    c = _case(18, 400, [8] * 20, 0.0, chain=True)
    for f in c["q_start"][:-1]:
        for i in range(1, 8):
            c["tokens"][f + i] = c["logits"][f + i - 1, :400].argmax()
    c["max_path"] = most
    count, _, _ = _check(torch, cq, c)
    assert (count == most).all()


def test_a_residual_of_nothing_keeps_the_distribution():
    """Draft probabilities of 1 everywhere (no distribution): whatever is taken away, nothing would be left."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(19, 6000, [4] * 10, 1.0, draft=True)
    c["draft"][:] = 1.0
    c["u_accept"][:] = 0.999
    _check(torch, cq, c)
    c["draft"][:] = 0.0                                  # nothing was drawn from it: kept where p > 0
    _check(torch, cq, c)


def test_captured_and_on_another_stream():
    torch, cq = torch_cuda(), cq_built()
    c = _case(20, 20000, [9] * 30, 0.8, draft=True)
    want = [x.clone() for x in _run(torch, cq, c)]
    t = {k: dev(torch, v) for k, v in c.items() if isinstance(v, np.ndarray)}
    call = lambda: cq.tree_verify_t(t["logits"], t["tokens"], t["parent"], t["q_start"], t["temperature"], t["u_accept"],
                                    t["u_sample"], 64, draft=t["draft"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        got = call()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            held = call()
    for _ in range(3):
        for x in held:
            x.fill_(-5)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(a, d) for a, b, d in zip(want, got, held))


def test_sums_of_rejected_residuals_past_64_bits():
    """A flat distribution of 200000 tokens (a sum of 2^62.6 units) and drafts that all lie where it does not: the
    residuals that were taken away add up to more than 2^64."""
    torch, cq = torch_cuda(), cq_built()
    V = 200000
    c = _case(21, V, [9, 12], 1.0, draft=True, spread=0.0)
    c["logits"][:] = 0.0
    c["draft"][:] = 0.0
    rng = np.random.default_rng(3)
    for f, n in zip(c["q_start"][:-1], (9, 12)):
        at = rng.permutation(V)[:16]
        c["draft"][f:f + n, at] = 1.0 / 16
        c["parent"][f + 1:f + n], c["tokens"][f + 1:f + n] = 0, at[:n - 1]
    c["u_accept"][:] = 0.9
    count, _, nxt = _check(torch, cq, c)
    assert count.tolist() == [1, 1]


@pytest.mark.parametrize("V", [262144, 262143])
@pytest.mark.parametrize("draft", [False, True])
def test_flat_rows_of_the_largest_vocabulary(V, draft):
    """Every value at its largest: the largest sums there are. u = (k + 1/2) / V falls into the middle of token k."""
    torch, cq = torch_cuda(), cq_built()
    c = _case(22, V, [1, 3, 2], 1.0, draft=draft, spread=0.0, chain=True)
    c["logits"][:] = -7.5
    if draft:
        c["draft"][:] = 1.0 / V
    c["u_accept"][:] = 0.5
    c["u_sample"][:] = [0.5 / V, (V // 2 + 0.5) / V, (V - 0.5) / V]
    got = [x.cpu().numpy() for x in _run(torch, cq, c)]
    if not draft:                                        # (with it the drafts are kept: u q < p for u = 1/2)
        assert got[0].tolist() == [1, 1, 1]
        want = [0, V // 2, V - 1]
        # a rejected draft takes its own step away in front of the token, at most one of two
        assert all(abs(int(g) - w) <= 2 for g, w in zip(got[2], want)) and got[2][0] == 0
    else:
        assert got[0].tolist() == [1, 3, 2] and got[2].tolist() == [0, V // 2, V - 1]
    if V == 262144:                                      # (whose borders 64 bits hold exactly)
        _check(torch, cq, c)
