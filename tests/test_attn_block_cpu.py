"""The attention layer's own bookkeeping -- lengths, pages, what may be kept -- with its calls replaced by their
definitions on the host."""
import types

import numpy as np
import pytest

import kv_ref
import tree_ref
from gemm_gguf_block_gb300 import attn_block, cq

torch = pytest.importorskip("torch")
HIDDEN, HEADS, D, P = 64, 2, 64, 16


def _definitions():
    def plan(past, new, table, free, page, pages, tokens):
        got = kv_ref.plan(past.numpy(), new.numpy(), table.numpy(), free.numpy(), page, pages, tokens)
        table.copy_(torch.from_numpy(got[0]))
        return tuple(torch.from_numpy(x) for x in got[1:])

    def append(cache, k, v, slots):
        for q, s, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v)):
            kv_ref.append(q.numpy(), s.numpy(), x.reshape(-1, cache.kv_heads, D).numpy(), slots.numpy())

    def tree_plan(kv_len, q_start, parent):
        mask, pos, _ = tree_ref.tree_plan(kv_len.numpy(), q_start.numpy(), parent.numpy(), parent.shape[0])
        return torch.from_numpy(mask.view(np.int64)), torch.from_numpy(pos)

    def move(cache, table, kv_len, q_start, count, path):
        if count.dtype != torch.int32 or count.shape != kv_len.shape or path.dtype != torch.int32 or path.shape[1] > 64:
            raise cq.CqError("cq_kv_move", cq.ERR_SHAPE)
        for q, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            new_len, _ = tree_ref.move(q.numpy(), s.numpy(), table.numpy(), kv_len.numpy(), q_start.numpy(), count.numpy(), path.numpy())
        return torch.from_numpy(new_len)

    def release(table, old, new, page, pages, capacity):
        return tuple(torch.from_numpy(np.array(x, np.int32)) for x in
                     tree_ref.release(table.numpy(), old.numpy(), new.numpy(), page, pages, capacity))

    return types.SimpleNamespace(**{
        **vars(cq), "attn_workspace_t": lambda *a: None, "quantize_act_t": lambda x, f: x,
        "gemv_t": lambda w, x, f, k: x @ w, "gemm_t": lambda w, x, f, k: x @ w, "kv_plan_t": plan, "kv_append_t": append,
        "tree_plan_t": tree_plan, "attn_paged_t": lambda q, *a, **k: (torch.zeros(q.shape), None),
        "attn_tree_t": lambda q, *a, **k: (torch.zeros(q.shape), None), "kv_move_t": move, "kv_release_t": release})


@pytest.fixture
def block(monkeypatch):
    """Two requests of 40 tokens after their prompts, on pages of 16."""
    monkeypatch.setattr(attn_block, "cq", _definitions())
    g = torch.Generator().manual_seed(0)
    b = attn_block.AttentionBlock(torch.randn(HIDDEN, 3 * HEADS * D, generator=g), torch.randn(HEADS * D, HIDDEN, generator=g),
                                  cq.FMT["q8_0"], HIDDEN, HEADS, HEADS, D, requests=2, num_pages=12)
    b.gen = g
    b.step(_tokens(b, 80), [40, 40])
    return b


def _tokens(b, n):
    return torch.randn(n, HIDDEN, generator=b.gen)


def _tree_step(b, new):
    parents = np.concatenate([tree_ref.random_parents(np.random.default_rng(n), n) if n else [] for n in new])
    b.step(_tokens(b, sum(new)), new, torch.from_numpy(parents.astype(np.int32)))


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def _pages(b):
    """The requests' pages; every page is a request's or free, none twice."""
    mine = [b.table[r, :-(-n // P)].tolist() for r, n in enumerate(b.past)]
    assert sorted(sum(mine, []) + b.free[b.taken:].tolist()) == list(range(b.cache.num_pages))
    return mine


def _state(b):
    return (list(b.past), b.taken, b.free.clone(), b.table.clone(), b.cache.k.clone(), b.cache.v.clone(),
            b.cache.k_scale.clone(), b.cache.v_scale.clone())


def _same(a, b):
    return all(torch.equal(x, y) if isinstance(x, torch.Tensor) else x == y for x, y in zip(a, b))


def test_a_step_is_kept_once(block):
    """The rows have moved: a second call with the path 0, 2, 4 would put token 4's where token 2's is."""
    _tree_step(block, [20, 20])
    path = torch.tensor([[0, 2, 4], [0, 3, 17]], dtype=torch.int32)
    with pytest.raises(cq.CqError):
        block.keep(_i32(3), path)                        # a refusal leaves the step to be kept
    block.keep(_i32(3, 3), path)
    assert block.past == [43, 43]
    _pages(block)
    was = _state(block)
    with pytest.raises(cq.CqError):
        block.keep(_i32(3, 3), path)
    assert _same(was, _state(block))
    _tree_step(block, [5, 1])
    block.keep(_i32(2, 1), torch.tensor([[0, 3], [0, -1]], dtype=torch.int32))
    assert block.past == [45, 44]
    _pages(block)


def test_nothing_to_keep_before_a_step(monkeypatch):
    monkeypatch.setattr(attn_block, "cq", _definitions())
    b = attn_block.AttentionBlock(torch.zeros(HIDDEN, 3 * HEADS * D), torch.zeros(HEADS * D, HIDDEN), cq.FMT["q8_0"], HIDDEN,
                                  HEADS, HEADS, D, requests=1, num_pages=2)
    with pytest.raises(cq.CqError):
        b.keep(_i32(0), torch.zeros((1, 1), dtype=torch.int32))


@pytest.mark.parametrize("wide", [False, True])
def test_a_request_ends_between_a_step_and_its_keep(block, wide):
    """Its accepted tokens held the text's end: the others are kept, its pages stay given back and untouched, its place
    serves a new prompt."""
    new = [20, 70] if wide else [20, 20]                 # (a prompt keeps all its tokens, unless it has ended)
    _tree_step(block, new)
    rows = block.cache.k.numpy().astype(np.float32)
    ended = block.table[1, :-(-(40 + new[1]) // P)].tolist()
    first = block.table[0].tolist()
    block.end(1)
    was = block.cache.k[ended].clone()
    block.keep(_i32(3, 3), torch.tensor([[0, 2, 4], [0, 5, 6]], dtype=torch.int32))
    assert block.past == [43, 0]
    assert torch.equal(block.cache.k[ended], was)        # nothing moved in pages that were given back
    mine = _pages(block)
    assert mine[0] == first[:3]
    at = lambda i: (first[i // P], i % P)                # request 0: tokens 0, 2 and 4 of the step at 40, 41, 42
    scale = block.cache.k_scale.numpy()
    for i, token in ((40, 40), (41, 42), (42, 44)):
        (p, row), (src, srow) = at(i), at(token)
        assert np.abs(block.cache.k[p, :, row].numpy() * scale[p][:, None] - rows[src, :, srow] * scale[src][:, None]).max() <= scale[p].max()
    block.step(_tokens(block, 31), [1, 30])
    assert block.past == [44, 30]
    _pages(block)


def test_all_requests_end_before_keep(block):
    _tree_step(block, [9, 9])
    block.end(0)
    block.end(1)
    block.end(1)
    block.keep(_i32(1, 1), torch.zeros((2, 1), dtype=torch.int32))
    assert block.past == [0, 0] and block.taken == 0
    _pages(block)


def test_an_end_does_not_outlive_its_step(block):
    """A request that ended before a step takes part in it as any other."""
    block.end(1)
    _tree_step(block, [4, 12])
    block.keep(_i32(2, 2), torch.tensor([[0, 3], [0, 7]], dtype=torch.int32))
    assert block.past == [42, 2]
    _pages(block)
    with pytest.raises(cq.CqError):
        block.end(1)
        block.keep(_i32(2, 2), torch.zeros((2, 2), dtype=torch.int32))


@pytest.mark.parametrize("count", [torch.ones(1, dtype=torch.int32), torch.ones(2, dtype=torch.int64), torch.ones((2, 1), dtype=torch.int32)])
def test_keep_after_an_end_refuses_what_it_refuses_else(block, count):
    _tree_step(block, [9, 9])
    block.end(0)
    was = _state(block)
    with pytest.raises(cq.CqError):
        block.keep(count, torch.zeros((2, 1), dtype=torch.int32))
    assert _same(was, _state(block))
    block.keep(_i32(1, 1), torch.zeros((2, 1), dtype=torch.int32))
    assert block.past == [0, 41]


@pytest.mark.parametrize("r", [-1, -2, 2, 100])
def test_end_refuses_requests_that_are_not_there(block, r):
    _tree_step(block, [9, 9])
    was = _state(block)
    with pytest.raises(cq.CqError):
        block.end(r)
    assert _same(was, _state(block))
    block.keep(_i32(2, 2), torch.tensor([[0, 3], [0, 7]], dtype=torch.int32))
    assert block.past == [42, 42]


@pytest.mark.parametrize("seed", range(6))
def test_any_order_of_steps_keeps_and_ends(monkeypatch, seed):
    """Random orders of the three calls, refused ones among them, against lists of the requests' keys: lengths, pages (each a
    request's or free, none twice), and every stored row within six steps of its page's scale (half a step a raise)."""
    monkeypatch.setattr(attn_block, "cq", _definitions())
    rng, R = np.random.default_rng(seed), 3
    g = torch.Generator().manual_seed(seed)
    b = attn_block.AttentionBlock(torch.randn(HIDDEN, 3 * HEADS * D, generator=g), torch.randn(HEADS * D, HIDDEN, generator=g),
                                  cq.FMT["q8_0"], HIDDEN, HEADS, HEADS, D, requests=R, num_pages=40)
    b.gen = g
    want, open_step = [[] for _ in range(R)], None       # keys of each request; (new tokens, lengths before, ended since)
    for _ in range(40):
        op = rng.choice(["step", "tree", "keep", "keep", "end"])
        if op in ("step", "tree"):
            new = [int(rng.choice([0, 1, 3, 12, 30, 70])) for _ in range(R)]
            parents = [tree_ref.random_parents(rng, n) if n else [] for n in new]
            x = _tokens(b, sum(new))
            if sum(new) == 0 or sum(-(-(len(w) + n) // P) for w, n in zip(want, new)) > 40:
                with pytest.raises(cq.CqError):
                    b.step(x, new)
                continue
            b.step(x, new, torch.from_numpy(np.concatenate(parents).astype(np.int32)) if op == "tree" else None)
            open_step = (new, [len(w) for w in want], set())
            k = (x @ b.wqkv)[:, HEADS * D:2 * HEADS * D].reshape(-1, HEADS, D).split(new)
            want = [w + list(rows) for w, rows in zip(want, k)]
        elif op == "keep":
            most = int(rng.integers(1, 20))
            new = open_step[0] if open_step else [0] * R
            paths = [np.sort(rng.permutation(n)[:int(rng.integers(0, min(n, most) + 1))]).tolist() if n <= 64 else [] for n in new]
            args = (_i32(*map(len, paths)), torch.tensor([(p + [-1] * most)[:most] for p in paths], dtype=torch.int32))
            if open_step is None:
                with pytest.raises(cq.CqError):
                    b.keep(*args)
                continue
            b.keep(*args)
            for r, (n, base) in enumerate(zip(*open_step[:2])):
                if r not in open_step[2] and n <= 64:
                    want[r] = want[r][:base] + [want[r][base + i] for i in paths[r]]
            open_step = None
        else:
            r = int(rng.integers(R))
            b.end(r)
            want[r] = []
            if open_step:
                open_step[2].add(r)
        assert b.past == [len(w) for w in want]
        _pages(b)
        for r, w in enumerate(want):
            for i, row in enumerate(w):
                scale = b.cache.k_scale[int(b.table[r, i // P])][:, None]
                assert ((b.cache.k[int(b.table[r, i // P]), :, i % P] * scale - row).abs() <= 6 * scale).all()
