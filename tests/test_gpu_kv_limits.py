"""The cache calls at the ends of their ranges: lengths, token counts and scales."""
import numpy as np
import pytest

import kv_ref
from helpers import cq_built, dev, torch_cuda

pytestmark = pytest.mark.gpu

INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("R", [4, 600])
def test_plan_lengths_whose_sum_passes_32_bits(P, R):
    """Tokens past the table get no slot wherever their position lies; one that 32 bits do not hold is -1."""
    torch, cq = torch_cuda(), cq_built()
    past, new = np.full(R, 5, np.int32), np.full(R, 3, np.int32)
    past[[0, 2, R - 1]] = INT_MAX, INT_MAX - 20, INT_MAX
    new[[0, 2, R - 1]] = 2, 40, 17
    wide = 4
    table = np.zeros((R, wide), np.int32)
    table[:, 0] = np.arange(R)
    T = int(new.sum()) + 2
    t = dev(torch, table)
    kv, q_start, slots, pos, used = (x.cpu().numpy() for x in cq.kv_plan_t(
        dev(torch, past), dev(torch, new), t, dev(torch, np.arange(R, 2 * R, dtype=np.int32)), P, 2 * R, T))
    assert np.array_equal(t.cpu().numpy(), table)
    assert np.array_equal(kv, np.minimum(past.astype(np.int64) + new, wide * P))
    assert np.array_equal(q_start, np.concatenate([[0], np.cumsum(new)]))
    assert used.tolist() == [0, cq.DEV_KV_BLOCKS]
    at = np.concatenate([np.arange(n, dtype=np.int64) + a for a, n in zip(past, new)])
    r = np.repeat(np.arange(R), new)
    inside = at < wide * P
    assert np.array_equal(slots[:-2], np.where(inside, table[r, np.where(inside, at // P, 0)] * np.int64(P) + at % P, -1))
    assert np.array_equal(pos[:-2], np.where(at <= INT_MAX, at, -1))
    assert (slots[-2:] == -1).all() and (pos[-2:] == -1).all()


def test_plan_sum_of_two_largest_lengths():
    torch, cq = torch_cuda(), cq_built()
    one = dev(torch, np.array([INT_MAX], np.int32))
    table = dev(torch, np.zeros((1, 2), np.int32))
    kv, q_start, slots, pos, used = cq.kv_plan_t(one, one, table, one[:0], 16, 4, 100)
    assert kv.tolist() == [32] and q_start.tolist() == [0, 100]
    assert (slots == -1).all() and pos.tolist() == [INT_MAX] + [-1] * 99
    assert used.tolist() == [0, cq.DEV_KV_BLOCKS | cq.DEV_KV_TOKENS]


@pytest.mark.parametrize("T", [INT_MAX, INT_MAX - 3000])
def test_plan_of_as_many_tokens_as_it_takes(T):
    """The largest T: every entry is written, the last ones as the first (26 GB of outputs)."""
    torch, cq = torch_cuda(), cq_built()
    P = 128
    past, new = np.array([7, INT_MAX // 2], np.int32), np.array([300, 5], np.int32)
    table, free = np.array([[0, -1, -1], [0, 0, 0]], np.int32), np.array([2, 1], np.int32)
    t = dev(torch, table)
    kv, q_start, slots, pos, used = cq.kv_plan_t(dev(torch, past), dev(torch, new), t, dev(torch, free), P, 3, T)
    assert t.tolist() == [[0, 2, 1], [0, 0, 0]] and kv.tolist() == [307, 3 * P] and q_start.tolist() == [0, 300, 305]
    assert used.tolist() == [2, cq.DEV_KV_BLOCKS]
    at = np.arange(7, 307)
    assert slots[:305].tolist() == (np.array([0, 2, 1])[at // P] * P + at % P).tolist() + [-1] * 5
    assert pos[:305].tolist() == at.tolist() + list(range(INT_MAX // 2, INT_MAX // 2 + 5))
    for x in (slots, pos):
        for i in range(305, T, 1 << 28):
            assert bool((x[i:i + (1 << 28)] == -1).all())
    del slots, pos, x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("growth", [1.0, 1.004, 1.03, 1.2])
def test_a_page_filled_token_by_token(P, growth):
    """Every call that raises a page's scale rounds its rows again: bits as the rule has them after each, and what is read
    back lies within half a step of every scale since its row was stored (fp32's roundings add 2^-15 of it) of what was
    given."""
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng([P, int(1000 * growth)])
    H, D = 2, 64
    x = (np.clip(rng.standard_normal((P, H, D)), -3, 3) * growth ** np.arange(P)[:, None, None]).astype(np.float32)
    if growth > 1.0:
        x[:, :, 0] = (3.0 * growth ** np.arange(P))[:, None]
    cache = cq.KVCache.empty(2, H, P, D)
    q, s = np.zeros((2, H, P, D), np.int8), np.zeros((2, H), np.float32)
    slots, tx, bound, raised = np.arange(P, 2 * P), dev(torch, x), np.zeros((P, H)), 0
    for t in range(P):
        old = s[1].copy()
        cq.kv_append_t(cache, tx[t:t + 1], tx[t:t + 1], dev(torch, slots[t:t + 1]))
        kv_ref.append(q, s, x[t:t + 1], slots[t:t + 1])
        raised += int(t > 0 and (s[1] > old).all())
        bound[:t] += np.where(s[1] > old, s[1].astype(np.float64) / 2, 0.0)
        bound[t] = s[1].astype(np.float64) / 2
        for got, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            assert np.array_equal(scale.cpu().numpy(), s) and np.array_equal(got.cpu().numpy(), q)
    assert raised == P - 1 or growth == 1.0
    for back in cq.kv_read_t(cache, dev(torch, slots)):
        off = np.abs(back.cpu().numpy().astype(np.float64) - x)
        assert (off <= bound[:, :, None] * (1 + 2.0 ** -15)).all()
