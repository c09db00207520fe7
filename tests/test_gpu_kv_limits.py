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
