"""Orders of an attention layer's calls that a decoder comes to: requests that end between a step and its keep()."""
import pytest

from helpers import cq_built, torch_cuda

pytestmark = pytest.mark.gpu


def _block(prompts):
    from gemm_gguf_block_gb300 import attn_block
    return attn_block.tree_demo(hidden=256, q_heads=4, kv_heads=2, head_dim=64, vocab=500, prompts=prompts, steps=1)[0]


def _attends(block, new):
    first = 0
    for r, n in enumerate(new):
        if n:
            want = block.dense(r, first, n)
            assert ((block.attended[first:first + n].double() - want).norm() <= 1e-5 * want.norm()).item(), r
        first += n


def _pages(block):
    mine = [block.table[r, :-(-n // 16)].tolist() for r, n in enumerate(block.past)]
    assert sorted(sum(mine, []) + block.free[block.taken:].tolist()) == list(range(block.cache.num_pages))


@pytest.mark.parametrize("gone", [0, 1, 2])
def test_a_request_ends_between_a_step_and_its_keep(gone):
    """The others are kept, every page is a request's or free, and a new prompt takes its place beside them."""
    torch, cq = torch_cuda(), cq_built()
    block = _block((30, 41, 20))
    parent = torch.tensor([-1, 0, 0, 1, 1, 2, 2, 3, 3, 4, 4, 5, 5, 6, 6] * 3, dtype=torch.int32, device="cuda")
    past = list(block.past)
    block.step(torch.randn(45, 256, device="cuda"), [15] * 3, parent)
    _attends(block, [15] * 3)
    before, slots = cq.kv_read_t(block.cache, block.slots), block.slots.clone()
    block.end(gone)
    path = torch.tensor([[0, 2, 6, 13]] * 3, dtype=torch.int32, device="cuda")
    block.keep(torch.tensor([4] * 3, dtype=torch.int32, device="cuda"), path)
    assert block.past == [0 if r == gone else n + 4 for r, n in enumerate(past)]
    _pages(block)
    after = cq.kv_read_t(block.cache, slots)
    assert all(torch.equal(a[15 * gone:15 * gone + 15], b[15 * gone:15 * gone + 15]) for a, b in zip(before, after))
    for r in range(3):
        if r != gone:                                    # within the steps of the pages' scales
            pos = torch.arange(past[r], past[r] + 4, device="cuda")
            page = block.table[r, pos // 16].long()
            rows = cq.kv_read_t(block.cache, page * 16 + pos % 16)
            at = 15 * r + path[r].long()
            for was, now, s in zip(before, rows, (block.cache.k_scale, block.cache.v_scale)):
                assert ((now - was[at]).abs() <= 0.51 * s[page][:, :, None]).all()
    new = [1, 1, 1]
    new[gone] = 37
    block.step(torch.randn(39, 256, device="cuda"), new)
    _attends(block, new)
    _pages(block)
    assert cq.cq_read_global_status() == (cq.OK, 0)


def test_a_prompt_beside_trees_goes_through_the_verification_unflagged():
    """Plan, attention, verification and move of one batch: a prompt of more than TREE_MAX tokens, a tree, a request
    that takes no part. The prompt has no drafts to verify: count 0, no token, no flag; it keeps its tokens."""
    torch, cq = torch_cuda(), cq_built()
    import numpy as np
    import tree_ref
    block = _block((30, 9, 20))
    block.end(0)
    past = list(block.past)
    parent = torch.tensor([7] * 70 + [-1, 0, 0, 1, 1, 2], dtype=torch.int32, device="cuda")      # (a prompt's are not read)
    y = block.step(torch.randn(76, 256, device="cuda"), [70, 6, 0], parent)
    _attends(block, [70, 6, 0])
    logits = (y @ torch.randn(256, 300, device="cuda"))
    logits *= 3.0 / logits.std()
    tokens = torch.randint(0, 300, (76,), dtype=torch.int32, device="cuda")
    tokens[71:73] = logits[70].topk(2).indices
    tokens[73:75] = logits[71].topk(2).indices
    tokens[75] = logits[72].argmax()
    for temp in (0.0, 0.8):
        args = (logits, tokens, parent, block.q_start, torch.full((3,), temp, device="cuda"), torch.rand(76, device="cuda"),
                torch.rand(3, device="cuda"))
        count, path, token = cq.tree_verify_t(*args, 6)
        a = [x.cpu().numpy() for x in args]              # the tree by itself
        want = tree_ref.verify(a[0][70:], a[1][70:], a[2][70:], np.array([0, 6]), a[4][1:2], a[5][70:], a[6][1:2], 6)
        assert count.tolist() == [0, want[0][0], 0] and token.tolist() == [-1, want[2][0], -1]
        assert path.tolist() == [[-1] * 6, want[1][0].tolist(), [-1] * 6]
        assert cq.cq_read_global_status() == (cq.OK, 0)
    block.keep(count, path)
    assert block.past == [70, past[1] + int(want[0][0]), past[2]]
    _pages(block)
    assert cq.cq_read_global_status() == (cq.OK, 0)


def test_well_formed_calls_flag_nothing():
    """Each call by itself with what it documents as well-formed, the status read after each; one malformed parent, one
    malformed path and a row without a distribution are flagged, with their bits and no others."""
    torch, cq = torch_cuda(), cq_built()
    i32, f32 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.float32, device="cuda")
    cache = cq.KVCache.empty(4, 2, 16, 64)
    kv, start, table = torch.tensor([5], **i32), torch.tensor([0, 3], **i32), torch.tensor([[1, 2]], **i32)
    parent, pos = torch.tensor([-1, 0, 0], **i32), torch.tensor([2, 3, 3], **i32)
    logits, u = torch.zeros(3, 10, **f32), torch.zeros(3, **f32)
    mask, _ = cq.tree_plan_t(kv, start, parent)
    verify = lambda z, p: cq.tree_verify_t(z, torch.tensor([1, 2, 3], **i32), p, start, torch.ones(1, **f32), u, u[:1], 3)
    move = lambda path: cq.kv_move_t(cache, table, kv, start, torch.tensor([2], **i32), path)
    good = [lambda: cq.tree_plan_t(kv, start, parent), lambda: cq.qk_rope_t(torch.zeros(3, 4, 64, **f32), torch.zeros(3, 2, 64, **f32), pos, None),
            lambda: cq.attn_tree_t(torch.zeros(3, 4, 64, **f32), cache, table, kv, start, mask, 3), lambda: verify(logits, parent),
            lambda: move(torch.tensor([[0, 2, -1]], **i32)), lambda: cq.kv_release_t(table, kv, kv, 16, 4, 3)]
    for call in good:
        call()
        assert cq.cq_read_global_status() == (cq.OK, 0)
    bad = [(lambda: cq.tree_plan_t(kv, start, parent + 1), cq.DEV_TREE), (lambda: verify(logits, parent + 1), cq.DEV_TREE),
           (lambda: move(torch.tensor([[0, 3, -1]], **i32)), cq.DEV_TREE),
           (lambda: verify(logits / 0.0, parent), cq.DEV_LOGITS),
           (lambda: cq.attn_tree_t(torch.zeros(3, 4, 64, **f32), cache, table + 3, kv, start, mask, 3), cq.DEV_KV_PAGE)]
    for call, bits in bad:
        call()
        assert cq.cq_read_global_status() == (cq.ERR_DEVICE_STATUS, bits)
