"""A run of tree decoding: plan, masks, projections, norm and rotation, append, attention, LM head, verification, rows
moved, pages given back, again and again."""
import numpy as np
import pytest

import tree_ref
from helpers import cq_built, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,shape", [("q8_0", dict(hidden=1024, q_heads=16, kv_heads=4, head_dim=64)),
                                       ("q4_0", dict(hidden=512, q_heads=8, kv_heads=2, head_dim=128, drafts=40))])
def test_steps(fmt, shape):
    """Attention within fp32 of 64 bits (1e-5 as the layer's other tests derive it; the norms bring queries and keys to
    about 1, less than there), every verification as its definition in 64 bits says, no page lost."""
    torch, cq = torch_cuda(), cq_built()
    from gemm_gguf_block_gb300 import attn_block
    block, worst, kept = attn_block.tree_demo(vocab=4000, prompts=(150, 33, 1), steps=8, fmt=fmt, **shape)
    assert worst <= 1e-5
    total = np.zeros(3, int)
    for args, count, path, token in kept:
        a = [x.cpu().numpy() for x in args]
        want = tree_ref.verify(*a, path.shape[1])
        assert np.array_equal(count.cpu().numpy(), want[0]) and np.array_equal(path.cpu().numpy(), want[1])
        assert np.array_equal(token.cpu().numpy(), want[2]) and want[3] == 0
        total += want[0]
    assert block.past == (np.array([150, 33, 1]) + total).tolist() and total.max() > 8
    assert block.taken == sum(-(-n // 16) for n in block.past)
    # every page is a request's or free, and none twice
    mine = [block.table[r, :-(-n // 16)].tolist() for r, n in enumerate(block.past)]
    free = block.free[block.taken:].tolist()
    assert sorted(sum(mine, []) + free) == list(range(block.cache.num_pages))
    block.end(1)
    assert block.past[1] == 0 and block.taken == sum(-(-n // 16) for n in block.past)
    free = block.free[block.taken:].tolist()
    assert sorted(mine[0] + mine[2] + free) == list(range(block.cache.num_pages))
    # its place and its pages serve a new prompt, beside a token of another request
    x = torch.randn(41, block.hidden, device="cuda")
    block.step(x, [0, 40, 1])
    for r, first, n in ((1, 0, 40), (2, 40, 1)):
        want = block.dense(r, first, n)
        assert ((block.attended[first:first + n].double() - want).norm() <= 1e-5 * want.norm()).item()
    assert cq.cq_read_global_status() == (cq.OK, 0)


def test_kept_rows_are_the_tokens_own():
    """After keep, the cache holds each kept token's row where a chain of them would have it, within the steps of its
    pages' scales: at most s / 2 for the append, s / 2 for the move and s / 2 for a scale that grew."""
    torch, cq = torch_cuda(), cq_built()
    from gemm_gguf_block_gb300 import attn_block
    block, _, _ = attn_block.tree_demo(hidden=256, q_heads=4, kv_heads=2, head_dim=64, vocab=500, prompts=(30, 9), steps=1)
    past = list(block.past)
    x = torch.randn(2 * 20, 256, device="cuda")
    parent = torch.tensor([-1, 0, 0, 0, 1, 1, 2, 3, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14] * 2, dtype=torch.int32, device="cuda")
    block.step(x, [20, 20], parent)
    before = cq.kv_read_t(block.cache, block.slots)
    path = torch.tensor([[0, 2, 6, 11, 16, -1], [0, 3, 8, 13, 18, -1]], dtype=torch.int32, device="cuda")
    block.keep(torch.tensor([5, 5], dtype=torch.int32, device="cuda"), path)
    assert block.past == [past[0] + 5, past[1] + 5]
    for r in range(2):
        pos = torch.arange(past[r], past[r] + 5, device="cuda")
        page = block.table[r, pos // 16].long()
        rows = cq.kv_read_t(block.cache, page * 16 + pos % 16)
        at = 20 * r + path[r, :5].long()
        for was, now, s in zip(before, rows, (block.cache.k_scale, block.cache.v_scale)):
            assert ((now - was[at]).abs() <= 0.51 * s[page][:, :, None]).all()


def test_refusals_leave_the_block_as_it_is():
    torch, cq = torch_cuda(), cq_built()
    from gemm_gguf_block_gb300 import attn_block
    block, _, _ = attn_block.tree_demo(hidden=256, q_heads=4, kv_heads=2, head_dim=64, vocab=500, prompts=(30, 9), steps=1)
    past, k = list(block.past), block.cache.k.clone()
    with pytest.raises(cq.CqError):
        block.keep(torch.tensor([1], dtype=torch.int32, device="cuda"), torch.zeros((2, 4), dtype=torch.int32, device="cuda"))
    with pytest.raises(cq.CqError):
        block.keep(torch.tensor([1, 1], dtype=torch.int32, device="cuda"), torch.zeros((2, 65), dtype=torch.int32, device="cuda"))
    with pytest.raises(cq.CqError):
        block.keep(torch.tensor([1, 1], dtype=torch.int32), torch.zeros((2, 4), dtype=torch.int32, device="cuda"))
    assert block.past == past and torch.equal(block.cache.k, k)


def test_helpers_refuse_tensors_on_the_host_and_of_other_types():
    torch, cq = torch_cuda(), cq_built()
    i32, f32 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.float32, device="cuda")
    cache = cq.KVCache.empty(4, 2, 16, 64)
    kv, start, table = torch.tensor([5], **i32), torch.tensor([0, 3], **i32), torch.tensor([[1, 2]], **i32)
    parent = torch.tensor([-1, 0, 0], **i32)
    mask, _ = cq.tree_plan_t(kv, start, parent)
    calls = [
        (cq.tree_plan_t, dict(kv_len=kv, q_start=start, parent=parent)),
        (cq.qk_rope_t, dict(q=torch.zeros(3, 4, 64, **f32), k=torch.zeros(3, 2, 64, **f32), positions=parent,
                            freqs=torch.ones(32, dtype=torch.float64, device="cuda"), q_norm=torch.ones(64, **f32),
                            k_norm=torch.ones(64, **f32), q_out=torch.zeros(3, 4, 64, **f32),
                            k_out=torch.zeros(3, 2, 64, **f32))),
        (cq.attn_tree_t, dict(q=torch.zeros(3, 4, 64, **f32), cache=cache, block_table=table, kv_len=kv, q_start=start,
                              mask=mask, max_new=3, out=torch.zeros(3, 4, 64, **f32), lse=torch.zeros(3, 4, **f32),
                              ws=cq.attn_workspace_t(4, 2, 64))),
        (cq.tree_verify_t, dict(logits=torch.zeros(3, 10, **f32), tokens=parent, parent=parent, q_start=start,
                                temperature=torch.ones(1, **f32), u_accept=torch.zeros(3, **f32),
                                u_sample=torch.zeros(1, **f32), max_path=3, draft=torch.zeros(3, 10, **f32))),
        (cq.kv_move_t, dict(cache=cache, block_table=table, kv_len=kv, q_start=start, count=torch.tensor([1], **i32),
                            path=torch.zeros((1, 3), **i32), new_len=torch.zeros(1, **i32))),
        (cq.kv_release_t, dict(block_table=table, old_len=kv, new_len=kv, page_size=16, num_pages=4, capacity=3)),
    ]
    for call, args in calls:
        call(**args)
        for name, x in args.items():
            if isinstance(x, torch.Tensor):
                with pytest.raises(cq.CqError):
                    call(**{**args, name: x.cpu()})
                if name != "ws":
                    with pytest.raises(cq.CqError):
                        call(**{**args, name: x.to(torch.int16)})
    assert cq.cq_read_global_status()[0] in (cq.OK, cq.ERR_DEVICE_STATUS)


def test_a_prompt_beside_trees_keeps_its_tokens():
    """A step with a prompt of more than TREE_MAX tokens, a tree and a request that takes no part: verification gives
    the prompt count 0 (it has no drafts), and keep() leaves it whole."""
    torch, cq = torch_cuda(), cq_built()
    from gemm_gguf_block_gb300 import attn_block
    block, _, _ = attn_block.tree_demo(hidden=256, q_heads=4, kv_heads=2, head_dim=64, vocab=500, prompts=(30, 9, 20), steps=1)
    block.end(0)
    past, taken = list(block.past), block.taken
    new = [70, 6, 0]
    parent = torch.tensor([-1] * 70 + [-1, 0, 0, 1, 1, 2], dtype=torch.int32, device="cuda")
    block.step(torch.randn(76, 256, device="cuda"), new, parent)
    for r, first, n in ((0, 0, 70), (1, 70, 6)):
        want = block.dense(r, first, n)
        assert ((block.attended[first:first + n].double() - want).norm() <= 1e-5 * want.norm()).item()
    before = cq.kv_read_t(block.cache, block.slots)
    path = torch.tensor([[-1, -1, -1], [0, 2, 5], [-1, -1, -1]], dtype=torch.int32, device="cuda")
    block.keep(torch.tensor([0, 3, 0], dtype=torch.int32, device="cuda"), path)
    assert block.past == [70, past[1] + 3, past[2]]
    assert block.taken == sum(-(-n // 16) for n in block.past)
    after = cq.kv_read_t(block.cache, block.slots)
    assert all(torch.equal(a[:70], b[:70]) for a, b in zip(before, after))
    assert cq.cq_read_global_status() == (cq.OK, 0)
