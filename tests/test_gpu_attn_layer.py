"""The attention layer: what it refuses, and how near its attention is."""
import pytest

from helpers import cq_built, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,new", [(3, [1, 1]), (1, [1, 1]), (2, [2]), (2, [1, 1, 0]), (0, [0, 0]), (1, [2, -1])])
def test_token_counts_that_do_not_fit_are_refused(rows, new):
    """... before anything is written: rows of no request would be left undefined, missing ones would be counted."""
    torch = torch_cuda()
    cq_built()
    from gemm_gguf_block_gb300 import attn_block, cq
    block, _ = attn_block.demo(hidden=256, q_heads=4, kv_heads=1, head_dim=64, prompts=(5, 20), steps=3)
    before = block.cache.k.clone(), block.table.clone()
    with pytest.raises(cq.CqError):
        block.step(torch.zeros(rows, 256, device="cuda"), new)
    assert torch.equal(block.cache.k, before[0]) and torch.equal(block.table, before[1])
    assert block.past == [8, 23]
    assert torch.isfinite(block.step(torch.zeros(1, 256, device="cuda"), [0, 1])).all() and block.past == [8, 24]


@pytest.mark.parametrize("fmt,shape", [("q8_0", dict(hidden=2048, q_heads=32, kv_heads=8, head_dim=64)),
                                       ("q4_0", dict(hidden=1024, q_heads=8, kv_heads=2, head_dim=128))])
def test_layer_within_fp32(fmt, shape):
    """The attention's error over a layer's results (2-norm against 64 bits) is fp32's. A score is a sum of D terms of
    about 4 / sqrt(D): queries taken to 22 bits move it by 2^-24 of a term each, 2.4e-7 in all, sums and factors by some
    2^-24 of their size, 5e-7, exponentials by 2^-22 of themselves: about 1e-6 of each probability. 1e-5 is ten times
    that; probabilities held to 11 bits would give 1.4e-4."""
    torch_cuda()
    cq_built()
    from gemm_gguf_block_gb300 import attn_block
    _, worst = attn_block.demo(prompts=(150, 33), steps=18, fmt=fmt, **shape)
    assert worst <= 1e-5
