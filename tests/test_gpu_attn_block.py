"""The calls of an attention layer together: projections, plan, append, attention, output projection."""
import pytest

from helpers import cq_built, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,shape", [("q8_0", dict(hidden=2048, q_heads=32, kv_heads=8, head_dim=64)),
                                       ("q4_0", dict(hidden=1024, q_heads=8, kv_heads=2, head_dim=128)),
                                       ("q4_k", dict(hidden=1024, q_heads=4, kv_heads=4, head_dim=64))])
def test_layer_against_its_own_cache(fmt, shape):
    """Every call's attention against 64 bits from the cache read back. The bound: queries and keys have values of
    about 2, so the terms of a score add up to A = sum |q k| / sqrt(D) of about 30; a score is off by at most 2^-18 A
    (see kv_ref.attend), a probability by twice that, 2.4e-4, and the sums by (n / 16 + 64) 2^-23."""
    torch_cuda()
    cq_built()
    from gemm_gguf_block_gb300 import attn_block, cq
    block, worst = attn_block.demo(prompts=(150, 33), steps=18, fmt=fmt, **shape)
    assert block.past == [168, 51]
    assert block.used.tolist()[1] == 0 and block.taken == 11 + 4
    assert block.positions.tolist() == [167, 50]
    assert worst <= 2.5e-4
    assert cq.cq_read_global_status() == (cq.OK, 0)


def test_pages_run_out_before_anything_is_written():
    torch = torch_cuda()
    cq_built()
    from gemm_gguf_block_gb300 import attn_block, cq
    block, _ = attn_block.demo(hidden=256, q_heads=4, kv_heads=1, head_dim=64, prompts=(16,), steps=16)
    assert block.taken == 2
    before = block.cache.k.clone()
    with pytest.raises(cq.CqError):
        block.step(torch.zeros(1, 256, device="cuda"), [1])
    assert torch.equal(block.cache.k, before) and block.past == [32]
