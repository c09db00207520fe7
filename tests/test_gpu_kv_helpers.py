"""The tensor helpers of the cache and attention calls refuse what is not on the cache's device."""
import pytest

from helpers import cq_built, torch_cuda

pytestmark = pytest.mark.gpu


def _refused(cq, call, args):
    """The call with each tensor in turn on the host (before any launch: the library would get a host address)."""
    import torch
    for name, x in args.items():
        if isinstance(x, torch.Tensor):
            with pytest.raises(cq.CqError):
                call(**{**args, name: x.cpu()})


def test_tensors_on_the_host_are_refused():
    torch, cq = torch_cuda(), cq_built()
    cache = cq.KVCache.empty(4, 2, 16, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    past, new = torch.zeros(2, **i32), torch.full((2,), 3, **i32)
    plan = dict(past_len=past, new_len=new, block_table=torch.full((2, 2), -1, **i32),
                free_pages=torch.arange(4, **i32), page_size=16, num_pages=4, tokens=6)
    kv_len, q_start, slots, _, used = cq.kv_plan_t(**plan)
    x = torch.randn(6, 128, device="cuda")
    append = dict(cache=cache, k=x, v=x, slots=slots)
    cq.kv_append_t(**append)
    attend = dict(q=torch.randn(6, 4, 64, device="cuda"), cache=cache, block_table=plan["block_table"], kv_len=kv_len,
                  q_start=q_start, max_new=3, max_kv=3, ws=cq.attn_workspace_t(4, 2, 64),
                  out=torch.empty(6, 4, 64, device="cuda"), lse=torch.empty(6, 4, device="cuda"))
    out, _ = cq.attn_paged_t(**attend)
    assert used.tolist() == [2, 0] and torch.isfinite(out).all()
    _refused(cq, cq.kv_plan_t, plan)
    _refused(cq, cq.kv_append_t, append)
    _refused(cq, cq.kv_read_t, dict(cache=cache, slots=slots))
    _refused(cq, cq.attn_paged_t, attend)
    host = cq.KVCache.empty(4, 2, 16, 64, "cpu")
    for call, args in ((cq.kv_append_t, append), (cq.kv_read_t, dict(slots=slots)), (cq.attn_paged_t, attend)):
        with pytest.raises(cq.CqError):
            call(**{**args, "cache": host})
    for i in range(4):
        parts = [cache.k, cache.v, cache.k_scale, cache.v_scale]
        parts[i] = parts[i].cpu()
        with pytest.raises(cq.CqError):
            cq.KVCache(*parts)


def test_a_workspace_is_as_large_as_its_memory():
    """Its size counts bytes, and one whose elements share memory is refused."""
    torch, cq = torch_cuda(), cq_built()
    cache = cq.KVCache.empty(4, 2, 16, 64)
    need = cq.cq_attn_workspace_size(4, 2, 64)
    table, kv, start = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([[0]], [5], [0, 1]))
    q = torch.randn(1, 4, 64, device="cuda")

    def call(ws):
        return cq.attn_paged_t(q, cache, table, kv, start, 1, 5, ws=ws)
    want = call(torch.zeros(need, dtype=torch.uint8, device="cuda"))
    assert need % 4 == 0
    got = call(torch.zeros(need // 4, dtype=torch.float32, device="cuda"))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for ws in (torch.zeros(need - 1, dtype=torch.uint8, device="cuda"), torch.zeros(need // 4 - 1, device="cuda"),
               torch.zeros(1, dtype=torch.uint8, device="cuda").expand(need),
               torch.zeros(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(cq.CqError):
            call(ws)
