"""What attention under masks keeps of its probabilities and sums, in each of its kernels and whatever stands beside a
request, against 64 bits."""
import numpy as np
import pytest

import kv_ref
import tree_ref
from helpers import cq_built, dev, torch_cuda
from test_gpu_attn import _case

pytestmark = pytest.mark.gpu


def _attend(torch, cq, c, masks, max_new):
    return cq.attn_tree_t(c["q"], c["cache"], dev(torch, c["table"]), dev(torch, c["kv"]), dev(torch, c["q_start"]),
                          dev(torch, masks.view(np.int64)), max_new)


# rows of a kv head: 12 the rows kernel's, 80 a tile of 128 rows, 160 two of them; trees beside prompts, short ones and (by
# the bound of new tokens) long ones
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,bound", [([3, 2], 3), ([20, 3], 20), ([40, 3, 20], 40), ([12, 70], 70), ([3, 64, 90], 90), ([3, 64, 90], 3000)])
def test_binary16_probabilities_of_trees_have_21_bits(D, new, bound):
    """Few visible keys and small scores, so that the probabilities' own rounding is what an error would come from.

    Per output, over kv_ref.attend's bound for scores, exponentials and fp32 sums (2 e_s of av >= the sum of p |v|, e_s
    from the small scores of these queries): of two binary16 parts the first is off by less than a step of 2^-10, the second
    by half a step of 11 bits of that: 2^-21 av; parts that are subnormal by 2^-25 each, where the row's largest p |v| is 2^7 at
    least: 2^-31 a key of it (127 steps of the scale). One part of 11 bits is 2^-12 av off, about 2^-13 typically: far outside
    where few keys are seen. A prompt beside them is held to kv_ref.attend's bound for 11 bits.
    """
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng([D, len(new), new[0]])
    past = [0, 1, 2][:len(new)]
    kv = [a + n for a, n in zip(past, new)]
    c = _case(torch, cq, [D, new[0]], "f16", 8, 2, D, 16, kv, new, spread=0.05)
    masks = np.zeros(c["T"], np.uint64)
    for r, n in enumerate(new):
        first = int(c["q_start"][r])
        if n <= 64:
            masks[first:first + n] = tree_ref.tree_plan([n], [0, n], tree_ref.random_parents(rng, n), n)[0]
    out, _ = _attend(torch, cq, c, masks, bound)
    got, q = out.float().cpu().numpy().astype(np.float64), c["q"].float().cpu().numpy()
    scale = float(np.float32(D ** -0.5))
    for r, n in enumerate(new):
        first, base = int(c["q_start"][r]), past[r]
        for t in range(n):
            seen = np.arange(base + t + 1) if n > 64 else \
                np.array(list(range(base)) + [base + j for j in range(n) if int(masks[first + t]) >> j & 1])
            page, row = c["table"][r][seen // 16], seen % 16
            k1, v1 = c["k"][page, :, row][:, :, None], c["v"][page, :, row][:, :, None]
            want, _, e32, _ = kv_ref.attend(q[first + t:first + t + 1], k1, v1, c["ks"][page], c["vs"][page],
                                            np.arange(len(seen))[None], [len(seen)], [0, 1], scale, False, 0, "f32" if n <= 64 else "f16")
            av = np.abs(v1[:, :, 0].astype(np.float64) * c["vs"][page][:, :, None]).max(0)      # at least the sum of p |v|
            av = np.repeat(av, 4, 0)
            most = e32[0]
            if n <= 64:
                most = most + 2.0 ** -21 * av + len(seen) * 2.0 ** -31 * 127 * c["vs"][page].max() + \
                    2.0 ** -11 * np.abs(want[0]) + 2.0 ** -24
            off = np.abs(got[first + t] - want[0])
            assert (off <= most).all(), f"request {r} token {t}: worst {(off / most).max():.2f} of its bound"


@pytest.mark.parametrize("D,n,R", [(64, 1, 57), (128, 2, 57), (64, 20, 12), (128, 20, 12), (128, 60, 6)])
def test_fp32_sums_of_long_contexts_round(D, n, R):
    """40000 keys, enough requests that none is split over the keys, and values of one sign between 100 and 127 steps: sums
    that are cut off at each addition lose some 2^-25 of themselves 2500 times over, 1e-5 (rows kernel) to 5e-5 of every result.

    Bound, relative to the result: every probability may be off by 2 e_s (as in kv_ref.attend, e_s = 2^-18 A + 64 * 2^-23, A =
    the largest scale |q| |k|), which moves a weighted mean of values in [100, 127] by 2 e_s * 27 / 100 at most; sums that
    are cut off between two that round: 32 additions of 2^-23 at full size = 2^-18 (the smaller parts of P have sums of their
    own); up to 2500 additions that round, each within 2^-24 either way, of numbers that grow: taken as independent, five
    deviations of sqrt(2500 / 3) * 2^-24 / sqrt(3) = 5 * 1e-6; the division and the result's rounding 2^-22.
    """
    torch, cq = torch_cuda(), cq_built()
    kv, P, H, Hq = 40000, 64, 8, 32
    rng = np.random.default_rng([D, n])
    pages = kv // P
    k = rng.integers(-127, 128, (pages, H, P, D)).astype(np.int8)
    v = rng.integers(100, 128, (pages, H, P, D)).astype(np.int8)
    ks, vs = np.full((pages, H), 0.01, np.float32), np.full((pages, H), 0.5, np.float32)
    cache = cq.KVCache(*(dev(torch, x) for x in (k, v, ks, vs)))
    q = dev(torch, (rng.standard_normal((n, Hq, D)) * 0.3).astype(np.float32)).repeat(R, 1, 1)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(R, 1)             # all read the same pages
    mask = tree_ref.tree_plan([n], [0, n], tree_ref.random_parents(rng, n), n)[0]
    out, _ = cq.attn_tree_t(q, cache, table, torch.full((R,), kv, dtype=torch.int32, device="cuda"),
                            torch.arange(R + 1, dtype=torch.int32, device="cuda") * n, dev(torch, mask.view(np.int64)).repeat(R), n)
    out = out.double().view(R, n, Hq, D)
    assert torch.equal(out, out[:1].expand_as(out))
    for h in (0, H - 1):
        kk = dev(torch, k[:, h]).double().view(kv, D) * float(ks[0, 0])
        vv = dev(torch, v[:, h]).double().view(kv, D) * 0.5
        qq = q[:n, h * 4:h * 4 + 4].double()
        z = torch.einsum("ngd,kd->ngk", qq, kk) * D ** -0.5
        hide = torch.zeros((n, kv), dtype=torch.bool, device="cuda")
        hide[:, kv - n:] = (dev(torch, mask.view(np.int64))[:, None] >> torch.arange(n, device="cuda")) & 1 == 0
        want = torch.softmax(z.masked_fill_(hide[:, None], -float("inf")), -1) @ vv
        A = (torch.einsum("ngd,kd->ngk", qq.abs(), kk.abs()) * D ** -0.5).max().item()
        es = 2.0 ** -18 * A + 64 * 2.0 ** -23
        most = 2 * es * 0.27 + 2.0 ** -18 + 5e-6 + 2.0 ** -22
        off = ((out[0, :, h * 4:h * 4 + 4] - want).abs() / want).max().item()
        assert off <= most, f"{off:.2e} of {most:.2e}"


@pytest.mark.parametrize("dtype,D,n,R,kv", [("f16", 64, 1, 57, 262144), ("f16", 128, 3, 57, 262144), ("f16", 64, 20, 12, 262144),
                                            ("f16", 128, 60, 12, 262144), ("bf16", 64, 20, 12, 524288), ("bf16", 128, 60, 12, 524288)])
def test_16_bit_sums_of_very_long_contexts_round(dtype, D, n, R, kv):
    """As above, where what is cut off passes the result's own rounding: contexts of a quarter and half a million keys.

    Bound: half a step of the result; the probabilities' errors as above, and of bfloat16's 11 bits 2^-12 (their roundings
    do not fall into step: a mean of them is far less); sums that are cut off go over 512 additions (binary16: 4096 keys,
    two parts) or 2048 (bfloat16: 32768 keys) and grow evenly, so that they are half their size on average, each off by at
    most 2^-23 for the sum and as much for the products that are cut off beside it: 2^-14 and 2^-12; and 5e-6 for those
    that round."""
    torch, cq = torch_cuda(), cq_built()
    P, H, Hq = 64, 8, 32
    g = torch.Generator(device="cuda")
    g.manual_seed(kv + D + n)
    shape = (kv // P, H, P, D)
    k = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8, device="cuda")
    v = torch.randint(100, 128, shape, generator=g, dtype=torch.int8, device="cuda")
    s = torch.tensor([0.01, 0.5018], device="cuda")
    cache = cq.KVCache(k, v, s[:1].expand(shape[0], H).contiguous(), s[1:].expand(shape[0], H).contiguous())
    dt = torch.float16 if dtype == "f16" else torch.bfloat16
    q = (torch.randn(n, Hq, D, generator=g, device="cuda") * 0.3).to(dt)
    table = torch.arange(shape[0], dtype=torch.int32, device="cuda").repeat(R, 1)
    mask = torch.tensor([1 << i | 1 for i in range(n)], dtype=torch.int64, device="cuda")
    out, _ = cq.attn_tree_t(q.repeat(R, 1, 1), cache, table, torch.full((R,), kv, dtype=torch.int32, device="cuda"),
                            torch.arange(R + 1, dtype=torch.int32, device="cuda") * n, mask.repeat(R), n)
    out = out.view(R, n, Hq, D)
    h = H - 1
    kk, vv = (x[:, h].reshape(kv, D).double() * y.double() for x, y in ((k, s[0]), (v, s[1])))
    t = slice(0, n, max(n // 6, 1))
    qq = q[t, h * 4:].double()
    z = torch.einsum("ngd,kd->ngk", qq, kk) * D ** -0.5
    z[:, :, kv - n:].masked_fill_(((mask[t, None] >> torch.arange(n, device="cuda")) & 1 == 0)[:, None], -float("inf"))
    want = torch.softmax(z, -1) @ vv
    A = (qq.abs().sum(-1).max() * kk.abs().max() * D ** -0.5).item()
    es = 2.0 ** -18 * A + 64 * 2.0 ** -23
    most = 2 * es * 0.27 + (2.0 ** -14 if dtype == "f16" else 2 * 2.0 ** -12) + 5e-6
    half = torch.finfo(dt).eps / 2 * torch.exp2(torch.floor(torch.log2(want)))
    off = (out[:, t, h * 4:].double() - want).abs()       # all requests read the same
    assert (off <= half + most * want).all(), f"{(off / (half + most * want)).max().item():.2f} of its bound"


@pytest.mark.parametrize("D", [64, 128])
def test_binary16_prompts_over_very_long_contexts_round(D):
    """The same for a prompt in a call that has two row tiles a CTA (by the bound of new tokens): 100 tokens over a quarter of a
    million keys each, requests enough that none is split over its keys.

    Bound: half a step of the result; probabilities of 11 bits 2^-12, as of bfloat16 above; sums that are cut off over 512
    additions (8192 keys): 2^-14; scores and exponentials as above, and 5e-6."""
    torch, cq = torch_cuda(), cq_built()
    P, H, Hq, n, R, kv = 64, 8, 16, 100, 12, 262144
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    shape = (kv // P, H, P, D)
    k = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8, device="cuda")
    v = torch.randint(100, 128, shape, generator=g, dtype=torch.int8, device="cuda")
    s = torch.tensor([0.01, 0.5018], device="cuda")
    cache = cq.KVCache(k, v, s[:1].expand(shape[0], H).contiguous(), s[1:].expand(shape[0], H).contiguous())
    q = (torch.randn(n, Hq, D, generator=g, device="cuda") * 0.3).half()
    table = torch.arange(shape[0], dtype=torch.int32, device="cuda").repeat(R, 1)
    out, _ = cq.attn_tree_t(q.repeat(R, 1, 1), cache, table, torch.full((R,), kv, dtype=torch.int32, device="cuda"),
                            torch.arange(R + 1, dtype=torch.int32, device="cuda") * n,
                            torch.zeros(R * n, dtype=torch.int64, device="cuda"), 3000)
    t, h = torch.tensor([0, 41, 99], device="cuda"), H - 1
    kk, vv = (x[:, h].reshape(kv, D).double() * y.double() for x, y in ((k, s[0]), (v, s[1])))
    qq = q[t, h * 2:].double()
    z = torch.einsum("ngd,kd->ngk", qq, kk) * D ** -0.5
    for i, at in enumerate(t.tolist()):
        z[i, :, kv - n + at + 1:] = -float("inf")
    want = torch.softmax(z, -1) @ vv
    A = (qq.abs().sum(-1).max() * kk.abs().max() * D ** -0.5).item()
    most = 2 * (2.0 ** -18 * A + 64 * 2.0 ** -23) * 0.27 + 2.0 ** -12 + 2.0 ** -14 + 5e-6
    half = 2.0 ** -11 * torch.exp2(torch.floor(torch.log2(want)))
    off = (out.view(R, n, Hq, D)[:, t, h * 2:].double() - want).abs()
    assert (off <= half + most * want).all(), f"{(off / (half + most * want)).max().item():.2f} of its bound"
