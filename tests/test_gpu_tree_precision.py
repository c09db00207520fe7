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
