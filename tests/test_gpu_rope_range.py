"""Norm and rotation at the ends of what the call takes: frequencies of either sign at far positions, rows of tiny values."""
import numpy as np
import pytest

import tree_ref
from helpers import cq_built, dev, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_negative_frequencies_are_the_positive_ones_turned_back(D, adjacent):
    """Turning (a, b) by -phi is turning (a, -b) by phi with b's sign changed: the same products and roundings, so the
    same bits, at any position. And against the formula: angles to 2^-31 of a turn at 2^31, sine and cosine 5.2 u, products
    and their sum 2 u, the result's rounding 1 u, with u = 2^-24: 8.2 u (|a| + |b|), and 2 pi 2^-31 = 0.05 u."""
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng(D)
    half = D // 2
    freqs = np.concatenate([10.0 ** rng.uniform(-8, 0, half - 6), [0.05 * 2 * np.pi, 1e-3, 3.0, 1e-18, 1e6, 2.0 ** 30]])
    pos = np.concatenate([2 ** 31 - 1 - rng.integers(0, 1000, 40), rng.integers(0, 2 ** 31, 40), [0, 1, 2 ** 30]]).astype(np.int32)
    x = rng.standard_normal((len(pos), 2, D)).astype(np.float32)
    b = np.arange(1, D, 2) if adjacent else np.arange(half, D)
    back = x.copy()
    back[..., b] *= -1
    run = lambda v, f: cq.qk_rope_t(dev(torch, v), dev(torch, v[:, :1]), dev(torch, pos), dev(torch, f), adjacent=adjacent)[0].cpu().numpy()
    got, want = run(x, -freqs), run(back, freqs)
    want[..., b] *= -1
    assert np.array_equal(got, want), f"largest difference {np.abs(got - want).max():.2e}"
    ref, _ = tree_ref.rope(x, None, 0.0, pos, -freqs, adjacent, 2.0 ** -24)
    far = freqs > 10                                     # (angles that long doubles of 64 bits do not hold)
    ia = np.arange(0, D, 2) if adjacent else np.arange(half)
    size = np.abs(x.astype(np.longdouble))
    size[..., ia] = size[..., b] = size[..., ia] + size[..., b]
    size[..., ia[far]] = size[..., b[far]] = np.inf
    assert (np.abs(got - ref) <= 8.25 * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("scale", [1e-13, 1e-15, 1e-19, 1e-25, 1e-36, 1e-40])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-30, 1e-26])
@pytest.mark.parametrize("D", [64, 128])
def test_norms_of_tiny_rows(scale, eps, D):
    """Rows whose squares are below fp32's smallest numbers, beside ordinary ones, with an eps that does not hide it."""
    torch, cq = torch_cuda(), cq_built()
    rng = np.random.default_rng([D, int(-np.log10(scale))])
    x = rng.standard_normal((19, 4, D))
    x[:, 1:] *= scale
    x[:, 2] *= 10.0 ** -rng.uniform(0, 2, (19, 1))
    x = x.astype(np.float32)
    w = (1 + 0.3 * rng.standard_normal(D)).astype(np.float32)
    pos = rng.integers(0, 100000, 19).astype(np.int32)
    freqs = 10000.0 ** (-2.0 * np.arange(D // 2) / D)
    q, k = cq.qk_rope_t(dev(torch, x), dev(torch, x[:, 1:2]), dev(torch, pos), dev(torch, freqs), q_norm=dev(torch, w), k_norm=dev(torch, w), eps=eps)
    want, bound = tree_ref.rope(x, w, eps, pos, freqs, False, 2.0 ** -24)
    off = np.abs(q.cpu().numpy().astype(np.longdouble) - want)
    assert (off <= bound).all(), f"worst {(off / bound).max():.2f} of its bound"
    assert torch.equal(k[:, 0], q[:, 1])
