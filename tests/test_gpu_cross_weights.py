"""Softmax weights of cross attention without tiles: they enter the product with V to 2^-15 (fp32 for one query, two bf16
terms for more), so that a row has the same precision alone, among others of its sequence and in a small call's blocks
of eight; and a value that is infinite is that in every row with a weight for it.

Bounds: O is rounded to bf16 once (2^-8 |O|).  A weight's upper half leaves less than 2^-7 of it, which is rounded to bf16
(2^-8 of that) and 2^-20 of the weight too large; exponentials, fp32 sums of weights and of products add less than 2^-17
at these lengths: below 2^-14 (A + |O|) together, A = sum_j p_j |v_j|.  Scores are off as in test_gpu_cross.py.
"""
import pytest
import torch

from tests.test_gpu_cross import Problem

pytestmark = pytest.mark.gpu

# (B, H, Sq, Sk): one query, two to eight, blocks of eight in small calls; runs of one step, of many, cut in shares
SIZES = [(2, 8, 1, 77), (2, 3, 2, 640), (3, 5, 3, 1500), (1, 2, 5, 9000), (4, 16, 8, 300), (2, 2, 40, 300), (1, 8, 64, 77),
         (1, 1, 100, 2000)]


def without_tiles(lib, B, H, Sq, Sk, ragged=False):
    assert lib.testing_cross_plan(B, H, Sq, Sk, ragged)[0] == 0


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("mag", [0.3, 1.0, 4.0])  # many alike weights, unlike ones, a few
def test_weights_keep_their_lower_bits(lib, size, mag):
    without_tiles(lib, *size)
    p = Problem(*size, mag=mag)
    out, lse = p.run(lib)
    lib.check_device_error()
    o, _, a, e = p.reference()
    tol = 2.0 ** -8 * (1 + 2.0 ** -7) * o.abs() + 2.0 ** -14 * (a + o.abs()) + 4 * e.transpose(1, 2)[..., None] * a
    err = (out.double() - o).abs()
    assert bool((err <= tol).all()), (err - tol).max().item()
    p.check(out, lse)


@pytest.mark.parametrize("size", SIZES)
def test_infinite_values(lib, size):
    B, H, Sq, Sk = size
    without_tiles(lib, *size)
    p = Problem(*size, mag=0.3)
    p.qn[:] = p.qr[:] = 0.0  # weights that one bf16 holds exactly
    clean = p.run(lib)
    p.v[0, 3, 0, 5], p.v[-1, Sk - 1, 1 % H, 100] = float("inf"), float("-inf")
    out, lse = p.run(lib)
    lib.check_device_error()
    assert bool((out[0, :, 0, 5] == float("inf")).all()) and bool((out[-1, :, 1 % H, 100] == float("-inf")).all())
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[0, :, 0, 5] = keep[-1, :, 1 % H, 100] = False
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse, clean[1])
    p = Problem(*size, mag=1.0)  # and weights of any bits
    p.v[0, 3, 0, 5], p.v[-1, Sk - 1, 1 % H, 100] = float("inf"), float("-inf")
    out, _ = p.run(lib)
    assert bool((out[0, :, 0, 5] == float("inf")).all()) and bool((out[-1, :, 1 % H, 100] == float("-inf")).all())
