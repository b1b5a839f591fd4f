"""Cross attention at the edges: batches whose empty key tiles the backward's CTAs pass over (more sequences than a
warp has lanes, runs without a key), tensors whose offsets pass 32 bits, and both directions under the
bounds-checked build (the normal build's outputs bit for bit, and a store past a reported end caught).
Bounds as in test_gpu_cross.py and test_gpu_cross_backward.py."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import cross_ref as ref
from tests.test_gpu_cross import SCALE, Problem
from tests.test_gpu_cross_backward import NAMES, Grad

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def lengths(kind, B, Sk):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, Sk + 1, (B,), generator=g)
    if kind == "first 40 empty":
        lens[:40] = 0
    elif kind == "last 40 empty":
        lens[-40:] = 0
    elif kind == "one":
        lens[:] = 0
        lens[B // 2] = Sk
    elif kind == "none":
        lens[:] = 0
    return lens.tolist()


@pytest.mark.parametrize("kind", ["any", "first 40 empty", "last 40 empty", "one", "none"])
@pytest.mark.parametrize("B,H,Sq,Sk", [(70, 3, 40, 300), (97, 2, 130, 140)])
def test_key_tiles_passed_over(lib, B, H, Sq, Sk, kind):
    p = Grad(lib, B, H, Sq, Sk, lens=lengths(kind, B, Sk))
    p.check(p.out, p.lse)
    grads = p.backward(lib)
    lib.check_device_error()
    p.check_grads(grads)


def test_key_tiles_passed_over_with_shares(lib):
    p = Grad(lib, 2, 16, 2048, 300, lens=[300, 100])
    grads = p.backward(lib)
    lib.check_device_error()
    p.check_grads(grads)


def test_offsets_past_32_bits(lib):
    # 128 heads x 140000 keys: 4.6 GB and 2.3e9 elements in K, V and their gradients.  The additions of 1094 tiles are
    # off by 2^-14 of their terms' sum at most, which is within the 0.02 of the rounded weights' 2^-8 in the bounds
    H, Sq, Sk = 128, 3, 140000
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    x = rnd(1, Sq, H, 128), rnd(1, Sq, H, 64), rnd(1, Sk, H, 128), rnd(1, Sk, 64), rnd(1, Sk, H, 128)
    d_out = rnd(1, Sq, H, 128)
    out, lse = lib.mla_cross_attention(*x, softmax_scale=SCALE)
    grads = lib.mla_cross_attention_backward(*x, out, lse, d_out, softmax_scale=SCALE)
    lib.check_device_error()
    for h in (0, 127):
        one = [t[:, :, h:h + 1] if t.dim() == 4 else t for t in x]
        o, l, a, e = ref.forward(*one, None, SCALE)
        e = 2.0 ** -16 * e
        tol = 2.0 ** -8 * (o.abs() + (1 + 2.0 ** -7) * (a + o.abs())) + 4 * e.transpose(1, 2)[..., None] * a
        assert bool(((out[:, :, h:h + 1].double() - o).abs() <= tol).all())
        assert bool(((lse[:, h:h + 1].double() - l).abs() <= e + 2.0 ** -18).all())
        want, bounds = ref.backward(*one, None, SCALE, out[:, :, h:h + 1], lse[:, h:h + 1], d_out[:, :, h:h + 1])
        for i in (0, 1, 2, 4):
            got = grads[i][:, :, h:h + 1].double()
            assert bool(((got - want[i]).abs() <= 2.0 ** -8 * want[i].abs() + 1.02 * bounds[i]).all()), (NAMES[i], h)
    # the rope key's, a sum over the heads, at its first and last keys
    for at in (slice(0, 200), slice(Sk - 200, Sk)):
        k = [t[:, at] for t in x[2:]]
        want, bounds = ref.backward(*x[:2], *k, None, SCALE, out, lse, d_out)
        assert bool(((grads[3][:, at].double() - want[3]).abs() <= 2.0 ** -8 * want[3].abs() + 1.02 * bounds[3]).all())


CHILD = r"""
import os, sys
import numpy as np
sys.path.insert(0, os.environ["MLA_REPO"])
from tests.test_gpu_cross_edges import CASES, run
from mla_flash_attention_gb300 import binding
assert binding.testing_bounds_checked()
res = {}
for k, case in enumerate(CASES):
    for i, a in enumerate(run(binding, case)):
        res["%d_%d" % (k, i)] = a
    binding.check_device_error()
    binding.testing_bounds_shrink(256)  # out and dq_nope reported one row short
    try:
        run(binding, case)
    finally:
        binding.testing_bounds_shrink(0)
    try:
        binding.check_device_error()
        raise SystemExit("%r: a store past the reported end was not caught" % (case,))
    except binding.MLAError as e:
        assert e.status == 6, e
np.savez(sys.argv[1], **res)
print("child ok")
"""

# whole and ragged tiles; keys in shares; both kinds of shares in the backward; passed-over tiles; no keys
CASES = [(2, 3, 300, 260, None), (1, 2, 5, 6000, None), (1, 1, 1500, 1700, None), (40, 4, 17, 200, "any"), (3, 2, 9, 50, "none")]


def run(lib, case):
    B, H, Sq, Sk, kind = case
    p = Problem(B, H, Sq, Sk, lens=None if kind is None else lengths(kind, B, Sk))
    out, lse = p.run(lib)
    grads = lib.mla_cross_attention_backward(*p.args()[:5], out, lse, out, p.lens, softmax_scale=SCALE)
    torch.cuda.synchronize()
    return [t.view(torch.uint8).cpu().numpy() for t in (out, lse, *grads)]


def test_bounds_checked_build(lib, tmp_path):
    from mla_flash_attention_gb300 import build

    path = str(tmp_path / "out.npz")
    env = dict(os.environ, MLA_GB300_LIB=build.build(debug=True), MLA_REPO=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD, path], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    got = np.load(path)
    for k, case in enumerate(CASES):
        for i, a in enumerate(run(lib, case)):
            assert np.array_equal(got["%d_%d" % (k, i)], a), (case, i)
    lib.check_device_error()
