"""Stores of the gradient of cross attention by tiles: under the bounds-checked build, alone, with key lengths (the walk past key
tiles that hold no key, their zeros, queries without a key, tiles that end inside a sequence) and with both kinds
of shares; and into gradients and a workspace that are 16-byte aligned but not 32.  The cases ask the library's plan for
the form that they mean.  Bounds as in test_gpu_cross_backward.py."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests.test_gpu_cross_backward import Grad
from tests.test_gpu_cross_edges import ROOT, lengths

pytestmark = pytest.mark.gpu

# (B, H, Sq, Sk, lengths, shares of the query tiles, of the key tiles); more units than SMs where lengths are given, but once
CASES = [(70, 3, 40, 300, "any", 1, 1), (97, 2, 130, 140, "none", 1, 1), (97, 2, 130, 140, "first 40 empty", 1, 1),
         (40, 4, 33, 600, "last 40 empty", 1, 1), (30, 3, 300, 385, "one", 1, 1), (5, 2, 70, 200, "any", 1, 1),
         (2, 16, 2048, 300, "any", 2, 1), (1, 1, 60, 3000, None, 1, 6), (1, 1, 2500, 140, None, 5, 1), (2, 1, 130, 3000, "any", 1, 6)]

CHILD = r"""
import os, sys
import numpy as np, torch
sys.path.insert(0, os.environ["MLA_REPO"])
from tests.test_gpu_cross_backward_bounds import CASES, problem, run
from mla_flash_attention_gb300 import binding
assert binding.testing_bounds_checked()
res = {}
for k, case in enumerate(CASES):
    p = problem(binding, case)
    for i, a in enumerate(run(binding, p)):
        res["%d_%d" % (k, i)] = a
    binding.check_device_error()
    binding.testing_bounds_shrink(256)  # dq_nope reported one row short
    try:
        run(binding, p)
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


def problem(lib, case):
    B, H, Sq, Sk, kind, query_shares, key_shares = case
    form, q, k = lib.testing_cross_backward_plan(B, H, Sq, Sk)
    assert (form, q > 1, k > 1) == (1, query_shares > 1, key_shares > 1), (case, form, q, k)
    return Grad(lib, B, H, Sq, Sk, lens=None if kind is None else lengths(kind, B, Sk))


def run(lib, p):
    grads = p.backward(lib)
    torch.cuda.synchronize()
    return [t.view(torch.uint8).cpu().numpy() for t in grads]


def test_bounds_checked_build(lib, tmp_path):
    from mla_flash_attention_gb300 import build

    path = str(tmp_path / "out.npz")
    env = dict(os.environ, MLA_GB300_LIB=build.build(debug=True), MLA_REPO=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD, path], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    got = np.load(path)
    for k, case in enumerate(CASES):
        for i, a in enumerate(run(lib, problem(lib, case))):
            assert np.array_equal(got["%d_%d" % (k, i)], a), (case, i)
    lib.check_device_error()


@pytest.mark.parametrize("case", CASES)
def test_values(lib, case):
    p = problem(lib, case)
    grads = p.backward(lib)
    lib.check_device_error()
    p.check_grads(grads)


def half_aligned(shape, dtype=torch.bfloat16):
    """A contiguous tensor 16 bytes past a 32-byte boundary."""
    n, each = int(np.prod(shape)), torch.empty((), dtype=dtype).element_size()
    buf = torch.full((n * each + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    at = (16 - buf.data_ptr()) % 32
    t = buf[at:at + n * each].view(dtype).view(shape)
    assert t.data_ptr() % 32 == 16
    return t


@pytest.mark.parametrize("B,H,Sq,Sk,lens", [(2, 5, 150, 280, [280, 131]), (1, 1, 60, 3000, None), (2, 4, 20, 130, [130, 7])])
def test_alignment_of_sixteen_bytes(lib, B, H, Sq, Sk, lens):
    p = Grad(lib, B, H, Sq, Sk, lens=lens)
    want = p.backward(lib)
    grads = [half_aligned(t.shape) for t in p.args()[:5]]
    ws = half_aligned((lib.cross_attention_backward_workspace_size(B, H, Sq, Sk),), torch.uint8)
    p.backward(lib, grads=grads, workspace=ws)
    lib.check_device_error()
    assert all(torch.equal(a, b) for a, b in zip(want, grads))
    p.check_grads(grads)
    x = [half_aligned(t.shape) for t in p.args()[:5]]  # the operands too
    for a, b in zip(x, p.args()):
        a.copy_(b)
    out, lse = half_aligned(p.out.shape), half_aligned(p.lse.shape, torch.float32)
    lib.mla_cross_attention(*x, p.lens, softmax_scale=p.scale, out=out, lse=lse)
    assert torch.equal(out, p.out) and torch.equal(lse, p.lse)
    again = lib.mla_cross_attention_backward(*x, out, lse, p.d_out, p.lens, softmax_scale=p.scale)
    lib.check_device_error()
    assert all(torch.equal(a, b) for a, b in zip(want, again))
