"""The norm, append and tree kernels under the bounds-checked build (MLA_DEBUG): they run clean, with
the normal build's outputs bit for bit, and the checks catch a store past a reported end."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from gen import make_decode

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import os, sys
import numpy as np
sys.path.insert(0, os.environ["MLA_REPO"])
from tests.test_gpu_rope_bounds_build import CASES, run
from mla_flash_attention_gb300 import binding
assert binding.testing_bounds_checked()
res = {}
for name in CASES:
    for i, a in enumerate(run(binding, name)):
        res["%s_%d" % (name, i)] = a
    binding.check_device_error()
    for rows in CASES[name]:  # an output reported so many bytes short
        binding.testing_bounds_shrink(rows)
        try:
            run(binding, name)
        finally:
            binding.testing_bounds_shrink(0)
        try:
            binding.check_device_error()
            raise SystemExit("%s: a store past the reported end was not caught" % name)
        except binding.MLAError as e:
            assert e.status == 6, e
np.savez(sys.argv[1], **res)
print("child ok")
"""

# one row of q_nope / dq / out reported missing; the append's places are checked page by page anyway
CASES = {"norm_rope": [256], "norm_rope_grad": [384], "append": [], "tree_bf16": [1024], "tree_fp8": [1024]}


def run(lib, name):
    g = torch.Generator(device="cuda").manual_seed(1)

    def rnd(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    turns = lib.rope_turns(10000.0 ** (-np.arange(0, 64, 2) / 64), "cuda")
    if name.startswith("norm"):
        q, kn, kr, w = rnd(2, 37, 5, 192), rnd(2, 37, 5, 128), rnd(2, 37, 64), [rnd(d) for d in (128, 64, 128, 64)]
        kw = dict(zip(("q_nope_weight", "q_rope_weight", "k_nope_weight", "k_rope_weight"), w), rope_turns=turns,
                  positions=torch.arange(74, device="cuda", dtype=torch.int32).view(2, 37))
        if name == "norm_rope":
            out = lib.mla_qk_norm_rope(q, kn, kr, **kw)
        else:
            out = lib.mla_qk_norm_rope_backward(rnd(2, 37, 5, 128), rnd(2, 37, 5, 64), rnd(2, 37, 5, 128),
                                                rnd(2, 37, 64, dtype=torch.float32), q, kn, kr, **kw)
    else:
        from mla_flash_attention_gb300.testing import decode_to_device

        # two query tiles, splits merged by both kernels, padding rows and a padded tile
        inp = make_decode(3, 40, 5, [5, 130, 7000], fp8=name == "tree_fp8", seed=70)
        d = decode_to_device(inp, torch.device("cuda"))
        if name == "append":
            lib.mla_rope_append(rnd(3, 5, 576), *d["args"][2:5], rope_turns=turns)
            out = [d["args"][2]]
        else:
            mask, _ = lib.tree_mask_from_parents([-1, 0, 0, 1, 3])
            new = torch.tensor([5, 2, 5], dtype=torch.int32, device="cuda")
            out = lib.mla_decode_tree(*d["args"], mask.cuda(), **d["kwargs"], new_lens=new, softmax_scale=0.07)
    torch.cuda.synchronize()
    return [t.view(torch.uint8).cpu().numpy() for t in out]


def test_clean_identical_and_live(lib, tmp_path):
    from mla_flash_attention_gb300 import build

    path = str(tmp_path / "out.npz")
    env = dict(os.environ, MLA_GB300_LIB=build.build(debug=True), MLA_REPO=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD, path], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    got = np.load(path)
    for name in CASES:
        for i, a in enumerate(run(lib, name)):
            assert np.array_equal(got["%s_%d" % (name, i)], a), (name, i)
    lib.check_device_error()
