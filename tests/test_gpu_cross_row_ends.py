"""Cross attention by tiles where a sequence's queries, or its keys, end inside a warp's 32 rows: some lanes of the warp
store a row, or zero one, and others do not, between loads of tensor memory that the whole warp makes together.  With
heads enough that both directions take tiles: one query tile, two, a last block of one, shares; values against the
definition, and the bounds-checked build (whose checks part the lanes further) bit for bit as the normal one.  Bounds as in
test_gpu_cross.py and test_gpu_cross_backward.py."""
import os
import subprocess
import sys

import numpy as np
import pytest

from tests.test_gpu_cross_backward import Grad
from tests.test_gpu_cross_edges import CHILD, ROOT, lengths, run

pytestmark = pytest.mark.gpu

CASES = [(4, 40, 70, 333, "any"), (4, 40, 150, 280, "any"), (3, 50, 257, 130, None), (2, 40, 300, 260, "any"),
         (2, 2, 500, 2000, None), (1, 4, 100, 5000, None)]


@pytest.mark.parametrize("case", CASES)
def test_values(lib, case):
    B, H, Sq, Sk, kind = case
    p = Grad(lib, B, H, Sq, Sk, lens=None if kind is None else lengths(kind, B, Sk))
    p.check(p.out, p.lse)
    grads = p.backward(lib)
    lib.check_device_error()
    p.check_grads(grads)


def test_bounds_checked_build(lib, tmp_path):
    from mla_flash_attention_gb300 import build

    path = str(tmp_path / "out.npz")
    env = dict(os.environ, MLA_GB300_LIB=build.build(debug=True), MLA_REPO=ROOT)
    child = CHILD.replace("tests.test_gpu_cross_edges", "tests.test_gpu_cross_row_ends")
    r = subprocess.run([sys.executable, "-c", child, path], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    got = np.load(path)
    for k, case in enumerate(CASES):
        for i, a in enumerate(run(lib, case)):
            assert np.array_equal(got["%d_%d" % (k, i)], a), (case, i)
    lib.check_device_error()
