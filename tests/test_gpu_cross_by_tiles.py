"""Cross attention by key tiles: every case says which form it means -- one query tile (whose key tiles alternate
between the two score buffers, joined at the end), two, or two with a last block of one -- and whether its keys are cut
in shares, and asks the library's plan before it runs, so that a change of the rule that picks forms fails here and does not
leave a form without its tests.  Bounds as in test_gpu_cross.py.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import test_gpu_cross_launch_order as launch_order
from tests.test_gpu_cross import DV, SCALE, Problem
from tests.test_gpu_cross_edges import CHILD, ROOT, lengths, run

pytestmark = pytest.mark.gpu

ONE, TWO = 1, 2  # query tiles

# (B, H, Sq, Sk, query tiles, shares of the keys): what the tests below mean by their sizes
SHAPES = [
    (2, 80, 9, 500, ONE, 1), (2, 80, 31, 333, ONE, 1), (2, 80, 33, 700, ONE, 1), (1, 160, 100, 900, ONE, 1),
    (1, 152, 127, 256, ONE, 1), (1, 152, 128, 257, ONE, 1), (1, 152, 128, 1, ONE, 1), (4, 40, 70, 129, ONE, 1),
    (1, 160, 129, 300, TWO, 1), (2, 80, 200, 900, TWO, 1), (2, 80, 256, 511, TWO, 1), (1, 80, 257, 130, TWO, 1),
    (1, 80, 300, 900, TWO, 1), (1, 80, 385, 640, TWO, 1), (1, 80, 512, 385, TWO, 1), (1, 160, 513, 1, TWO, 1),
    (1, 30, 1000, 64, TWO, 1), (1, 304, 300, 260, TWO, 1)]
CUT = [(1, 3, 40, 9097, ONE), (1, 4, 100, 5000, ONE), (1, 2, 130, 5000, TWO), (2, 1, 300, 3000, TWO), (2, 2, 500, 2000, TWO)]
MANY = [(1, 160, 100, 900, ONE, 1), (2, 80, 200, 900, TWO, 1), (1, 80, 300, 900, TWO, 1)]  # every tile of a score buffer's
SMALL = [(2, 80, 70, 333, ONE, 1), (2, 80, 150, 280, TWO, 1), (1, 80, 300, 280, TWO, 1)]
PLANNED = ([(s[:4], s[4:], r) for s in SHAPES + MANY + SMALL for r in (False, True)] +
           [(s[:4], s[4:], r) for s in CUT for r in (False, True)])


def planned(lib, B, H, Sq, Sk, form, shares=None, ragged=False):
    got = lib.testing_cross_plan(B, H, Sq, Sk, ragged)
    assert got[0] == form and (got[1] == shares if shares else got[1] > 1), (B, H, Sq, Sk, got)


def solve(lib, shape, lens=None, **kw):
    planned(lib, *shape, ragged=lens is not None)
    p = Problem(*shape[:4], lens=lens, **kw)
    got = p.run(lib)
    lib.check_device_error()
    return p, got


@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(lib, shape):
    p, got = solve(lib, shape)
    p.check(*got)
    assert all(torch.equal(a, b) for a, b in zip(got, p.run(lib)))


@pytest.mark.parametrize("shape", CUT)
def test_keys_cut_in_shares(lib, shape):
    p, got = solve(lib, shape)
    p.check(*got)
    p, got = solve(lib, shape, lens=lengths("any", shape[0], shape[3]))
    p.check(*got)


ROWS = [(20, 30, ONE), (128, 30, ONE), (200, 20, TWO), (300, 20, TWO)]
LENS = [(300, [300, 0, 1, 127, 128, 129, 255, 256, 257]), (700, [-3, 701, 2 ** 31 - 1, -2 ** 31, 699, 513, 384, 385])]
PLANNED += [((len(lens), H, Sq, Sk), (form, 1), True) for Sq, H, form in ROWS for Sk, lens in LENS]


@pytest.mark.parametrize("Sq,H,form", ROWS)
@pytest.mark.parametrize("Sk,lens", LENS)
def test_key_lengths_with_nan_behind_them(lib, Sq, H, form, Sk, lens):
    p, got = solve(lib, (len(lens), H, Sq, Sk, form, 1), lens=lens)
    p.check(*got)


def ramp(kind, Sk):
    """A column of the keys, a value a key tile: its product with 4 or -4 in the queries adds 26 to a tile's scores in
    units of log2 (more than the 8 that a running maximum may lag), or 3.3 (less, so that it rises every third tile)."""
    tile = torch.arange(Sk, device="cuda") // 128
    if kind == "slow":
        return tile * 8
    if kind == "by turns":  # the two score buffers' maxima far apart, the higher one's growing
        return torch.where(tile % 2 == 0, tile * 64, 0)
    if kind == "last":
        return torch.where(tile == tile[-1], 256, 0)
    return tile * 64


@pytest.mark.parametrize("kind", ["fast", "slow", "by turns", "last"])
@pytest.mark.parametrize("ends", [False, True])
@pytest.mark.parametrize("shape", MANY)
def test_rising_and_falling_maxima(lib, shape, kind, ends):
    B, H, Sq, Sk = shape[:4]
    planned(lib, *shape, ragged=ends)
    p = Problem(B, H, Sq, Sk, mag=0.3, lens=[Sk - 3] * B if ends else None)  # (or ending inside the last tile)
    # rows that rise, rows that fall, in every warp
    p.qn[..., 0] = torch.where(torch.arange(Sq, device="cuda") % 2 == 0, 4.0, -4.0)[:, None].bfloat16()
    p.kn[..., 0] = ramp(kind, Sk)[:, None].bfloat16()
    if ends:
        p.kn[:, Sk - 3:] = float("nan")
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)


@pytest.mark.parametrize("mag,scale", [(0.0, SCALE), (1e-20, SCALE), (30.0, SCALE), (1.0, 1e-6), (1.0, 3.0)])
@pytest.mark.parametrize("shape", SMALL)
def test_magnitudes_and_scales(lib, shape, mag, scale):
    B, Sk = shape[0], shape[3]
    p, got = solve(lib, shape, lens=([Sk, 200] * B)[:B], mag=mag, scale=scale)
    p.check(*got)


@pytest.mark.parametrize("shape", SMALL)
def test_non_finite_values_stay_in_their_row_head_and_sequence(lib, shape):
    B, H, Sq, Sk = shape[:4]
    p, clean = solve(lib, shape)
    p.v[0, 5, 1, 7] = float("nan")
    p.v[0, 250, 3, 100] = float("inf")
    p.kn[-1, 200, 2, 3] = float("inf")
    p.qn[-1, 9, 0, 0] = float("nan")
    p.qr[-1, Sq - 1, 4, 63] = float("nan")
    out, lse = p.run(lib)
    lib.check_device_error()
    assert bool(torch.isnan(out[0, :, 1, 7]).all()) and bool(torch.isinf(out[0, :, 3, 100]).all())
    assert not bool(torch.isfinite(out[-1, :, 2].float()).all())
    for i, h in ((9, 0), (Sq - 1, 4)):
        assert bool(torch.isnan(out[-1, i, h]).all()) and bool(torch.isnan(lse[-1, h, i]))
    keep = torch.ones(B, Sq, H, DV, dtype=torch.bool, device="cuda")
    keep[0, :, 1, 7] = keep[0, :, 3, 100] = keep[-1, :, 2] = keep[-1, 9, 0] = keep[-1, Sq - 1, 4] = False
    assert torch.equal(out[keep], clean[0][keep])
    keep = keep[..., 0].transpose(1, 2)
    assert torch.equal(lse[keep], clean[1][keep])


@pytest.mark.parametrize("shape", SMALL)
def test_scores_of_minus_infinity(lib, shape):
    B, H, Sq, Sk = shape[:4]
    planned(lib, *shape)
    p = Problem(B, H, Sq, Sk)
    p.qn[..., 0] = 1.0
    p.kn[:, :128, 3, 0] = float("-inf")  # a head whose first tile no query sees
    p.kn[:, 128:, 4, 0] = float("-inf")  # those behind the first
    p.kn[:, :, 5, 0] = float("-inf")     # no key at all
    out, lse = p.run(lib)
    lib.check_device_error()
    assert not bool(out[:, :, 5].any()) and bool(torch.isneginf(lse[:, 5]).all())
    for h, keys in ((3, slice(128, Sk)), (4, slice(0, 128))):
        q = Problem(B, 1, Sq, 1)  # the same over the keys that have a weight
        q.qn, q.qr, q.kn, q.v = p.qn[:, :, h:h + 1], p.qr[:, :, h:h + 1], p.kn[:, keys, h:h + 1], p.v[:, keys, h:h + 1]
        q.kr, q.Sk = p.kr[:, keys], q.kn.shape[1]
        q.check(out[:, :, h:h + 1], lse[:, h:h + 1])
    others = [h for h in range(H) if not 3 <= h <= 5]
    assert bool(torch.isfinite(out[:, :, others].float()).all()) and bool(torch.isfinite(lse[:, others]).all())


@pytest.mark.parametrize("shape", SMALL)
def test_writes_only_its_outputs(lib, shape):
    from tests.test_gpu_canaries import Guarded

    B, H, Sq, Sk = shape[:4]
    for lens in (None, lengths("any", B, Sk), [0] * B):
        planned(lib, *shape, ragged=lens is not None)
        p = Problem(B, H, Sq, Sk, lens=lens)
        out, lse = Guarded((B, Sq, H, DV), torch.bfloat16), Guarded((B, H, Sq), torch.float32)
        p.run(lib, out=out.t, lse=lse.t)
        lib.check_device_error()
        assert out.intact() and lse.intact()
        p.check(out.t, lse.t)


BETWEEN = [(8, 20, 60, 300, ONE, 1), (4, 40, 150, 200, TWO, 1), (2, 40, 300, 257, TWO, 1)]
SQUARE = [(1, 160, 100, 100, ONE, 1), (2, 80, 300, 300, TWO, 1)]
CAPTURED = [(2, 80, 70, 333, ONE, 1), (1, 80, 300, 700, TWO, 1)]
PLANNED += [(s[:4], s[4:], True) for s in BETWEEN + CAPTURED] + [(s[:4], s[4:], False) for s in SQUARE]


@pytest.mark.parametrize("shape", BETWEEN)
def test_back_to_back_with_the_calls_around_it(lib, shape):
    planned(lib, *shape, ragged=True)
    launch_order.test_back_to_back(lib, *shape[:4])


@pytest.mark.parametrize("shape", SQUARE)
def test_square_without_mask_is_the_prefill(lib, shape):
    p, got = solve(lib, shape)
    p.check(*got)
    p.check(*lib.mla_prefill(*p.args()[:5], softmax_scale=SCALE, causal=False))


def test_captured_replayed_and_on_side_streams(lib):
    shapes = CAPTURED
    lens = [[333, 17], [650]]
    for s in shapes:
        planned(lib, *s, ragged=True)
    ps, new = ([Problem(*s[:4], lens=[x - d for x in n], seed=k) for s, n in zip(shapes, lens)] for k, d in ((1, 0), (2, 5)))
    sides = [torch.cuda.Stream() for _ in shapes]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [[p.run(lib, stream=s) for _ in range(3)][-1] for p, s in zip(ps, sides)]  # both at once
    for p, g, s in zip(ps, got, sides):
        s.synchronize()
        p.check(*g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [p.run(lib) for p in ps]
    for p, q in zip(ps, new):
        for a, b in zip(p.args(), q.args()):
            a.copy_(b)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    lib.check_device_error()
    for q, g in zip(new, got):
        q.check(*g)


# each form's own stores of rows, of rows that see no key, and of partial results (the gradient of each runs too)
CASES = [(4, 40, 70, 333, "any"), (40, 4, 100, 130, "none"), (2, 80, 150, 280, None), (40, 4, 290, 200, "first 40 empty"),
         (1, 80, 513, 129, None), (1, 3, 40, 9097, None), (2, 1, 300, 3000, "any")]
FORMS = [(ONE, 1), (ONE, 1), (TWO, 1), (TWO, 1), (TWO, 1), (ONE, None), (TWO, None)]
PLANNED += [(c[:4], f, c[4] is not None) for c, f in zip(CASES, FORMS)]


def test_bounds_checked_build(lib, tmp_path):
    from mla_flash_attention_gb300 import build

    for c, f in zip(CASES, FORMS):
        planned(lib, *c[:4], *f, ragged=c[4] is not None)
    path = str(tmp_path / "out.npz")
    env = dict(os.environ, MLA_GB300_LIB=build.build(debug=True), MLA_REPO=ROOT)
    child = CHILD.replace("tests.test_gpu_cross_edges", "tests.test_gpu_cross_by_tiles")
    r = subprocess.run([sys.executable, "-c", child, path], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    got = np.load(path)
    for k, case in enumerate(CASES):
        for i, a in enumerate(run(lib, case)):
            assert np.array_equal(got["%d_%d" % (k, i)], a), (case, i)
    lib.check_device_error()
