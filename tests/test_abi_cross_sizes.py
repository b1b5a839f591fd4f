"""The largest counts of queries and keys that cross attention takes: one more than 2^31 - 512, and what the binding passes for
a size past an int's range, is refused by the calls and by both size queries, although one head of one sequence is
within every other limit."""
import pytest

from tests.test_abi_cross import BACKWARD, BACKWARD0, FORWARD, FORWARD0
from tests.test_abi_rope import I, Z, call, clib  # noqa: F401

LARGEST = 2 ** 31 - 512
REFUSED = [{n: v} for n in ("Sq", "Sk") for v in (LARGEST + 1, 2 ** 31 - 256, 2 ** 31 - 128, 2 ** 31 - 1)]
QUERIES = ["mla_cross_attention_workspace_size", "mla_cross_attention_backward_workspace_size"]


@pytest.mark.parametrize("kw", REFUSED)
@pytest.mark.parametrize("name,spec,defaults", [("mla_cross_attention", FORWARD, FORWARD0),
                                                ("mla_cross_attention_backward", BACKWARD, BACKWARD0)])
def test_calls_refuse(clib, name, spec, defaults, kw):  # noqa: F811
    assert call(getattr(clib, name), spec, defaults, **dict(dict(B=1, H=1, Sq=1, Sk=1, ws=16), **kw)) == 2
    assert clib.mla_last_error() == (name + ": problem too large").encode()


@pytest.mark.parametrize("kw", REFUSED)
@pytest.mark.parametrize("name", QUERIES)
def test_size_queries_refuse(clib, name, kw):  # noqa: F811
    f = getattr(clib, name)
    f.restype, f.argtypes = Z, [I, I, I, I]
    size = dict(dict(Sq=1, Sk=1), **kw)
    assert f(1, 1, size["Sq"], size["Sk"]) == 0
    assert clib.mla_last_error() == (name + ": problem too large").encode()


@pytest.mark.gpu
def test_largest_counts_have_a_size(lib):
    # (a query of the size alone: host arithmetic.  The keys' partial results of one query, and the rope keys' gradient)
    assert 128 * 4 * 2 <= lib.cross_attention_workspace_size(1, 1, 1, LARGEST) < 2 ** 24
    assert lib.cross_attention_backward_workspace_size(1, 1, 1, LARGEST) >= 64 * 4 * LARGEST
    assert lib.cross_attention_backward_workspace_size(1, 1, LARGEST, 1) >= 2 * 4 * LARGEST
    for n in (LARGEST + 1, 2 ** 31 - 1):
        assert lib.cross_attention_workspace_size(1, 1, 1, n) == lib.cross_attention_workspace_size(1, 1, n, 1) == 0
        assert lib.cross_attention_backward_workspace_size(1, 1, 1, n) == 0
        assert lib.cross_attention_backward_workspace_size(1, 1, n, 1) == 0
