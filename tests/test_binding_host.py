"""The binding's host-side helpers as a program sets torch up (CPU only)."""
import pytest
import torch


@pytest.fixture(scope="module")
def binding():
    import os

    from mla_flash_attention_gb300 import build

    if not (os.path.exists(build.LIB) and os.path.exists(build.MARSHAL)):
        build.build()
    from mla_flash_attention_gb300 import binding

    return binding


def test_tree_masks_under_another_default_device(binding):
    # a program that sets torch's default device to its GPU ("meta" stands for it here)
    parents = torch.tensor([[-1, 0, 0, 1], [-1, -1, 1, 2]])
    want = binding.tree_mask_from_parents(parents)
    torch.set_default_device("meta")
    try:
        got = binding.tree_mask_from_parents(parents)
    finally:
        torch.set_default_device(None)
    for g, w in zip(got, want):
        assert g.device.type == "cpu" and torch.equal(g, w)


def test_calls_of_the_plain_binding_without_the_marshalling_module(binding):
    # built for another torch, say: the attention calls do not need it, the ones it marshals say so
    import os
    import subprocess
    import sys

    code = """
import sys
sys.modules["mla_flash_attention_gb300._marshal"] = None
from mla_flash_attention_gb300 import binding
assert binding.version() > 0 and callable(binding.mla_prefill)
for call in (lambda: binding.mla_qk_norm_rope(None, positions=None, rope_turns=None),
             lambda: binding.mla_qk_norm_rope_backward(None, None, None, None, positions=None, rope_turns=None),
             lambda: binding.mla_rope_append(None, None, None, None, rope_turns=None),
             lambda: binding.mla_decode_tree(None, None, None, None, None, None, softmax_scale=1.0)):
    try:
        call()
    except ImportError as e:
        assert "build()" in str(e)
    else:
        raise SystemExit("no ImportError")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
