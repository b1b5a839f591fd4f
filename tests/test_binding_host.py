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
