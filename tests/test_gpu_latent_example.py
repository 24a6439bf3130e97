"""The example block: both forms of the attention agree on the cache it leaves, and its pages are what they should be."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompt", [100, 96, 15])
def test_example_block(prompt):
    import latent_moe_block as ex
    absorbed, expanded, y, y1, n_live, b = ex.main(prompt, seed=prompt)
    # each form is within 4e-3 of the definition (its own test); the folded query and the projected output add a bf16
    # rounding each (2^-9 / sqrt(3) of their norm, twice)
    assert float((absorbed.float() - expanded.float()).norm() / expanded.float().norm()) <= 8e-3 + 2 * 1.2e-3
    assert y.shape == (prompt, b.cfg.H) and bool(torch.isfinite(y.float()).all())
    assert y1.shape == (4, b.cfg.H) and bool(torch.isfinite(y1.float()).all())
    # two sequences of prompt + 1 tokens left, the prompt's full pages shared
    full = prompt // ex.PAGE
    assert n_live == full + 2 * (-(-(prompt + 1) // ex.PAGE) - full)
    assert int((b.refs > 0).sum()) == n_live and bool((b.refs[n_live:] == 0).all())
    assert b.lens.tolist() == [prompt + 1, 0, 0, prompt + 1]
