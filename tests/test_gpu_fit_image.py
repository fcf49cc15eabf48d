"""The example that trains with the loss and the training operators together."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_the_example_fits_its_image():
    import fit_image

    losses, norms = fit_image.fit(steps=60, size=64, width=256, blocks=2)
    assert torch.isfinite(losses).all() and torch.isfinite(norms).all()
    assert float(losses[-5:].mean()) < 0.5 * float(losses[0])
