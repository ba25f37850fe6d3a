"""The training example: quantisation, the block-scaled products and the
orthogonalised update together lower the loss."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_train_block8():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    from train_block8 import train
    losses = train(steps=40, width=200, tokens=520)
    assert all(l == l for l in losses)
    assert sum(losses[-5:]) < 0.5 * sum(losses[:5]), losses
