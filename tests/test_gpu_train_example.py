"""The draft-head training example: the losses and the overlap together."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_training_raises_the_accepted_length():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from train_draft_head import train
    first, last, kl0, kl1, tau0, tau1 = train(steps=120)
    assert last < 0.7 * first and kl1 < 0.7 * kl0 and tau1 > tau0 + 0.2
