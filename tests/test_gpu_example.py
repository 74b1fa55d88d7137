"""The example trains: its policy finds the rewarded words, and the same seed gives the same
run bit for bit (every operator's sums have a fixed order)."""

import os
import sys

import pytest

from tests.gpu_util import announce, require_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


def test_policy_training_learns():
    require_gpu()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import policy_training
    announce("example policy training, 30 steps")
    rewards = policy_training.train(steps=30)
    # one word in 64 is right by chance: 2048 tokens give 0.016 +- 0.003
    assert rewards[0] < 0.05
    assert sum(rewards[-5:]) / 5 > 0.3
    announce("example policy training again, 5 steps")
    assert policy_training.train(steps=5) == rewards[:5]
