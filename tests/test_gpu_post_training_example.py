"""The post-training example learns: the operators together, from hidden states to updated weights."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", ["8", "32"])
def test_policy_training_raises_the_reward(bits):
    from linear_cross_entropy_tiled_gb300.examples import post_training
    h = post_training.main(["--loss", "policy", "--steps", "25", "--state-bits", bits])
    assert 0.4 < h[0][0] < 0.6                       # half of the tokens drawn are even
    assert sum(x[0] for x in h[-3:]) / 3 > h[0][0] + 0.1


@pytest.mark.parametrize("bits", ["8", "32"])
def test_preference_training_separates_the_pairs(bits):
    from linear_cross_entropy_tiled_gb300.examples import post_training
    h = post_training.main(["--loss", "preference", "--steps", "25", "--state-bits", bits])
    assert h[0][1] == pytest.approx(0.6931, abs=1e-3)   # log 2 at the starting model
    assert h[-1][0] > 0.9 and h[-1][1] < 0.6
