"""Gates on logits where fp32 keys say less than usual: the smallest fp32 numbers, whose keys drop more than a
margin relative to them covers. Choice and tables are those of the 64-bit scores."""
import numpy as np
import pytest

from test_gpu_gate import check, device, pytestmark  # noqa: F401  (pytestmark: these need a GPU too)

TINY = np.float32(2.0 ** -149)


@pytest.mark.parametrize("E", [32, 64, 160, 256, 384, 1024])
@pytest.mark.parametrize("k", [1, 8])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_among_the_smallest_numbers(E, k, score):
    rng = np.random.default_rng(E + k)
    l = np.zeros((40, E), np.float32)
    l[0, :3] = np.float32([5, 3, 7]) * TINY                   # one lane's, the others far below
    l[0, 3:] = -1.0
    for t in range(1, 30):                                    # all within a few, or a few hundred, steps
        l[t] = rng.integers(-4 << t % 8, 4 << t % 8, E).astype(np.float32) * TINY
    for t in range(30, 36):                                   # on either side of the smallest normal one
        l[t] = (rng.integers(1 << 23, (1 << 23) + 400, E) - 200).astype(np.float32) * TINY
    l[36:] = rng.permutation(E).astype(np.float32) * TINY     # no two alike
    check(device(), l, k, dict(score=score))
