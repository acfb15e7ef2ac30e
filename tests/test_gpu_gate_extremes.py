"""Gates on logits where fp32 scores or keys say less than usual: the smallest fp32 numbers, whose keys drop
more than a margin relative to them covers, and sigmoid scores below the smallest normal numbers, which
fp32 rounds to 0 while their sums still order groups. Choice and tables are those of the 64-bit scores."""
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


@pytest.mark.parametrize("top", [1, 2])
def test_groups_of_scores_that_fp32_rounds_to_zero(top):
    # two scores of 3.0e-39 are more than one of 3.1e-39, although fp32 has 0 for one of the two
    l = np.float32([[-88.70, -88.73, -88.69, -200.0]])
    _, idx, _ = check(device(), l, 1, dict(score="sigmoid", n_group=2, topk_group=1, group_top=top))
    assert idx[0, 0] == (0 if top == 2 else 2)


@pytest.mark.parametrize("E,G,Gk", [(32, 4, 1), (64, 8, 3), (256, 8, 4), (160, 8, 3), (60, 5, 2), (1001, 7, 3)])
@pytest.mark.parametrize("renorm", [0, 1])
def test_groups_of_the_smallest_scores(E, G, Gk, renorm):
    rng = np.random.default_rng(E)
    l = (-88.72 + 0.05 * rng.standard_normal((64, E))).astype(np.float32)
    l[::2] = np.where(rng.random((32, E)) < 0.8, np.float32(-200.0), l[::2])   # few of them a group
    l[40:50] -= 10.0                                                           # below every fp32 number
    l[50:60] += rng.uniform(-16, 4, (10, E)).astype(np.float32)
    rule = dict(score="sigmoid", n_group=G, topk_group=Gk, group_top=2, renorm=renorm)
    check(device(), l, 2, rule)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 64, 160])
def test_ratios_of_scores_that_are_far_apart(score, E):
    """Experts taken for their bias: one score is far above the smallest fp32 numbers, another below them, and
    their ratio is a number like any other."""
    rng = np.random.default_rng(E)
    l = rng.uniform(-130, -40, (60, E)).astype(np.float32)
    l[:, 0] = 3.0                                             # what softmax's scores are relative to
    l[::3] += 20.0
    b = np.linspace(8, 9, E, dtype=np.float32)
    b[0] = -100.0                                             # and no token takes
    check(device(), l, 4, dict(score=score), b)
