"""Routing where 32 bits mislead: the choice is the formulas', and weights are within 1e-6 of themselves.  Inputs are picked on
the CPU for what 32 bits make of them."""
import numpy as np
import pytest
import torch

from tests import moe_oracle as mo
from tests.test_moe_route import check

F = np.float32


def sigmoid(z):
    return 1 / (1 + np.exp(-np.asarray(z, np.float64)))


def opposite_biases(big, rows=100):
    """Rows of 4 groups of two experts with biases +big and -big, which cancel in a group's sum; and the biases.  Group 0 is
    the best and group 1 the next.  Rounding score + bias takes both scores of group 0 down and both of group 1 up, so that
    32 bits have the sums the other way round, a step of +-big apart, which is more than scores of 1 are rounded by."""
    rng = np.random.default_rng(1)
    step = float(np.spacing(F(big)))
    cell = rng.integers(int(0.55 / step), int(0.9 / step), (rows, 2))
    down, up = rng.uniform(0.3, 0.42, (rows, 2)), rng.uniform(0.58, 0.7, (rows, 2))
    first, second = (cell + down) * step, (cell - [0, 1] + up) * step
    p = np.concatenate([first, second], 1)
    z = np.concatenate([np.log(p / (1 - p)), np.tile([-5.0, -5.0, -6.0, -6.0], (rows, 1))], 1).astype(F)
    return z, np.tile([big, -big], 4)


def test_the_inputs_mislead_32_bits():
    for big in (100.0, 1000.0):
        z, b = opposite_biases(big)
        c = F(sigmoid(z)) + F(b)
        assert np.all((c[:, 2] + c[:, 3]) - (c[:, 0] + c[:, 1]) >= 0.9 * np.spacing(F(big)))
        ids, _ = mo.route(z, 2, "sigmoid", b, 4, 1, 2, True, 1.0)
        assert np.all(ids == [0, 1])


@pytest.mark.gpu
@pytest.mark.parametrize("big", [100.0, 1000.0])
def test_groups_whose_biases_cancel(qk, big):
    z, b = opposite_biases(big)
    check(qk, z, 2, "sigmoid", b, 4, 1, 2)
    check(qk, z, 2, "sigmoid", b, 4, 2, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_an_expert_behind_the_next_one(qk, score):
    """The choice is undecided between the last that is chosen and one that 32 bits put two places behind it: a large score
    that its bias takes back to the others' size, beside small ones that are exact."""
    rng = np.random.default_rng(2)
    rows = []
    for _ in range(4000):
        top = F(rng.uniform(1.5, 4))
        z = np.array([top, -15.0, -15.015, -18, -18, -18, -18, -18], F)
        p = sigmoid(z)
        if score == "softmax":
            z[1:3] += top
            z[3] = top - F(rng.uniform(0.8, 2))          # (its bias takes it out)
            p = np.exp(z.astype(np.float64)) / np.exp(z.astype(np.float64)).sum()
        below = p[0] - float(F(p[0]))
        # exact: first, by a little; in 32 bits: behind both others
        b = -(p[0] - p[1] - 5e-9)
        b0 = F(b)
        c = p[0] + float(b0)
        if below > 1e-8 and c > p[1] + 2e-9 and float(F(F(p[0]) + b0)) < p[2] - 2e-9:
            rows.append((z, b0))
        if len(rows) == 12:
            break
    assert len(rows) == 12
    for z, b0 in rows:
        bias = np.zeros(8)
        bias[0], bias[3] = b0, -10
        check(qk, z[None], 1, score, bias, renorm=False)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("low", [-np.inf, float(np.finfo(F).min), -1e4])
def test_experts_that_a_bias_masks(qk, score, low):
    rng = np.random.default_rng(3)
    z = rng.standard_normal((50, 64))
    bias = 0.1 * rng.standard_normal(64)
    bias[rng.permutation(64)[:40]] = low
    check(qk, z, 8, score, bias)
    check(qk, z, 8, score, bias, 8, 3, 2)
    check(qk, z, 8, score, bias, 8, 3, 1)
    few = bias[:12].copy()
    few[::2] = low                                # and chosen all the same, where nothing else is left
    check(qk, z[:, :12], 12, score, few)
    check(qk, z[:, :12], 5, score, few, 6, 3, 2)
    bias[:16] = low                               # whole groups, too
    check(qk, z, 8, score, bias, 8, 5, 2)


@pytest.mark.gpu
def test_scores_below_the_normal_numbers(qk):
    """Sums of two scores that 32 bits hold in a few bits, or as zero."""
    rng = np.random.default_rng(4)
    z = F(-100 + 12 * rng.random((400, 16)))
    check(qk, z, 2, "sigmoid", None, 8, 2, 2)
    z[:, 0] = 0                                   # softmax: the others lie that far below
    check(qk, z, 4, "softmax", None, 8, 2, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [64, 512, 1024])
def test_weights_of_logits_far_apart(qk, renorm, E):
    """Chosen logits 20 to 80 below the largest, whose differences 32 bits round."""
    rng = np.random.default_rng(5)
    z = F(rng.uniform(-150, -100, (60, E)))
    for i in range(7):
        z[:, i] = F(10.1 + rng.random(60) - 12 * i)
    check(qk, z, 7, "softmax", renorm=renorm)
    check(qk, F(rng.uniform(-3, 3, (60, E))), 7, "softmax", renorm=renorm)
    check(qk, z - 60, 7, "sigmoid", renorm=True)


@pytest.mark.gpu
def test_small_sigmoids_beside_larger_ones(qk):
    """Scores below 32 bits' range that are within it over their sum."""
    rng = np.random.default_rng(6)
    z = F(rng.uniform(-95, -84, (200, 8)))
    z[:, 0] = F(rng.uniform(-28, -8, 200))
    check(qk, z, 8, "sigmoid")
    z[:, 1] = F(rng.uniform(-12, 12, 200))
    check(qk, z, 8, "sigmoid")
    check(qk, z, 8, "sigmoid", renorm=False)
    check(qk, F(rng.uniform(-60, 60, (200, 8))), 8, "sigmoid")
