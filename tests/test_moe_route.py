"""Expert routing against the formulas in 64 bits: ids equal, weights within 1e-6 of themselves (each is a quotient of
32-bit exponentials: an argument rounded by 2^-24 of at most 20, an exponential, a sum of up to 32 and a division)."""
import numpy as np
import pytest
import torch

from tests import moe_oracle as mo

pytestmark = pytest.mark.gpu


def check(qk, z, top_k, score="softmax", bias=None, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0, dtype="f32"):
    t = torch.from_numpy(np.asarray(z, np.float32)).to(mo.TORCH[dtype])
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32))
    ids, w = qk.moe_route(t.cuda(), top_k, score=score, bias=None if b is None else b.cuda(), n_groups=groups, top_groups=top_groups,
                          group_top=group_top, renorm=renorm, scale=scale)
    want, ww = mo.route(t.double().numpy(), top_k, score, None if b is None else b.double().numpy(), groups, top_groups, group_top,
                        renorm, scale)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert np.array_equal(ids.cpu().numpy(), want)
    err = np.abs(w.double().cpu().numpy() - ww)
    assert np.all(err <= 1e-6 * np.abs(ww) + 1e-38), (err / np.maximum(np.abs(ww), 1e-30)).max()
    return ids, w


@pytest.mark.parametrize("T,E,k", [(1, 128, 8), (3, 8, 2), (7, 1, 1), (5, 60, 4), (2, 1024, 32), (130, 160, 6), (4, 33, 33 - 1), (9, 512, 10), (6, 5, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_matches_the_formula(qk, T, E, k, score, biased, dtype):
    rng = np.random.default_rng(T * 1000 + E)
    check(qk, 2 * rng.standard_normal((T, E)), k, score, 0.2 * rng.standard_normal(E) if biased else None, renorm=E != 60,
          scale=2.5 if E == 160 else 1.0, dtype=dtype)


@pytest.mark.parametrize("E,groups,top_groups,k", [(256, 8, 4, 8), (64, 4, 1, 16), (60, 6, 3, 5), (32, 32, 7, 7), (1024, 16, 3, 32), (160, 8, 8, 6)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score,biased", [("sigmoid", True), ("sigmoid", False), ("softmax", False), ("softmax", True)])
def test_groups(qk, E, groups, top_groups, k, group_top, score, biased):
    if group_top > E // groups:
        group_top = 1
    rng = np.random.default_rng(E + groups)
    check(qk, 1.5 * rng.standard_normal((50, E)), k, score, 0.1 * rng.standard_normal(E) if biased else None, groups, top_groups, group_top)


def test_equal_values(qk):
    """Ties go to the lowest index, of experts and of groups, with a bias too."""
    rng = np.random.default_rng(5)
    z = rng.integers(-2, 3, (40, 128)).astype(np.float64)
    for score in ("softmax", "sigmoid"):
        check(qk, z, 8, score)
        check(qk, z, 8, score, bias=np.zeros(128))
        check(qk, z, 8, score, bias=rng.integers(0, 2, 128))
        check(qk, np.zeros((3, 64)), 6, score, groups=8, top_groups=2, group_top=2)
        check(qk, np.zeros((3, 64)), 6, score, bias=np.ones(64), groups=8, top_groups=2)


def test_order_beyond_32_bits(qk):
    """Scores + biases that differ by less than an fp32 step of them."""
    rng = np.random.default_rng(6)
    T, E = 64, 256
    z = np.float32(rng.standard_normal((T, E)))
    for score in ("sigmoid", "softmax"):
        # a bias that lifts every score of the first token to about the same value
        p = 1 / (1 + np.exp(-z[0].astype(np.float64))) if score == "sigmoid" else np.exp(z[0].astype(np.float64)) / np.exp(z[0].astype(np.float64)).sum()
        bias = np.float32(1.0 - p)
        rows = z + np.float32(1e-7) * np.arange(T, dtype=np.float32)[:, None]
        check(qk, rows, 8, score, bias)
        check(qk, rows, 8, score, bias, groups=8, top_groups=3, group_top=2)


def test_masked_experts(qk):
    """-infinity is a score of 0: chosen last, with a weight of 0; a row of nothing else gets the first ids and no weight."""
    rng = np.random.default_rng(7)
    z = rng.standard_normal((6, 64))
    z[0, 3:] = -np.inf
    z[1] = -np.inf
    z[2, ::2] = -np.inf
    z[3, 5] = np.finfo(np.float32).min
    z[4] = np.finfo(np.float32).min
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            for bias in (None, np.zeros(64), 0.1 * rng.standard_normal(64)):
                ids, w = check(qk, z, 8, score, bias, renorm=renorm)
                assert torch.all(w[1] == 0)


def test_far_logits(qk):
    """Scores under fp32's range still share their sum."""
    rng = np.random.default_rng(8)
    z = rng.standard_normal((4, 64))
    z[0] -= 200
    z[1] += 3e4
    z[2] -= 95
    check(qk, z, 4, "sigmoid")
    check(qk, z, 4, "softmax")


def test_nothing_to_route_by(qk):
    z = torch.randn(5, 64)
    z[1, 7], z[3, 0] = float("nan"), float("inf")
    ids, w = qk.moe_route(z.cuda(), 4)
    for t in (1, 3):
        assert ids[t].tolist() == [0, 1, 2, 3] and torch.isnan(w[t]).all()
    assert torch.isfinite(w[[0, 2, 4]]).all()
    ids, w = qk.moe_route(z.cuda(), 4, score="sigmoid")
    assert torch.isnan(w[1]).all() and ids[1].tolist() == [0, 1, 2, 3]
    assert ids[3, 0] == 0 and torch.isfinite(w[3]).all()
    bias = torch.zeros(64)
    bias[9] = float("nan")
    ids, w = qk.moe_route(z.cuda(), 4, score="sigmoid", bias=bias.cuda())
    assert torch.isnan(w).all() and ids.tolist() == [[0, 1, 2, 3]] * 5
    bias[9], z = -float("inf"), torch.zeros(5, 64)
    ids, w = qk.moe_route(z.cuda(), 10, score="sigmoid", bias=bias.cuda())
    assert 9 not in ids.tolist()[0]


def test_strides_streams_outputs_and_graphs(qk):
    rng = np.random.default_rng(9)
    z = torch.from_numpy(rng.standard_normal((20, 140)).astype(np.float32)).cuda()
    want = qk.moe_route(z[:, 5:133].contiguous(), 6)
    ids, w = torch.full((22, 6), -9, dtype=torch.int32, device="cuda"), torch.full((22, 6), -9.0, device="cuda")
    qk.moe_route(z[:, 5:133], 6, ids=ids[:20], weights=w[:20])
    assert torch.equal(ids[:20], want[0]) and torch.equal(w[:20], want[1]) and torch.all(ids[20:] == -9) and torch.all(w[20:] == -9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = qk.moe_route(z[:, 5:133], 6, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = qk.moe_route(z[:, 5:133], 6)
    z.copy_(z.flip(0))
    graph.replay()
    assert torch.equal(got[0], want[0].flip(0)) and torch.equal(got[1], want[1].flip(0))
    empty = qk.moe_route(z[:0], 6)
    assert empty[0].shape == (0, 6) and empty[1].shape == (0, 6)
