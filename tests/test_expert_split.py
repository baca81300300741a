"""Calls whose experts go by the few-token form, by the many-token form, or by both: each side of the rule that splits them."""
import numpy as np
import pytest
import torch

from tests import moe_oracle as mo
from tests.test_moe_ffn import Case, bits

pytestmark = pytest.mark.gpu


def split(counts):
    """The rule, restated: the number of sets of each form, and which experts the many-token form takes."""
    counts = np.asarray(counts)
    rows = -(-counts // 16)
    parts = -(-counts // 128)
    per = np.where(counts > 0, (-(-counts // np.maximum(parts, 1)) + 31) // 32 * 32, 1)
    tiles = -(-counts // per)
    many = counts >= 16
    few_sets, many_sets = rows[~many].sum(), rows[many].sum()
    if many_sets <= few_sets // 4:
        tiled = np.zeros_like(many)
    elif 2 * few_sets <= tiles[many].sum():
        tiled = counts > 0
    else:
        tiled = many
    return rows[~tiled].sum(), tiles[tiled].sum(), tiled


COUNTS = {
    "both": [1, 130, 15, 8, 300, 7, 2, 9, 11, 0, 16, 3],
    "both, many small ones": [1 + i % 15 for i in range(40)] + [200, 17],
    "just not all by few tokens": [5] * 8 + [33],
    "all by few tokens": [5] * 8 + [32],
    "all by few tokens, none of 16": [15] * 9 + [1],
    "just not all by many": [3] * 3 + [128] * 4 + [32],
    "all by many": [3] * 3 + [128] * 5 + [32],
    "all by many, one left": [1, 200, 0, 16],
}
FORMS = {"both": (True, True), "all by few": (True, False), "all by many": (False, True), "just not": (True, True)}


def case(qk, counts, k, gate, down, xt, yt, seed):
    """Assignments in random order, k a token: an expert's tokens have places of other experts beside them."""
    ids = np.repeat(np.arange(len(counts)), counts).astype(np.int32)
    np.random.default_rng(seed).shuffle(ids)
    ids = np.concatenate([ids, -np.ones(-len(ids) % k, np.int32)]).reshape(-1, k)
    return Case(qk, len(ids), len(counts), k, 288, 80, 136, gate, down, xt, yt, seed=seed, ids=ids)


@pytest.mark.parametrize("name", COUNTS)
@pytest.mark.parametrize("gate,down,xt,yt", [("q4_k", "q6_k", "f32", "f32"), ("q8_0", "q4_k", "bf16", "bf16"), ("q6_k", "q8_0", "f16", "f32"),
                                             ("q4_k", "q4_k", "bf16", "bf16"), ("q4_k", "q8_0", "f16", "bf16")])
@pytest.mark.parametrize("k", [1, 3])
def test_each_side_of_the_rule(qk, name, gate, down, xt, yt, k):
    counts = COUNTS[name]
    few, many, tiled = split(counts)
    assert (few > 0, many > 0) == next(v for n, v in FORMS.items() if name.startswith(n))
    c = case(qk, counts, k, gate, down, xt, yt, len(name))
    ws = qk.moe_ffn_workspace(len(c.ids), k, c.E, c.K, c.F, c.N)
    ws.fill_(0xff)                                  # NaN wherever nothing was written
    y = c.call(workspace=ws)
    assert ws[:12].cpu().view(torch.int32).tolist() == [few, many, sum(counts)]
    # what is rounded with bf16 rows and outputs is the many-token form's weights, no other
    dw = None
    if xt == yt == "bf16":
        dw = [mo.rounded_weights(c.b[n].fmt, c.b[n].w.cpu().numpy(), c.w[n]) * tiled[:, None, None] for n in ("gate", "up", "down")]
    rows = sorted({int(np.argwhere(c.ids == e)[i][0]) for e in range(c.E) for i in (0, -1) if counts[e]} | set(range(0, len(c.ids), 9)))
    want, bound = mo.ffn(c.xv[rows], c.ids[rows], c.p[rows], c.w["gate"], c.w["up"], c.w["down"], xt, yt, dw)
    assert np.all(np.abs(y[rows].double().cpu().numpy() - want) <= bound)
    assert torch.equal(bits(y), bits(c.call())) and qk.device_error() == 0


def test_both_forms_in_a_graph(qk):
    """One graph, replayed with ids that go by either form, by both, by none and past the last."""
    counts = COUNTS["both"]
    c = case(qk, counts, 2, "q4_k", "q6_k", "f32", "f32", 1)
    T, E = len(c.ids), c.E
    x, ids, p = c.x.cuda(), torch.from_numpy(c.ids).cuda(), torch.from_numpy(c.p).cuda()
    args = (c.b["gate"], c.b["up"], c.b["down"], E, c.F, c.N)
    ws = qk.moe_ffn_workspace(T, 2, E, c.K, c.F, c.N)
    y = torch.empty(T, c.N, device="cuda")
    qk.moe_ffn(x, ids, p, *args, y=y, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qk.moe_ffn(x, ids, p, *args, y=y, workspace=ws)
    g = torch.Generator().manual_seed(1)
    live = torch.randint(0, E, (T, 2), generator=g).int()
    one = torch.full((T, 2), -1, dtype=torch.int32)
    one[::40] = 3
    past = live.clone()
    past[::7, 1] = E
    for new in (torch.from_numpy(c.ids), live, torch.zeros(T, 2).int(), torch.full((T, 2), -1).int(), one, past, torch.from_numpy(c.ids)):
        ids.copy_(new)
        ws.fill_(0xff)
        graph.replay()
        assert qk.device_error() == (9 if (new == E).any() else 0)
        assert torch.equal(bits(y), bits(qk.moe_ffn(x, ids, p, *args)))
        qk.device_error()
        assert torch.equal(torch.isnan(y).any(1).cpu(), (new == E).any(1))
