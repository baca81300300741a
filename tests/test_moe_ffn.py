"""The experts' feed-forward products against the formulas in 64 bits, with derived bounds (moe_oracle.ffn)."""
import numpy as np
import pytest
import torch

from tests import moe_oracle as mo

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.uint8)


class Case:
    """Weights, rows and routing of a call; `call` runs it, `check` holds its rows to the bound."""

    def __init__(self, qk, T, E, k, K, F, N, gate="q4_k", down="q4_k", x_type="f32", y_type=None, seed=0, ids=None, scale=1.0):
        self.qk, self.E, self.K, self.F, self.N = qk, E, K, F, N
        self.x_type, self.y_type = x_type, y_type or x_type
        rng = np.random.default_rng(seed)
        self.b, self.w = {}, {}
        for i, (name, fmt, rows, cols) in enumerate((("gate", gate, F, K), ("up", gate, F, K), ("down", down, N, F))):
            b, self.w[name] = mo.expert_weights(fmt, E, rows, cols, seed * 10 + i)
            self.b[name] = qk.ExpertWeights(fmt, torch.from_numpy(b).cuda())
        self.x, self.xv = mo.as_rows(scale * rng.standard_normal((T, K)), x_type)
        self.ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if ids is None else np.asarray(ids, np.int32)
        self.p = rng.random((T, k)).astype(np.float32) + 0.1

    def call(self, x=None, ids=None, **kw):
        x = self.x.cuda() if x is None else x
        ids = torch.from_numpy(self.ids if ids is None else np.asarray(ids, np.int32)).cuda()
        kw.setdefault("y", torch.empty(x.shape[0], self.N, dtype=mo.TORCH[self.y_type], device="cuda"))
        return self.qk.moe_ffn(x, ids, torch.from_numpy(self.p).cuda(), self.b["gate"], self.b["up"], self.b["down"], self.E, self.F,
                               self.N, **kw)

    def check(self, y, rows=None):
        rows = range(len(self.ids)) if rows is None else rows
        rows = list(rows)
        want, bound = mo.ffn(self.xv[rows], self.ids[rows], self.p[rows], self.w["gate"], self.w["up"], self.w["down"], self.x_type, self.y_type)
        err = np.abs(y[rows].double().cpu().numpy() - want)
        assert np.all(err <= bound), f"worst {np.nanmax(err / bound):.3g} of the bound, at {np.unravel_index(np.nanargmax(err / bound), err.shape)}"


CASES = [
    # T, E, k, K, F, N, gate, down, x type, y type
    (1, 8, 2, 256, 64, 256, "q4_k", "q4_k", "f32", "f32"),
    (1, 16, 8, 2048, 96, 512, "q4_k", "q6_k", "f32", "f32"),
    (2, 4, 3, 576, 288, 576, "q8_0", "q8_0", "f32", "f32"),
    (3, 4, 2, 300, 77, 45, "q4_k", "q8_0", "f32", "f32"),            # nothing a whole number of anything
    (5, 3, 1, 33, 7, 1, "q8_0", "q6_k", "f32", "f32"),
    (1, 1, 1, 1, 1, 1, "q8_0", "q4_k", "f32", "f32"),
    (20, 2, 1, 512, 256, 130, "q4_k", "q4_k", "f32", "f32"),         # two columns sets an expert
    (70, 2, 2, 256, 256, 256, "q6_k", "q4_k", "f32", "f32"),         # several sets an expert
    (64, 32, 4, 256, 256, 64, "q4_k", "q6_k", "bf16", "bf16"),
    (33, 8, 4, 896, 352, 96, "q8_0", "q4_k", "f16", "f16"),
    (40, 8, 8, 1024, 40, 200, "q4_k", "q8_0", "bf16", "bf16"),
    (9, 5, 2, 768, 512, 64, "q6_k", "q6_k", "bf16", "f32"),
    (9, 5, 2, 768, 512, 64, "q6_k", "q6_k", "f32", "f16"),
    (300, 4, 2, 256, 64, 64, "q4_k", "q4_k", "bf16", "bf16"),        # 150 tokens an expert
    (300, 4, 2, 320, 96, 160, "q8_0", "q6_k", "f32", "f32"),
    (260, 2, 1, 512, 128, 384, "q4_k", "q8_0", "f16", "f16"),
]


@pytest.mark.parametrize("T,E,k,K,F,N,gate,down,xt,yt", CASES)
def test_matches_the_formula(qk, T, E, k, K, F, N, gate, down, xt, yt):
    c = Case(qk, T, E, k, K, F, N, gate, down, xt, yt, seed=T + K + F)
    y = c.call()
    c.check(y)
    assert torch.equal(bits(y), bits(c.call())), "a call's bits repeat"
    assert qk.device_error() == 0


def test_uneven_experts(qk):
    """One expert has nearly all tokens, some have none, one token is sent to one expert twice."""
    T = 150
    ids = np.zeros((T, 2), np.int32)
    ids[:, 1] = 5
    ids[::40, 1], ids[3] = 2, (7, 7)
    for xt in ("f32", "bf16"):
        c = Case(qk, T, 9, 2, 512, 160, 192, "q4_k", "q6_k", xt, seed=3, ids=ids)
        c.check(c.call())


def test_skipped_and_bad_ids(qk):
    T = 12
    rng = np.random.default_rng(1)
    ids = rng.integers(0, 6, (T, 3)).astype(np.int32)
    ids[2], ids[5, 1], ids[7, 0] = -1, -7, -2 ** 31
    c = Case(qk, T, 6, 3, 512, 64, 100, "q4_k", "q8_0", "f32", seed=4, ids=ids)
    y = c.call()
    c.check(y)
    assert torch.all(y[2] == 0) and qk.device_error() == 0
    bad = ids.copy()
    bad[4, 2], bad[9, 0] = 6, 2 ** 31 - 1
    z = c.call(ids=bad)
    assert torch.isnan(z[4]).all() and torch.isnan(z[9]).all() and qk.device_error() == 9
    c.check(z, [t for t in range(T) if t not in (4, 9)])
    assert qk.device_error() == 0


def test_every_token_skipped(qk):
    c = Case(qk, 5, 4, 2, 256, 64, 64, ids=-np.ones((5, 2)))
    assert torch.all(c.call() == 0) and qk.device_error() == 0


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_a_bad_row_stays_alone(qk, value, xt):
    T, ids = 40, np.zeros((40, 1), np.int32)
    c = Case(qk, T, 2, 1, 512, 64, 96, "q4_k", "q4_k", xt, seed=5, ids=ids)
    x = c.x.clone()
    x[17, 100] = value
    y = c.call(x=x.cuda())
    assert not torch.isfinite(y[17]).any()
    c.check(y, [t for t in range(T) if t != 17])


@pytest.mark.parametrize("xt,scale", [("f32", 2.0 ** 60), ("f32", 2.0 ** -60), ("bf16", 2.0 ** 50), ("bf16", 2.0 ** -40), ("f16", 2.0 ** -12)])
def test_scale_of_a_row(qk, xt, scale):
    """Rows far from 1: |h| goes with the square where gate is large, so the tolerance is the bound's."""
    c = Case(qk, 6, 4, 2, 512, 64, 64, "q8_0", "q8_0", xt, "f32", seed=6, scale=scale)
    c.check(c.call())


def test_fused_gate_and_up(qk):
    """Gate and up as halves of one tensor [E][2F][K], and experts further into a tensor."""
    E, F, K, N = 4, 48, 512, 64
    c = Case(qk, 10, E, 2, K, F, N, "q4_k", "q6_k", "f32", seed=7)
    rb = c.b["gate"].w.numel() // (E * F)
    g, u = (c.b[n].w.reshape(E, F, rb) for n in ("gate", "up"))
    fused = torch.cat([torch.zeros(3, rb, dtype=torch.uint8, device="cuda"), torch.cat([g, u], 1).reshape(-1, rb)]).contiguous()
    want = c.call()
    c.b["gate"], c.b["up"] = qk.ExpertWeights("q4_k", fused, 3, 2 * F), qk.ExpertWeights("q4_k", fused, 3 + F, 2 * F)
    assert torch.equal(bits(c.call()), bits(want))


@pytest.mark.parametrize("fmt", ["q8_0", "q6_k"])
@pytest.mark.parametrize("off", [2, 6, 14])
def test_weights_off_16_bytes(qk, fmt, off):
    c = Case(qk, 40, 3, 2, 544, 64, 96, fmt, fmt, "f32", seed=8)
    want = c.call()
    for n in ("gate", "up", "down"):
        b = c.b[n].w.reshape(-1)
        t = torch.empty(b.numel() + off, dtype=torch.uint8, device="cuda")
        t[off:] = b
        c.b[n] = qk.ExpertWeights(fmt, t[off:])
    assert torch.equal(bits(c.call()), bits(want))


def test_columns_behind_the_last_have_no_effect(qk):
    """Bytes of a row's last block that stand for columns past K."""
    c = Case(qk, 7, 3, 2, 300, 40, 64, "q4_k", "q4_k", "f32", seed=9)
    want = c.call()
    b = c.b["gate"].w.reshape(-1, 2, 144).clone()
    b[:, 1, 16 + 32:] = 0xa5                    # nibbles of columns 320 and above
    c.b["gate"] = qk.ExpertWeights("q4_k", b)
    assert torch.equal(bits(c.call()), bits(want))


@pytest.mark.parametrize("xt", ["f32", "f16"])
def test_strides_and_rows_behind(qk, xt):
    c = Case(qk, 21, 4, 2, 320, 64, 72, "q8_0", "q4_k", xt, seed=10)
    want = c.call()
    for pad in (1, 3, 8):
        x = torch.zeros(21, 320 + pad, dtype=mo.TORCH[xt], device="cuda")
        x[:, pad:] = c.x.cuda()
        y = torch.full((24, 72 + pad), 7.0, dtype=mo.TORCH[xt], device="cuda")
        c.call(x=x[:, pad:], y=y[:, :72])
        assert torch.equal(bits(y[:21, :72]), bits(want))
        assert torch.all(y[21:] == 7) and torch.all(y[:, 72:] == 7)


def test_no_tokens(qk):
    c = Case(qk, 3, 4, 2, 256, 64, 64)
    y = torch.full((2, 64), 3.0, device="cuda")
    c.p = c.p[:0]
    c.call(x=torch.empty(0, 256, device="cuda"), ids=np.zeros((0, 2)), y=y)
    assert torch.all(y == 3)


def test_streams_and_graphs(qk):
    """On another stream, and captured and replayed with new rows and ids; a dirty workspace has no effect."""
    c = Case(qk, 48, 8, 2, 512, 96, 64, "q4_k", "q8_0", "bf16", seed=11)
    want = c.call()
    ws = qk.moe_ffn_workspace(48, 2, 8, 512, 96, 64)
    ws.fill_(0xff)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = c.call(workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(bits(y), bits(want))
    x, ids, p = c.x.cuda(), torch.from_numpy(c.ids).cuda(), torch.from_numpy(c.p).cuda()
    y = torch.zeros_like(want)
    args = (c.b["gate"], c.b["up"], c.b["down"], c.E, c.F, c.N)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qk.moe_ffn(x, ids, p, *args, y=y, workspace=ws)
    graph.replay()
    assert torch.equal(bits(y), bits(want))
    x.copy_(x.flip(0)), ids.copy_(ids.flip(0)), p.copy_(p.flip(0))
    graph.replay()
    assert torch.equal(bits(y), bits(qk.moe_ffn(x, ids, p, *args)))


def test_programmatic_launch(qk):
    c = Case(qk, 30, 8, 2, 512, 96, 64, seed=12)
    want = c.call()
    was = qk.set_programmatic_launch(True)
    try:
        ys = [c.call() for _ in range(6)]
    finally:
        qk.set_programmatic_launch(was)
    assert all(torch.equal(bits(y), bits(want)) for y in ys)
