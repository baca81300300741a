"""Low-rank adapters against the formula in 64 bits, with derived bounds (moe_oracle.lora)."""
import numpy as np
import pytest
import torch

from tests import moe_oracle as mo

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.uint8)


class Case:
    def __init__(self, qk, T, n, rank, K, N, x_type="f32", w_type="f16", y_type=None, ids=None, seed=0, scaled=True):
        rng = np.random.default_rng(seed)
        self.qk, self.y_type = qk, y_type or x_type
        self.x, self.xv = mo.as_rows(rng.standard_normal((T, K)), x_type)
        self.y, self.yv = mo.as_rows(rng.standard_normal((T, N)), self.y_type)
        self.A, self.Av = mo.as_rows(rng.standard_normal((n, rank, K)) * K ** -0.5, w_type)
        self.B, self.Bv = mo.as_rows(rng.standard_normal((n, N, rank)), w_type)
        self.ids = rng.integers(-1, n, T).astype(np.int32) if ids is None else np.asarray(ids, np.int32)
        self.s = (0.5 + rng.random(n)).astype(np.float32) if scaled else None

    def call(self, x=None, y=None, ids=None, **kw):
        return self.qk.lora(self.x.cuda() if x is None else x, self.y.cuda() if y is None else y, self.A.cuda(), self.B.cuda(),
                            torch.from_numpy(self.ids if ids is None else np.asarray(ids, np.int32)).cuda(),
                            scales=None if self.s is None else torch.from_numpy(self.s).cuda(), **kw)

    def check(self, out, rows=None):
        rows = list(range(len(self.ids)) if rows is None else rows)
        want, bound = mo.lora(self.xv[rows], self.yv[rows], self.Av, self.Bv, self.ids[rows], self.s, self.y_type)
        err = np.abs(out[rows].double().cpu().numpy() - want)
        assert np.all(err <= bound), f"worst excess {np.nanmax(err - bound):.3g} at {np.unravel_index(np.nanargmax(err - bound), err.shape)}"


CASES = [
    # T, adapters, rank, K, N, x, adapters, y
    (1, 1, 16, 4096, 512, "f32", "f16", "f32"), (1, 3, 8, 896, 640, "f32", "bf16", "f32"), (7, 4, 16, 576, 576, "bf16", "bf16", "bf16"),
    (64, 48, 16, 512, 256, "f32", "bf16", "f32"), (33, 5, 4, 300, 77, "f32", "f16", "f32"), (17, 2, 1, 33, 1, "f32", "f32", "f32"),
    (1, 1, 1, 1, 1, "f16", "f16", "f16"), (20, 3, 64, 256, 130, "f16", "f16", "f16"), (20, 3, 100, 256, 64, "bf16", "bf16", "f32"),
    (12, 2, 256, 512, 100, "f32", "f32", "f32"), (19, 2, 24, 1000, 200, "f16", "f32", "f16"), (15, 2, 33, 64, 40, "f32", "bf16", "bf16"),
    (700, 3, 16, 256, 144, "bf16", "bf16", "bf16"), (650, 3, 64, 128, 96, "f32", "f16", "f32"), (350, 40, 32, 96, 96, "f16", "f16", "f16"),
    (500, 2, 130, 72, 50, "f32", "f32", "f32"), (400, 7, 8, 520, 264, "f32", "f16", "f32"), (330, 2, 12, 200, 100, "bf16", "f32", "bf16"),
]


@pytest.mark.parametrize("T,n,rank,K,N,xt,wt,yt", CASES)
def test_matches_the_formula(qk, T, n, rank, K, N, xt, wt, yt):
    c = Case(qk, T, n, rank, K, N, xt, wt, yt, seed=T + rank, scaled=T % 2 == 1)
    out = c.call()
    c.check(out)
    assert torch.equal(bits(out), bits(c.call())), "a call's bits repeat"
    assert qk.device_error() == 0


@pytest.mark.parametrize("T", [1, 40, 700])
def test_no_adapter_and_bad_ids(qk, T):
    c = Case(qk, T, 3, 16, 256, 200, "f32", "bf16", seed=2, ids=-np.ones(T))
    assert torch.equal(bits(c.call()), bits(c.y.cuda()))
    ids = np.arange(T) % 4 - 1
    bad = ids.copy()
    bad[0], bad[T - 1] = 3, 2 ** 31 - 1
    c.ids = ids.astype(np.int32)
    out = c.call(ids=bad)
    assert torch.isnan(out[[0, T - 1]]).all() and qk.device_error() == 9
    c.check(out, range(1, T - 1))
    y = c.y.cuda()
    c.call(y=y, ids=bad, out=y)
    assert torch.isnan(y[[0, T - 1]]).all() and torch.equal(bits(y[1:T - 1]), bits(out[1:T - 1])) and qk.device_error() == 9


@pytest.mark.parametrize("yt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [5, 700])
def test_in_place_strides_and_rows_behind(qk, T, yt):
    c = Case(qk, T, 4, 16, 160, 72, yt, "f16", seed=3)
    want = c.call()
    for pad in (1, 4, 8):
        x = torch.zeros(T, 160 + pad, dtype=c.x.dtype, device="cuda")
        x[:, pad:] = c.x.cuda()
        y = torch.full((T + 2, 72 + pad), 7.0, dtype=c.y.dtype, device="cuda")
        y[:T, :72] = c.y.cuda()
        got = c.call(x=x[:, pad:], y=y[:T, :72], out=y[:T, :72])
        assert got.data_ptr() == y.data_ptr()
        assert torch.equal(bits(y[:T, :72]), bits(want)) and torch.all(y[T:] == 7) and torch.all(y[:, 72:] == 7)


@pytest.mark.parametrize("T", [48, 640])
def test_a_bad_row_stays_alone(qk, T):
    """A NaN or an infinity in one token's x, or in an adapter, reaches no other row."""
    c = Case(qk, T, 3, 16, 256, 96, "bf16", "bf16", seed=4, ids=np.arange(T) % 3)
    x = c.x.clone()
    x[7, 3], x[20, 200] = float("nan"), float("inf")
    out = c.call(x=x.cuda())
    assert not torch.isfinite(out[[7, 20]].float()).any()
    c.check(out, [t for t in range(T) if t not in (7, 20)])
    c.A[1] = float("nan")
    out = c.call()
    assert torch.isnan(out[1::3].float()).all()
    c.check(out, [t for t in range(T) if t % 3 != 1])


def test_one_token_at_a_time_gives_the_batch(qk):
    """Rows do not depend on their neighbours."""
    c = Case(qk, 40, 5, 16, 512, 96, "f32", "f16", seed=5)
    out = c.call()
    for t in range(0, 40, 7):
        one = c.call(x=c.x[t:t + 1].cuda(), y=c.y[t:t + 1].cuda(), ids=c.ids[t:t + 1])
        assert torch.equal(bits(one), bits(out[t:t + 1]))


def test_streams_graphs_and_programmatic_launch(qk):
    c = Case(qk, 50, 4, 16, 256, 128, "bf16", "bf16", seed=6)
    want = c.call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.call(stream=side)
    side.synchronize()
    assert torch.equal(bits(got), bits(want))
    x, y, A, B, ids, s = c.x.cuda(), c.y.cuda(), c.A.cuda(), c.B.cuda(), torch.from_numpy(c.ids).cuda(), torch.from_numpy(c.s).cuda()
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qk.lora(x, y, A, B, ids, scales=s, out=out)
    x.copy_(x.flip(0)), y.copy_(y.flip(0)), ids.copy_(ids.flip(0))
    graph.replay()
    assert torch.equal(bits(out), bits(want.flip(0)))
    was = qk.set_programmatic_launch(True)
    try:
        z = c.y.cuda()
        for _ in range(4):
            z = qk.lora(c.x.cuda(), z, A, B, torch.from_numpy(c.ids).cuda(), scales=s, out=z)
    finally:
        qk.set_programmatic_launch(was)
    w = c.y.cuda()
    for _ in range(4):
        w = c.call(y=w)
    assert torch.equal(bits(z), bits(w))
    assert qk.lora(x[:0], y[:0], A, B, ids[:0]).shape == (0, 128)
