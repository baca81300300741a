"""The forms that the experts' products and the adapters' take at different sizes, and their edges."""
import numpy as np
import pytest
import torch

from tests import moe_oracle as mo
from tests.test_lora import Case as LoraCase
from tests.test_moe_ffn import Case, bits

pytestmark = pytest.mark.gpu


# up to 24 assignments: no plan
@pytest.mark.parametrize("gate", ["q4_k", "q8_0", "q6_k"])
@pytest.mark.parametrize("down", ["q4_k", "q8_0", "q6_k"])
@pytest.mark.parametrize("T,k,K,F,N", [(1, 8, 512, 160, 96), (3, 2, 290, 49, 33), (1, 24, 64, 16, 8), (2, 1, 2400, 300, 1)])
def test_few_assignments(qk, gate, down, T, k, K, F, N):
    for xt, yt in (("f32", "f32"), ("f16", "bf16")):           # (outputs reach 1.2e6, past fp16's range)
        c = Case(qk, T, 24, k, K, F, N, gate, down, xt, yt, seed=T + K)
        y = c.call()
        c.check(y)
        assert torch.equal(bits(y), bits(c.call())) and qk.device_error() == 0


def test_few_assignments_of_one_expert(qk):
    """An id that repeats in a token, and ids that are skipped or bad next to it."""
    ids = np.array([[2, 2, 2, -1], [-1, -1, -1, -1], [0, 2, -5, 2], [1, 0, 1, 0]], np.int32)
    c = Case(qk, 4, 3, 4, 512, 64, 70, "q4_k", "q6_k", "f32", seed=3, ids=ids)
    y = c.call()
    c.check(y)
    assert torch.all(y[1] == 0) and qk.device_error() == 0
    bad = ids.copy()
    bad[2, 2] = 3
    z = c.call(ids=bad)
    assert torch.isnan(z[2]).all() and qk.device_error() == 9 and torch.equal(bits(z[[0, 1, 3]]), bits(y[[0, 1, 3]]))


@pytest.mark.parametrize("K,F", [(8448, 32), (32, 8448), (8192, 32), (32, 8192)])
def test_long_rows_of_few_assignments(qk, K, F):
    """Rows that shared memory has no room for go by the plan; its edge does not."""
    c = Case(qk, 2, 2, 2, K, F, 40, "q4_k", "q8_0", "f32", seed=5)
    c.check(c.call())


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_row_among_few(qk, value):
    c = Case(qk, 3, 4, 2, 512, 64, 96, "q4_k", "q4_k", "f32", seed=5)
    want = c.call()
    x = c.x.clone()
    x[1, 100] = value
    y = c.call(x=x.cuda())
    assert not torch.isfinite(y[1]).any() and torch.equal(bits(y[[0, 2]]), bits(want[[0, 2]]))


@pytest.mark.parametrize("T", [1, 3])
def test_few_assignments_strides_streams_and_graphs(qk, T):
    c = Case(qk, T, 6, 3, 300, 40, 72, "q8_0", "q4_k", "f16", seed=10)
    want = c.call()
    for pad in (1, 3, 8):
        x = torch.zeros(T, 300 + pad, dtype=torch.float16, device="cuda")
        x[:, pad:] = c.x.cuda()
        y = torch.full((T + 2, 72 + pad), 7.0, dtype=torch.float16, device="cuda")
        c.call(x=x[:, pad:], y=y[:, :72])
        assert torch.equal(bits(y[:T, :72]), bits(want)) and torch.all(y[T:] == 7) and torch.all(y[:, 72:] == 7)
    ws = qk.moe_ffn_workspace(T, 3, 6, 300, 40, 72)
    ws.fill_(0xff)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = c.call(workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(bits(y), bits(want))
    x, ids, p = c.x.cuda(), torch.from_numpy(c.ids).cuda(), torch.from_numpy(c.p).cuda()
    args = (c.b["gate"], c.b["up"], c.b["down"], c.E, c.F, c.N)
    graph = torch.cuda.CUDAGraph()
    was = qk.set_programmatic_launch(True)
    try:
        with torch.cuda.graph(graph):
            # two calls that share their workspace, one after the other
            y = qk.moe_ffn(x, ids, p, *args, workspace=ws, y=torch.zeros_like(want))
            z = qk.moe_ffn(x, ids, p, *args, workspace=ws, y=torch.zeros_like(want))
        for shift in (0, 1, 2):
            x.copy_(x.roll(shift, 1)), ids.copy_((ids + shift) % 6)
            graph.replay()
            w = qk.moe_ffn(x, ids, p, *args)
            assert torch.equal(bits(y), bits(w)) and torch.equal(bits(z), bits(w))
    finally:
        qk.set_programmatic_launch(was)


# more assignments, few tokens an expert: every format and both numbers of pieces
@pytest.mark.parametrize("gate,down", [("q4_k", "q6_k"), ("q8_0", "q4_k"), ("q6_k", "q8_0")])
@pytest.mark.parametrize("T,k,xt,yt", [(13, 2, "f32", "f32"), (15, 4, "bf16", "bf16"), (9, 3, "f16", "f32"), (25, 1, "f32", "bf16")])
def test_few_tokens_an_expert(qk, gate, down, T, k, xt, yt):
    c = Case(qk, T, 9, k, 800, 136, 88, gate, down, xt, yt, seed=T)
    y = c.call()
    c.check(y)
    assert torch.equal(bits(y), bits(c.call())) and qk.device_error() == 0


@pytest.mark.parametrize("gate,down", [("q4_k", "q6_k"), ("q8_0", "q4_k"), ("q6_k", "q8_0")])
@pytest.mark.parametrize("xt,yt", [("f32", "f32"), ("bf16", "bf16"), ("f16", "bf16"), ("bf16", "f32")])
def test_both_forms_in_a_call(qk, gate, down, xt, yt):
    """Experts of 1, 15, 16, 17, 128, 129 and 300 tokens next to one another."""
    counts = [1, 15, 16, 17, 128, 129, 300, 0, 3]
    ids = np.repeat(np.arange(len(counts)), counts).astype(np.int32)
    np.random.default_rng(0).shuffle(ids)
    c = Case(qk, len(ids), len(counts), 1, 288, 80, 136, gate, down, xt, yt, seed=2, ids=ids[:, None])
    y = c.call()
    rows = list(range(0, len(ids), 5)) + [int(np.flatnonzero(ids == e)[0]) for e in range(9) if counts[e]]
    dw = None
    if xt == yt == "bf16":
        dw = [mo.rounded_weights(c.b[n].fmt, c.b[n].w.cpu().numpy(), c.w[n]) for n in ("gate", "up", "down")]
    want, bound = mo.ffn(c.xv[rows], c.ids[rows], c.p[rows], c.w["gate"], c.w["up"], c.w["down"], xt, yt, dw)
    assert np.all(np.abs(y[rows].double().cpu().numpy() - want) <= bound)
    assert torch.equal(bits(y), bits(c.call())) and qk.device_error() == 0


def test_more_places_than_a_warp_has_lanes(qk):
    """40 experts a token: a row's places are looked up 32 at a time, parts summed eight at a time."""
    for T in (2, 40):
        c = Case(qk, T, 45, 40, 256, 32, 48, "q8_0", "q8_0", "f32", seed=T)
        c.check(c.call())


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("chunk", [0, 2])
def test_a_chunk_that_never_comes(qk, xt, chunk):
    """The wait for it runs out, the call ends and says so, and the next one is as ever."""
    c = Case(qk, 300, 4, 2, 512, 256, 256, "q4_k", "q4_k", xt, seed=9)
    want = c.call()
    limit = qk.set_wait_limit_ns(20_000_000)
    qk.debug_moe_skip_chunk(chunk)
    try:
        c.call()
        assert qk.device_error() == 6
    finally:
        qk.debug_moe_skip_chunk(-1)
        qk.set_wait_limit_ns(limit)
    assert torch.equal(bits(c.call()), bits(want)) and qk.device_error() == 0


TYPES = ["f32", "f16", "bf16"]


@pytest.mark.parametrize("xt", TYPES)
@pytest.mark.parametrize("wt", TYPES)
@pytest.mark.parametrize("T,n,rank,K,N", [(1, 3, 8, 104, 40), (2, 5, 64, 296, 72), (31, 40, 16, 32, 8), (65, 9, 24, 520, 264), (270, 64, 40, 136, 104)])
def test_adapters_of_every_type(qk, xt, wt, T, n, rank, K, N):
    """Whole vectors (K, N and ranks of 8) with tails of every other length, outputs of both widths."""
    for yt in ("f32", "bf16" if xt == "bf16" else "f16"):
        c = LoraCase(qk, T, n, rank, K, N, xt, wt, yt, seed=T)
        out = c.call()
        c.check(out)
        assert torch.equal(bits(out), bits(c.call())) and qk.device_error() == 0


@pytest.mark.parametrize("xt,wt", [("f32", "bf16"), ("bf16", "f16"), ("f16", "f16")])
@pytest.mark.parametrize("T", [40, 300])
def test_adapters_off_their_vectors(qk, xt, wt, T):
    """Bits do not depend on alignment or strides, and with adapters off 16 bytes the bound holds."""
    c = LoraCase(qk, T, 5, 40, 136, 72, xt, wt, seed=7)
    want = c.call()
    for pad in (1, 4):
        x = torch.zeros(T, 136 + pad, dtype=c.x.dtype, device="cuda")
        x[:, pad:] = c.x.cuda()
        out = torch.full((T + 1, 72 + pad), 5.0, dtype=c.y.dtype, device="cuda")
        c.call(x=x[:, pad:], out=out[:T, :72])
        assert torch.equal(bits(out[:T, :72]), bits(want)) and torch.all(out[T:] == 5) and torch.all(out[:, 72:] == 5)


@pytest.mark.parametrize("T", [3, 33, 300])
def test_adapters_without_a_workspace(qk, T):
    """One launch; too small a workspace is none, and one off its alignment is refused."""
    c = LoraCase(qk, T, 5, 16, 200, 72, "bf16", "bf16", seed=8)
    empty = torch.empty(256, dtype=torch.uint8, device="cuda")[:1]
    out = c.call(workspace=empty)
    c.check(out)
    big = torch.empty(T * 64 * 4 + 512, dtype=torch.uint8, device="cuda")
    with pytest.raises((ValueError, RuntimeError)):
        c.call(workspace=big[1:])


def test_adapters_streams_and_graphs(qk):
    for T, xt in ((7, "bf16"), (90, "f16"), (300, "f32")):
        c = LoraCase(qk, T, 6, 16, 256, 96, xt, "bf16" if xt != "f16" else "f16", seed=T)
        want = c.call()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y = c.call(stream=side)
        side.synchronize()
        assert torch.equal(bits(y), bits(want))
        x, y0, A, B, s = c.x.cuda(), c.y.cuda(), c.A.cuda(), c.B.cuda(), torch.from_numpy(c.s).cuda()
        ids = torch.from_numpy(c.ids).cuda()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = qk.lora(x, y0, A, B, ids, scales=s)
        for _ in range(3):
            x.copy_(x.flip(0)), ids.copy_((ids + 2) % 7 - 1)
            graph.replay()
            assert torch.equal(bits(out), bits(qk.lora(x, y0, A, B, ids, scales=s)))


def test_two_streams_at_once(qk):
    """Calls that run beside one another, each with its workspace."""
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for T in (2, 40, 200):
        cs = [Case(qk, T, 8, 2, 512, 96, 64, "q4_k", "q8_0", xt, seed=i) for i, xt in enumerate(("f32", "bf16"))]
        ls = [LoraCase(qk, T, 5, 16, 512, 96, xt, "bf16", seed=i) for i, xt in enumerate(("f32", "bf16"))]
        want = [[bits(c.call()) for c in cs], [bits(c.call()) for c in ls]]
        ws = [qk.moe_ffn_workspace(T, 2, 8, 512, 96, 64) for _ in sides]
        torch.cuda.synchronize()
        got = [([], []), ([], [])]
        for _ in range(8):
            for i, side in enumerate(sides):
                got[0][i].append(cs[i].call(workspace=ws[i], stream=side)), got[1][i].append(ls[i].call(stream=side))
        torch.cuda.synchronize()
        for o in range(2):
            for i in range(2):
                assert all(torch.equal(bits(y), want[o][i]) for y in got[o][i])
    assert qk.device_error() == 0


def test_rows_far_apart(qk):
    """Rows of x whose offsets pass 32 bits."""
    T, ld = 20, (1 << 27) + 8
    big = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    for k in (1, 2):                                            # 20 assignments, and 40
        c = Case(qk, T, 4, k, 256, 64, 48, "q4_k", "q8_0", "bf16", seed=k)
        x = big.as_strided((T, 256), (ld, 1))
        x.copy_(c.x)
        assert torch.equal(bits(c.call(x=x)), bits(c.call()))
        l = LoraCase(qk, T, 4, 8 * k * k, 256, 48, "bf16", "bf16", seed=k)
        x.copy_(l.x)
        assert torch.equal(bits(l.call(x=x)), bits(l.call()))
        x = big.as_strided((T, 64), (ld, 1))
        z = torch.randn(T, 64).bfloat16().cuda()
        x.copy_(z)
        assert all(torch.equal(a, b) for a, b in zip(qk.moe_route(x, 4), qk.moe_route(z, 4)))
    assert qk.device_error() == 0


def test_experts_behind_32_bits(qk):
    """The last experts of a tensor of 4.6 GB, in each form."""
    E, F, K, N, last = 1024, 2048, 2048, 32, 8
    c = Case(qk, 30, last, 1, K, F, N, "q8_0", "q8_0", "f32", seed=1)
    need = F * (K // 32 * 34)
    w = torch.zeros(E * need, dtype=torch.uint8, device="cuda")
    d = torch.zeros(E * N * (F // 32 * 34), dtype=torch.uint8, device="cuda")
    w[-last * need:], d[-c.b["down"].w.numel():] = c.b["gate"].w.reshape(-1), c.b["down"].w.reshape(-1)
    c.b["up"] = c.b["gate"]
    far = [qk.ExpertWeights("q8_0", t) for t in (w, w, d)]
    for ids in ([7], [6] * 30, [i % 8 for i in range(30)]):      # one assignment, 30 tokens an expert, four
        x, ids = c.x[:len(ids)].cuda(), torch.tensor(ids, dtype=torch.int32).cuda()[:, None]
        p = torch.from_numpy(c.p[:len(ids)]).cuda()
        near = qk.moe_ffn(x, ids, p, c.b["gate"], c.b["up"], c.b["down"], last, F, N)
        assert torch.equal(bits(qk.moe_ffn(x, ids + E - last, p, *far, E, F, N)), bits(near))
    assert qk.device_error() == 0
