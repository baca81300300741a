"""Norm + rotation, the append to the 4-bit cache and attention over it,
against the 64-bit oracle (tests/kv4_oracle.py).

Tolerances (u = 2^-24, the fp32 rounding; o(t) the output type's rounding:
2^-24, 2^-11, 2^-8 relative for fp32, fp16, bf16, with fp16's subnormal step
2^-24 as an absolute term):

* norm + rotation: a sum of up to 512 squares in a tree of depth <= 16 + 5,
  halved by the square root, then two products, a rotation product and a sum:
  below 2^-19 of the magnitudes a result is made of, plus o(t).
* attention, fp32 queries: a score is a sum of up to 256 products with 22-bit
  pieces, accumulated in at most 32 + 8 steps: e = 2^-18 * A, A the largest sum
  of magnitudes of a row's scores; a probability is off by 2e + 2^-20, and up
  to 64 accumulation steps a warp and the joins add 2^-17:
  |o - ref| <= (2^-17 A + 2^-16) S, S = sum p |v|.
* attention, 16-bit queries: keys, values and probabilities rounded once to
  fp16 (2^-11 each at most): |o - ref| <= (2^-10 A + 2^-9) S + o(t) |ref|, and
  over a whole output, where such roundings are independent, a 2-norm within
  1.5e-3 (fp16) or 5e-3 (bf16) of the reference's.
"""
import numpy as np
import pytest
import torch

from tests import kv4_oracle as ko

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
OUT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def f64(t):
    return t.detach().double().cpu().numpy()


def rand(seed, *shape, scale=1.0, dtype="f32"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(DT[dtype]).cuda()


def table(n_pos, rot):
    inv = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(n_pos)[:, None] * inv
    return torch.from_numpy(np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)).cuda()


def close(got, ref, bound, what):
    got = f64(got)
    assert got.shape == ref.shape
    worst = (np.abs(got - ref) - bound).max()
    assert np.all(np.abs(got - ref) <= bound), f"{what}: worst excess {worst:.3e}"


# ---------------------------------------------------------------- norm + rotation

@pytest.mark.parametrize("T,nq,nk,D,rot,interleaved,norm,dtype,out", [
    (1, 32, 8, 128, 128, False, True, "f32", "f32"),
    (37, 9, 3, 64, 64, True, False, "f32", "f32"),
    (5, 14, 2, 64, 32, False, True, "f16", "f16"),
    (129, 4, 4, 96, 72, False, True, "bf16", "bf16"),
    (3, 8, 1, 256, 256, False, True, "f32", "bf16"),
    (7, 3, 1, 80, 80, False, True, "f32", "f16"),
    (6, 2, 0, 512, 250, True, True, "bf16", "f32"),
    (4, 1, 2, 30, 10, False, True, "f32", "f32"),
    (2, 1, 1, 2, 2, True, False, "f16", "f16"),
    (3, 5, 1, 128, 0, False, True, "f32", "f32"),
])
def test_norm_rope(qk, T, nq, nk, D, rot, interleaved, norm, dtype, out):
    x = rand(T + D, T, (nq + nk) * D, dtype=dtype)
    tab = table(300, rot) if rot else None
    pos = torch.randint(0, 300, (T,), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda()
    wq = 1 + rand(2, D, scale=0.3) if norm else None
    wk = 1 + rand(3, D, scale=0.3) if norm else None
    y = torch.empty(T, (nq + nk) * D, dtype=DT[out], device="cuda")
    qk.norm_rope(x, nq, nk, D, pos, tab, wq, wk, eps=1e-5, interleaved=interleaved, y=y)
    h = f64(x).reshape(T, nq + nk, D)
    args = (1e-5, None if tab is None else f64(tab), pos.cpu().numpy(), rot, interleaved)
    rq, mq = ko.norm_rope(h[:, :nq], f64(wq) if norm else None, *args)
    rk, mk = ko.norm_rope(h[:, nq:], f64(wk) if norm else None, *args)
    ref = np.concatenate([rq, rk], 1).reshape(T, -1)
    mag = np.concatenate([mq, mk], 1).reshape(T, -1)
    close(y, ref, 2.0 ** -19 * mag + OUT[out] * np.abs(ref) + 2.0 ** -24, "norm_rope")
    assert qk.device_error() == 0


def test_norm_rope_strided_rows_and_in_place(qk):
    """Rows inside a wider buffer, at an offset that rules out wide loads, and in place; the rest is untouched."""
    T, nq, nk, D = 11, 3, 2, 64
    w = (nq + nk) * D
    for off in (0, 1, 4):
        for dtype in ("f32", "bf16"):
            buf = rand(off, T, w + 37, dtype=dtype)
            keep = buf.clone()
            tab, pos = table(50, D), torch.arange(T, dtype=torch.int32).cuda()
            x = buf[:, off:off + w]
            ref = qk.norm_rope(x.contiguous(), nq, nk, D, pos, tab)
            got = qk.norm_rope(x, nq, nk, D, pos, tab, y=x)
            assert torch.equal(got, ref)
            assert torch.equal(buf[:, :off], keep[:, :off]) and torch.equal(buf[:, off + w:], keep[:, off + w:])


def test_norm_rope_bad_position_and_non_finite(qk):
    x = rand(0, 4, 2 * 64)
    x[2, 5] = float("nan")
    pos = torch.tensor([0, 50, 3, -1], dtype=torch.int32).cuda()
    y = qk.norm_rope(x, 1, 1, 64, pos, table(50, 64), q_weight=torch.ones(64).cuda())
    assert qk.device_error() == 9 and qk.device_error() == 0
    bad = torch.isnan(y)
    assert bad[1].all() and bad[3].all() and not bad[0].any()
    assert bad[2, :64].all() and not bad[2, 64:].any()


def test_empty_calls(qk):
    e = torch.empty(0, 128, device="cuda")
    i32, i64 = torch.empty(0, dtype=torch.int32).cuda(), torch.empty(0, dtype=torch.int64).cuda()
    tab = table(4, 64)
    assert qk.norm_rope(e, 1, 1, 64, i32, tab).shape == (0, 128)
    cache = qk.kv_cache_q4(1, 2, 16, 64)
    assert qk.kv_append_q4(cache, e, e, e, i32, i64, tab).shape == (0, 128)
    assert qk.kv_read_q4(cache, i64)[0].shape == (0, 128)
    assert qk.attn_q4(cache, e, torch.empty(0, 1, dtype=torch.int32).cuda(), i32).shape == (0, 128)


# ---------------------------------------------------------------- rotation tables

@pytest.mark.parametrize("kw", [
    dict(), dict(freq_scale=0.125, base=500000.0), dict(amplitude=1.25, freq_scale=0.25, orig_ctx=4096),
    dict(orig_ctx=8192, freq_scale=1 / 16, beta_fast=16.0, beta_slow=2.0), dict(factors=True)])
def test_rope_table(qk, kw):
    """Long positions against 64 bits; the ramp from its definition."""
    kw = dict(kw)
    n, rot = 131072, 96
    factors = 1 + np.arange(rot // 2, dtype=np.float32) / 7 if kw.pop("factors", False) else None
    got = f64(qk.rope_table(n, rot, freq_factors=None if factors is None else torch.from_numpy(factors).cuda(), **kw))
    i = np.arange(rot // 2)
    base, s, amp = kw.get("base", 10000.0), kw.get("freq_scale", 1.0), kw.get("amplitude", 1.0)
    f = base ** (-2.0 * i / rot)
    if factors is not None:
        f = f / factors
    if kw.get("orig_ctx"):
        def dim(t):
            return rot * np.log(kw["orig_ctx"] / (t * 2 * np.pi)) / (2 * np.log(base))
        lo = max(0, np.floor(dim(kw.get("beta_fast", 32.0))))
        hi = min(rot - 1, np.ceil(dim(kw.get("beta_slow", 1.0))))
        m = 1 - np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        f = f * (s * (1 - m) + m)
        assert m[0] == 1 and m[-1] < 1     # the fastest pairs are kept, the slowest interpolated
    else:
        f = f * s
    a = np.arange(n)[:, None] * f
    assert np.abs(got - amp * np.stack([np.cos(a), np.sin(a)], -1)).max() <= 4e-7 * amp


# ---------------------------------------------------------------- append and read back

@pytest.mark.parametrize("T,nq,nkv,D,page,rot,interleaved,norm,dtype", [
    (1, 32, 8, 128, 16, 128, False, True, "f32"),
    (70, 9, 3, 64, 48, 64, True, False, "f32"),
    (33, 4, 4, 96, 32, 72, False, True, "bf16"),
    (19, 8, 1, 256, 64, 256, False, True, "f16"),
    (40, 0, 2, 128, 16, 0, False, False, "f32"),
])
def test_append(qk, T, nq, nkv, D, page, rot, interleaved, norm, dtype):
    pages = 2 + -(-T // page)
    g = torch.Generator().manual_seed(T)
    cache = torch.randint(0, 256, (pages, nkv, page // 16, 18 * D), dtype=torch.uint8, generator=g).cuda()
    before = cache.cpu().numpy()
    slots = torch.randperm(pages * page, generator=g)[:T].long()
    pos = torch.randint(0, 200, (T,), generator=g).int()
    qkv = rand(T, T, (nq + 2 * nkv) * D, scale=2.0, dtype=dtype)
    q, k, v = qkv.split([nq * D, nkv * D, nkv * D], 1)
    tab = table(200, rot) if rot else None
    wq = 1 + rand(2, D, scale=0.3) if norm else None
    wk = 1 + rand(3, D, scale=0.3) if norm else None
    qo = qk.kv_append_q4(cache, q if nq else None, k, v, pos.cuda(), slots.cuda(), tab, wq, wk, eps=1e-5,
                         interleaved=interleaved)
    kr, vr = qk.kv_read_q4(cache, slots.cuda(), dtype=torch.float32)
    assert qk.device_error() == 0
    args = (1e-5, None if tab is None else f64(tab), pos.numpy(), rot, interleaved)
    if nq:
        ref, mag = ko.norm_rope(f64(q).reshape(T, nq, D), f64(wq) if norm else None, *args)
        close(qo, ref.reshape(T, -1),
              (2.0 ** -19 * mag + OUT[dtype] * np.abs(ref) + 2.0 ** -24).reshape(T, -1), "queries")
    # values: the definition, exactly
    vn, vd = ko.quantise(f64(v).reshape(T, nkv, D))
    want = ((vn.astype(np.float64) - 8) * np.repeat(vd.astype(np.float64), 32, -1)).reshape(T, -1)
    assert np.array_equal(f64(vr), want)
    # keys: the definition, but for a scale one fp16 step off and a nibble whose value lies on its edge
    x, _ = ko.norm_rope(f64(k).reshape(T, nkv, D), f64(wk) if norm else None, *args)
    kn, kd = ko.quantise(x)
    step = np.repeat(np.abs(kd.astype(np.float64)), 32, -1)
    ref = (kn.astype(np.float64) - 8) * np.repeat(kd.astype(np.float64), 32, -1)
    off = np.abs(f64(kr).reshape(T, nkv, D) - ref)
    assert np.all(off <= step * 1.01)
    assert (off > 2.0 ** -9 * np.abs(ref)).mean() < 1e-4
    # every other byte is as it was
    after = cache.cpu().numpy()
    kb, _, vb, _, sk, sv = ko.places(D)
    mine = np.zeros(before.shape, bool)
    for s in slots.tolist():
        p, o = divmod(s, page)
        for cols in (kb[o % 16], vb[o % 16], sk[o % 16], sk[o % 16] + 1, sv[o % 16], sv[o % 16] + 1):
            mine[p, :, o // 16, cols] = True
    assert np.array_equal(before[~mine], after[~mine])


def test_append_extreme_groups(qk):
    """Zero groups, ties of both signs, scales past fp16's range, NaN and infinities."""
    D = 64
    x = torch.zeros(8, D)
    x[1, :32] = torch.linspace(-1, 1, 32)                  # a tie: the positive value sets the scale
    x[2, 0], x[2, 1] = -3.0, 1.0
    x[3, :] = 1e6                                          # |d| is held to 65504
    x[4, 3] = float("nan")
    x[5, 40] = float("inf")
    x[6, :] = 1e-9                                         # the scale underflows to 0
    x[7, :32] = torch.arange(32) * 1e-3
    cache = qk.kv_cache_q4(1, 1, 16, D)
    slots = torch.arange(8).cuda()
    qk.kv_append_q4(cache, None, x.cuda(), x.cuda(), None, slots, None)
    for r in qk.kv_read_q4(cache, slots, dtype=torch.float32):
        r = r.cpu()
        assert (r[0] == 0).all() and (r[6] == 0).all()
        assert r[1, 31] == 1.0 and r[1, 0] == -0.875
        assert r[2, 0] == -3.0 and abs(float(r[2, 1]) - 1.125) < 1e-3
        assert (r[3] == 8 * 65504.0).all()
        assert torch.isnan(r[4, :32]).all() and (r[4, 32:] == 0).all()
        assert torch.isnan(r[5, 32:]).all() and (r[5, :32] == 0).all()


def test_append_slots(qk):
    """Negative slots store nothing, slots beyond the cache report; a bad position stores a NaN key."""
    D, T = 64, 5
    cache = qk.kv_cache_q4(2, 1, 16, D)
    x = rand(1, T, D)
    slots = torch.tensor([3, -1, 32, 31, 1 << 40]).cuda()
    pos = torch.tensor([0, 1, 2, 99, 3], dtype=torch.int32).cuda()
    q = qk.kv_append_q4(cache, x, x, x, pos, slots, table(10, D))
    assert qk.device_error() == 9
    assert torch.isnan(q[3]).all() and not torch.isnan(q[[0, 1, 2, 4]]).any()
    k, v = qk.kv_read_q4(cache, torch.arange(32).cuda(), dtype=torch.float32)
    assert torch.isnan(k[31]).all() and not torch.isnan(v).any() and (v[31] != 0).any()
    others = [s for s in range(32) if s not in (3, 31)]
    assert (k[others] == 0).all() and (v[others] == 0).all() and (k[3] != 0).any()
    k, _ = qk.kv_read_q4(cache, torch.tensor([-7, 32]).cuda())
    assert (k[0] == 0).all() and torch.isnan(k[1]).all() and qk.device_error() == 9


# ---------------------------------------------------------------- attention

def make_cache(seed, lens, nkv, D, page, spare=3, garbage=True):
    """A paged cache of random keys and values; slots past each length hold garbage, NaN scales among it."""
    g = np.random.default_rng(seed)
    need = [-(-max(l, 0) // page) for l in lens]
    pages = sum(need) + spare
    order = g.permutation(pages)
    width = max(max(need), 1)
    tab = np.full((len(lens), width), -1, np.int32)
    cache = g.integers(0, 256, (pages, nkv, page // 16, 18 * D), dtype=np.uint8)
    keys, vals, at = [], [], 0
    for b, n in enumerate(need):
        tab[b, :n] = order[at:at + n]
        at += n
        k = g.standard_normal((n, nkv, page, D)) * np.exp(0.5 * g.standard_normal((1, nkv, 1, D)))
        v = g.standard_normal((n, nkv, page, D))
        kn, kd = ko.quantise(k)
        vn, vd = ko.quantise(v)
        if garbage and n:
            tail = np.arange(page) >= lens[b] - (n - 1) * page
            kd[-1, :, tail] = np.float16(np.nan)
            vd[-1, :, tail] = np.float16(np.inf)
        blocks = ko.pack(kn, kd, vn, vd)
        cache[tab[b, :n]] = blocks
        k, v = ko.unpack(blocks)        # [n][nkv][page/16][16][D]
        keys.append(k.reshape(n, nkv, page, D).transpose(0, 2, 1, 3).reshape(n * page, nkv, D)[:max(lens[b], 0)])
        vals.append(v.reshape(n, nkv, page, D).transpose(0, 2, 1, 3).reshape(n * page, nkv, D)[:max(lens[b], 0)])
    return torch.from_numpy(cache).cuda(), torch.from_numpy(tab).cuda(), keys, vals


def check_attn(qk, lens, new, nq, nkv, D, page, window=0, dtype="f32", out=None, seed=0, split=True, max_len=0,
               scale=None, qscale=1.5):
    cache, tab, keys, vals = make_cache(seed, lens, nkv, D, page)
    T = sum(new)
    q = rand(seed + 1, T, nq * D, scale=qscale, dtype=dtype)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    ws = qk.attn_q4_workspace(len(lens), nq, nkv, D, max(new), max(lens)) if split else None
    o = torch.full((T, nq * D), 7.0, dtype=DT[out or dtype], device="cuda")
    scale = D ** -0.5 if scale is None else scale
    qk.attn_q4(cache, q, tab, torch.tensor(lens, dtype=torch.int32).cuda(), q_start=starts, max_q=max(new),
               max_len=max_len, scale=scale, window=window, out=o, workspace=ws)
    assert qk.device_error() == 0
    at, refs, bounds = 0, [], []
    u = OUT[out or dtype]
    for b, (L, n) in enumerate(zip(lens, new)):
        x = f64(q[at:at + n]).reshape(n, nq, D)
        at += n
        ref, A, S = ko.attention(x, keys[b], vals[b], L - n + np.arange(n), scale, window)
        e = (2.0 ** -17 * A + 2.0 ** -16 if dtype == "f32" else 2.0 ** -10 * A + 2.0 ** -9)[..., None] * S
        refs.append(ref.reshape(n, nq * D))
        bounds.append((e + u * np.abs(ref)).reshape(n, nq * D) + 2.0 ** -24)
    ref = np.concatenate(refs)
    close(o, ref, np.concatenate(bounds), "attention")
    norm = np.linalg.norm(ref)
    if norm > 0:
        rel = np.linalg.norm(f64(o) - ref) / norm
        limit = 1e-5 if "f32" == dtype == (out or dtype) else 5e-3 if "bf16" in (dtype, out) else 1.5e-3
        assert rel <= limit, f"2-norm {rel:.2e}"
    if ws is not None:     # its counters are zero again: a second call gives the same bits
        o2 = qk.attn_q4(cache, q, tab, torch.tensor(lens, dtype=torch.int32).cuda(), q_start=starts, max_q=max(new),
                        max_len=max_len, scale=scale, window=window, out=torch.empty_like(o), workspace=ws)
        assert torch.equal(o, o2)
    return o


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("nq,nkv,D,page", [(9, 3, 64, 16), (32, 8, 128, 64), (4, 4, 96, 48), (8, 1, 256, 32),
                                           (24, 2, 128, 16), (20, 1, 64, 256)])
def test_attn_single_tokens(qk, nq, nkv, D, page, dtype):
    check_attn(qk, [1, 15, 16, 17, 300, 700], [1] * 6, nq, nkv, D, page, dtype=dtype, seed=D + nq)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 31, 33, 127, 129, 2049, 5000])
def test_attn_one_sequence_lengths(qk, L, dtype):
    check_attn(qk, [L], [1], 8, 2, 128, 32, dtype=dtype, seed=L)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,new,nq,nkv,D,page,window", [
    ([40], [40], 8, 2, 128, 16, 0),                # a whole prompt
    ([333, 64, 5], [64, 64, 5], 4, 2, 64, 32, 0),
    ([200, 17, 90], [3, 1, 33], 6, 3, 96, 48, 0),  # decode beside chunks
    ([300, 150], [130, 150], 4, 1, 128, 64, 0),    # more than one row tile
    ([280, 150], [130, 20], 2, 1, 256, 32, 0),
    ([300, 150, 40], [70, 20, 40], 4, 4, 64, 16, 37),
])
def test_attn_chunks(qk, lens, new, nq, nkv, D, page, window, dtype):
    check_attn(qk, lens, new, nq, nkv, D, page, window=window, dtype=dtype, seed=sum(lens))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,new,nq,nkv,D,page,window", [
    ([2000], [64], 4, 2, 128, 16, 0),              # parts that are no whole number of key tiles of the whole
    ([1999], [47], 4, 1, 96, 48, 0),
    ([3000, 0, 700, 50], [64, 0, 64, 1], 4, 2, 64, 32, 0),
    ([2500, 2400], [200, 3], 4, 2, 128, 64, 700),
    ([1030], [1030], 2, 1, 64, 16, 0),
    ([16000], [40], 2, 1, 128, 64, 0),
    ([777] * 40, [33] * 40, 2, 2, 64, 16, 0),      # more heads than may be cut
])
def test_attn_cut_chunks(qk, lens, new, nq, nkv, D, page, window, dtype):
    check_attn(qk, lens, new, nq, nkv, D, page, window=window, dtype=dtype, seed=sum(new))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("qscale,scale", [(1e-3, None), (60.0, None), (1.5, -0.1), (1e20, 1e-21)])
def test_attn_chunks_flat_and_peaked(qk, dtype, qscale, scale):
    check_attn(qk, [500], [50], 4, 2, 128, 32, dtype=dtype, qscale=qscale if dtype == "f32" else min(qscale, 60.0),
               scale=scale if dtype == "f32" or scale != 1e-21 else None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attn_cut_faults(qk, dtype):
    """A page out of range, or a block that never comes, in one part of a cut head: the rows that see it are NaN, the
    other sequence is as it was, and the workspace stays usable."""
    D, page, n = 128, 16, 80
    cache, tab, _, _ = make_cache(4, [2100, 90], 2, D, page)
    lens = torch.tensor([2100, 90], dtype=torch.int32).cuda()
    q = rand(3, 2 * n, 4 * D, dtype=dtype)
    ws = qk.attn_q4_workspace(2, 4, 2, D, n, 2100)
    ref = qk.attn_q4(cache, q, tab, lens, max_q=n, workspace=ws).reshape(2, n, 4, D)
    assert not torch.isnan(ref).any() and qk.device_error() == 0
    t = tab.clone()
    t[0, 70] = cache.shape[0]
    o = qk.attn_q4(cache, q, t, lens, max_q=n, workspace=ws).reshape(2, n, 4, D)
    assert qk.device_error() == 9 and torch.isnan(o[0]).all() and torch.equal(o[1], ref[1])
    limit = qk.set_wait_limit_ns(20_000_000)
    qk.debug_attn_skip_block(1)
    try:
        o = qk.attn_q4(cache, q, tab, lens, max_q=n, workspace=ws).reshape(2, n, 4, D)
        assert qk.device_error() == 6
    finally:
        qk.debug_attn_skip_block(-1)
        qk.set_wait_limit_ns(limit)
    assert torch.isnan(o[0, 0, 0]).all() and torch.equal(o[1], ref[1])
    o = qk.attn_q4(cache, q, tab, lens, max_q=n, workspace=ws).reshape(2, n, 4, D)
    assert torch.equal(o, ref) and qk.device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_cut_chunks_programmatic_and_graph(qk, dtype):
    """Append and cut attention calls one after another, of other lengths on one workspace, under programmatic launch
    and from a captured graph: the plain calls' bits."""
    D, nkv, nq, page, n = 128, 2, 4, 16, 70
    cache, tab, _, _ = make_cache(6, [1800, 900], nkv, D, page)
    rot = table(2048, D)
    qkv = rand(1, 2 * n, (nq + 2 * nkv) * D, dtype=dtype)
    q, k, v = qkv.split([nq * D, nkv * D, nkv * D], 1)
    ws = qk.attn_q4_workspace(2, nq, nkv, D, n, 1800)
    lens = [torch.tensor(x, dtype=torch.int32).cuda() for x in ([1800, 900], [600, 880], [90, 71])]
    steps = []
    for l in lens:
        at = (l[:, None] - n + torch.arange(n, dtype=torch.int32).cuda()).long()
        slots = tab.long().gather(1, at // page) * page + at % page
        steps.append((l, at.int().reshape(-1), slots.reshape(-1)))
    base = cache.clone()
    outs = [torch.empty(2 * n, nq * D, dtype=DT[dtype], device="cuda") for _ in lens]
    qo = torch.empty(2 * n, nq * D, dtype=DT[dtype], device="cuda")

    def run():
        for (l, pos, slots), o in zip(steps, outs):
            qk.kv_append_q4(cache, q, k, v, pos, slots, rot, q_out=qo)
            qk.attn_q4(cache, qo, tab, l, max_q=n, max_len=1800, out=o, workspace=ws)

    run()
    want = [o.clone() for o in outs]
    qk.set_programmatic_launch(True)
    try:
        for _ in range(10):
            cache.copy_(base)
            for o in outs:
                o.zero_()
            run()
            assert all(torch.equal(o, w) for o, w in zip(outs, want))
    finally:
        qk.set_programmatic_launch(False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            run()
    for _ in range(3):
        cache.copy_(base)
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert qk.device_error() == 0


def test_attn_fp32_chunk_strides(qk):
    """fp32 rows and outputs off 16-byte boundaries."""
    D, nq, n = 64, 6, 40
    cache, tab, _, _ = make_cache(5, [90, 200], 2, D, 32)
    lens = torch.tensor([90, 200], dtype=torch.int32).cuda()
    q = rand(1, 2 * n, nq * D + 9)[:, 3:3 + nq * D]
    ref = qk.attn_q4(cache, q.contiguous(), tab, lens, max_q=n)
    out = torch.full((2 * n, nq * D + 3), 5.0, device="cuda")
    qk.attn_q4(cache, q, tab, lens, max_q=n, out=out[:, 1:1 + nq * D])
    assert torch.equal(out[:, 1:1 + nq * D], ref)
    assert (out[:, 0] == 5).all() and (out[:, 1 + nq * D:] == 5).all()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("window", [1, 2, 16, 100, 100000])
def test_attn_window(qk, window, dtype):
    check_attn(qk, [1, 99, 100, 101, 640], [1] * 5, 4, 2, 64, 32, window=window, dtype=dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attn_rows_without_keys_are_zero(qk, dtype):
    """A sequence of no keys, and chunks longer than their sequence: the first rows see nothing."""
    o = check_attn(qk, [0, 3, 50], [1, 8, 2], 4, 2, 64, 16, dtype=dtype)
    assert (o[0] == 0).all() and (o[1:6] == 0).all() and (o[6:] != 0).any(1).all()


def test_attn_split_and_hints(qk):
    """No workspace, a small one, and a length hint far from the lengths give the same answer to rounding."""
    for kw in (dict(split=False), dict(max_len=64), dict(max_len=100000)):
        check_attn(qk, [4000, 77], [1, 1], 8, 2, 128, 16, seed=3, **kw)
        check_attn(qk, [2000, 77], [9, 1], 8, 2, 128, 16, seed=3, dtype="bf16", **kw)


def test_attn_one_workspace_for_calls_of_all_shapes(qk):
    """A workspace serves calls of other shapes in turn: none leaves anything where another's counters are."""
    ws = torch.zeros(8 << 20, dtype=torch.uint8, device="cuda")
    calls = []
    for i, (lens, n, nq, nkv, D, dtype) in enumerate([([3000], 1, 8, 1, 128, "f32"), ([900] * 40, 1, 16, 8, 64, "bf16"),
                                                      ([2500, 800], 5, 4, 2, 256, "f16"), ([5000], 1, 3, 3, 96, "f32")]):
        cache, tab, _, _ = make_cache(i, lens, nkv, D, 64)
        q = rand(i, len(lens) * n, nq * D, dtype=dtype)
        args = (cache, q, tab, torch.tensor(lens, dtype=torch.int32).cuda(), None, n, max(lens))
        calls.append((args, qk.attn_q4(*args, workspace=torch.zeros_like(ws))))
    for _ in range(3):
        for args, want in calls:
            assert torch.equal(qk.attn_q4(*args, workspace=ws), want)


@pytest.mark.parametrize("dtype,out", [("f32", "bf16"), ("f16", "f32"), ("bf16", "f16")])
def test_attn_output_types(qk, dtype, out):
    check_attn(qk, [77, 130], [1, 40], 4, 2, 64, 16, dtype=dtype, out=out)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("qscale", [1e-3, 30.0])
def test_attn_flat_and_peaked(qk, dtype, qscale):
    """Nearly equal probabilities, and one that takes all; also a negative scale."""
    check_attn(qk, [500, 60], [1, 20], 8, 2, 128, 32, dtype=dtype, qscale=qscale, seed=5)
    check_attn(qk, [130], [1], 4, 2, 64, 32, dtype=dtype, qscale=qscale, seed=6, scale=-0.3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vscale", [1e-4, 6e4])
def test_attn_value_magnitudes(qk, vscale, dtype):
    """Tiny values and values whose scales are near fp16's limit keep their relative accuracy."""
    D, page, nkv, L = 64, 32, 1, 200
    g = np.random.default_rng(1)
    pages = -(-L // page)
    k, v = g.standard_normal((2, pages, nkv, page, D))
    blocks = ko.pack(*ko.quantise(k), *ko.quantise(v * vscale))
    kk, vv = (t.transpose(0, 2, 3, 1, 4).reshape(-1, nkv, D)[:L] for t in ko.unpack(blocks))
    for n in (1, 70):
        q = rand(2, n, 4 * D, dtype=dtype)
        tab = torch.arange(pages, dtype=torch.int32).reshape(1, -1).cuda()
        o = qk.attn_q4(torch.from_numpy(blocks).cuda(), q, tab, torch.tensor([L], dtype=torch.int32).cuda(), max_q=n,
                       out=torch.empty(n, 4 * D, device="cuda"))
        ref, A, S = ko.attention(f64(q).reshape(n, 4, D), kk, vv, L - n + np.arange(n), D ** -0.5, 0)
        e = (2.0 ** -17 * A + 2.0 ** -16 if dtype == "f32" else 2.0 ** -10 * A + 2.0 ** -9)[..., None] * S
        close(o, ref.reshape(n, -1), (e + 2.0 ** -24 * np.abs(ref)).reshape(n, -1), f"values x {vscale}")


@pytest.mark.parametrize("n", [1, 70])
def test_attn_non_finite(qk, n):
    """A NaN query row, a NaN key and an infinite value reach the rows that see them and no others."""
    D, L = 64, 100
    cache, tab, _, _ = make_cache(1, [L], 2, D, 16)
    lens = torch.tensor([L], dtype=torch.int32).cuda()
    q = rand(3, n, 4 * D, dtype="f16")
    q[n - 1, 3 * D + 1] = float("nan")
    o = qk.attn_q4(cache, q, tab, lens, max_q=n)
    assert torch.isnan(o[n - 1, 3 * D:]).all() and not torch.isnan(o[n - 1, :3 * D]).any()
    assert not torch.isnan(o[:n - 1]).any()
    q[n - 1, 3 * D + 1] = 0
    x = torch.full((1, 2 * D), float("nan"), device="cuda")
    qk.kv_append_q4(cache, None, x, x, None, torch.tensor([int(tab[0, 0]) * 16 + 3]).cuda(), None)
    o = qk.attn_q4(cache, q, tab, lens, max_q=n)
    assert torch.isnan(o).all()
    o = qk.attn_q4(cache, q, tab, lens, max_q=n, window=20)
    assert not torch.isnan(o).any()


@pytest.mark.parametrize("dtype,n", [("f32", 1), ("bf16", 1), ("bf16", 80)])
def test_attn_bad_indices(qk, dtype, n):
    """Pages, lengths and row ranges out of range poison their sequence and nothing else."""
    D, page = 64, 16
    cache, tab, _, _ = make_cache(2, [100, 100, 100, 100], 2, D, page)
    good = torch.tensor([100] * 4, dtype=torch.int32).cuda()
    q = rand(3, 4 * n, 4 * D, dtype=dtype)
    ws = qk.attn_q4_workspace(4, 4, 2, D, n, 100)
    ref = qk.attn_q4(cache, q, tab, good, max_q=n, workspace=ws).reshape(4, n, -1)
    assert not torch.isnan(ref).any() and qk.device_error() == 0
    for page_id in (-1, cache.shape[0]):
        t = tab.clone()
        t[1, 2] = page_id
        o = qk.attn_q4(cache, q, t, good, max_q=n, workspace=ws).reshape(4, n, -1)
        assert qk.device_error() == 9
        sees = 100 - n + torch.arange(n) >= 2 * page      # the rows that see the page's keys
        assert torch.isnan(o[1][sees.cuda()]).all() and torch.equal(o[[0, 2, 3]], ref[[0, 2, 3]])
    for bad in (-1, tab.shape[1] * page + 1):
        lens = good.clone()
        lens[2] = bad
        o = qk.attn_q4(cache, q, tab, lens, max_q=n, workspace=ws).reshape(4, n, -1)
        assert qk.device_error() == 9
        assert torch.isnan(o[2]).all() and torch.equal(o[[0, 1, 3]], ref[[0, 1, 3]])
    starts = torch.tensor([0, n, 2 * n, 3 * n, 4 * n + 1], dtype=torch.int32).cuda()
    o = qk.attn_q4(cache, q, tab, good, q_start=starts, max_q=n, workspace=ws).reshape(4, n, -1)
    assert qk.device_error() == 9
    assert torch.isnan(o[3]).all() and torch.equal(o[:3], ref[:3])
    o = qk.attn_q4(cache, q, tab, good, max_q=n, workspace=ws).reshape(4, n, -1)
    assert torch.equal(o, ref) and qk.device_error() == 0      # the workspace is usable after all of it


@pytest.mark.parametrize("n", [1, 40])
def test_attn_strides_and_streams(qk, n):
    """Strided queries, outputs and page tables, and another stream than the current one."""
    D, nq = 64, 6
    cache, tab, _, _ = make_cache(5, [90, 200], 2, D, 32)
    lens = torch.tensor([90, 200], dtype=torch.int32).cuda()
    wide = rand(1, 2 * n, nq * D + 10, dtype="bf16")
    q = wide[:, 3:3 + nq * D]
    ref = qk.attn_q4(cache, q.contiguous(), tab, lens, max_q=n)
    big = torch.full((2, 20), 123456, dtype=torch.int32).cuda()
    big[:, :tab.shape[1]] = tab
    out = torch.full((2 * n, nq * D + 4), 5.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    qk.attn_q4(cache, q, big[:, :tab.shape[1]], lens, max_q=n, out=out[:, 1:1 + nq * D], stream=s)
    s.synchronize()
    assert torch.equal(out[:, 1:1 + nq * D], ref)
    assert (out[:, 0] == 5).all() and (out[:, 1 + nq * D:] == 5).all()


def test_cache_past_32_bit_offsets(qk):
    """Pages beyond 4 GiB of the cache, appended to, read back and attended over."""
    D, page, nkv = 128, 64, 8
    pages = (5 << 30) // (nkv * page // 16 * 18 * D)
    cache = torch.empty(pages, nkv, page // 16, 18 * D, dtype=torch.uint8, device="cuda")
    small = qk.kv_cache_q4(2, nkv, page, D)
    tab = torch.tensor([[pages - 1, pages - 5]], dtype=torch.int32).cuda()
    L = 100
    k, v = rand(1, L, nkv * D), rand(2, L, nkv * D)
    j = torch.arange(L).cuda()
    slots = tab[0].long()[j // page] * page + j % page
    lens = torch.tensor([L], dtype=torch.int32).cuda()
    q = rand(3, 2, 32 * D, dtype="bf16")
    got = []
    for c, t, s in ((cache, tab, slots), (small, torch.tensor([[0, 1]], dtype=torch.int32).cuda(), j)):
        qk.kv_append_q4(c, None, k, v, None, s, None)
        got.append((*qk.kv_read_q4(c, s), qk.attn_q4(c, q, t, lens, max_q=2),
                    qk.attn_q4(c, q.repeat(40, 1), t, lens, max_q=80)))
    for x, y in zip(*got):
        assert torch.equal(x, y) and not torch.isnan(x).any()
    assert qk.device_error() == 0


def test_programmatic_launch_and_graph(qk):
    """The chain append -> attention under programmatic launch and in a captured graph gives the plain calls' bits."""
    D, nkv, nq, page = 128, 2, 8, 16
    tab = torch.arange(8, dtype=torch.int32).reshape(1, 8).cuda()
    rot = table(128, D)
    qkv = rand(1, 1, (nq + 2 * nkv) * D)
    q, k, v = qkv.split([nq * D, nkv * D, nkv * D], 1)
    pos, slot = torch.tensor([99], dtype=torch.int32).cuda(), torch.tensor([99]).cuda()
    lens = torch.tensor([100], dtype=torch.int32).cuda()
    first = torch.randn(100, nkv * D, generator=torch.Generator().manual_seed(2)).cuda()
    ws = qk.attn_q4_workspace(1, nq, nkv, D, 1, 128)
    qo, out = torch.empty(1, nq * D, device="cuda"), torch.empty(1, nq * D, device="cuda")

    def fresh():
        cache = qk.kv_cache_q4(8, nkv, page, D)
        qk.kv_append_q4(cache, None, first, first, None, torch.arange(100).cuda(), None)
        return cache

    def step(cache):
        qk.kv_append_q4(cache, q, k, v, pos, slot, rot, q_out=qo)
        qk.attn_q4(cache, qo, tab, lens, max_len=128, out=out, workspace=ws)

    step(fresh())
    want = out.clone()
    cache = fresh()
    qk.set_programmatic_launch(True)
    try:
        for _ in range(20):
            out.zero_()
            step(cache)
            assert torch.equal(out, want)
    finally:
        qk.set_programmatic_launch(False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step(cache)
    out.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype,n", [("f32", 1), ("bf16", 1), ("bf16", 80)])
def test_attn_timeout_is_reported(qk, dtype, n):
    """A block that is never copied: the bounded waits run out, the call ends, the error word says so, the thread
    block's rows are NaN, and the next call is right."""
    cache, tab, _, _ = make_cache(1, [300, 200], 2, 64, 16)
    lens = torch.tensor([300, 200], dtype=torch.int32).cuda()
    q = rand(3, 2 * n, 4 * 64, dtype=dtype)
    want = qk.attn_q4(cache, q, tab, lens, max_q=n)
    limit = qk.set_wait_limit_ns(20_000_000)
    qk.debug_attn_skip_block(1)
    try:
        got = qk.attn_q4(cache, q, tab, lens, max_q=n)
        assert qk.device_error() == 6
    finally:
        qk.debug_attn_skip_block(-1)
        qk.set_wait_limit_ns(limit)
    assert torch.isnan(got[0, :2 * 64]).all() and torch.equal(got[n:], want[n:])
    assert torch.equal(qk.attn_q4(cache, q, tab, lens, max_q=n), want) and qk.device_error() == 0


# ---------------------------------------------------------------- refusals of the binding

def test_binding_refuses(qk):
    cache = qk.kv_cache_q4(2, 2, 16, 64)
    q, kv = torch.zeros(3, 256, device="cuda"), torch.zeros(3, 128, device="cuda")
    i32, i64 = torch.zeros(3, dtype=torch.int32).cuda(), torch.zeros(3, dtype=torch.int64).cuda()
    tab, pages = table(4, 64), torch.zeros(3, 2, dtype=torch.int32).cuda()
    bad = [
        lambda: qk.norm_rope(q.cpu(), 2, 2, 64, i32, tab),
        lambda: qk.norm_rope(q, 2, 1, 64, i32, tab),
        lambda: qk.norm_rope(q.double(), 2, 2, 64, i32, tab),
        lambda: qk.norm_rope(q, 2, 2, 64, i32[:2], tab),
        lambda: qk.norm_rope(q, 2, 2, 64, i64, tab),
        lambda: qk.norm_rope(q, 2, 2, 64, None, tab),
        lambda: qk.norm_rope(q, 4, 4, 32, i32, tab),
        lambda: qk.norm_rope(q, 2, 2, 64, i32, tab, q_weight=torch.ones(63).cuda()),
        lambda: qk.norm_rope(q, 2, 2, 64, i32, tab, y=torch.empty(2, 256, device="cuda")),
        lambda: qk.norm_rope(q.t().contiguous().t(), 2, 2, 64, i32, tab),
        lambda: qk.kv_append_q4(cache, q, kv, kv[:2], i32, i64, tab),
        lambda: qk.kv_append_q4(cache, q, kv, kv.half(), i32, i64, tab),
        lambda: qk.kv_append_q4(cache, q, kv, kv, i32, i32, tab),
        lambda: qk.kv_append_q4(cache, q[:, :100], kv, kv, i32, i64, tab),
        lambda: qk.kv_append_q4(cache[:, :, :, :64], q, kv, kv, i32, i64, tab),
        lambda: qk.kv_read_q4(cache, i64, dtype=torch.float64),
        lambda: qk.attn_q4(cache, q[:, :192], pages, i32),
        lambda: qk.attn_q4(cache, q, pages[:2], i32),
        lambda: qk.attn_q4(cache, q, pages.long(), i32),
        lambda: qk.attn_q4(cache, q, pages, i32, q_start=i32),
        lambda: qk.attn_q4(cache, q, pages, i32, out=torch.empty(2, 256, device="cuda")),
        lambda: qk.kv_cache_q4(1, 1, 24, 64),
        lambda: qk.kv_cache_q4(1, 1, 16, 80),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was accepted")
    with pytest.raises(qk.QKError) as e:
        qk.attn_q4(cache, q, pages, i32, max_q=2)
    assert e.value.status == 2
    with pytest.raises(qk.QKError) as e:
        qk.attn_q4(cache, q, pages, i32, scale=float("inf"))
    assert e.value.status == 2
