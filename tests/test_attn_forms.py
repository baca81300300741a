"""The forms of the attention operators that large calls, odd rows and mixed types take, against the 64-bit oracle, with
the tolerances that tests/test_attn_ops.py derives."""
import ctypes

import numpy as np
import pytest
import torch

from tests import kv4_oracle as ko
from tests.test_attn_ops import DT, OUT, check_attn, close, f64, make_cache, rand, table

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- norm + rotation: several heads a lane

@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f32", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("nq,nk,D,rot,interleaved,norm", [
    (32, 8, 128, 128, False, "qk"),     # a lane goes from queries to keys
    (13, 5, 128, 96, True, "qk"),
    (20, 21, 96, 72, False, "qk"),
    (40, 7, 64, 64, True, "q"),         # and to rows without a norm
    (40, 7, 64, 64, False, "k"),
    (17, 3, 256, 128, True, "k"),
    (9, 9, 256, 256, False, ""),
    (70, 0, 64, 32, False, "q"),
])
def test_norm_rope_many_tokens(qk, nq, nk, D, rot, interleaved, norm, dtype, out):
    T = 400
    x = rand(T + D, T, (nq + nk) * D, dtype=dtype)
    tab = table(300, rot)
    pos = torch.randint(0, 300, (T,), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda()
    wq = 1 + rand(2, D, scale=0.3) if "q" in norm else None
    wk = 1 + rand(3, D, scale=0.3) if "k" in norm else None
    y = torch.empty(T, (nq + nk) * D, dtype=DT[out], device="cuda")
    qk.norm_rope(x, nq, nk, D, pos, tab, wq, wk, eps=1e-5, interleaved=interleaved, y=y)
    h = f64(x).reshape(T, nq + nk, D)
    args = (1e-5, f64(tab), pos.cpu().numpy(), rot, interleaved)
    rq, mq = ko.norm_rope(h[:, :nq], None if wq is None else f64(wq), *args)
    rk, mk = ko.norm_rope(h[:, nq:], None if wk is None else f64(wk), *args)
    ref, mag = np.concatenate([rq, rk], 1).reshape(T, -1), np.concatenate([mq, mk], 1).reshape(T, -1)
    close(y, ref, 2.0 ** -19 * mag + OUT[out] * np.abs(ref) + 2.0 ** -24, "norm_rope")
    assert qk.device_error() == 0


# ---------------------------------------------------------------- append

def strided(t, pad, off):
    """The same rows inside a wider buffer."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), 3.0, dtype=t.dtype, device="cuda")
    buf[:, off:off + t.shape[1]] = t
    return buf[:, off:off + t.shape[1]]


def check_append(qk, T, nq, nkv, D, page, rot, interleaved, norm, dtype, out=None, pad=0, off=0, shift=0, seed=0):
    """One append and its read-back: queries and keys within rounding, values exactly, no other byte changed.  shift:
    weights and table begin off a 16-byte boundary."""
    pages = 2 + -(-T // page)
    g = torch.Generator().manual_seed(T + seed)
    cache = torch.randint(0, 256, (pages, nkv, page // 16, 18 * D), dtype=torch.uint8, generator=g).cuda()
    before = cache.clone()
    slots = torch.randperm(pages * page, generator=g)[:T].long()
    pos = torch.randint(0, 200, (T,), generator=g).int()
    q, k, v = (strided(rand(seed + i, T, n * D, scale=2.0, dtype=dtype), pad, off) for i, n in enumerate((nq, nkv, nkv)))

    def shifted(t, n=1):
        flat = torch.empty(t.numel() + n * shift, device="cuda")
        flat[n * shift:] = t.reshape(-1)
        return flat[n * shift:].reshape(t.shape)

    tab = shifted(table(200, rot), 2) if rot else None      # a pair of floats is 8 bytes
    wq = shifted(1 + rand(2, D, scale=0.3)) if norm else None
    wk = shifted(1 + rand(3, D, scale=0.3)) if norm else None
    qo = strided(torch.zeros(T, nq * D, dtype=DT[out or dtype], device="cuda"), pad, off)
    got = qk.kv_append_q4(cache, q, k, v, pos.cuda(), slots.cuda(), tab, wq, wk, eps=1e-5, interleaved=interleaved, q_out=qo)
    assert got is qo
    kr, vr = qk.kv_read_q4(cache, slots.cuda(), dtype=torch.float32)
    assert qk.device_error() == 0
    args = (1e-5, None if tab is None else f64(tab), pos.numpy(), rot, interleaved)
    ref, mag = ko.norm_rope(f64(q).reshape(T, nq, D), f64(wq) if norm else None, *args)
    close(qo, ref.reshape(T, -1), (2.0 ** -19 * mag + OUT[out or dtype] * np.abs(ref) + 2.0 ** -24).reshape(T, -1), "queries")
    vn, vd = ko.quantise(f64(v).reshape(T, nkv, D))
    assert np.array_equal(f64(vr), ((vn.astype(np.float64) - 8) * np.repeat(vd.astype(np.float64), 32, -1)).reshape(T, -1))
    x, _ = ko.norm_rope(f64(k).reshape(T, nkv, D), f64(wk) if norm else None, *args)
    kn, kd = ko.quantise(x)
    step = np.repeat(np.abs(kd.astype(np.float64)), 32, -1)
    ref = (kn.astype(np.float64) - 8) * np.repeat(kd.astype(np.float64), 32, -1)
    miss = np.abs(f64(kr).reshape(T, nkv, D) - ref)
    assert np.all(miss <= step * 1.01)
    assert (miss > 2.0 ** -9 * np.abs(ref)).mean() < 1e-4
    # every other slot's bytes are as they were
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[slots] = False
    rest = rest.nonzero().reshape(-1).cuda()
    for a, b in zip(qk.kv_read_q4(cache, rest, dtype=torch.float32), qk.kv_read_q4(before, rest, dtype=torch.float32)):
        assert torch.equal(a.nan_to_num(1e9), b.nan_to_num(1e9))
    if pad:
        wide = qo.as_strided((T, nq * D + pad), (nq * D + pad, 1), qo.storage_offset() - off)
        assert (wide[:, :off] == 3).all() and (wide[:, off + nq * D:] == 3).all()


@pytest.mark.parametrize("T,nq,nkv,D,page,rot,interleaved,norm,dtype", [
    (3000, 12, 12, 128, 64, 128, False, True, "f32"),      # lanes go from keys to values, blocks from token to token
    (3000, 6, 9, 128, 48, 128, True, True, "bf16"),
    (2600, 5, 18, 96, 32, 72, False, True, "f16"),
    (2500, 3, 6, 256, 64, 256, True, True, "f32"),
    (700, 7, 11, 128, 16, 64, False, False, "f16"),
    (2600, 14, 2, 64, 64, 64, False, True, "bf16"),
    (400, 33, 17, 64, 16, 64, True, True, "f32"),
])
def test_append_many_tokens(qk, T, nq, nkv, D, page, rot, interleaved, norm, dtype):
    check_append(qk, T, nq, nkv, D, page, rot, interleaved, norm, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,nq,nkv,D,rot,pad,off,shift", [
    (37, 9, 3, 64, 36, 0, 0, 0),        # a rotation that is no multiple of 8
    (21, 4, 1, 256, 250, 0, 0, 0),
    (37, 4, 2, 128, 128, 5, 3, 0),      # rows off every boundary
    (37, 2, 2, 96, 96, 2, 2, 0),
    (37, 4, 2, 128, 64, 4, 0, 1),       # weights and table off 16 bytes
    (300, 6, 3, 128, 126, 1, 1, 1),
    (19, 3, 1, 256, 2, 0, 0, 0),
])
def test_append_general_form(qk, T, nq, nkv, D, rot, pad, off, shift, interleaved, dtype):
    check_append(qk, T, nq, nkv, D, 32, rot, interleaved, True, dtype, pad=pad, off=off, shift=shift, seed=rot)


@pytest.mark.parametrize("T", [1, 50, 2500])
@pytest.mark.parametrize("dtype,out", [("f32", "bf16"), ("f32", "f16"), ("bf16", "f32"), ("f16", "bf16")])
def test_append_queries_of_another_type(qk, T, dtype, out):
    """fp32 rows, as the products here write them, with 16-bit queries for the attention, and the other way."""
    check_append(qk, T, 8, 2, 128, 64, 128, False, True, dtype, out=out)
    if T < 100:
        check_append(qk, T, 8, 2, 128, 64, 100, True, True, dtype, out=out, pad=3, off=1)


def test_fp32_prompt_through_16_bit_queries(qk):
    """An fp32 prompt appended with bf16 queries out, and attention in bf16 with fp32 out, against 64 bits over what the
    cache holds."""
    T, nq, nkv, D, page = 300, 8, 2, 128, 64
    pages = -(-T // page)
    cache = qk.kv_cache_q4(pages, nkv, page, D)
    qkv = rand(3, T, (nq + 2 * nkv) * D)
    q, k, v = qkv.split([nq * D, nkv * D, nkv * D], 1)
    slots = torch.arange(T).cuda()
    qo = qk.kv_append_q4(cache, q, k, v, slots.int(), slots, table(T, D), q_out=torch.empty(T, nq * D, dtype=torch.bfloat16, device="cuda"))
    tab, lens = torch.arange(pages, dtype=torch.int32).reshape(1, -1).cuda(), torch.tensor([T], dtype=torch.int32).cuda()
    o = qk.attn_q4(cache, qo, tab, lens, max_q=T, out=torch.empty(T, nq * D, device="cuda"))
    kr, vr = (f64(t).reshape(T, nkv, D) for t in qk.kv_read_q4(cache, slots, dtype=torch.float32))
    ref, A, S = ko.attention(f64(qo).reshape(T, nq, D), kr, vr, np.arange(T), D ** -0.5, 0)
    close(o, ref.reshape(T, -1), ((2.0 ** -10 * A + 2.0 ** -9)[..., None] * S).reshape(T, -1) + 2.0 ** -24, "attention")
    assert qk.device_error() == 0


# ---------------------------------------------------------------- read-back

def test_read_types_and_strides(qk):
    """The three types are the exact values rounded once; rows off 16-byte boundaries (by the C interface), keys or values
    alone; the rest of the rows is untouched."""
    nkv, D, page, T = 3, 96, 48, 70
    cache, _, _, _ = make_cache(7, [T], nkv, D, page, garbage=False)
    slots = torch.randint(0, cache.shape[0] * page, (T,), generator=torch.Generator().manual_seed(2)).cuda()
    cache[:, :, :, 16 * D:] = torch.from_numpy(np.random.default_rng(1).normal(0, 0.2, (*cache.shape[:3], D))
                                               .astype(np.float16).view(np.uint8)).cuda()
    want = qk.kv_read_q4(cache, slots, dtype=torch.float32)
    k, v = ko.unpack(cache.cpu().numpy())
    at = slots.cpu().numpy()
    for got, all_ in zip(want, (k, v)):
        ref = all_.transpose(0, 2, 3, 1, 4).reshape(-1, nkv * D)[at]
        assert np.array_equal(f64(got), ref)
    for dtype in ("f16", "bf16"):
        for got, ref in zip(qk.kv_read_q4(cache, slots, dtype=DT[dtype]), want):
            assert torch.equal(got, ref.to(DT[dtype]))
    lib = qk.load()
    c = qk._KVCacheQ4(cache.data_ptr(), cache.shape[0], nkv, D, page)
    for code, dtype in enumerate(("f32", "f16", "bf16")):
        for off in (0, 1):
            ld = nkv * D + 5
            bufs = [torch.full((T * ld + 1,), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
            for use_k, use_v in ((1, 1), (1, 0), (0, 1)):
                for b in bufs:
                    b.fill_(7.0)
                at = [b.data_ptr() + off * b.element_size() if on else None for b, on in zip(bufs, (use_k, use_v))]
                torch.cuda.synchronize()
                assert lib.qk_kv_read_q4(ctypes.byref(c), slots.data_ptr(), T, at[0], ld, at[1], ld, code, None) == 0
                torch.cuda.synchronize()
                for b, on, ref in zip(bufs, (use_k, use_v), want):
                    rows = b[off:off + T * ld].reshape(T, ld)
                    assert torch.equal(rows[:, :nkv * D], ref.to(DT[dtype])) if on else (b == 7).all()
                    assert (rows[:, nkv * D:] == 7).all() and (off == 0 or b[0] == 7)
    assert qk.device_error() == 0


# ---------------------------------------------------------------- attention of 5 to 32 rows a head, in batches

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,new,nq,nkv,D", [
    (60, 4, 16, 4, 128),       # four tokens, four heads a key head: two column sets in 16 bits, four in fp32
    (60, 3, 16, 4, 64),
    (60, 5, 12, 4, 96),
    (120, 4, 3, 1, 256),
    (130, 8, 4, 1, 128),       # more than one tile of rows
    (3, 2, 9, 3, 96),          # few heads: one set in 16 bits, two in fp32
    (3, 1, 2, 1, 256),
])
def test_attn_batches_of_few_rows(qk, B, new, nq, nkv, D, dtype):
    lens = [new + (37 * b) % 90 for b in range(B)]
    check_attn(qk, lens, [new if b % 4 else 1 + b % new for b in range(B)], nq, nkv, D, 16, dtype=dtype, seed=B + D)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attn_batches_of_few_rows_long(qk, dtype):
    """The same column sets with long sequences and a window."""
    check_attn(qk, [700 - b for b in range(60)], [4] * 60, 16, 4, 128, 64, dtype=dtype, window=300, seed=9)


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("split", [False, True])
def test_fp16_chunks_keep_fp32_accuracy(qk, D, split):
    """fp16 queries of chunks are exact operands, keys and values exact in two pieces and probabilities in 22 bits: with
    fp32 out, what fp32 queries have, 1e-5 of the 2-norm.  (Rounded to 11 bits, as few rows and bf16 chunks are: 4e-4.)"""
    lens, n, nq, nkv, page = [1500, 200], 60, 4, 2, 32
    cache, tab, keys, vals = make_cache(D, lens, nkv, D, page)
    q = rand(1, 2 * n, nq * D, scale=1.5, dtype="f16")
    ws = qk.attn_q4_workspace(2, nq, nkv, D, n, max(lens)) if split else None
    o = qk.attn_q4(cache, q, tab, torch.tensor(lens, dtype=torch.int32).cuda(), max_q=n,
                   out=torch.empty(2 * n, nq * D, device="cuda"), workspace=ws)
    for b, L in enumerate(lens):
        x = f64(q[b * n:b * n + n]).reshape(n, nq, D)
        ref = ko.attention(x, keys[b], vals[b], L - n + np.arange(n), D ** -0.5, 0)[0].reshape(n, -1)
        assert np.linalg.norm(f64(o[b * n:b * n + n]) - ref) <= 1e-5 * np.linalg.norm(ref)
    assert qk.device_error() == 0
