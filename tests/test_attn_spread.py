"""Attention over a cache whose scales differ much: between the channel groups of a key or value, between the tokens of a
block, and with one large token that a row does not see, or that has no weight.

References are the 64-bit oracle's.  Outputs are fp32, so what is off is the kernel's own:

* element by element the bounds of tests/test_attn_ops.py, (2^-17 A + 2^-16) S with fp32 queries and (2^-10 A + 2^-9) S
  with 16-bit ones, where S = sum p |v| is the channel's own: a group of small values has small bounds;
* over each group of 32 channels, where the roundings of a few hundred keys are independent, a 2-norm within 2^-9 of the
  reference's (16-bit queries: keys, values and probabilities rounded to 11 bits, each less than 2^-11), and 1e-5 with
  fp32 queries.  Few rows keep, of an fp32 query's probability, 32 bits less the powers of two between its key's value
  scale and the largest: 2^(r-32) more.  An fp32 query is held in 24 bits below its row's largest, so one 2^-r below
  that adds 2^(r-22) A to its score.
"""
import numpy as np
import pytest
import torch

from tests import kv4_oracle as ko
from tests.test_attn_ops import DT, close, f64, rand

pytestmark = pytest.mark.gpu

PAGE, L = 32, 400
LATE = 340        # a token in the middle of its block of 16


def spread(kind, r, k, v, q):
    """k, v [L][nkv][D] and q [n][nq][D] with scales 2^r apart; the number of rows that are looked at."""
    n, D = q.shape[0], q.shape[2]
    big = 2.0 ** r
    if kind == "key groups":            # every score has its parts of both groups
        k[..., :32] *= big
        q[..., :32] /= big
    elif kind == "value groups":
        v[..., :32] *= big
    elif kind == "late key":            # rows before it do not see it
        k[LATE] *= big
        n -= L - LATE
    elif kind == "late value":
        v[LATE] *= big
        n -= L - LATE
    else:                               # a value of a key that no row gives weight to
        assert kind == "ignored value"
        q[:] = (q / 256 + 1) * np.log(2)
        k[5] = -60 / np.sqrt(D)           # 2^-60 below the others, which are small
        v[5] *= big
    return k, v, q, n


KINDS = ["key groups", "value groups", "late key", "late value", "ignored value"]


@pytest.mark.parametrize("r", [0, 12, 16, 20])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,D,n", [("bf16", 64, 80), ("bf16", 96, 80), ("bf16", 128, 300), ("f16", 128, 80),
                                       ("f32", 64, 80), ("f32", 96, 80), ("f32", 128, 300), ("bf16", 128, 70),
                                       ("f32", 128, 9), ("f16", 64, 9), ("bf16", 256, 70)])
def test_scales_apart(qk, dtype, D, n, kind, r):
    nkv, rep = 1, 2
    g = np.random.default_rng(r + D + n)
    k, v = g.standard_normal((2, L, nkv, D))
    k, v = k * 2.0 ** -6, v * 2.0 ** -6          # the largest scales stay below fp16's limit
    if kind.startswith("late") and n <= L - LATE:
        pytest.skip("no row before the late token")
    if kind == "key groups" and dtype == "f32" and r > 12:
        pytest.skip("the small queries have no bits left")
    q0 = f64(rand(n + r, n, nkv * rep * D, scale=1.5 * 2.0 ** 6)).reshape(n, nkv * rep, D)
    k, v, q0, rows = spread(kind, r, k, v, q0)
    as_pages = [np.concatenate([t, np.zeros((-L % PAGE, nkv, D))]).reshape(-1, PAGE, nkv, D).transpose(0, 2, 1, 3) for t in (k, v)]
    blocks = ko.pack(*ko.quantise(as_pages[0]), *ko.quantise(as_pages[1]))
    k, v = (t.reshape(-1, nkv, PAGE, D).transpose(0, 2, 1, 3).reshape(-1, nkv, D)[:L] for t in ko.unpack(blocks))
    q = torch.from_numpy(q0.reshape(n, -1)).to(DT[dtype]).cuda()
    tab = torch.arange(len(blocks), dtype=torch.int32).reshape(1, -1).cuda()
    o = qk.attn_q4(torch.from_numpy(blocks).cuda(), q, tab, torch.tensor([L], dtype=torch.int32).cuda(), max_q=n,
                   out=torch.empty(n, nkv * rep * D, device="cuda"))
    assert qk.device_error() == 0
    ref, A, S = ko.attention(f64(q).reshape(n, nkv * rep, D), k, v, L - n + np.arange(n), D ** -0.5, 0)
    got, ref, A, S = f64(o).reshape(ref.shape)[:rows], ref[:rows], A[:rows], S[:rows]
    chunk = n * rep > 32 and D <= 128
    few = 0.0 if chunk or dtype != "f32" else 2.0 ** (r - 32)
    if kind == "key groups" and dtype == "f32":
        few += 2.0 ** (r - 22) * A[..., None]
    e = (2.0 ** -17 * A + 2.0 ** -16 if dtype == "f32" else 2.0 ** -10 * A + 2.0 ** -9)[..., None] * S
    close(torch.from_numpy(got), ref, e + few * S + 2.0 ** -24 * np.abs(ref), kind)
    limit = 1e-5 + np.max(few) if dtype == "f32" else 2.0 ** -9
    for at in range(0, D, 32):
        x, y = got[..., at:at + 32], ref[..., at:at + 32]
        rel = np.linalg.norm(x - y) / np.linalg.norm(y)
        assert rel <= limit, f"{kind}, channels {at}..: 2-norm {rel:.2e}"


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [8, 70])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_value_scale_not_finite(qk, n, dtype, bad):
    """A value group without a finite scale: its 32 channels are NaN in the rows that see the key (in chunks the whole
    rows), all else is as without it."""
    D, nq, late = 128, 4, L - 3
    pages = -(-L // PAGE)
    cache = qk.kv_cache_q4(pages, 1, PAGE, D)
    k, v, q = rand(1, L, D), rand(2, L, D), rand(3, n, nq * D, dtype=dtype)
    tab = torch.arange(pages, dtype=torch.int32).reshape(1, -1).cuda()
    lens = torch.tensor([L], dtype=torch.int32).cuda()

    def attention():
        qk.kv_append_q4(cache, None, k, v, None, torch.arange(L).cuda(), None)
        return qk.attn_q4(cache, q, tab, lens, max_q=n).reshape(n, nq, D)

    want = attention()
    v[late, 40] = bad
    got = attention()
    sees = n - (L - late)
    assert torch.equal(got[:sees], want[:sees]) and torch.isnan(got[sees:, :, 32:64]).all()
    others = torch.cat([got[sees:, :, :32], got[sees:, :, 64:]], -1)
    if n * nq > 32:
        assert torch.isnan(others).all()
    else:
        assert torch.equal(others, torch.cat([want[sees:, :, :32], want[sees:, :, 64:]], -1))
    assert qk.device_error() == 0
