"""Attention of chunks whose rows move their softmax reference at chosen key tiles, against the 64-bit oracle.

The tolerance is that of tests/test_attn_ops.py: |o - ref| <= (2^-17 A + 2^-16) S with fp32 queries, (2^-10 A + 2^-9) S
with 16-bit ones, and the output's own rounding.  A row whose earlier sums kept their old reference would be off by
about S.
"""
import numpy as np
import pytest
import torch

from tests import kv4_oracle as ko
from tests.test_attn_ops import DT, OUT, close, f64, rand

pytestmark = pytest.mark.gpu

TILE = 64      # keys a tile of the chunk forms
PAGE = 64


def rising_cache(seed, jumps, tiles, nkv, D):
    """Keys of one direction, one level higher from each tile of `jumps` on; random values."""
    g = np.random.default_rng(seed)
    level = np.array([sum(t >= j for j in jumps) for t in range(tiles)])
    k = np.repeat(level, TILE)[:, None, None] + 0.1 * g.standard_normal((tiles * TILE, nkv, D))
    v = g.standard_normal((tiles * TILE, nkv, D))
    as_pages = [t.reshape(-1, PAGE, nkv, D).transpose(0, 2, 1, 3) for t in (k, v)]
    blocks = ko.pack(*ko.quantise(as_pages[0]), *ko.quantise(as_pages[1]))
    k, v = (t.reshape(-1, nkv, PAGE, D).transpose(0, 2, 1, 3).reshape(-1, nkv, D) for t in ko.unpack(blocks))
    return torch.from_numpy(blocks).cuda(), k, v


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("jumps", [(4,), (8,), (4, 8), (3, 4, 5, 8, 12), (0, 4, 7, 11), tuple(range(1, 14))])
def test_reference_moves_at_tile(qk, jumps, D, dtype):
    """Tiles 4, 8 and 12 are those at which the fp32 form empties its accumulator into the sum."""
    nkv, nq, n, tiles = 2, 4, 40, 14
    L = tiles * TILE
    cache, k, v = rising_cache(D + len(jumps), jumps, tiles, nkv, D)
    # a level is 16, 8, 4, 2 powers of two, from row to row
    up = 16 * np.log(2) / np.sqrt(D) * 2.0 ** -(np.arange(n) % 4)
    q = rand(len(jumps), n, nq * D, scale=0.05)
    q = ((1 + q) * torch.from_numpy(up).float().cuda()[:, None]).to(DT[dtype])
    tab = torch.arange(L // PAGE, dtype=torch.int32).reshape(1, -1).cuda()
    o = qk.attn_q4(cache, q, tab, torch.tensor([L], dtype=torch.int32).cuda(), max_q=n,
                   out=torch.empty(n, nq * D, device="cuda"))
    ref, A, S = ko.attention(f64(q).reshape(n, nq, D), k, v, L - n + np.arange(n), D ** -0.5, 0)
    e = (2.0 ** -17 * A + 2.0 ** -16 if dtype == "f32" else 2.0 ** -10 * A + 2.0 ** -9)[..., None] * S
    close(o, ref.reshape(n, -1), (e + OUT["f32"] * np.abs(ref)).reshape(n, -1) + 2.0 ** -24, "attention")
    assert qk.device_error() == 0
