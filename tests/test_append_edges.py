"""What the append stores for values next to a nibble's edge, wherever the rows lie: floor(x / d + 8.5) in fp32, the
quotient and the sum each rounded, byte for byte."""
import numpy as np
import pytest
import torch

from tests import kv4_oracle as ko
from tests.test_attn_ops import table

pytestmark = pytest.mark.gpu


def edge_rows(seed, T, heads, D):
    """fp32 rows whose groups hold a value that sets the scale and others on an edge, one step below it and one above."""
    g = np.random.default_rng(seed)
    d = (g.uniform(0.5, 1, (T, heads, D // 32, 1)) * 2.0 ** g.integers(-13, 9, (T, heads, D // 32, 1))).astype(np.float16)
    d = d.astype(np.float32) * np.where(g.random(d.shape) < 0.5, 1, -1).astype(np.float32)
    x = ((g.integers(1, 16, (T, heads, D // 32, 32)) - np.float32(8.5)) * d).astype(np.float32)      # exact
    side = g.integers(-1, 2, x.shape)
    x = np.where(side < 0, np.nextafter(x, np.float32(-np.inf)), np.where(side > 0, np.nextafter(x, np.float32(np.inf)), x))
    x[..., 5:6] = -8 * d
    return x.reshape(T, heads * D).astype(np.float32)


def quantise32(x):
    """Nibbles and scales as kv4_oracle.quantise, in fp32."""
    _, d = ko.quantise(x)
    g, e = np.asarray(x, np.float32).reshape(*d.shape, 32), d.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        n = np.clip(np.floor((g / e).astype(np.float32) + np.float32(8.5)), 0, 15)
    return np.where(e == 0, 8, n).reshape(x.shape).astype(np.uint8), d


def place(x, off, pad):
    """The rows inside a wider buffer, `off` elements from its start."""
    buf = torch.zeros(x.shape[0], x.shape[1] + pad, device="cuda")
    buf[:, off:off + x.shape[1]] = torch.from_numpy(x).cuda()
    return buf[:, off:off + x.shape[1]]


@pytest.mark.parametrize("nkv,D", [(8, 128), (3, 64), (2, 96), (1, 256)])
def test_edges(qk, nkv, D):
    T, page = 300, 32
    k, v = edge_rows(D, T, nkv, D), edge_rows(D + 1, T, nkv, D)
    pages = -(-T // page)
    as_pages = [np.concatenate([t.reshape(T, nkv, D), np.zeros((pages * page - T, nkv, D))]).reshape(pages, page, nkv, D)
                .transpose(0, 2, 1, 3) for t in (k, v)]
    want = ko.pack(*quantise32(as_pages[0]), *quantise32(as_pages[1]))
    exact = ko.pack(*ko.quantise(as_pages[0]), *ko.quantise(as_pages[1]))
    assert (want != exact).any()        # the rows hold values that the roundings carry over an edge
    empty = ko.pack(*ko.quantise(as_pages[0] * 0), *ko.quantise(as_pages[1] * 0))
    for off, pad in ((0, 0), (4, 4), (1, 1), (2, 7)):      # the last two rule out wide loads
        cache = torch.from_numpy(empty).cuda()
        qk.kv_append_q4(cache, None, place(k, off, pad), place(v, off, pad), None, torch.arange(T).cuda(), None)
        got = cache.cpu().numpy()
        assert (got != want).sum() == 0, f"offset {off}"


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_keys_are_the_same_bytes_anywhere(qk, interleaved):
    """Without a norm every product and sum is rounded by itself: rows off a boundary are stored as aligned ones."""
    T, nkv, D, page = 200, 4, 128, 64
    g = torch.Generator().manual_seed(4)
    k = torch.randn(T, nkv * D, generator=g).numpy()
    pos = torch.randint(0, 500, (T,), generator=g).int().cuda()
    got = []
    for off, pad in ((0, 0), (3, 5)):
        cache = qk.kv_cache_q4(-(-T // page), nkv, page, D)
        kv = place(k, off, pad)
        qk.kv_append_q4(cache, None, kv, kv, pos, torch.arange(T).cuda(), table(500, D), interleaved=interleaved)
        got.append(cache)
    assert torch.equal(*got) and qk.device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("nkv,D,rot", [(4, 128, 128), (8, 64, 32), (3, 96, 72), (2, 256, 256), (2, 256, 64), (5, 128, 0)])
def test_normed_keys_are_the_same_bytes_anywhere(qk, nkv, D, rot, interleaved, dtype):
    """A key's squares are added in one order whichever form takes its row, so its norm has the same bits."""
    T, page = 3000, 64
    g = torch.Generator().manual_seed(4)
    k = torch.randn(T, nkv * D, generator=g)
    if dtype == "bf16":
        k = k.bfloat16()
    pos, w = torch.randint(0, 500, (T,), generator=g).int().cuda(), (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    got = []
    for off, pad in ((0, 0), (3, 5)):
        cache = qk.kv_cache_q4(-(-T // page), nkv, page, D)
        buf = torch.zeros(T, nkv * D + pad, dtype=k.dtype, device="cuda")
        kv = buf[:, off:off + nkv * D]
        kv.copy_(k)
        qk.kv_append_q4(cache, None, kv, kv, pos, torch.arange(T).cuda(), table(500, rot) if rot else None, k_weight=w,
                        interleaved=interleaved)
        got.append(cache)
    assert (got[0] != got[1]).sum() == 0 and qk.device_error() == 0
