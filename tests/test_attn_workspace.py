"""The size of the attention's workspace: what a call of these sizes and any length can make use of."""
import pytest
import torch

from quantised_gguf_weight_gb300 import build as qbuild


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    from quantised_gguf_weight_gb300 import qk as _qk
    return _qk.load()


@pytest.mark.parametrize("B,nq,nkv,D,max_q", [(1, 32, 8, 128, 1), (16, 14, 2, 64, 1), (1, 8, 1, 256, 4), (4, 32, 8, 128, 64),
                                              (1, 32, 8, 128, 300), (2, 4, 4, 96, 40), (64, 32, 8, 128, 1), (400, 32, 8, 128, 1)])
def test_length_zero_is_any_length(lib, B, nq, nkv, D, max_q):
    f = lib.qk_attn_q4_workspace_bytes
    lengths = [f(B, nq, nkv, D, max_q, n) for n in (1, 100, 257, 700, 1500, 3000, 10001, 40000, 131072, 1 << 20)]
    assert f(B, nq, nkv, D, max_q, 0) == max(lengths)
    assert f(B, nq, nkv, D, max_q, -1) == 0
    assert (max(lengths) > 0) == (B < 64)


@pytest.mark.gpu
@pytest.mark.parametrize("max_q", [1, 64])
def test_default_workspace_splits(qk, max_q):
    """A workspace made without a length is large enough for parts, and a long sequence leaves some in it."""
    D, nkv, nq, page, L = 128, 2, 8, 64, 6000
    pages = -(-L // page)
    cache = qk.kv_cache_q4(pages, nkv, page, D)
    g = torch.Generator().manual_seed(1)
    kv = torch.randn(L, nkv * D, generator=g).cuda()
    qk.kv_append_q4(cache, None, kv, kv, None, torch.arange(L).cuda(), None)
    q = torch.randn(max_q, nq * D, generator=g).cuda()
    tab, lens = torch.arange(pages, dtype=torch.int32).reshape(1, -1).cuda(), torch.tensor([L], dtype=torch.int32).cuda()
    ws = qk.attn_q4_workspace(1, nq, nkv, D, max_q)
    out = qk.attn_q4(cache, q, tab, lens, max_q=max_q, workspace=ws)
    assert ws.numel() == qk.attn_q4_workspace(1, nq, nkv, D, max_q, L).numel() and ws.any()
    assert torch.equal(out, qk.attn_q4(cache, q, tab, lens, max_q=max_q, workspace=qk.attn_q4_workspace(1, nq, nkv, D, max_q, L)))
    assert qk.device_error() == 0
