"""Outputs and workspaces that a call on another stream makes for itself are that stream's memory: the current stream is
not given them while the call may still be running."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def weights(rows, K):
    from quantised_gguf_weight_gb300 import synth
    return torch.from_numpy(synth.weights("q4_k", rows, K, seed=3)).cuda()


def calls(qk):
    """name -> a call that makes its output, given a stream."""
    w, K, R = weights(256, 256), 256, 256
    x, big = torch.randn(4, K, device="cuda"), torch.randn(64, K, device="cuda")
    i32 = torch.arange(64, dtype=torch.int32).cuda()
    i64, tab = i32.long(), qk.rope_table(64, 64)
    cache = qk.kv_cache_q4(4, 2, 16, 64)
    rows = torch.randn(64, 4 * 64, device="cuda")
    kv = torch.randn(64, 2 * 64, device="cuda")
    pages, lens = torch.arange(4, dtype=torch.int32).reshape(1, 4).cuda(), torch.tensor([64], dtype=torch.int32).cuda()
    return {
        "qmatvec": lambda s: qk.qmatvec_q4_k(w, 0, R, K, x, stream=s),
        "swiglu": lambda s: qk.qmatvec_swiglu("q4_k", w, 0, R // 2, R // 2, K, x, stream=s),
        "gemm": lambda s: qk.qgemm_q4_k(w, 0, R, K, big, stream=s),
        "gemm swiglu": lambda s: qk.qgemm_swiglu("q4_k", w, 0, R // 2, R // 2, K, big, stream=s),
        "rope table": lambda s: qk.rope_table(64, 64, stream=s),
        "norm_rope": lambda s: qk.norm_rope(rows, 2, 2, 64, i32, tab, stream=s),
        "append": lambda s: qk.kv_append_q4(cache, rows, kv, kv, i32, i64, tab, stream=s),
        "read": lambda s: qk.kv_read_q4(cache, i64, stream=s),
        "attention": lambda s: qk.attn_q4(cache, rows, pages, lens, max_q=64, stream=s),
    }


NAMES = ["qmatvec", "swiglu", "gemm", "gemm swiglu", "rope table", "norm_rope", "append", "read", "attention"]


@pytest.mark.parametrize("by_handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_output_is_not_reused(qk, name, by_handle):
    call = calls(qk)[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = call(side.cuda_stream if by_handle else side)
    side.synchronize()
    tensors, wants = (got, want) if isinstance(got, tuple) else ((got,), (want,))
    assert all(torch.equal(t, w) for t, w in zip(tensors, wants))
    places, shape, dtype = {t.data_ptr() for t in tensors}, tensors[0].shape, tensors[0].dtype
    del got, tensors
    mine = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(8)]
    assert not places & {t.data_ptr() for t in mine}


def test_gemm_workspace_is_the_streams(qk, monkeypatch):
    """The GEMM's own workspace is dropped when the call returns."""
    made, empty = [], qk._empty

    def watch(*a):
        t = empty(*a)
        made.append((t.data_ptr(), t.numel(), t.dtype))
        return t

    monkeypatch.setattr(qk, "_empty", watch)
    w, x = weights(256, 256), torch.randn(64, 256, device="cuda")
    y = torch.empty(64, 256, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    qk.qgemm_q4_k(w, 0, 256, 256, x, y=y, ldy=256, stream=side)
    side.synchronize()
    assert made
    for at, n, dtype in made:
        mine = [torch.empty(n, dtype=dtype, device="cuda") for _ in range(8)]
        assert at not in {t.data_ptr() for t in mine}


def test_default_stream_by_handle(qk):
    """Handle 0 is the default stream."""
    x = torch.randn(3, 128, device="cuda")
    tab, pos = qk.rope_table(8, 64, stream=0), torch.arange(3, dtype=torch.int32).cuda()
    assert np.array_equal(tab.cpu().numpy(), qk.rope_table(8, 64).cpu().numpy())
    assert torch.equal(qk.norm_rope(x, 1, 1, 64, pos, tab, stream=0), qk.norm_rope(x, 1, 1, 64, pos, tab))
