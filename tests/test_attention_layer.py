"""The example's layer: its steps against plain 64-bit attention over what its cache holds."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_steps(example):
    qk = example.qk
    layer = example.random_layer(width=512, n_q=6, n_kv=2, head_dim=64, n_pages=24, page_tokens=16, max_len=256)
    pages = example.Pages(24, 16, 2, 160)
    g = torch.Generator().manual_seed(7)
    D, rep, q_rows, kv_rows = 64, 3, 6 * 64, 2 * 64
    for new in ([70, 33], [1, 1], [1, 40], [3, 0], [1, 1]):
        x = torch.randn(sum(new), 512, generator=g).cuda()
        step = pages.extend(new)
        got = layer.step(x, **step)
        qkv = layer._matmul(layer.w_qkv, q_rows + 2 * kv_rows, 512, x)
        q = qk.norm_rope(qkv[:, :q_rows], 6, 0, D, step["positions"], layer.table, q_weight=layer.q_norm).double()
        mixed, at = torch.empty_like(q), 0
        for b, n in enumerate(new):
            L = pages.lens[b]
            j = torch.arange(L)
            slots = (pages.table[b][j // 16].long() * 16 + j % 16).cuda()
            k, v = (t.double().reshape(L, 2, D) for t in qk.kv_read_q4(layer.cache, slots, dtype=torch.float32))
            z = torch.einsum("thrd,khd->thrk", q[at:at + n].reshape(n, 2, rep, D), k) * D ** -0.5
            seen = torch.arange(L).cuda() <= (L - n + torch.arange(n).cuda())[:, None]
            p = z.masked_fill(~seen[:, None, None], -torch.inf).softmax(-1)
            mixed[at:at + n] = torch.einsum("thrk,khd->thrd", p, v).reshape(n, q_rows)
            at += n
        want = layer._matmul(layer.w_out, 512, q_rows, mixed.float().contiguous())
        # the attention's 1e-5; the matrix products of more than 8 rows round their inputs to bf16
        limit = 1e-4 if sum(new) <= qk.MAX_BATCH else 2.0 ** -8
        assert ((got - want).norm() / want.norm()).item() <= limit
        assert qk.device_error() == 0
