"""The example's layer: each operator of a step against the formulas in 64 bits, on what the step gave it."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import oracle as orc
from tests import moe_oracle as mo

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def f64(t):
    return t.double().cpu().numpy()


def test_steps(example):
    qk = example.qk
    E, width, hidden = 8, 512, 128
    layer = example.random_layer(width=width, hidden=hidden, n_experts=E, top_k=2, n_adapters=4, rank=8, max_tokens=300)
    w = [orc.decode(fmt, p.w.cpu().numpy(), cols, n_rows_total=E * rows).reshape(E, rows, cols)
         for p, fmt, rows, cols in ((layer.gate, "q4_k", hidden, width), (layer.up, "q4_k", hidden, width), (layer.down, "q6_k", width, hidden))]
    g = torch.Generator().manual_seed(3)
    for T in (1, 5, 40, 300):
        x = torch.randn(T, width, generator=g).cuda()
        adapters = torch.randint(-1, 4, (T,), generator=g).int().cuda()
        few = T <= qk.MAX_BATCH
        plain = (qk.qmatvec_q4_k if few else qk.qgemm_q4_k)(layer.w_in, 0, width, width, x)
        h = layer.project(x, adapters)
        want, bound = mo.lora(f64(x), f64(plain), f64(layer.A), f64(layer.B), f64(adapters).astype(int), f64(layer.scales), "f32")
        assert np.all(np.abs(f64(h) - want) <= bound)
        logits, ids, weights = layer.route(h)
        want_ids, want_weights = mo.route(f64(logits), 2, "softmax", None, 1, 1, 1, True, 1.0)
        assert np.array_equal(ids.cpu().numpy(), want_ids) and np.all(np.abs(f64(weights) - want_weights) <= 1e-6)
        rows = list(range(0, T, 7))
        y = layer.experts(h, ids, weights)
        want, bound = mo.ffn(f64(h)[rows], want_ids[rows], f64(weights)[rows], *w, "f32", "f32")
        assert np.all(np.abs(f64(y)[rows] - want) <= bound)
        assert torch.equal(layer.step(x, adapters), h + y)
        assert qk.device_error() == 0


def test_a_step_in_a_graph(example):
    """All operators of a step captured, and replayed with other rows, adapters and so other experts."""
    qk = example.qk
    layer = example.random_layer(width=512, hidden=128, n_experts=8, top_k=2, n_adapters=4, rank=8, max_tokens=64)
    g = torch.Generator().manual_seed(4)
    for T in (2, 33):
        x = torch.randn(T, 512, generator=g).cuda()
        adapters = torch.randint(-1, 4, (T,), generator=g).int().cuda()
        layer.step(x, adapters)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = layer.step(x, adapters)
        for _ in range(3):
            x.copy_(torch.randn(T, 512, generator=g)), adapters.copy_(torch.randint(-1, 4, (T,), generator=g))
            graph.replay()
            assert torch.equal(y, layer.step(x, adapters))
    assert qk.device_error() == 0
