"""Argument checks of routing, the experts' products and the adapters (no GPU): the status comes before any launch."""
import ctypes

import pytest
import torch

from quantised_gguf_weight_gb300 import build as qbuild

FAKE = 0x10000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def qk():
    qbuild.build()
    from quantised_gguf_weight_gb300 import qk as _qk
    _qk.load()
    return _qk


def caller(fn, ok):
    return lambda **kw: fn(*dict(ok, **kw).values())


def test_route_statuses(qk):
    call = caller(qk.load().qk_moe_route,
                  dict(logits=FAKE, ld=0, type=0, T=3, E=64, k=8, score=0, bias=None, groups=8, top_groups=4, group_top=2, renorm=1,
                       scale=1.0, ids=FAKE, weights=FAKE, stream=None))
    assert call(logits=None) == 1 and call(ids=None) == 1 and call(weights=None) == 1
    for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(k=33), dict(groups=0), dict(groups=7), dict(top_groups=0), dict(top_groups=9),
               dict(group_top=0), dict(group_top=3), dict(groups=64, top_groups=8), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(ld=63)):
        assert call(**kw) == 2, kw
    assert call(logits=FAKE + 2) == 3 and call(ids=FAKE + 2) == 3 and call(weights=FAKE + 1) == 3 and call(bias=FAKE + 2) == 3
    assert call(type=3) == 10 and call(score=2) == 10 and call(type=1, logits=FAKE + 1) == 3
    assert call(E=2048, groups=1, top_groups=1) == 8 and call(E=64, k=40, groups=1, top_groups=1) == 8 and call(T=1 << 40) == 8
    assert call(E=128, groups=64, top_groups=8) == 8
    assert call(T=0, logits=None) == 0


def weights(qk, w=FAKE, fmt=1, off=0, per=0):
    return ctypes.pointer(qk._ExpertWeights(w, fmt, off, per))


def test_ffn_statuses(qk):
    g = weights(qk)
    call = caller(qk.load().qk_moe_ffn,
                  dict(gate=g, up=g, down=g, E=8, K=256, F=64, N=256, x=FAKE, ldx=0, x_type=0, T=2, ids=FAKE, weights=FAKE, k=2,
                       y=FAKE, ldy=0, y_type=0, ws=FAKE, bytes=1 << 40, stream=None))
    for n in ("gate", "up", "down", "x", "ids", "weights", "y"):
        assert call(**{n: None}) == 1, n
    assert call(down=weights(qk, None)) == 1
    for kw in (dict(E=0), dict(K=0), dict(F=0), dict(N=-1), dict(T=-1), dict(k=0), dict(ldx=255), dict(ldy=255),
               dict(up=weights(qk, off=-1)), dict(gate=weights(qk, per=63)), dict(down=weights(qk, per=255))):
        assert call(**kw) == 2, kw
    assert call(gate=weights(qk, FAKE + 2)) == 3 and call(down=weights(qk, FAKE + 1, 0)) == 3 and call(x=FAKE + 2) == 3
    assert call(y=FAKE + 1, y_type=2) == 3 and call(ids=FAKE + 2) == 3 and call(weights=FAKE + 2) == 3
    assert call(ws=None) == 7 and call(ws=FAKE + 16) == 7 and call(bytes=100) == 7
    need = qk.load().qk_moe_ffn_workspace_bytes(2, 2, 8, 256, 64, 256)
    assert need > 0
    assert call(E=1025) == 8 and call(K=1 << 25, ldx=0) == 8 and call(T=1 << 28) == 8
    assert call(gate=weights(qk, off=1 << 62)) == 8 and call(gate=weights(qk, per=1 << 40)) == 8
    assert call(x_type=3) == 10 and call(y_type=-1) == 10 and call(gate=weights(qk, fmt=3), up=weights(qk, fmt=3)) == 10
    assert call(up=weights(qk, fmt=0)) == 10
    assert call(T=0, x=None) == 0


def test_ffn_strict_blocks(qk):
    g = weights(qk)
    args = [g, g, g, 8, 300, 256, 256, FAKE, 0, 0, 2, FAKE, FAKE, 2, FAKE, 0, 0, None, 0, None]
    assert qk.load().qk_moe_ffn(*args) == 7
    was = qk.set_strict_blocks(True)
    try:
        assert qk.load().qk_moe_ffn(*args) == 2
        args[4] = 256
        assert qk.load().qk_moe_ffn(*args) == 7
    finally:
        qk.set_strict_blocks(was)


def test_workspace_of_nothing(qk):
    f = qk.load().qk_moe_ffn_workspace_bytes
    for a in ((0, 2, 8, 256, 64, 256), (2, 0, 8, 256, 64, 256), (2, 2, 0, 256, 64, 256), (2, 2, 8, 0, 64, 256), (1 << 40, 2, 8, 256, 64, 256)):
        assert f(*a) == 0
    sizes = [f(T, 2, 8, 256, 64, 256) for T in (1, 2, 3, 10, 100, 1000)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_lora_statuses(qk):
    call = caller(qk.load().qk_lora,
                  dict(x=FAKE, ldx=0, x_type=0, T=3, K=64, A=FAKE, B=FAKE, w_type=1, n=2, rank=8, N=64, ids=FAKE, scales=None, y=FAKE,
                       ldy=0, out=2 * FAKE, ldo=0, y_type=0, ws=None, bytes=0, stream=None))
    for n in ("x", "A", "B", "ids", "y", "out"):
        assert call(**{n: None}) == 1, n
    for kw in (dict(T=-1), dict(K=0), dict(N=0), dict(n=0), dict(rank=0), dict(ldx=63), dict(ldy=63), dict(ldo=63), dict(out=FAKE, ldo=80)):
        assert call(**kw) == 2, kw
    assert call(x=FAKE + 2) == 3 and call(A=FAKE + 1) == 3 and call(B=FAKE + 1) == 3 and call(ids=FAKE + 2) == 3
    assert call(scales=FAKE + 2) == 3 and call(y=FAKE + 2) == 3 and call(out=FAKE + 3) == 3
    assert call(rank=257) == 8 and call(T=1 << 40) == 8 and call(K=1 << 25) == 8 and call(N=1 << 25) == 8
    assert call(x_type=3) == 10 and call(w_type=-1) == 10 and call(y_type=7) == 10
    assert call(T=0, x=None) == 0
    f = qk.load().qk_lora_workspace_bytes
    assert f(0, 8) == f(4096, 0) == f(4096, 257) == 0 and f(4096, 64) == 4096 * 64 * 4 and f(4096, 65) == 4096 * 128 * 4 and f(1, 8) == 64


def test_binding_refuses_host_tensors(qk):
    z, i = torch.zeros(2, 8), torch.zeros(2, 2, dtype=torch.int32)
    w = qk.ExpertWeights("q8_0", torch.zeros(8 * 34, dtype=torch.uint8))
    for f in (lambda: qk.moe_route(z, 2), lambda: qk.moe_ffn(z, i, torch.zeros(2, 2), w, w, w, 1, 8),
              lambda: qk.lora(z, z, torch.zeros(1, 2, 8), torch.zeros(1, 8, 2), i[:, 0])):
        with pytest.raises((ValueError, RuntimeError)):
            f()
    with pytest.raises(ValueError):
        qk.moe_route(z, 2, score="tanh")
    with pytest.raises(ValueError):
        qk.moe_ffn(z, i, torch.zeros(2, 2), qk.ExpertWeights("q5_k", w.w), w, w, 1, 8)
