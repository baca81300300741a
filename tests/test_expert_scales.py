"""Rows of weights whose blocks' scales lie far apart, and rows of h near the least numbers: the header's bounds."""
import numpy as np
import pytest
import torch

from oracle import oracle as orc
from tests import moe_oracle as mo
from tests.test_moe_ffn import Case

pytestmark = pytest.mark.gpu

PER, SIZE = {"q8_0": 32, "q4_k": 256, "q6_k": 256}, {"q8_0": 34, "q4_k": 144, "q6_k": 210}
D_AT = {"q8_0": [0], "q4_k": [0, 2], "q6_k": [208]}


def far_apart(c, name, fmt, rows, up):
    """The first 256 columns' scales up by 2^up, the others' down by 2^-3 (fp16's subnormals among them)."""
    b = c.b[name].w.cpu().numpy().reshape(c.E * rows, -1, SIZE[fmt]).copy()
    first = 256 // PER[fmt]
    for at in D_AT[fmt]:
        d = b[..., at:at + 2].copy().view(np.float16)[..., 0].astype(np.float64)
        d[:, :first] *= 2.0 ** up
        d[:, first:] *= 2.0 ** -3
        assert np.abs(d).max() < 65504
        b[..., at:at + 2] = d.astype(np.float16)[..., None].view(np.uint8)
    b = b.reshape(c.E * rows, -1)
    c.b[name] = c.qk.ExpertWeights(fmt, torch.from_numpy(b).cuda())
    c.w[name] = orc.decode(fmt, b, c.K, n_rows_total=c.E * rows).reshape(c.E, rows, c.K)
    # what the many-token form's weights may be off by
    w, d = np.abs(c.w[name]), [np.abs(b.reshape(c.E, rows, -1, SIZE[fmt])[..., at:at + 2].copy().view(np.float16)[..., 0].astype(np.float64))
                               for at in D_AT[fmt]]
    if fmt == "q4_k":
        made = w + 2 * np.repeat(63 * d[1], 256, axis=2)[..., :c.K]
        largest = (945 * d[0] + 63 * d[1]).max(2)
    else:
        made, largest = w, ({"q8_0": 128, "q6_k": 4096}[fmt] * d[0]).max(2)
    low = 2.0 ** -29 * largest[..., None]
    fine = 2.0 ** -22 * w + 2.0 ** -24 * made + low
    return fine, 2.0 ** -11 * (1 + 2.0 ** -10) * (w + made) + low


@pytest.mark.parametrize("fmt,up", [("q8_0", 14), ("q4_k", 12), ("q6_k", 12)])
@pytest.mark.parametrize("T,k,E", [(2, 1, 2), (14, 3, 3), (48, 1, 2)])
@pytest.mark.parametrize("xt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("one", [False, True])
def test_blocks_far_apart(qk, fmt, up, T, k, E, xt, one):
    """No token has anything in the columns of the large blocks: the small ones are all of gate and up.  one: each token has
    one column, so that gate and up are single weights and the bound all but theirs."""
    c = Case(qk, T, E, k, 512, 40, 64, fmt, "q8_0", xt, seed=T)
    ids = np.stack([np.arange(k) + (0 if k == E else t % (E - k + 1)) for t in range(T)]).astype(np.int32)
    c.ids, c.xv = ids, c.xv * (np.arange(512) >= 256)
    if one:
        c.xv *= np.arange(512) == 256 + 5 * np.arange(T)[:, None]
    c.x = torch.from_numpy(c.xv).to(mo.TORCH[xt])
    dw = [far_apart(c, n, fmt, 40, up) for n in ("gate", "up")]
    y = c.call()
    fine = [d[xt == "bf16"] for d in dw] + [(2.0 ** -11 if xt == "bf16" else 2.0 ** -21) * np.abs(c.w["down"]) + 2.0 ** -29 * np.abs(c.w["down"]).max()]
    want, bound = mo.ffn(c.xv, c.ids, c.p, c.w["gate"], c.w["up"], c.w["down"], xt, xt, fine if T >= 16 else None)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= bound)
    assert qk.device_error() == 0


def test_h_near_the_least_numbers(qk):
    """One token, one column of x and one expert: g = 2^-60, u = 2^-60 d q and so h = 2^-61 u are exact, 18 bits of 2^-121.
    Down has one quant of 1 in each sub-block; column f of h is read through row f, whatever it is scaled by."""
    K, F, N = 32, 64, 64
    gate = np.zeros((F, 34), np.uint8)
    gate[:, :2], gate[:, 2] = np.array([1.0], np.float16).view(np.uint8), 1
    up = gate.copy()
    q = 65 + np.arange(F) % 60
    up[:, :2], up[:, 2] = np.array([1 + 1023 / 1024], np.float16).view(np.uint8), q
    down = np.zeros((N, 144), np.uint8)
    down[:, :2] = np.array([1.0], np.float16).view(np.uint8)
    down[:, 4:6] = 1                                           # scales of sub-blocks 0 and 1
    for f in range(F):
        down[f, 16 + f % 32] = 1 << 4 * (f // 32)
    w = [qk.ExpertWeights(n, torch.from_numpy(b).cuda()) for n, b in (("q8_0", gate), ("q8_0", up), ("q4_k", down))]
    assert np.array_equal(orc.decode("q4_k", down, F, n_rows_total=N), np.eye(F))
    x = torch.zeros(1, K)
    x[0, 0] = 2.0 ** -60
    y = qk.moe_ffn(x.cuda(), torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.ones(1, 1).cuda(), *w, 1, F, N)
    want = 2.0 ** -121 * (1 + 1023 / 1024) * q
    err = np.abs(y[0].double().cpu().numpy() - want)
    assert np.all(err <= 2.0 ** -138 + 2.0 ** -24 * want) and qk.device_error() == 0
