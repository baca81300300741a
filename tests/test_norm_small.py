"""Norms of rows so small that their mean square is subnormal in fp32, without an eps: the rows come out at their weights'
size, in the wide form and in the general one."""
import numpy as np
import pytest
import torch

from tests import kv4_oracle as ko
from tests.test_attn_ops import close, f64, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("off", [0, 1])       # 1 rules out wide loads
@pytest.mark.parametrize("D", [64, 96, 128, 256, 80])
@pytest.mark.parametrize("size", [1e-17, 3e-20, 1e-20])
def test_small_rows(qk, size, D, off):
    """A square is rounded to 2^-149, half of that off at most: 2^-150 / size^2 of a row's mean, half of it after the
    square root, besides the 2^-19 of test_norm_rope."""
    T, heads = 9, 3
    buf = rand(D, T, heads * D + 4, scale=size)
    x = buf[:, off:off + heads * D]
    w = 1 + rand(2, D, scale=0.3)
    y = qk.norm_rope(x, heads, 0, D, None, None, q_weight=w, eps=0.0)
    ref, mag = ko.norm_rope(f64(x).reshape(T, heads, D), f64(w), 0.0, None, None, 0, False)
    close(y, ref.reshape(T, -1), ((2.0 ** -19 + 2.0 ** -150 / size ** 2) * mag + 2.0 ** -24).reshape(T, -1), "norm")
    assert np.isfinite(f64(y)).all()
