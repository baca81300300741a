"""The many-token form of the experts' products: thread blocks that take several items, one after the other."""
import numpy as np
import pytest
import torch

from tests import moe_oracle as mo
from tests.test_moe_ffn import Case, bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("N", [200, 130])
def test_a_token_keeps_its_own_scale(qk, xt, N):
    """Tokens far apart in size, next to one another in a thread block's items: 180 experts of 20 tokens are more items
    than there are pairs of thread blocks, and the last tile of N rows leaves lanes without a row."""
    E, per = 180, 20
    T = E * per // 2
    ids = np.random.default_rng(1).permutation(np.repeat(np.arange(E), per)).reshape(T, 2)
    c = Case(qk, T, E, 2, 256, 72, N, "q4_k", "q8_0", xt, "f32", seed=3, ids=ids)
    x = c.xv * 2.0 ** np.random.default_rng(2).integers(-15, 16, (T, 1))
    c.x, c.xv = mo.as_rows(x, xt)
    y = c.call()
    c.check(y, range(0, T, 3))
    for _ in range(4):
        assert torch.equal(bits(y), bits(c.call()))
    assert qk.device_error() == 0
