"""What lies between an adapter's two products: A x is held to 22 bits, to 16 only with bf16 adapters and outputs."""
import pytest
import torch

from tests import moe_oracle as mo

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("wt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("yt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,rank,N", [(1, 16, 64), (40, 16, 64), (40, 16, 67), (300, 64, 40), (300, 100, 40)])
def test_ranks_that_nearly_cancel(qk, xt, wt, yt, T, rank, N):
    """Two ranks whose values differ in the 18th to 20th bit, beside columns of B that take one from the other.  Everything
    else is exact: A x is 1 + (1 + k / 128) 2^-9, and 7 2^-20 more in one of them, all sums are whole multiples of 2^-20
    below 2^2, B is a power of two.  A x to 2^-22 of itself in each, then, and a product's sum cut at 2^-23 of its
    largest part (< 2), leave an error below 2 2^-22 2 + 2 2^-23, of b (2^-17 for 2^-22 with bf16 adapters and outputs)."""
    n, K = 5, 64
    x = torch.zeros(T, K)
    x[:, 0], x[:, 9], x[:, 41] = 1, 2.0 ** -9, 2.0 ** -20
    A, B = torch.zeros(n, rank, K), torch.zeros(n, N, rank)
    k = torch.tensor([1.0, 37, 64, 99, 126])
    for r in (3, 12):
        A[:, r, 0], A[:, r, 9] = 1, 1 + k / 128
    A[:, 12, 41] = 7
    b = 2.0 ** (torch.arange(N) % 4).float()
    B[:, :, 12], B[:, :, 3] = b, -b
    ids = (torch.arange(T) % (n + 1) - 1).int()
    if T == 1:
        ids[0] = 1
    scale = 2.0 ** 12
    x, A, B = x.to(mo.TORCH[xt]), A.to(mo.TORCH[wt]), B.to(mo.TORCH[wt])
    assert float(x[0, 41]) == 2.0 ** -20 and float(A[3, 12, 9]) == 1 + 99 / 128
    out = qk.lora(x.cuda(), torch.zeros(T, N, dtype=mo.TORCH[yt]).cuda(), A.cuda(), B.cuda(), ids.cuda(),
                  scales=torch.full((n,), scale).cuda()).double().cpu()
    want = (ids >= 0)[:, None] * (b * 7 * 2.0 ** -20 * scale).double()
    held = 2.0 ** -17 if wt == yt == "bf16" else 2.0 ** -22
    bound = (ids >= 0)[:, None] * (b * scale).double() * (2 * held * 2 + 2 * 2.0 ** -23)
    bound = bound + mo.HALF_STEP[yt] * (want + bound)
    assert torch.all((out - want).abs() <= bound), ((out - want).abs() / bound.clamp(min=1e-30)).max()
    assert qk.device_error() == 0
