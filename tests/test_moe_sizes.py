"""Sizes of workspaces, and calls whose arguments were taken wrongly (no GPU)."""
import random

from tests.test_moe_abi import FAKE, caller, qk  # noqa: F401


def test_a_workspace_serves_smaller_calls(qk):
    """A buffer for some sizes is enough for every call of at most these, ids that repeat in a token among them."""
    f = qk.load().qk_moe_ffn_workspace_bytes
    assert f(16, 8, 1, 64, 32, 64) >= f(15, 8, 1, 64, 32, 64)
    rng = random.Random(1)
    for _ in range(20000):
        big = [rng.choice([1, 3, 15, 16, 17, 24, 25, 40, 1000]), rng.choice([1, 2, 8, 25, 64]), rng.choice([1, 2, 8, 64, 1024]),
               *(rng.choice([1, 64, 128, 129, 256, 300, 1000, 8192, 8193, 9000]) for _ in range(3))]
        small = [v if rng.random() < 0.4 else rng.randint(1, v) for v in big]
        assert f(*small) <= f(*big), (small, big)


def test_workspace_sizes_that_no_call_has(qk):
    """Sizes that a call refuses as too large have no workspace; the largest that it takes have one beyond 2^32."""
    f = qk.load().qk_moe_ffn_workspace_bytes
    for a in ((1 << 28, 2, 8, 256, 64, 256), (2, 2, 1025, 256, 64, 256), (2, 2, 8, (1 << 24) + 1, 64, 256),
              (2, 2, 8, 256, (1 << 24) + 1, 256), (2, 2, 8, 256, 64, (1 << 24) + 1),
              ((1 << 31) - 1, 1, 8, (1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1)):
        assert f(*a) == 0, a
    assert f(1 << 28, 1, 1024, 1 << 24, 1 << 24, 1 << 24) > 1 << 52


def test_one_row_in_place_has_no_stride(qk):
    """A single token's row may be given with any distance to the next."""
    call = caller(qk.load().qk_lora,
                  dict(x=FAKE, ldx=0, x_type=0, T=1, K=64, A=FAKE, B=FAKE, w_type=1, n=2, rank=8, N=64, ids=None, scales=None, y=FAKE,
                       ldy=0, out=FAKE, ldo=80, y_type=0, ws=None, bytes=0, stream=None))
    assert call() == 1 and call(ldo=0) == 1           # only the ids are missing
    assert call(T=2) == 2 and call(ldo=63) == 2


def test_adapters_workspace(qk):
    """A buffer for some tokens and ranks serves fewer of either."""
    sizes = [[qk.lora_workspace(T, r, "cpu").numel() for r in range(1, 257)] for T in (1, 2, 15, 16, 300, 4096)]
    assert all(a <= b for row in sizes for a, b in zip(row, row[1:]))
    assert all(a <= b for m, n in zip(sizes, sizes[1:]) for a, b in zip(m, n))
    assert sizes[5][63] == 4096 * 64 * 4 and qk.lora_workspace(0, 8, "cpu").numel() == 256
