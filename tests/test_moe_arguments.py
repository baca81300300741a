"""Arguments that the binding has to refuse or take as they are meant."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_renorm_without_a_truth_value(qk):
    """An error in asking for it is raised as it is, before anything is launched."""
    z = torch.randn(3, 16).cuda()
    with pytest.raises(RuntimeError, match="ambiguous"):
        qk.moe_route(z, 2, renorm=torch.tensor([1, 2]))
    ids, w = qk.moe_route(z, 2, renorm=torch.tensor([0]))
    assert torch.equal(w, qk.moe_route(z, 2, renorm=False)[1]) and qk.device_error() == 0


def test_interleaved_without_a_truth_value(qk):
    """The same of the rotation's order of pairs."""
    x, pos, slots = torch.randn(2, 64).cuda(), torch.zeros(2, dtype=torch.int32).cuda(), torch.arange(2).cuda()
    table, cache = qk.rope_table(4, 64), qk.kv_cache_q4(1, 1, 16, 64)
    was = cache.clone()
    with pytest.raises(RuntimeError, match="ambiguous"):
        qk.norm_rope(x, 1, 0, 64, pos, table, interleaved=torch.tensor([0, 1]))
    with pytest.raises(RuntimeError, match="ambiguous"):
        qk.kv_append_q4(cache, None, x, x, pos, slots, table, interleaved=torch.tensor([0, 1]))
    assert torch.equal(cache, was) and qk.device_error() == 0


def test_one_row_in_place(qk):
    """The first row of a longer buffer, given as y by itself and as out with the rows behind it."""
    x, A, B = torch.randn(1, 64).cuda(), torch.randn(2, 8, 64).cuda(), torch.randn(2, 48, 8).cuda()
    ids = torch.ones(1, dtype=torch.int32).cuda()
    buf = torch.randn(3, 80).cuda()
    y, behind = buf[:1, :48].clone(), buf[1:].clone()
    qk.lora(x, buf[:1, :48], A, B, ids, out=buf[:, :48])
    assert torch.equal(buf[:1, :48], qk.lora(x, y, A, B, ids)) and torch.equal(buf[1:], behind)


def test_adapters_with_a_workspace_of_ones_own(qk):
    """A buffer for more, and with anything in it, gives the bits that one made by the call gives."""
    for T, rank, dtype in ((1, 64, torch.float16), (40, 16, torch.bfloat16), (300, 100, torch.float32)):
        x, y = torch.randn(T, 96).to(dtype).cuda(), torch.randn(T, 40).to(dtype).cuda()
        A, B = torch.randn(3, rank, 96).to(dtype).cuda(), torch.randn(3, 40, rank).to(dtype).cuda()
        ids = (torch.arange(T) % 4 - 1).int().cuda()
        ws = qk.lora_workspace(2 * T, rank)
        ws.fill_(0xff)
        assert torch.equal(qk.lora(x, y, A, B, ids, workspace=ws), qk.lora(x, y, A, B, ids))
    assert qk.device_error() == 0


@pytest.mark.parametrize("T", [1, 12, 40, 300])
def test_experts_in_place(qk, T):
    """y is x, or rows that lie across x's, in calls of every form."""
    from tests.test_moe_ffn import Case, bits
    for xt in ("f32", "bf16"):
        c = Case(qk, T, 9, 3, 256, 64, 256, "q4_k", "q8_0", xt, seed=T)
        want = c.call()
        x = c.x.cuda()
        assert c.call(x=x, y=x).data_ptr() == x.data_ptr() and torch.equal(bits(x), bits(want))
        buf = torch.zeros(T + 1, 256, dtype=c.x.dtype, device="cuda")
        buf[:T] = c.x.cuda()
        y = buf.reshape(-1)[128:128 + T * 256].reshape(T, 256)
        c.call(x=buf[:T], y=y)
        assert torch.equal(bits(y), bits(want))
    assert qk.device_error() == 0
