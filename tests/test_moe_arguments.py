"""Arguments of routing, experts and adapters that the binding has to refuse or take as they are meant."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_one_row_in_place(qk):
    """The first row of a longer buffer, given as y by itself and as out with the rows behind it."""
    x, A, B = torch.randn(1, 64).cuda(), torch.randn(2, 8, 64).cuda(), torch.randn(2, 48, 8).cuda()
    ids = torch.ones(1, dtype=torch.int32).cuda()
    buf = torch.randn(3, 80).cuda()
    y, behind = buf[:1, :48].clone(), buf[1:].clone()
    qk.lora(x, buf[:1, :48], A, B, ids, out=buf[:, :48])
    assert torch.equal(buf[:1, :48], qk.lora(x, y, A, B, ids)) and torch.equal(buf[1:], behind)
