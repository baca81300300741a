"""Calls from several host threads at once, each with its stream, output and workspace.  ctypes lets go of Python's lock during a
call; every status has to be QK_OK and every output what one thread gets."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def at_once(calls, times):
    """calls: functions that return a status; each thread repeats its own.  The statuses that came."""
    seen, gate = [set() for _ in calls], threading.Barrier(len(calls))

    def loop(i):
        gate.wait()
        for _ in range(times):
            seen[i].add(calls[i]())

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return seen


def test_adapters_of_two_ranks(qk):
    """One kernel, with more shared memory for one thread's rank than for the other's."""
    K, N, T = 64, 64, 16
    calls, outs = [], []
    for rank in (256, 64, 200, 40):
        x, y, out = (torch.randn(T, K).cuda() for _ in range(3))
        A, B = torch.randn(2, rank, K).cuda(), torch.randn(2, N, rank).cuda()
        ids = (torch.arange(T) % 3 - 1).int().cuda()
        s = torch.cuda.Stream()
        want = qk.lora(x, y, A, B, ids, workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
        outs.append((out, want, x, y, A, B, ids, s))
        args = (x.data_ptr(), 0, 0, T, K, A.data_ptr(), B.data_ptr(), 0, 2, rank, N, ids.data_ptr(), None, y.data_ptr(), 0, out.data_ptr(),
                0, 0, None, 0, s.cuda_stream)
        calls.append(lambda args=args: qk.load().qk_lora(*args))
    torch.cuda.synchronize()
    assert at_once(calls, 1500) == [{0}] * 4
    assert all(torch.equal(o[0], o[1]) for o in outs) and qk.device_error() == 0
