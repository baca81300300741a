"""Calls from several host threads at once, each with its stream, output and workspace.  ctypes lets go of Python's lock during a
call; every status has to be QK_OK and every output what one thread gets."""
import os
import subprocess
import sys
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


FIRST = '''
import ctypes, sys, torch
sys.path.insert(0, sys.argv[1])
from quantised_gguf_weight_gb300 import qk, synth
from tests.test_host_threads import at_once
lib, E, T, K, F = qk.load(), 2, 64, 256, 64
w = torch.from_numpy(synth.weights("q8_0", E * K, K, seed=1)).cuda()
e = [qk._ExpertWeights(w.data_ptr(), 0, 0, 0) for _ in range(3)]
calls, keep = [], []
for i in range(8):
    x, y = torch.randn(T, K).cuda(), torch.empty(T, K).cuda()
    ids, p, ws = (torch.arange(T) % E).int().cuda(), torch.ones(T).cuda(), qk.moe_ffn_workspace(T, 1, E, K, F)
    s = torch.cuda.Stream()
    keep.append((x, y, ids, p, ws, s))
    a = (*map(ctypes.byref, e), E, K, F, K, x.data_ptr(), 0, 0, T, ids.data_ptr(), p.data_ptr(), 1, y.data_ptr(), 0, 0, ws.data_ptr(),
         ws.numel(), s.cuda_stream)
    calls.append(lambda a=a: lib.qk_moe_ffn(*a))
torch.cuda.synchronize()
print(at_once(calls, 1))
'''


def test_first_calls_at_once(qk):
    """A process whose first calls, which look up the driver's tensor maps, come from eight threads."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", FIRST, root], cwd=root, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        assert r.stdout.strip() == str([{0}] * 8)


def test_products_of_two_widths(qk):
    """The same of the GEMV, whose shared memory goes with K: both threads' first calls of their size."""
    from quantised_gguf_weight_gb300 import synth
    code = FIRST.split("lib, E")[0] + '''
lib, calls, keep = qk.load(), [], []
for i, K in enumerate((8192, 256, 4096, 512)):
    w, x, y = torch.from_numpy(synth.weights("q4_k", 64, K, seed=1)).cuda(), torch.randn(1, K).cuda(), torch.empty(1, 64).cuda()
    s = torch.cuda.Stream()
    keep.append((w, x, y, s))
    calls.append(lambda a=(w.data_ptr(), 0, 64, K, x.data_ptr(), 1, y.data_ptr(), 0, s.cuda_stream): lib.qmatvec_q4_k(*a))
torch.cuda.synchronize()
print(at_once(calls, 1))
'''
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", code, root], cwd=root, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        assert r.stdout.strip() == str([{0}] * 4)
