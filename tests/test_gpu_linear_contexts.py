"""Threads and driver contexts that call the tensor-map kernels: a thread without a context gets the
device's primary one, a thread with one of its own keeps it (in a process of its own, since contexts
outlive a failing test).  And the kernels' waits, which end when nothing arrives."""
import os
import subprocess
import sys
import time

import pytest
import torch

import sparse_mixture_experts_26_b200 as moe

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HEAD = """
import ctypes, threading, torch
import sparse_mixture_experts_26_b200 as moe
cu = ctypes.CDLL("libcuda.so.1")
P = ctypes.c_void_p
def ok(code):
    assert code == 0, code
def current():
    c = P()
    ok(cu.cuCtxGetCurrent(ctypes.byref(c)))
    return c.value
def in_thread(f):
    errors = []
    def body():
        try:
            f()
        except BaseException as e:
            errors.append(repr(e))
    t = threading.Thread(target=body)
    t.start()
    t.join()
    assert not errors, errors
torch.cuda.init()
x = torch.ones(5, 64, device="cuda").bfloat16()
W = torch.ones(1, 40, 64, device="cuda").bfloat16()
torch.cuda.synchronize()
"""

LOST = """
def body():
    ws = moe.alloc_grouped_linear_workspace(5, 64, 40, 1)
    for _ in range(3):
        y = torch.zeros(5, 40, dtype=torch.bfloat16, device="cuda")
        stream = torch.cuda.current_stream()
        ok(cu.cuCtxSetCurrent(None))
        assert current() is None
        code = moe._lib.moe_grouped_linear(x.data_ptr(), None, W.data_ptr(), None, None, 5, 64, 40,
                                           1, 0, 1, 1, y.data_ptr(), ws.data_ptr(), ws.numel(),
                                           stream.cuda_stream)
        assert code == 0, code
        torch.cuda.synchronize()
        assert bool((y == 64).all())
in_thread(body)
"""

# The call of the second thread ends where its tensor map is refused (a stride of 2^41 bytes), before
# anything is launched; that the driver refuses it is checked first.
OWN = """
def body():
    ctx = P()
    ok(cu.cuCtxCreate_v2(ctypes.byref(ctx), 0, 0))
    try:
        assert current() == ctx.value
        n = 1 << 20
        m = (ctypes.c_uint64 * 17)()
        at = (ctypes.addressof(m) + 63) // 64 * 64
        u64, u32 = ctypes.c_uint64, ctypes.c_uint32
        code = cu.cuTensorMapEncodeTiled(P(at), 9, 3, P(n), (u64 * 3)(n, n, 1),
                                         (u64 * 2)(2 * n, 2 * n * n), (u32 * 3)(64, 128, 1),
                                         (u32 * 3)(1, 1, 1), 0, 3, 3, 0)
        assert code == 1, code
        code = moe._lib.moe_grouped_linear(n, None, n, None, None, 1, n, n, 1, 0, 1, 1, n, n,
                                           1 << 60, None)
        assert code == 1, code
        assert current() == ctx.value
    finally:
        cu.cuCtxDestroy_v2(ctx)
in_thread(body)
"""


@pytest.mark.parametrize("body", [LOST, OWN], ids=["a_thread_that_lost_its_context",
                                                   "a_thread_with_its_own_context"])
def test_contexts_of_calling_threads(body):
    run = subprocess.run([sys.executable, "-c", HEAD + body + "print('done')"], cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "done", run.stderr


def test_the_sleeping_wait_gives_up_too():
    """The self-test's barrier is waited for twice, by polling and asleep, each up to the limit."""
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    moe.moe_selftest_wait_timeout(ws, 0.01)  # the library is loaded
    t0 = time.perf_counter()
    assert moe.moe_selftest_wait_timeout(ws, 0.5) == (2, 2)
    assert 1.0 <= time.perf_counter() - t0 < 5.0
    assert moe.moe_device_status(ws) & 1 and moe.moe_device_status(ws) == 0
    assert not bool(ws.any())
