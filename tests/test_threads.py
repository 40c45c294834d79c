"""Calls from several host threads at once: sizes that share a kernel and differ in the shared memory they launch it with.

The C calls are made as directly as ctypes can, so that they overlap (it gives up the interpreter's lock for each).
"""
import ctypes
import threading

import pytest
import torch

import row_wise_online_gb300 as rwo
from row_wise_online_gb300 import train
from train_util import BF

pytestmark = pytest.mark.gpu
CALLS = 10000


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def at_once(makes):
    """Each call from a thread and on a stream of its own, many times.  make(stream): a function, its arguments, and what they point to."""
    streams = [torch.cuda.Stream() for _ in makes]
    calls = [make(s.cuda_stream) for make, s in zip(makes, streams)]
    torch.cuda.synchronize()
    failed, start = [0] * len(calls), threading.Barrier(len(calls))

    def run(k):
        torch.cuda.set_device(0)
        fn, args, _ = calls[k]
        start.wait()
        for i in range(CALLS):
            failed[k] += fn(*args) != rwo.OK
            if i % 200 == 0:
                streams[k].synchronize()
        streams[k].synchronize()

    threads = [threading.Thread(target=run, args=(k,)) for k in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert failed == [0] * len(calls)
    assert rwo.get_status() == rwo.OK


def vp(t):
    return ctypes.c_void_p(t.data_ptr())


def test_norm_backward():
    def make(N):
        def of(stream):
            M = 64
            t = [torch.ones(M, N, device="cuda", dtype=BF) for _ in range(3)] + [torch.ones(N, device="cuda", dtype=BF), torch.ones(M, device="cuda"), torch.empty(N, device="cuda")]
            dy, h, dx, w, rstd, dw = (v.data_ptr() for v in t)
            ws = rwo.rms_norm_backward_workspace(M, N, BF)
            a = train._NormGrad(dy=dy, h=h, dx=dx, weight=w, rstd=rstd, dweight=dw)
            return rwo.capi().rms_norm_rows_backward, (ctypes.byref(a), M, N, rwo.BF16, vp(ws), ws.numel(), ctypes.c_void_p(stream)), (t, ws, a)
        return of

    at_once([make(N) for N in (2304, 4096, 3200)])


def test_embedding_backward():
    def make(V):
        def of(stream):
            T, D = 5000, 16
            dy, tok, grad = torch.ones(T, D, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda"), torch.empty(V, D, device="cuda")
            ws = rwo.embedding_backward_workspace(T, V, D)
            return (rwo.capi().embedding_rows_backward,
                    (vp(dy), 0, vp(tok), 8, vp(grad), 0, T, V, D, 1.0, 0, rwo.F32, rwo.F32, vp(ws), ws.numel(), ctypes.c_void_p(stream)), (dy, tok, grad, ws))
        return of

    at_once([make(V) for V in (50, 1000, 300)])


def test_loss():
    def make(N):
        def of(stream):
            x, labels, loss = torch.ones(16, N, device="cuda", dtype=BF), torch.zeros(16, dtype=torch.int64, device="cuda"), torch.empty(16, device="cuda")
            return (rwo.capi().cross_entropy_rows_grad,
                    (vp(x), 0, vp(labels), None, 1.0, 0.0, 0.0, vp(x), 0, vp(loss), None, 16, N, rwo.BF16, ctypes.c_void_p(stream)), (x, labels, loss))
        return of

    at_once([make(N) for N in (40000, 65536, 131072)])


@pytest.mark.parametrize("sizes", [(1024, 1536, 2048), (9000, 12000, 16000), (20000, 24000, 32000)])
def test_softmax(sizes):
    def make(N):
        def of(stream):
            x = torch.ones(64, N // 8 * 8, device="cuda", dtype=BF)
            y = torch.empty_like(x)
            return rwo.capi().softmax_rows, (vp(x), vp(y), *x.shape, rwo.BF16, ctypes.c_void_p(stream)), (x, y)
        return of

    at_once([make(N) for N in sizes])


def test_causal():
    def make(N):
        def of(stream):
            x = torch.ones(300, N, device="cuda", dtype=BF)
            y = torch.empty_like(x)
            return rwo.capi().softmax_rows_causal, (vp(x), vp(y), None, None, None, 300, N, N, 0, rwo.BF16, ctypes.c_void_p(stream)), (x, y)
        return of

    at_once([make(N) for N in (512, 2048, 4096)])
