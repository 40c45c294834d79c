"""The training-step calls without a GPU: every argument that the host can refuse is refused before anything is enqueued."""
import ctypes
import math

import pytest
import torch

import row_wise_online_gb300 as rwo
from row_wise_online_gb300 import _build, train

X = 0x10000  # never dereferenced: every call below fails validation first
BAD, ODD, NO, OK = rwo.ERR_INVALID_ARG, rwo.ERR_MISALIGNED, rwo.ERR_UNSUPPORTED, rwo.OK


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return rwo.capi()


def test_loss_faults(lib):
    def call(x=X, ldx=0, labels=X, up=None, gs=1.0, eps=0.0, z=0.0, g=X, ldg=0, loss=X, lse=None, M=4, N=100, dt=0):
        return lib.cross_entropy_rows_grad(x, ldx, labels, up, gs, eps, z, g, ldg, loss, lse, M, N, dt, None)

    assert call(N=0) == BAD and call(M=-1) == BAD and call(dt=3) == BAD and call(N=2 ** 31) == NO
    assert call(x=None) == BAD and call(labels=None) == BAD and call(g=None) == BAD and call(loss=None) == BAD
    assert call(ldx=99) == BAD and call(ldg=99) == BAD and call(ldx=2 ** 62) == BAD and call(ldx=-1) == BAD
    assert call(ldx=101, ldg=102) == BAD  # in place with two pitches
    for v in (math.nan, math.inf, -math.inf):
        assert call(gs=v) == BAD and call(eps=v) == BAD and call(z=v) == BAD
    assert call(eps=-0.1) == BAD and call(eps=1.0) == BAD and call(z=-1e-3) == BAD
    assert call(x=X + 2) == ODD and call(dt=1, g=X + 1) == ODD and call(labels=X + 4) == ODD and call(loss=X + 2) == ODD
    assert call(lse=X + 1) == ODD and call(up=X + 2) == ODD
    assert call(M=0, x=None, labels=None, g=None, loss=None) == OK and call(M=0, N=0) == BAD


def norm(M=4, N=256, dt=1, out=0, lib=None, **kw):
    return lib.rms_norm_rows(ctypes.byref(train._Norm(**{**dict(x=X, y=X + 0x8000, eps=1e-6), **kw})), M, N, dt, out, None)


def test_norm_faults(lib):
    assert lib.rms_norm_rows(None, 4, 4, 0, 0, None) == BAD
    assert norm(lib=lib, N=0) == BAD and norm(lib=lib, M=-1) == BAD and norm(lib=lib, dt=4) == BAD and norm(lib=lib, out=2) == BAD
    assert norm(lib=lib, N=2 ** 31) == NO
    assert norm(lib=lib, x=None) == BAD and norm(lib=lib, y=None) == BAD
    assert norm(lib=lib, residual=X) == BAD and norm(lib=lib, sum_out=X) == BAD  # one without the other
    assert norm(lib=lib, residual=X, sum_out=X + 0x8000) == BAD  # y and the sum in one place
    for v in (math.nan, math.inf):
        assert norm(lib=lib, eps=v) == BAD and norm(lib=lib, offset=v) == BAD
    assert norm(lib=lib, eps=-1.0) == BAD and norm(lib=lib, weight_f32=2) == BAD
    assert norm(lib=lib, group=128) == BAD  # scales belong to e4m3
    assert norm(lib=lib, out=1, group=64, scales=X) == NO and norm(lib=lib, out=1, group=-128, scales=X) == BAD and norm(lib=lib, out=1) == BAD
    for ld in ("ldx", "ldy"):
        assert norm(lib=lib, **{ld: 255}) == BAD and norm(lib=lib, **{ld: 2 ** 62}) == BAD
    assert norm(lib=lib, residual=X, sum_out=X, ld_residual=3) == BAD and norm(lib=lib, residual=X, sum_out=X, ld_sum=3) == BAD
    assert norm(lib=lib, x=X + 1) == ODD and norm(lib=lib, weight=X + 1) == ODD and norm(lib=lib, weight=X + 2, weight_f32=1) == ODD
    assert norm(lib=lib, rstd_out=X + 2) == ODD and norm(lib=lib, out=1, scales=X + 2) == ODD and norm(lib=lib, residual=X + 1, sum_out=X) == ODD
    assert norm(lib=lib, out=1, scales=X, y=X) == BAD and norm(lib=lib, out=1, scales=X, y=X + 64, residual=X + 64, sum_out=X) == BAD  # 8 bits over 16
    assert norm(lib=lib, y=X, ldx=300) == BAD  # in place with two pitches
    assert norm(lib=lib, residual=X + 64, sum_out=X, ldx=300) == BAD and norm(lib=lib, residual=X + 64, sum_out=X + 64, ld_sum=300) == BAD
    assert norm(lib=lib, M=0, x=None, y=None) == OK


def test_norm_grad_faults(lib):
    def call(M=4, N=256, dt=1, ws=X, n=2 ** 40, **kw):
        return lib.rms_norm_rows_backward(ctypes.byref(train._NormGrad(**{**dict(dy=X, h=X, rstd=X, dx=X), **kw})), M, N, dt, ws, n, None)

    assert lib.rms_norm_rows_backward(None, 4, 4, 0, X, 0, None) == BAD
    assert call(N=0) == BAD and call(M=-1) == BAD and call(dt=9) == BAD and call(N=2 ** 31) == NO
    for p in ("dy", "h", "rstd", "dx"):
        assert call(**{p: None}) == BAD
        assert call(**{p: X + 1}) == ODD
    assert call(sum_grad=X + 1) == ODD and call(weight=X + 2, weight_f32=1) == ODD and call(dweight=X + 2) == ODD
    for ld in ("ld_dy", "ldh", "ld_dx"):
        assert call(**{ld: 100}) == BAD
    assert call(sum_grad=X, ld_sum_grad=100) == BAD
    assert call(ldh=300) == BAD and call(dx=X + 64, sum_grad=X + 64, ld_dx=300) == BAD  # in place with two pitches
    assert call(offset=math.nan) == BAD and call(accumulate=2) == BAD and call(weight_f32=-1) == BAD
    assert call(M=0, dy=None, h=None, rstd=None, dx=None) == OK
    assert lib.rms_norm_backward_workspace(4, 0, 0) == -1 and lib.rms_norm_backward_workspace(4, 4, 5) == -1


def test_embedding_faults(lib):
    def look(table=X, ldt=0, tok=X, kb=8, y=X, ldy=0, T=4, V=10, D=64, scale=1.0, dt=1):
        return lib.embedding_rows(table, ldt, tok, kb, y, ldy, T, V, D, scale, dt, None)

    assert look(T=-1) == BAD and look(V=0) == BAD and look(D=0) == BAD and look(kb=2) == BAD and look(dt=3) == BAD and look(scale=math.inf) == BAD
    assert look(table=None) == BAD and look(tok=None) == BAD and look(y=None) == BAD and look(ldt=63) == BAD and look(ldy=63) == BAD
    assert look(tok=X + 4) == ODD and look(tok=X + 2, kb=4) == ODD and look(table=X + 1) == ODD and look(y=X + 1) == ODD
    assert look(T=0, table=None, tok=None, y=None) == OK and look(D=2 ** 30 + 1) == NO

    def grad(dy=X, ldd=0, tok=X, kb=8, g=X, ldg=0, T=4, V=10, D=64, scale=1.0, acc=0, dt=1, gdt=0, ws=X, n=2 ** 40):
        return lib.embedding_rows_backward(dy, ldd, tok, kb, g, ldg, T, V, D, scale, acc, dt, gdt, ws, n, None)

    assert grad(T=-1) == BAD and grad(V=0) == BAD and grad(D=0) == BAD and grad(kb=1) == BAD and grad(dt=3) == BAD and grad(gdt=3) == BAD
    assert grad(dt=1, gdt=2) == NO and grad(dt=0, gdt=1) == NO and grad(scale=math.nan) == BAD and grad(acc=2) == BAD
    assert grad(T=2 ** 24 + 1) == NO and grad(V=2 ** 31 - 1) == NO and grad(D=2 ** 30 + 1) == NO
    assert grad(dy=None) == BAD and grad(tok=None) == BAD and grad(g=None) == BAD and grad(ldd=63) == BAD and grad(ldg=63) == BAD
    assert grad(ws=None) == BAD and grad(n=10) == BAD and grad(ws=X + 128) == ODD
    assert grad(dy=X + 1) == ODD and grad(g=X + 2) == ODD and grad(tok=X + 4) == ODD
    assert grad(T=0, acc=1, dy=None, tok=None, g=None, ws=None, n=0) == OK
    assert lib.embedding_backward_workspace(4, 0, 4) == -1 and lib.embedding_backward_workspace(2 ** 25, 4, 4) == -1
    assert lib.embedding_backward_workspace(4, 4, 4) > 0


def test_grad_norm_faults(lib):
    def call(entries=((X, X, 5, 0, 0),), count=None, scale=1.0, limit=1.0, out=X, ws=X, n=2 ** 40):
        arr = (train._Grad * max(1, len(entries)))(*[train._Grad(*e) for e in entries])
        p = ctypes.cast(arr, ctypes.c_void_p) if entries else None
        count = len(entries) if count is None else count
        a = lib.clip_grad_norm(p, count, scale, limit, out, ws, n, None)
        if limit == 1.0:
            same = all(e[0] is not None and e[2] >= 0 for e in entries)
            b = lib.grad_norm(p, count, scale, out, ws, n, None) if a in (BAD, ODD, NO) and (not same or scale != 1.0 or not out or count < 0) else a
            assert b == a
        return a

    assert call(count=-1) == BAD and call(entries=(), count=1) == BAD and call(count=2 ** 21, entries=((X, X, 1, 0, 0),)) == NO
    assert call(scale=math.nan) == BAD and call(out=None) == BAD and call(out=X + 2) == ODD
    for limit in (0.0, -1.0, math.inf, math.nan):
        assert call(limit=limit) == BAD
    assert call(((None, X, 5, 0, 0),)) == BAD and call(((X, None, 5, 0, 0),)) == BAD and call(((X, X, -1, 0, 0),)) == BAD
    assert call(((X, X, 5, 7, 0),)) == BAD and call(((X, X, 5, 0, 7),)) == BAD and call(((X, X + 64, 5, 0, 1),)) == NO
    assert call(((X, X, 5, 1, 0),)) == BAD  # in place in another type
    assert call(((X + 2, X, 5, 0, 0),)) == ODD and call(((X, X + 2, 5, 1, 0),)) == ODD
    assert call(((X, X, 2 ** 41, 0, 0), (X, X, 2 ** 41 + 1, 0, 0))) == NO and call(((X, X, 2 ** 62, 0, 0),)) == NO


def test_structures_match_the_header():
    assert ctypes.sizeof(train._Norm) == 13 * 8 + 8 and ctypes.sizeof(train._NormGrad) == 13 * 8 + 8 and ctypes.sizeof(train._Grad) == 32
    for packed, whole, floats in ((train._NORM, train._Norm, 2), (train._NORM_GRAD, train._NormGrad, 1)):
        names = [n for n, _ in whole._fields_]
        a = whole.from_buffer_copy(packed.pack(*range(1, 14), *(0.5 * (k + 1) for k in range(floats))))
        assert ctypes.sizeof(whole) == packed.size
        assert [getattr(a, n) for n in names] == [*range(1, 14), *(0.5 * (k + 1) for k in range(floats))]


def test_binding_refuses_on_the_host():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    i = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: rwo.cross_entropy_rows_grad(x, i), lambda: rwo.rms_norm_rows(x, w), lambda: rwo.rms_norm_rows_e4m3(x, w),
                 lambda: rwo.rms_norm_rows_backward(x, x, x[:, 0], w), lambda: rwo.embedding_rows(x, i), lambda: rwo.embedding_rows_backward(x, i, 3),
                 lambda: rwo.grad_norm([x]), lambda: rwo.clip_grad_norm([x], 1.0)):
        with pytest.raises(ValueError):
            call()  # not CUDA tensors


@pytest.mark.gpu
def test_binding_refuses_on_the_device():
    _build.build()
    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(8, device="cuda")
    i, f = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda")
    bf = x.bfloat16()
    bad = [
        lambda: rwo.cross_entropy_rows_grad(x, i.int()), lambda: rwo.cross_entropy_rows_grad(x, i[:3]), lambda: rwo.cross_entropy_rows_grad(x, i.cpu()),
        lambda: rwo.cross_entropy_rows_grad(x, i, grad=bf), lambda: rwo.cross_entropy_rows_grad(x.t(), i[:1].expand(8)),
        lambda: rwo.cross_entropy_rows_grad(x[:1].expand(4, 8), i), lambda: rwo.cross_entropy_rows_grad(x, i, upstream=f[:2]),
        lambda: rwo.rms_norm_rows(x, w[:7]), lambda: rwo.rms_norm_rows(bf, w.half()), lambda: rwo.rms_norm_rows(x, w, residual=bf),
        lambda: rwo.rms_norm_rows(x, w, sum_out=x), lambda: rwo.rms_norm_rows(x[:, ::2], w[:4]), lambda: rwo.rms_norm_rows_e4m3(x, w, group=64),
        lambda: rwo.rms_norm_rows_e4m3(x, w, y=x), lambda: rwo.rms_norm_rows_e4m3(x, w, scales=f),
        lambda: rwo.rms_norm_rows_backward(bf, x, f, w), lambda: rwo.rms_norm_rows_backward(x, x, f[:3], w), lambda: rwo.rms_norm_rows_backward(x, x, f, w, accumulate=True),
        lambda: rwo.rms_norm_rows_backward(x, x, f, w, workspace=f), lambda: rwo.embedding_rows(x[0], i), lambda: rwo.embedding_rows(x, f),
        lambda: rwo.embedding_rows_backward(x, i), lambda: rwo.embedding_rows_backward(x, i[:2], 3), lambda: rwo.embedding_rows_backward(x, i, 3, accumulate=True),
        lambda: rwo.embedding_rows_backward(x, i, 3, grad=x), lambda: rwo.grad_norm([x, x.cpu()]), lambda: rwo.grad_norm([x.t()]), lambda: rwo.grad_norm([x.double()]),
        lambda: rwo.clip_grad_norm([x, w], 1.0, out=[x]), lambda: rwo.clip_grad_norm([x], 1.0, out=[bf]), lambda: rwo.clip_grad_norm([bf], 1.0, out=[bf.half()]),
        lambda: rwo.grad_norm([x], norm_out=f), lambda: rwo.grad_norm([x], workspace=f),
    ]
    for k, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            pytest.fail(f"call {k} was taken")
    for call in (lambda: rwo.clip_grad_norm([x], -1.0), lambda: rwo.cross_entropy_rows_grad(x, i, label_smoothing=1.5), lambda: rwo.rms_norm_rows(x, w, eps=-1.0),
                 lambda: rwo.embedding_rows_backward(bf, i, 3, dtype=torch.float16), lambda: rwo.grad_norm([x], workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(rwo.SoftmaxError):
            call()
    assert rwo.get_status() == OK
