"""The training step around the matrix products: the loss of the logits with its gradient (``cross_entropy_rows_grad``),
the root-mean-square norm of rows (``rms_norm_rows``, ``rms_norm_rows_e4m3``, ``rms_norm_rows_backward``), embedding
lookup and its gradient (``embedding_rows``, ``embedding_rows_backward``), and the norm of all gradients with clipping
(``grad_norm``, ``clip_grad_norm``).

As the rest of the package, this module only marshals arguments; the calls are described in
``include/softmax_rows.h``.  Every tensor of a call is on one CUDA device, which need not be the current one; the
work is enqueued on ``stream`` or on that device's current stream.  Matrices are contiguous, of any number of
dimensions, or 2-D with contiguous rows a pitch apart.  Workspaces are allocated for a call unless given; calls that
may run at the same time need one each.
"""
from __future__ import annotations

import array
import ctypes
import functools

import row_wise_online_gb300 as _rwo

from .decode import _on, _tensor

_vp, _i64, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float


class _Norm(ctypes.Structure):
    _fields_ = [("x", _vp), ("ldx", _i64), ("residual", _vp), ("ld_residual", _i64), ("sum_out", _vp), ("ld_sum", _i64),
                ("weight", _vp), ("weight_f32", _i64), ("y", _vp), ("ldy", _i64), ("scales", _vp), ("group", _i64),
                ("rstd_out", _vp), ("eps", _f32), ("offset", _f32)]


class _NormGrad(ctypes.Structure):
    _fields_ = [("dy", _vp), ("ld_dy", _i64), ("h", _vp), ("ldh", _i64), ("sum_grad", _vp), ("ld_sum_grad", _i64),
                ("rstd", _vp), ("weight", _vp), ("weight_f32", _i64), ("dx", _vp), ("ld_dx", _i64), ("dweight", _vp),
                ("accumulate", _i64), ("offset", _f32)]


class _Grad(ctypes.Structure):
    _fields_ = [("grad", _vp), ("out", _vp), ("n", _i64), ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


def _declare(lib) -> None:
    """Argument types of the calls of this module."""
    ci = ctypes.c_int
    lib.cross_entropy_rows_grad.argtypes = [_vp, _i64, _vp, _vp, _f32, _f32, _f32, _vp, _i64, _vp, _vp, _i64, _i64, ci, _vp]
    lib.rms_norm_rows.argtypes = [ctypes.POINTER(_Norm), _i64, _i64, ci, ci, _vp]
    lib.rms_norm_rows_backward.argtypes = [ctypes.POINTER(_NormGrad), _i64, _i64, ci, _vp, _i64, _vp]
    lib.rms_norm_backward_workspace.argtypes = [_i64, _i64, ci]
    lib.embedding_rows.argtypes = [_vp, _i64, _vp, ci, _vp, _i64, _i64, _i64, _i64, _f32, ci, _vp]
    lib.embedding_rows_backward.argtypes = [_vp, _i64, _vp, ci, _vp, _i64, _i64, _i64, _i64, _f32, ci, ci, ci, _vp, _i64, _vp]
    lib.embedding_backward_workspace.argtypes = [_i64] * 3
    lib.grad_norm.argtypes = [_vp, _i64, _f32, _vp, _vp, _i64, _vp]
    lib.clip_grad_norm.argtypes = [_vp, _i64, _f32, _f32, _vp, _vp, _i64, _vp]
    lib.grad_norm_workspace.argtypes = [_i64]
    for name in ("cross_entropy_rows_grad", "rms_norm_rows", "rms_norm_rows_backward", "embedding_rows", "embedding_rows_backward",
                 "grad_norm", "clip_grad_norm"):
        getattr(lib, name).restype = ci
    for name in ("rms_norm_backward_workspace", "embedding_backward_workspace", "grad_norm_workspace"):
        getattr(lib, name).restype = _i64


def _sizes(t, name):
    """(M, N) and the device of a matrix of rows along the last dimension."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() == 0:
        raise ValueError(f"{name} must have at least one dimension")
    N = int(t.shape[-1])
    return (t.numel() // N if N else 0), N, t.get_device()


def _matrix(t, name, shape, dtype, index):
    """Pointer and row pitch of a matrix of a shape and dtype on CUDA device ``index``."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on cuda:{index}")
    if t.is_contiguous():
        return t.data_ptr(), shape[-1]
    if t.dim() != 2 or (t.stride(1) != 1 and shape[1] > 1) or (shape[0] > 1 and t.stride(0) < shape[1]):
        raise ValueError(f"{name} must be contiguous, or 2-D with contiguous rows (stride(1) == 1, stride(0) >= N)")
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else shape[1]


def _weight(w, N, dtype, index):
    """Pointer of a norm's weight, and whether it is in 32 bits."""
    import torch

    if w is None:
        return None, 0
    f32 = w.dtype is torch.float32
    return _tensor(w, "weight", torch.float32 if f32 else dtype, (N,), index), int(f32)


def _scratch(workspace, need, device, index, what):
    """A workspace of at least ``need`` bytes: the given one, checked, or a new one."""
    import torch

    if need < 0:
        raise _rwo.SoftmaxError(_rwo.ERR_UNSUPPORTED, what)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.dtype is not torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != index:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{index}")
    return workspace


@functools.lru_cache(maxsize=4096)
def _bytes_of(name, index, *sizes):
    """Workspace bytes on device ``index``, which is current: a function of the sizes and the device alone."""
    return getattr(_rwo.capi(), name)(*sizes)


def _workspace(name, device, *sizes):
    import torch

    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        n = _bytes_of(name, torch.cuda.current_device(), *sizes)
        return _scratch(None, n, device, torch.cuda.current_device(), name)


def cross_entropy_rows_grad(x, labels, grad=None, loss=None, lse_out=None, upstream=None, grad_scale: float = 1.0,
                            label_smoothing: float = 0.0, z_loss: float = 0.0, stream=None):
    """Per-row cross-entropy loss (fp32) of logits x [..., N] and its gradient, in one pass.

    labels int64 [...], negative = ignored row (loss and gradient 0).  grad = d(sum of grad_scale * upstream * loss) / dx in
    x's dtype, upstream fp32 [...] (None: 1); grad may be x.  label_smoothing mixes in the mean over all N, z_loss adds
    z_loss * LSE^2 to a row's loss.  Returns (loss, grad) (and fills lse_out).
    """
    import torch

    M, N, index = _sizes(x, "x")
    dt, lead = _rwo._dtype_code(x), x.shape[:-1]
    xp, ldx = _matrix(x, "x", x.shape, x.dtype, index)
    lp = _tensor(labels, "labels", torch.int64, lead, index)
    up = _tensor(upstream, "upstream", torch.float32, lead, index)
    with _on(index, stream) as s:
        if grad is None:
            grad = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if loss is None:
            loss = torch.empty(lead, dtype=torch.float32, device=x.device)
        gp, ldg = _matrix(grad, "grad", x.shape, x.dtype, index)
        st = _rwo.capi().cross_entropy_rows_grad(xp, ldx, lp, up, grad_scale, label_smoothing, z_loss, gp, ldg,
                                                 _tensor(loss, "loss", torch.float32, lead, index),
                                                 _tensor(lse_out, "lse_out", torch.float32, lead, index), M, N, dt, s)
    _rwo._check(st, "cross_entropy_rows_grad")
    return loss, grad


def _norm(x, weight, residual, sum_out, y, scales, group, rstd_out, eps, offset, out, stream):
    import torch

    M, N, index = _sizes(x, "x")
    dt, lead = _rwo._dtype_code(x), x.shape[:-1]
    a = _Norm(group=group, eps=eps, offset=offset)
    a.x, a.ldx = _matrix(x, "x", x.shape, x.dtype, index)
    a.weight, a.weight_f32 = _weight(weight, N, x.dtype, index)
    a.rstd_out = _tensor(rstd_out, "rstd_out", torch.float32, lead, index)
    if residual is None and sum_out is not None:
        raise ValueError("sum_out without residual")
    if out and group not in (0, 128):
        raise ValueError("group must be 0 (a scale for each row) or 128")
    with _on(index, stream) as s:
        if residual is not None:
            a.residual, a.ld_residual = _matrix(residual, "residual", x.shape, x.dtype, index)
            if sum_out is None:
                sum_out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            a.sum_out, a.ld_sum = _matrix(sum_out, "sum_out", x.shape, x.dtype, index)
        if y is None:
            y = torch.empty(x.shape, dtype=torch.float8_e4m3fn if out else x.dtype, device=x.device)
        a.y, a.ldy = _matrix(y, "y", x.shape, torch.float8_e4m3fn if out else x.dtype, index)
        if out:
            shape = (*lead, -(-N // group) if group else 1)
            if scales is None:
                scales = torch.empty(shape, dtype=torch.float32, device=x.device)
            a.scales = _tensor(scales, "scales", torch.float32, shape, index)
        st = _rwo.capi().rms_norm_rows(a, M, N, dt, out, s)
    _rwo._check(st, "rms_norm_rows")
    return y, scales, sum_out


def rms_norm_rows(x, weight=None, residual=None, y=None, sum_out=None, rstd_out=None, eps: float = 1e-6, offset: float = 0.0,
                  stream=None):
    """y = h / sqrt(mean(h^2) + eps) * (weight + offset) along the last dimension, h = x + residual (rounded to the dtype).

    weight [N] in x's dtype or fp32 (None: factor 1).  Returns (y, h); h is written to sum_out (default: a new tensor; may
    be x or residual) and is None without a residual.  rstd_out fp32 [...] keeps what the backward pass needs.
    """
    y, _, total = _norm(x, weight, residual, sum_out, y, None, 0, rstd_out, eps, offset, 0, stream)
    return y, total


def rms_norm_rows_e4m3(x, weight=None, residual=None, group: int = 128, y=None, scales=None, sum_out=None, rstd_out=None,
                       eps: float = 1e-6, offset: float = 0.0, stream=None):
    """rms_norm_rows with y in 8 bits (torch.float8_e4m3fn) and fp32 scales: the value is y * scale.

    group: 128 elements a scale (scales [..., ceil(N / 128)]), or 0 for one a row ([..., 1]).  Returns (y, scales, h).
    """
    return _norm(x, weight, residual, sum_out, y, scales, group, rstd_out, eps, offset, 1, stream)


def rms_norm_backward_workspace(rows: int, dim: int, dtype, device=None):
    """A workspace tensor for rms_norm_rows_backward calls of these sizes."""
    import torch

    return _workspace("rms_norm_backward_workspace", device, rows, dim, _rwo._dtype_code(torch.empty(0, dtype=dtype)))


def rms_norm_rows_backward(dy, h, rstd, weight=None, offset: float = 0.0, sum_grad=None, dx=None, dweight=None,
                           accumulate: bool = False, workspace=None, stream=None):
    """Gradients of rms_norm_rows: of x (and of residual alike), and of weight in fp32 (None without a weight).

    h is what the norm was taken of (x, or the sum), rstd its rstd_out, sum_grad the gradient that reaches h by its
    other uses.  dx may be dy, h or sum_grad.  accumulate adds to a given dweight.  Returns (dx, dweight).
    """
    import torch

    M, N, index = _sizes(h, "h")
    dt = _rwo._dtype_code(h)
    a = _NormGrad(offset=offset, accumulate=int(accumulate))
    a.h, a.ldh = _matrix(h, "h", h.shape, h.dtype, index)
    a.dy, a.ld_dy = _matrix(dy, "dy", h.shape, h.dtype, index)
    if sum_grad is not None:
        a.sum_grad, a.ld_sum_grad = _matrix(sum_grad, "sum_grad", h.shape, h.dtype, index)
    a.rstd = _tensor(rstd, "rstd", torch.float32, h.shape[:-1], index)
    a.weight, a.weight_f32 = _weight(weight, N, h.dtype, index)
    if dweight is None and accumulate:
        raise ValueError("accumulate needs a dweight to add to")
    with _on(index, stream) as s:
        if dx is None:
            dx = torch.empty(h.shape, dtype=h.dtype, device=h.device)
        a.dx, a.ld_dx = _matrix(dx, "dx", h.shape, h.dtype, index)
        if dweight is None and weight is not None:
            dweight = torch.empty(N, dtype=torch.float32, device=h.device)
        a.dweight = _tensor(dweight, "dweight", torch.float32, (N,), index)
        wp, wn = None, 0
        if dweight is not None:
            workspace = _scratch(workspace, _bytes_of("rms_norm_backward_workspace", index, M, N, dt), h.device, index, "rms_norm_rows_backward")
            wp, wn = workspace.data_ptr(), workspace.numel()
        st = _rwo.capi().rms_norm_rows_backward(a, M, N, dt, wp, wn, s)
    _rwo._check(st, "rms_norm_rows_backward")
    return dx, dweight


def _tokens(tokens, lead, index):
    """Pointer and element size of int32 or int64 tokens of a shape."""
    import torch

    if tokens.dtype is not torch.int64 and tokens.dtype is not torch.int32:
        raise ValueError("tokens must be int32 or int64")
    return _tensor(tokens, "tokens", tokens.dtype, lead, index), 8 if tokens.dtype is torch.int64 else 4


def embedding_rows(table, tokens, y=None, scale: float = 1.0, stream=None):
    """y[...] = scale * table[tokens[...]] for a table [V, D] and int32 or int64 tokens; a negative token gives zeros."""
    import torch

    if not table.is_cuda or table.dim() != 2:
        raise ValueError("table must be a 2-D CUDA tensor [V, D]")
    V, D = table.shape
    dt, index = _rwo._dtype_code(table), table.get_device()
    tp, ldt = _matrix(table, "table", table.shape, table.dtype, index)
    kp, kb = _tokens(tokens, tokens.shape, index)
    shape = (*tokens.shape, D)
    with _on(index, stream) as s:
        if y is None:
            y = torch.empty(shape, dtype=table.dtype, device=table.device)
        yp, ldy = _matrix(y, "y", shape, table.dtype, index)
        st = _rwo.capi().embedding_rows(tp, ldt, kp, kb, yp, ldy, tokens.numel(), V, D, scale, dt, s)
    _rwo._check(st, "embedding_rows")
    return y


def embedding_backward_workspace(tokens: int, num_rows: int, dim: int, device=None):
    """A workspace tensor for embedding_rows_backward calls of these sizes."""
    return _workspace("embedding_backward_workspace", device, tokens, num_rows, dim)


def embedding_rows_backward(dy, tokens, num_rows: int | None = None, grad=None, scale: float = 1.0, accumulate: bool = False,
                            dtype=None, workspace=None, stream=None):
    """Gradient [num_rows, D] of embedding_rows' table from dy [..., D]: dense, in ``dtype`` (default fp32; or dy's).

    accumulate adds to a given grad and leaves rows that no token names as they are.
    """
    import torch

    T, D, index = _sizes(dy, "dy")
    dt, lead = _rwo._dtype_code(dy), dy.shape[:-1]
    dp, ldd = _matrix(dy, "dy", dy.shape, dy.dtype, index)
    kp, kb = _tokens(tokens, lead, index)
    if grad is None and (num_rows is None or accumulate):
        raise ValueError("accumulate needs a grad to add to" if accumulate else "num_rows is needed to allocate grad")
    V = int(grad.shape[0]) if grad is not None else int(num_rows)
    if num_rows is not None and num_rows != V:
        raise ValueError(f"grad has {V} rows, num_rows is {num_rows}")
    with _on(index, stream) as s:
        if grad is None:
            grad = torch.empty((V, D), dtype=dtype or torch.float32, device=dy.device)
        gp, ldg = _matrix(grad, "grad", (V, D), dtype or grad.dtype, index)
        workspace = _scratch(workspace, _bytes_of("embedding_backward_workspace", index, T, V, D), dy.device, index, "embedding_rows_backward")
        st = _rwo.capi().embedding_rows_backward(dp, ldd, kp, kb, gp, ldg, T, V, D, scale, int(accumulate), dt, _rwo._dtype_code(grad),
                                                 workspace.data_ptr(), workspace.numel(), s)
    _rwo._check(st, "embedding_rows_backward")
    return grad


def grad_norm_workspace(count: int, device=None):
    """A workspace tensor for grad_norm and clip_grad_norm calls over this many tensors."""
    return _workspace("grad_norm_workspace", device, count)


@functools.lru_cache(maxsize=None)
def _codes():
    import torch

    return {torch.float32: _rwo.F32, torch.bfloat16: _rwo.BF16, torch.float16: _rwo.F16}


def _grads(tensors, out):
    """The list as the C call takes it (four 64-bit words a tensor: grad, out, n, types), and its device."""
    import torch

    if not tensors:
        return array.array("q"), torch.cuda.current_device()
    index, codes, words = tensors[0].get_device(), _codes(), []
    for t in tensors:
        code = codes.get(t.dtype)
        if code is None or t.get_device() != index or index < 0 or not t.is_contiguous():
            raise ValueError("gradients must be contiguous float32, bfloat16 or float16 tensors on one CUDA device")
        p = t.data_ptr()
        words += (p, p, t.numel(), code | code << 32)
    if out is not None:
        if len(out) != len(tensors):
            raise ValueError(f"out must have as many tensors as there are gradients ({len(tensors)})")
        for i, (t, o) in enumerate(zip(tensors, out)):
            if o.shape != t.shape or (o.dtype is not t.dtype and o.dtype is not torch.float32) or o.get_device() != index or not o.is_contiguous():
                raise ValueError("out must be contiguous tensors of the gradients' shapes, in their dtype or float32, on their device")
            words[4 * i + 1] = o.data_ptr()
            words[4 * i + 3] = codes[t.dtype] | codes[o.dtype] << 32
    return array.array("q", words), index


def _grad_norm(tensors, out, max_norm, scale, norm_out, workspace, stream):
    import torch

    tensors = list(tensors)
    words, index = _grads(tensors, out)
    n = len(tensors)
    with _on(index, stream) as s:
        if norm_out is None:
            norm_out = torch.empty((), dtype=torch.float32, device=f"cuda:{index}")
        np = _tensor(norm_out, "norm_out", torch.float32, norm_out.shape if norm_out.numel() == 1 else (), index)
        workspace = _scratch(workspace, _bytes_of("grad_norm_workspace", index, n), norm_out.device, index, "grad_norm")
        wp, wn, lp = workspace.data_ptr(), workspace.numel(), words.buffer_info()[0] if n else None
        if max_norm is None:
            st = _rwo.capi().grad_norm(lp, n, scale, np, wp, wn, s)
        else:
            st = _rwo.capi().clip_grad_norm(lp, n, scale, max_norm, np, wp, wn, s)
    _rwo._check(st, "grad_norm" if max_norm is None else "clip_grad_norm")
    return norm_out


def grad_norm(tensors, scale: float = 1.0, norm_out=None, workspace=None, stream=None):
    """|scale| * the 2-norm of all elements of a list of contiguous CUDA tensors (fp32, bf16, fp16), as a fp32 scalar on the device."""
    return _grad_norm(tensors, None, None, scale, norm_out, workspace, stream)


def clip_grad_norm(tensors, max_norm: float, out=None, scale: float = 1.0, norm_out=None, workspace=None, stream=None):
    """Scale gradients by ``scale * min(1, max_norm / norm)``, norm = grad_norm(tensors, scale), which is returned.

    In place, or into ``out``: as many tensors, in the gradients' dtypes or float32.  A norm that is inf or NaN limits nothing;
    in place, gradients whose factor is 1 are not touched.
    """
    return _grad_norm(tensors, out, float(max_norm), scale, norm_out, workspace, stream)
