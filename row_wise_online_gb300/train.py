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
import struct

import row_wise_online_gb300 as _rwo

from .decode import _raw_stream, _switched

_vp, _i64, _f32, _f64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_double


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


# The same structures packed in one go: filling a ctypes.Structure field by field takes 2 us of a call's 9.
_NORM, _NORM_GRAD = struct.Struct("=13q2f"), struct.Struct("=13qf4x")


def _declare(lib) -> None:
    """Argument types of the calls of this module."""
    ci = ctypes.c_int
    lib.cross_entropy_rows_grad.argtypes = [_vp, _i64, _vp, _vp, _f32, _f32, _f32, _vp, _i64, _vp, _vp, _i64, _i64, ci, _vp]
    lib.rms_norm_rows.argtypes = [_vp, _i64, _i64, ci, ci, _vp]
    lib.rms_norm_rows_backward.argtypes = [_vp, _i64, _i64, ci, _vp, _i64, _vp]
    lib.rms_norm_backward_workspace.argtypes = [_i64, _i64, ci]
    lib.embedding_rows.argtypes = [_vp, _i64, _vp, ci, _vp, _i64, _i64, _i64, _i64, _f32, ci, _vp]
    lib.embedding_rows_backward.argtypes = [_vp, _i64, _vp, ci, _vp, _i64, _i64, _i64, _i64, _f32, ci, ci, ci, _vp, _i64, _vp]
    lib.embedding_backward_workspace.argtypes = [_i64] * 3
    lib.grad_norm.argtypes = [_vp, _i64, _f32, _vp, _vp, _i64, _vp]
    lib.clip_grad_norm.argtypes = [_vp, _i64, _f32, _f64, _vp, _vp, _i64, _vp]
    lib.grad_norm_workspace.argtypes = [_i64]
    for name in ("cross_entropy_rows_grad", "rms_norm_rows", "rms_norm_rows_backward", "embedding_rows", "embedding_rows_backward",
                 "grad_norm", "clip_grad_norm"):
        getattr(lib, name).restype = ci
    for name in ("rms_norm_backward_workspace", "embedding_backward_workspace", "grad_norm_workspace"):
        getattr(lib, name).restype = _i64


@functools.lru_cache(maxsize=None)
def _codes():
    import torch

    return {torch.float32: _rwo.F32, torch.bfloat16: _rwo.BF16, torch.float16: _rwo.F16}


def _code(t) -> int:
    c = _codes().get(t.dtype)
    return _rwo._dtype_code(t) if c is None else c  # raises


@functools.lru_cache(maxsize=None)
def _current():
    """The current device, and a device's current stream as a pointer: torch's own short ways where it has them."""
    import torch

    return getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device), getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _stream_of(index, stream):
    """The stream's pointer where device ``index`` is current and the stream is its current one, else None: the call then
    makes itself again with both switched to."""
    if stream is not None:
        return None
    device, raw = _current()
    return raw(index) if device() == index else None


def _lead(t, name):
    """Shape, length N of the last dimension, rows M and device of a matrix of rows along it."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if not shape:
        raise ValueError(f"{name} must have at least one dimension")
    N = shape[-1]
    return shape, N, (t.numel() // N if N else 0), t.get_device()


def _pitch(t, name, shape):
    """Row pitch of a matrix."""
    if t.is_contiguous():
        return shape[-1]
    if len(shape) != 2 or (t.stride(1) != 1 and shape[1] > 1) or (shape[0] > 1 and t.stride(0) < shape[1]):
        raise ValueError(f"{name} must be contiguous, or 2-D with contiguous rows (stride(1) == 1, stride(0) >= N)")
    return t.stride(0) if shape[0] > 1 else shape[1]


def _matrix(t, name, shape, dtype, index):
    """Pointer and row pitch of a matrix of a shape and dtype on CUDA device ``index``."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on cuda:{index}")
    return t.data_ptr(), _pitch(t, name, shape)


def _vector(t, name, dtype, shape, index):
    """Pointer of a contiguous tensor of a dtype and shape on CUDA device ``index`` (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}")
    return t.data_ptr()


def _like(t, dtype=None):
    """A new contiguous tensor of t's shape."""
    import torch

    if dtype is None and t.is_contiguous():
        return torch.empty_like(t)  # 1 us less than spelling it out
    return torch.empty(t.shape, dtype=dtype or t.dtype, device=t.device)


def _weight(w, N, dtype, index):
    """Pointer of a norm's weight, and whether it is in 32 bits."""
    import torch

    if w is None:
        return 0, 0
    f32 = w.dtype is torch.float32
    return _vector(w, "weight", torch.float32 if f32 else dtype, (N,), index), int(f32)


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

    shape, N, M, index = _lead(x, "x")
    s = _stream_of(index, stream)
    if s is None:
        with _switched(index, stream):
            return cross_entropy_rows_grad(x, labels, grad, loss, lse_out, upstream, grad_scale, label_smoothing, z_loss)
    dt, lead, f32 = _code(x), shape[:-1], torch.float32
    xp, ldx = x.data_ptr(), _pitch(x, "x", shape)
    lp, up = _vector(labels, "labels", torch.int64, lead, index), _vector(upstream, "upstream", f32, lead, index)
    if grad is None:
        grad = _like(x)
        gp, ldg = grad.data_ptr(), N
    else:
        gp, ldg = _matrix(grad, "grad", shape, x.dtype, index)
    if loss is None:
        loss = torch.empty(lead, dtype=f32, device=x.device)
        op = loss.data_ptr()
    else:
        op = _vector(loss, "loss", f32, lead, index)
    st = _rwo.capi().cross_entropy_rows_grad(xp, ldx, lp, up, grad_scale, label_smoothing, z_loss, gp, ldg, op,
                                             _vector(lse_out, "lse_out", f32, lead, index), M, N, dt, s)
    if st:
        _rwo._check(st, "cross_entropy_rows_grad")
    return loss, grad


def _norm(x, weight, residual, sum_out, y, scales, group, rstd_out, eps, offset, out, stream):
    import torch

    shape, N, M, index = _lead(x, "x")
    s = _stream_of(index, stream)
    if s is None:
        with _switched(index, stream):
            return _norm(x, weight, residual, sum_out, y, scales, group, rstd_out, eps, offset, out, None)
    dt, lead, f32 = _code(x), shape[:-1], torch.float32
    xp, ldx = x.data_ptr(), _pitch(x, "x", shape)
    wp, wf = _weight(weight, N, x.dtype, index)
    rp = ldr = hp = ldh = sp = 0
    if residual is not None:
        rp, ldr = _matrix(residual, "residual", shape, x.dtype, index)
        if sum_out is None:
            sum_out = _like(x)
            hp, ldh = sum_out.data_ptr(), N
        else:
            hp, ldh = _matrix(sum_out, "sum_out", shape, x.dtype, index)
    elif sum_out is not None:
        raise ValueError("sum_out without residual")
    held = torch.float8_e4m3fn if out else None
    if y is None:
        y = _like(x, held)
        yp, ldy = y.data_ptr(), N
    else:
        yp, ldy = _matrix(y, "y", shape, held or x.dtype, index)
    if out:
        if group not in (0, 128):
            raise ValueError("group must be 0 (a scale for each row) or 128")
        parts = (*lead, -(-N // group) if group else 1)
        if scales is None:
            scales = torch.empty(parts, dtype=f32, device=x.device)
        sp = _vector(scales, "scales", f32, parts, index)
    st = _rwo.capi().rms_norm_rows(_NORM.pack(xp, ldx, rp, ldr, hp, ldh, wp, wf, yp, ldy, sp, group,
                                              _vector(rstd_out, "rstd_out", f32, lead, index), eps, offset), M, N, dt, out, s)
    if st:
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

    shape, N, M, index = _lead(h, "h")
    s = _stream_of(index, stream)
    if s is None:
        with _switched(index, stream):
            return rms_norm_rows_backward(dy, h, rstd, weight, offset, sum_grad, dx, dweight, accumulate, workspace)
    dt, f32 = _code(h), torch.float32
    hp, ldh = h.data_ptr(), _pitch(h, "h", shape)
    dp, ldd = _matrix(dy, "dy", shape, h.dtype, index)
    gp, ldg = (0, 0) if sum_grad is None else _matrix(sum_grad, "sum_grad", shape, h.dtype, index)
    wp, wf = _weight(weight, N, h.dtype, index)
    if dx is None:
        dx = _like(h)
        xp, ldx = dx.data_ptr(), N
    else:
        xp, ldx = _matrix(dx, "dx", shape, h.dtype, index)
    if dweight is None:
        if accumulate:
            raise ValueError("accumulate needs a dweight to add to")
        if weight is not None:
            dweight = torch.empty(N, dtype=f32, device=h.device)
    sp, sn = 0, 0
    if dweight is not None:
        workspace = _scratch(workspace, _bytes_of("rms_norm_backward_workspace", index, M, N, dt), h.device, index, "rms_norm_rows_backward")
        sp, sn = workspace.data_ptr(), workspace.numel()
    st = _rwo.capi().rms_norm_rows_backward(
        _NORM_GRAD.pack(dp, ldd, hp, ldh, gp, ldg, _vector(rstd, "rstd", f32, shape[:-1], index), wp, wf, xp, ldx,
                        _vector(dweight, "dweight", f32, (N,), index), 1 if accumulate else 0, offset), M, N, dt, sp, sn, s)
    if st:
        _rwo._check(st, "rms_norm_rows_backward")
    return dx, dweight


def _tokens(tokens, lead, index):
    """Pointer and element size of int32 or int64 tokens of a shape."""
    import torch

    if tokens.dtype is torch.int64:
        return _vector(tokens, "tokens", torch.int64, lead, index), 8
    if tokens.dtype is torch.int32:
        return _vector(tokens, "tokens", torch.int32, lead, index), 4
    raise ValueError("tokens must be int32 or int64")


def embedding_rows(table, tokens, y=None, scale: float = 1.0, stream=None):
    """y[...] = scale * table[tokens[...]] for a table [V, D] and int32 or int64 tokens; a negative token gives zeros."""
    import torch

    shape, D, V, index = _lead(table, "table")
    if len(shape) != 2:
        raise ValueError("table must be a 2-D CUDA tensor [V, D]")
    s = _stream_of(index, stream)
    if s is None:
        with _switched(index, stream):
            return embedding_rows(table, tokens, y, scale)
    dt = _code(table)
    tp, ldt = table.data_ptr(), _pitch(table, "table", shape)
    kp, kb = _tokens(tokens, tokens.shape, index)
    out = (*tokens.shape, D)
    if y is None:
        y = torch.empty(out, dtype=table.dtype, device=table.device)
        yp, ldy = y.data_ptr(), D
    else:
        yp, ldy = _matrix(y, "y", out, table.dtype, index)
    st = _rwo.capi().embedding_rows(tp, ldt, kp, kb, yp, ldy, tokens.numel(), shape[0], D, scale, dt, s)
    if st:
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

    shape, D, T, index = _lead(dy, "dy")
    s = _stream_of(index, stream)
    if s is None:
        with _switched(index, stream):
            return embedding_rows_backward(dy, tokens, num_rows, grad, scale, accumulate, dtype, workspace)
    dt = _code(dy)
    dp, ldd = dy.data_ptr(), _pitch(dy, "dy", shape)
    kp, kb = _tokens(tokens, shape[:-1], index)
    if grad is None:
        if accumulate or num_rows is None:
            raise ValueError("accumulate needs a grad to add to" if accumulate else "num_rows is needed to allocate grad")
        V = int(num_rows)
        grad = torch.empty((V, D), dtype=dtype or torch.float32, device=dy.device)
        gp, ldg = grad.data_ptr(), D
    else:
        V = grad.shape[0] if grad.dim() else 0
        if num_rows is not None and num_rows != V:
            raise ValueError(f"grad has {V} rows, num_rows is {num_rows}")
        gp, ldg = _matrix(grad, "grad", (V, D), dtype or grad.dtype, index)
    workspace = _scratch(workspace, _bytes_of("embedding_backward_workspace", index, T, V, D), dy.device, index, "embedding_rows_backward")
    st = _rwo.capi().embedding_rows_backward(dp, ldd, kp, kb, gp, ldg, T, V, D, scale, 1 if accumulate else 0, dt, _code(grad),
                                             workspace.data_ptr(), workspace.numel(), s)
    if st:
        _rwo._check(st, "embedding_rows_backward")
    return grad


def grad_norm_workspace(count: int, device=None):
    """A workspace tensor for grad_norm and clip_grad_norm calls over this many tensors."""
    return _workspace("grad_norm_workspace", device, count)


def _types(ts, index, error):
    """Type codes of contiguous tensors on a device: one number where all are of one type, else a list."""
    import torch

    kind, codes = torch.Tensor, _codes()
    # map() over the tensors' own methods: 0.25 us a tensor, where a loop with the same checks takes 0.45
    if index < 0 or set(map(kind.get_device, ts)) != {index} or not all(map(kind.is_contiguous, ts)):
        raise ValueError(error)
    kinds = {t.dtype for t in ts}
    if not kinds <= codes.keys():
        raise ValueError(error)
    return codes[kinds.pop()] if len(kinds) == 1 else [codes[t.dtype] for t in ts]


def _grads(tensors, out):
    """The list as the C call takes it (four 64-bit words a tensor: grad, out, n, types), and its device."""
    import torch

    n, kind, words = len(tensors), torch.Tensor, array.array
    if not n:
        return words("q"), torch.cuda.current_device()
    index = tensors[0].get_device()
    types = outs = _types(tensors, index, "gradients must be contiguous float32, bfloat16 or float16 tensors on one CUDA device")
    w = words("q", bytes(32 * n))
    w[0::4] = w[1::4] = words("q", map(kind.data_ptr, tensors))
    w[2::4] = words("q", map(kind.numel, tensors))
    if out is not None:
        error = "out must be contiguous tensors of the gradients' shapes, in their dtype or float32, on their device"
        if len(out) != n:
            raise ValueError(f"out must have as many tensors as there are gradients ({n})")
        outs = _types(out, index, error)
        if list(map(kind.size, out)) != list(map(kind.size, tensors)):
            raise ValueError(error)
        w[1::4] = words("q", map(kind.data_ptr, out))
    if isinstance(types, int) and isinstance(outs, int):
        pairs = {(types, outs)}
        w[3::4] = words("q", [types | outs << 32]) * n
    else:
        pairs = list(zip(*([v] * n if isinstance(v, int) else v for v in (types, outs))))
        w[3::4] = words("q", [a | b << 32 for a, b in pairs])
    if out is not None and any(b != a and b != _rwo.F32 for a, b in pairs):
        raise ValueError(error)
    return w, index


def _distinct(words):
    """Refuses a tensor that a call would scale twice."""
    to = words[1::4]
    if len(set(to)) != len(to):
        held = [p for p, n in zip(to, words[2::4]) if n]
        if len(set(held)) != len(held):
            raise ValueError("a gradient (or a tensor of out) is listed twice")


def _grad_norm(tensors, out, max_norm, scale, norm_out, workspace, stream):
    import torch

    tensors = tensors if isinstance(tensors, (list, tuple)) else list(tensors)
    words, index = _grads(tensors, out)
    if max_norm is not None:
        _distinct(words)
    s = _stream_of(index, stream)
    if s is None:
        with _switched(index, stream):
            return _grad_norm(tensors, out, max_norm, scale, norm_out, workspace, None)
    n = len(tensors)
    device = tensors[0].device if n else torch.device("cuda", index)
    if norm_out is None:
        norm_out = torch.empty((), dtype=torch.float32, device=device)
    np = _vector(norm_out, "norm_out", torch.float32, norm_out.shape if norm_out.numel() == 1 else (), index)
    workspace = _scratch(workspace, _bytes_of("grad_norm_workspace", index, n), device, index, "grad_norm")
    wp, wn, lp = workspace.data_ptr(), workspace.numel(), words.buffer_info()[0] if n else None
    if max_norm is None:
        st = _rwo.capi().grad_norm(lp, n, scale, np, wp, wn, s)
    else:
        st = _rwo.capi().clip_grad_norm(lp, n, scale, max_norm, np, wp, wn, s)
    if st:
        _rwo._check(st, "grad_norm" if max_norm is None else "clip_grad_norm")
    return norm_out


def grad_norm(tensors, scale: float = 1.0, norm_out=None, workspace=None, stream=None):
    """|scale| * the 2-norm of all elements of a list of contiguous CUDA tensors (fp32, bf16, fp16), as a fp32 scalar on the device."""
    return _grad_norm(tensors, None, None, scale, norm_out, workspace, stream)


def clip_grad_norm(tensors, max_norm: float, out=None, scale: float = 1.0, norm_out=None, workspace=None, stream=None):
    """Scale gradients, each listed once, by ``scale * min(1, max_norm / norm)``, norm = grad_norm(tensors, scale), which is returned.

    In place, or into ``out``: as many tensors, in the gradients' dtypes or float32, that overlap no other tensor of the call.  A norm that is inf or NaN limits nothing;
    in place, gradients whose factor is 1 are not touched.
    """
    return _grad_norm(tensors, out, float(max_norm), scale, norm_out, workspace, stream)
