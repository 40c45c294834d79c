"""The decoding step: a paged key/value cache held in 4 bits (``kv4_append``, ``kv4_gather``,
``attention_kv4``) and the processing of logits before their softmax (``logits_process_rows``).

As the rest of the package, this module only marshals arguments; the calls and the layout of the cache are
described in ``include/softmax_rows.h``.  Every tensor of a call is on one CUDA device, which need not be the
current one; the work is enqueued on ``stream`` or on that device's current stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import row_wise_online_gb300 as _rwo

KV4_FLAG_NEIGHBOURS = 1
LOGITS_OUT = {"logits": 0, "softmax": 1, "log_softmax": 2}

_vp, _i64 = ctypes.c_void_p, ctypes.c_int64


class _Cache(ctypes.Structure):
    _fields_ = [("data", _vp), ("page_table", _vp), ("seq_lens", _vp), ("cu_tokens", _vp)] + [
        (n, _i64) for n in ("num_pages", "page_size", "heads", "head_dim", "batch", "table_width", "tokens")]


class _Rows(ctypes.Structure):
    _fields_ = [("data", _vp), ("token_stride", _i64), ("head_stride", _i64)]


class _Logits(ctypes.Structure):
    _fields_ = [("x", _vp), ("ldx", _i64), ("y", _vp), ("ldy", _i64), ("lse_out", _vp), ("tokens", _vp),
                ("token_width", _i64), ("prompt_lens", _vp), ("token_lens", _vp), ("repetition", _vp),
                ("frequency", _vp), ("presence", _vp), ("bias_ids", _vp), ("bias_values", _vp), ("bias_count", _i64),
                ("mask", _vp), ("ld_mask", _i64), ("scale", _vp)]


def _declare(lib) -> None:
    """Argument types of the calls of this module."""
    rows, ci = ctypes.POINTER(_Rows), ctypes.c_int
    cache = ctypes.POINTER(_Cache)
    lib.kv4_append.argtypes = [cache, rows, rows, rows, rows, _i64, _vp, _i64, _i64, ci, ci, _vp]
    lib.kv4_gather.argtypes = [cache, rows, rows, ci, _vp]
    lib.attention_kv4.argtypes = [cache, rows, _vp, _vp, _i64, ctypes.c_float, ci, _vp, _i64, _vp]
    lib.attention_kv4_workspace.argtypes = [_i64] * 5
    lib.attention_kv4_workspace.restype = _i64
    lib.logits_process_rows.argtypes = [ctypes.POINTER(_Logits), _i64, _i64, ci, ci, _vp]
    for name in ("kv4_append", "kv4_gather", "attention_kv4", "logits_process_rows"):
        getattr(lib, name).restype = ci


def _tensor(t, name, dtype, shape, index):
    """Data pointer of a contiguous tensor of a dtype and shape on CUDA device ``index`` (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}")
    return t.data_ptr()


@contextlib.contextmanager
def _switched(index, stream):
    import torch

    s = stream
    if s is not None and not hasattr(s, "cuda_stream"):
        s = torch.cuda.ExternalStream(int(s), device=index)
    with torch.cuda.device(index), torch.cuda.stream(s):
        yield torch.cuda.current_stream(index).cuda_stream


class _Here:
    """The current device's current stream, where nothing has to be switched."""

    __slots__ = ("stream",)

    def __init__(self, stream):
        self.stream = stream

    def __enter__(self):
        return self.stream

    def __exit__(self, *exc):
        return False


def _on(index, stream):
    """Context: device ``index`` current, the stream's pointer; what torch allocates inside belongs to that stream."""
    import torch

    if stream is None and torch.cuda.current_device() == index:
        return _Here(_raw_stream(index))
    return _switched(index, stream)


def _raw_stream(index):
    """The device's current stream as a pointer (torch's own short way where it has one: 0.1 us instead of 1.4)."""
    import torch

    short = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return short(index) if short else torch.cuda.current_stream(index).cuda_stream


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(index, *sizes):
    """Of device ``index``, which is current: a function of the sizes and the device alone."""
    return _rwo.capi().attention_kv4_workspace(*sizes)


def _rows(t, name, heads, tokens, dim, dtype, index):
    """[tokens, heads, dim] with the elements of a head side by side."""
    if t.shape != (tokens, heads, dim) or t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {(tokens, heads, dim)} on cuda:{index}")
    s = t.stride()
    if s[2] != 1 and t.numel():
        raise ValueError(f"{name}: the elements of a head must be contiguous (stride(2) == 1)")
    return _Rows(t.data_ptr(), s[0] if tokens > 1 else heads * dim, s[1] if heads > 1 else dim)


def _paged(cache, page_table, seq_lens, cu_tokens, tokens):
    """The cache argument and its device: shapes and types checked, pointers taken."""
    import torch

    if cache.dtype is not torch.uint8 or cache.dim() != 4 or not cache.is_cuda or not cache.is_contiguous() or cache.shape[3] % 20:
        raise ValueError("cache must be a contiguous CUDA uint8 tensor [pages, heads, page_size / 16, 20 * head_dim] (kv4_cache_empty)")
    pages, heads, blocks, held = cache.shape
    if page_table.dim() != 2:
        raise ValueError("page_table must be a 2-D int32 tensor [batch, pages a sequence has room for]")
    batch, width = page_table.shape
    if cu_tokens is None and tokens != batch:
        raise ValueError(f"{tokens} rows for {batch} sequences: cu_tokens is needed where they are not one each")
    index, i32 = cache.get_device(), torch.int32
    return _Cache(cache.data_ptr(), _tensor(page_table, "page_table", i32, (batch, width), index),
                  _tensor(seq_lens, "seq_lens", i32, (batch,), index), _tensor(cu_tokens, "cu_tokens", i32, (batch + 1,), index),
                  pages, blocks * 16, heads, held // 20, batch, width, tokens), index


def kv4_cache_empty(num_pages: int, num_kv_heads: int, page_size: int, head_dim: int, device=None):
    """A zeroed cache [num_pages, num_kv_heads, page_size / 16, 20 * head_dim] of bytes: page_size a multiple of
    16, head_dim 64 or 128.  Room for num_pages * page_size tokens, 1.25 * head_dim bytes a token and head."""
    import torch

    if page_size < 16 or page_size % 16:
        raise ValueError("page_size must be a multiple of 16")
    if head_dim not in (64, 128):
        raise ValueError("head_dim must be 64 or 128")
    return torch.zeros((num_pages, num_kv_heads, page_size // 16, 20 * head_dim), dtype=torch.uint8, device=device or "cuda")


def kv4_append(k, v, cache, page_table, seq_lens, cu_tokens=None, q=None, q_out=None, cos_sin=None, interleaved: bool = False,
               stream=None):
    """Write new keys and values [T, kv_heads, d] (bf16 or fp16) into the 4-bit cache, keys rotated by their positions.

    page_table int32 [B, W] and seq_lens int32 [B] say where a sequence lies and how long it is with the new
    tokens; cu_tokens int32 [B + 1] where its rows are (None: one each).  cos_sin fp32 [positions, rotated]
    holds cosines, then sines; pairs are (i, i + rotated / 2), or neighbours if ``interleaved``.  With q
    [T, heads, d], also rotates q into q_out (default: a new tensor; q_out may be q) and returns it.
    """
    import torch

    if k.dim() != 3:
        raise ValueError("k must be a 3-D tensor [tokens, kv_heads, head_dim]")
    T = int(k.shape[0])
    c, index = _paged(cache, page_table, seq_lens, cu_tokens, T)
    dt, d = _rwo._dtype_code(k), cache.shape[3] // 20
    kr, vr = (_rows(t, n, c.heads, T, d, k.dtype, index) for t, n in ((k, "k"), (v, "v")))
    if q is None and q_out is not None:
        raise ValueError("q_out without q")
    positions = rotated = 0
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be a 2-D float32 tensor [positions, rotated]")
        positions, rotated = cos_sin.shape
    table = _tensor(cos_sin, "cos_sin", torch.float32, (positions, rotated), index)
    qr = qo = None
    heads = 0
    with _on(index, stream) as s:
        if q is not None:
            heads = int(q.shape[1]) if q.dim() == 3 else 0
            qr = _rows(q, "q", heads, T, d, k.dtype, index)
            if q_out is None:
                q_out = torch.empty((T, heads, d), dtype=q.dtype, device=q.device)
            qo = _rows(q_out, "q_out", heads, T, d, k.dtype, index)
        st = _rwo.capi().kv4_append(c, kr, vr, qr, qo, heads, table, positions, rotated, KV4_FLAG_NEIGHBOURS if interleaved else 0, dt, s)
    _rwo._check(st, "kv4_append")
    return q_out


def kv4_gather(cache, page_table, seq_lens, cu_tokens=None, num_tokens: int | None = None, k=None, v=None, dtype=None, stream=None):
    """The last cu_tokens[b + 1] - cu_tokens[b] tokens of each sequence (None: one) read back as bf16 or fp16.

    Returns (k, v), [num_tokens, kv_heads, d] in ``dtype`` (default bf16) unless given; num_tokens defaults to
    the given k's rows, or to one a sequence.  Rows that belong to no sequence are left as they were.
    attention_forward takes them a sequence at a time, [heads, n, d], heads repeated for their query heads.
    """
    import torch

    if num_tokens is None:
        if k is None and cu_tokens is not None:
            raise ValueError("num_tokens (cu_tokens' last entry) is needed to allocate k and v")
        num_tokens = int(k.shape[0]) if k is not None else int(page_table.shape[0])
    c, index = _paged(cache, page_table, seq_lens, cu_tokens, int(num_tokens))
    dtype = dtype or (k.dtype if k is not None else v.dtype if v is not None else torch.bfloat16)
    shape = (int(num_tokens), c.heads, c.head_dim)
    with _on(index, stream) as s:
        k = torch.empty(shape, dtype=dtype, device=cache.device) if k is None else k
        v = torch.empty(shape, dtype=dtype, device=cache.device) if v is None else v
        kr, vr = (_rows(t, n, shape[1], shape[0], shape[2], dtype, index) for t, n in ((k, "k"), (v, "v")))
        st = _rwo.capi().kv4_gather(c, kr, vr, _rwo._dtype_code(k), s)
    _rwo._check(st, "kv4_gather")
    return k, v


def attention_kv4_workspace(batch: int, tokens: int, num_heads: int, num_kv_heads: int, head_dim: int, device=None):
    """A workspace tensor for attention_kv4 calls of these sizes.  Calls that may run at the same time need one each."""
    import torch

    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        n = _workspace_bytes(torch.cuda.current_device(), batch, tokens, num_heads, num_kv_heads, head_dim)
        if n < 0:
            raise _rwo.SoftmaxError(_rwo.ERR_UNSUPPORTED, "attention_kv4_workspace")
        return torch.empty(n, dtype=torch.uint8, device=device)


def attention_kv4(q, cache, page_table, seq_lens, cu_tokens=None, o=None, lse_out=None, scale: float | None = None, workspace=None,
                  stream=None):
    """O = softmax(scale Q K^T) V of q [T, heads, d] (bf16 or fp16) over the 4-bit cache; row i of a sequence sees the
    tokens up to its own position.  scale defaults to 1/sqrt(d).  Returns o (and fills lse_out [T, heads] fp32).

    The workspace (attention_kv4_workspace) is allocated for the call unless given.
    """
    import torch

    if q.dim() != 3:
        raise ValueError("q must be a 3-D tensor [tokens, heads, head_dim]")
    T, heads = int(q.shape[0]), int(q.shape[1])
    c, index = _paged(cache, page_table, seq_lens, cu_tokens, T)
    dt, d = _rwo._dtype_code(q), cache.shape[3] // 20
    qr = _rows(q, "q", heads, T, d, q.dtype, index)
    lse = _tensor(lse_out, "lse_out", torch.float32, (T, heads), index)
    if workspace is not None and (workspace.dtype is not torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != index):
        raise ValueError("workspace must be a contiguous uint8 tensor on the cache's device")
    lib = _rwo.capi()
    with _on(index, stream) as s:
        if o is None:
            o = torch.empty((T, heads, d), dtype=q.dtype, device=q.device)
        op = _tensor(o, "o", q.dtype, (T, heads, d), index)
        if workspace is None:
            n = _workspace_bytes(index, page_table.shape[0], T, heads, cache.shape[1], d)
            workspace = torch.empty(max(n, 0), dtype=torch.uint8, device=q.device)
        st = lib.attention_kv4(c, qr, op, lse, heads, 0.0 if scale is None else float(scale), dt, workspace.data_ptr(),
                                       workspace.numel(), s)
    _rwo._check(st, "attention_kv4")
    return o


def logits_process_rows(x, y=None, out: str = "softmax", lse_out=None, tokens=None, prompt_lens=None, token_lens=None,
                        repetition=None, frequency=None, presence=None, bias_ids=None, bias_values=None, mask=None, scale=None,
                        stream=None):
    """Penalties for repeated tokens, biases, scale and mask on logits x [M, N] (rows may be pitched), then ``out``:
    "logits", "softmax" or "log_softmax".

    tokens int32 [M, L] (prompt, then generated; negative: absent) with prompt_lens and token_lens int32 [M];
    repetition, frequency, presence, scale fp32 [M]; bias_ids int32 and bias_values fp32 [M, K]; mask int32
    [M, words >= ceil(N / 32)], a set bit allows its token.  y defaults to a new contiguous tensor and may be x.
    """
    import torch

    if out not in LOGITS_OUT:
        raise ValueError(f"out must be one of {sorted(LOGITS_OUT)}")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    M, N, ldx = _rwo._rows_strided(x)
    dt, index = _rwo._dtype_code(x), x.get_device()
    a = _Logits(x=x.data_ptr(), ldx=ldx)
    if tokens is not None:
        if tokens.dim() != 2 or token_lens is None:
            raise ValueError("tokens must be a 2-D int32 tensor [M, L], with token_lens")
        a.token_width = int(tokens.shape[1])
        a.tokens = _tensor(tokens, "tokens", torch.int32, (M, a.token_width), index)
        a.token_lens = _tensor(token_lens, "token_lens", torch.int32, (M,), index)
        a.prompt_lens = _tensor(prompt_lens, "prompt_lens", torch.int32, (M,), index)
    elif any(t is not None for t in (prompt_lens, token_lens, repetition, frequency, presence)):
        raise ValueError("penalties need tokens")
    for n, t in (("repetition", repetition), ("frequency", frequency), ("presence", presence), ("scale", scale), ("lse_out", lse_out)):
        if t is not None:
            setattr(a, n, _tensor(t, n, torch.float32, (M,), index))
    if (bias_ids is None) != (bias_values is None):
        raise ValueError("bias_ids and bias_values go together")
    if bias_ids is not None:
        if bias_ids.dim() != 2:
            raise ValueError("bias_ids must be a 2-D int32 tensor [M, K]")
        a.bias_count = int(bias_ids.shape[1])
        a.bias_ids = _tensor(bias_ids, "bias_ids", torch.int32, (M, a.bias_count), index)
        a.bias_values = _tensor(bias_values, "bias_values", torch.float32, (M, a.bias_count), index)
    if mask is not None:
        a.ld_mask = int(mask.shape[1]) if mask.dim() == 2 else 0
        if a.ld_mask < (N + 31) // 32:
            raise ValueError("mask must be an int32 tensor [M, words] with a bit for each token")
        a.mask = _tensor(mask, "mask", torch.int32, (M, a.ld_mask), index)
    with _on(index, stream) as s:
        if y is None:
            y = torch.empty((M, N), dtype=x.dtype, device=x.device)
        if y.shape != (M, N) or y.dtype is not x.dtype or y.get_device() != index:
            raise ValueError("y must have x's shape, dtype and device")
        a.y, a.ldy = y.data_ptr(), _rwo._rows_strided(y)[2]
        st = _rwo.capi().logits_process_rows(a, M, N, dt, LOGITS_OUT[out], s)
    _rwo._check(st, "logits_process_rows")
    return y
