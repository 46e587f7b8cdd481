"""int8 rows and row sampling (rt_quantize_rows_int8, rt_matmul_int8,
rt_linear_int8, rt_sample_rows): the steps from a model's hidden state to its
next token.  No engine; device tensors in, device tensors out.

    w, w_scale = quantize_rows_int8(weights)                 # once: [n, k] -> int8 rows and their scales
    logits = linear_int8(hidden, w, w_scale)                 # [m, k] -> [m, n]
    token, prob = sample_rows(logits, u, temperature=0.8, top_k=50, top_p=0.9)

Matrices are 2-D with neighbouring elements in a row and any row stride.  The
work is enqueued on `stream` (default: torch's current stream on the tensors'
device); tensors made here belong to that stream.
"""
import contextlib
import ctypes

from . import _lib
from ._lib import SampleSettings

_T = {}  # torch and what is looked up in it once


def _torch():
    if not _T:
        import torch
        _T.update(torch=torch, floats={torch.float32: _lib.RT_DTYPE_FLOAT32, torch.bfloat16: _lib.RT_DTYPE_BFLOAT16,
                                       torch.float16: _lib.RT_DTYPE_FLOAT16},
                  raw=getattr(torch._C, "_cuda_getCurrentRawStream", None))
    return _T["torch"]


def _raise(status, what):
    raise _lib.ResidentTopKError(status, what)


def _place(x, stream):
    """(stream handle, context that makes x's device current and, with a stream of
    the caller's, torch's allocations that stream's; None if nothing is to be entered)."""
    torch = _torch()
    device = x.get_device()
    if device < 0:
        raise TypeError("a CUDA tensor is needed")
    if stream is not None:
        if stream.device_index != device:
            raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors on cuda:{device}")
        return stream.cuda_stream, torch.cuda.stream(stream)
    raw = _T["raw"]
    handle = raw(device) if raw is not None else torch.cuda.current_stream(device).cuda_stream
    if torch.cuda.current_device() != device:
        return handle, torch.cuda.device(device)
    return handle, None


def _matrix(t, name, dtypes, device):
    """Rows, columns and row stride of a 2-D CUDA tensor whose rows are dense and do not overlap."""
    torch = _T["torch"]
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {t.dim()}-D")
    dev = t.get_device()
    if dev != device:
        if dev < 0:
            raise TypeError(f"{name} must be a CUDA tensor")
        raise ValueError(f"{name} is on {t.device}, the call on cuda:{device}")
    rows, cols = t.shape
    ld, step = t.stride()
    if rows <= 1 or cols == 0:
        ld = cols
    if (step != 1 and cols > 1) or ld < cols:
        raise TypeError(f"{name} must have neighbouring elements in its rows and rows that do not overlap")
    return rows, cols, ld


def _vector(t, name, dtype, n, device):
    torch = _T["torch"]
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    dev = t.get_device()
    if dev != device:
        if dev < 0:
            raise TypeError(f"{name} must be a CUDA tensor")
        raise ValueError(f"{name} is on {t.device}, the call on cuda:{device}")
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must have shape [{n}], got {list(t.shape)}")
    if n > 1 and t.stride(0) != 1:
        raise TypeError(f"{name} must be contiguous")
    return t.data_ptr()


def _out_matrix(out, m, n, device):
    rows, cols, ld = _matrix(out, "out", _T["floats"], device)
    if rows != m or cols != n:
        raise ValueError(f"out must have shape [{m}, {n}], got {list(out.shape)}")
    return ld


def quantize_rows_int8(x, out=None, out_scale=None, stream=None):
    """Each row of x ([m, k] fp32, bf16 or fp16) as int8 codes and an fp32 scale:
    scale = max|x| / 127, codes = x / scale rounded to the nearest whole number,
    ties to even.  Returns (codes int8 [m, k], scale fp32 [m]).  The codes made here
    have a row stride that is a multiple of 16 with zeros behind each row, the
    layout the products read fastest.  A row with an infinity or NaN gets scale
    NaN and zero codes."""
    torch = _torch()
    handle, context = _place(x, stream) if isinstance(x, torch.Tensor) else _matrix(x, "x", (), 0)
    device = x.get_device()
    m, k, ld = _matrix(x, "x", _T["floats"], device)
    with context or contextlib.nullcontext():
        if out is None:
            pitch = (k + 15) // 16 * 16
            out = torch.empty((m, pitch), dtype=torch.int8, device=x.device)
            if pitch != k:
                out[:, k:].zero_()
                out = out[:, :k]
        if out_scale is None:
            out_scale = torch.empty(m, dtype=torch.float32, device=x.device)
        rows, cols, ldq = _matrix(out, "out", (torch.int8,), device)
        if (rows, cols) != (m, k):
            raise ValueError(f"out must have shape [{m}, {k}], got {list(out.shape)}")
        st = _lib.load().rt_quantize_rows_int8(x.data_ptr(), _T["floats"][x.dtype], m, k, ld, out.data_ptr(), ldq,
                                               _vector(out_scale, "out_scale", torch.float32, m, device), handle)
    if st:
        _raise(st, "quantize_rows_int8")
    return out, out_scale


def matmul_int8(a, a_scale, b, b_scale, bias=None, out=None, out_dtype=None, stream=None):
    """out[i, j] = sum(a[i] * b[j]) * a_scale[i] * b_scale[j] (+ bias[j]) for int8
    rows a [m, k] and b [n, k] with fp32 scales [m] and [n] and an fp32 bias [n].
    The sums are exact; the result is rounded once to out_dtype (default fp32), fp32, bf16
    or fp16.  Returns out [m, n]."""
    torch = _torch()
    handle, context = _place(a, stream) if isinstance(a, torch.Tensor) else _matrix(a, "a", (), 0)
    device = a.get_device()
    m, k, lda = _matrix(a, "a", (torch.int8,), device)
    n, kb, ldb = _matrix(b, "b", (torch.int8,), device)
    if kb != k:
        raise ValueError(f"a has rows of {k}, b rows of {kb}")
    sa = _vector(a_scale, "a_scale", torch.float32, m, device)
    sb = _vector(b_scale, "b_scale", torch.float32, n, device)
    pbias = None if bias is None else _vector(bias, "bias", torch.float32, n, device)
    out, st = _product(context, out, out_dtype or torch.float32, m, n, a.device, device,
                       lambda f, o, dt, ldo: f.rt_matmul_int8(a.data_ptr(), lda, sa, b.data_ptr(), ldb, sb, pbias, o,
                                                              dt, ldo, m, n, k, handle))
    if st:
        _raise(st, "matmul_int8")
    return out


def _product(context, out, out_dtype, m, n, where, device, call):
    if context is not None:
        with context:
            return _product(None, out, out_dtype, m, n, where, device, call)
    if out is None:
        if out_dtype not in _T["floats"]:
            raise TypeError(f"out_dtype must be torch.float32, torch.bfloat16 or torch.float16, got {out_dtype}")
        out = _T["torch"].empty((m, n), dtype=out_dtype, device=where)
        ldo = n
    else:
        ldo = _out_matrix(out, m, n, device)
    return out, call(_lib.load(), out.data_ptr(), _T["floats"][out.dtype], ldo)


def linear_int8(x, w, w_scale, bias=None, out=None, out_dtype=None, workspace=None, stream=None):
    """matmul_int8(*quantize_rows_int8(x), w, w_scale, bias): activations x [m, k]
    (fp32, bf16 or fp16), quantised row by row, times int8 rows w [n, k].  Returns
    out [m, n] in out_dtype (default: x's type).  `workspace`: a uint8 CUDA tensor
    of at least linear_int8_workspace(m, k) bytes, 16-byte aligned, for callers
    that keep one (one for each call that may run at the same time); by default
    one is taken from torch's allocator for the call."""
    torch = _torch()
    handle, context = _place(x, stream) if isinstance(x, torch.Tensor) else _matrix(x, "x", (), 0)
    device = x.get_device()
    m, k, ldx = _matrix(x, "x", _T["floats"], device)
    n, kw, ldw = _matrix(w, "w", (torch.int8,), device)
    if kw != k:
        raise ValueError(f"x has rows of {k}, w rows of {kw}")
    sw = _vector(w_scale, "w_scale", torch.float32, n, device)
    pbias = None if bias is None else _vector(bias, "bias", torch.float32, n, device)

    def call(lib, o, dt, ldo):
        need = lib.rt_linear_int8_workspace(m, k)
        if workspace is not None:
            ws, have = _workspace(workspace, device)
        elif need > 0:
            keep = torch.empty(need, dtype=torch.uint8, device=x.device)
            ws, have = keep.data_ptr(), need
        else:
            ws, have = None, 0
        return lib.rt_linear_int8(x.data_ptr(), _T["floats"][x.dtype], ldx, w.data_ptr(), ldw, sw, pbias, o, dt, ldo,
                                  m, n, k, ws, have, handle)

    out, st = _product(context, out, out_dtype or x.dtype, m, n, x.device, device, call)
    if st:
        _raise(st, "linear_int8")
    return out


def linear_int8_workspace(m, k):
    """Bytes of workspace linear_int8 needs for m activations of depth k."""
    need = _lib.load().rt_linear_int8_workspace(int(m), int(k))
    if need < 0:
        _raise(_lib.RT_EINVAL, "linear_int8_workspace")
    return need


def sample_rows_workspace(r, v):
    """Bytes of workspace sample_rows needs for r rows of v logits."""
    need = _lib.load().rt_sample_rows_workspace(int(r), int(v))
    if need < 0:
        _raise(_lib.RT_EINVAL, "sample_rows_workspace")
    return need


def _workspace(t, device):
    if not isinstance(t, _T["torch"].Tensor) or t.dtype != _T["torch"].uint8 or not t.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor")
    if t.get_device() != device:
        raise ValueError(f"workspace is on {t.device}, the call on cuda:{device}")
    return t.data_ptr(), t.numel()


def sample_rows(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out_token=None, out_prob=None,
                workspace=None, stream=None):
    """One token for each row of logits ([r, v] fp32, bf16 or fp16), drawn with the
    given random numbers u (fp32 [r] in [0, 1)).  Each setting is a number or a
    device tensor [r] (fp32; int32 for top_k).

    Tokens are ordered by logit (ties: the lower index first; NaN as -inf) and
    weigh exp((logit - largest) / temperature).  Kept are the first top_k of
    them (0: all), of those the shortest prefix with at least top_p of their
    weight (1: all), and of those the tokens that weigh at least min_p (0: all);
    the first always.  Drawn is the first token, in index order, at which the
    running weight of the kept ones exceeds u times their sum.  temperature 0
    takes the first token of the order.

    Returns (token int32 [r], prob fp32 [r], the drawn token's share of the kept
    weight); -1 and 0 for a row with no logit above -inf."""
    torch = _torch()
    handle, context = _place(logits, stream) if isinstance(logits, torch.Tensor) else _matrix(logits, "logits", (), 0)
    device = logits.get_device()
    r, v, ld = _matrix(logits, "logits", _T["floats"], device)
    pu = _vector(u, "u", torch.float32, r, device)
    s = SampleSettings()
    tensor = torch.Tensor
    if isinstance(temperature, tensor):
        s.temperatures = _vector(temperature, "temperature", torch.float32, r, device)
    else:
        s.temperature = temperature
    if isinstance(top_k, tensor):
        s.top_ks = _vector(top_k, "top_k", torch.int32, r, device)
    else:
        s.top_k = min(max(int(top_k), 0), 2147483647)
    if isinstance(top_p, tensor):
        s.top_ps = _vector(top_p, "top_p", torch.float32, r, device)
    else:
        s.top_p = top_p
    if isinstance(min_p, tensor):
        s.min_ps = _vector(min_p, "min_p", torch.float32, r, device)
    else:
        s.min_p = min_p
    with context or contextlib.nullcontext():
        lib = _lib.load()
        if out_token is None:
            out_token = torch.empty(r, dtype=torch.int32, device=logits.device)
        if out_prob is None:
            out_prob = torch.empty(r, dtype=torch.float32, device=logits.device)
        if workspace is not None:
            ws, have = _workspace(workspace, device)
        else:
            have = lib.rt_sample_rows_workspace(r, v)
            keep = torch.empty(have, dtype=torch.uint8, device=logits.device) if have > 0 else None
            ws = keep.data_ptr() if have > 0 else None
        st = lib.rt_sample_rows(logits.data_ptr(), _T["floats"][logits.dtype], r, v, ld, pu, ctypes.byref(s),
                                _vector(out_token, "out_token", torch.int32, r, device),
                                _vector(out_prob, "out_prob", torch.float32, r, device), ws, have, handle)
    if st:
        _raise(st, "sample_rows")
    return out_token, out_prob
