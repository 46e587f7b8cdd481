"""int8 rows and row sampling (rt_quantize_rows_int8, rt_matmul_int8,
rt_linear_int8, rt_sample_rows): the steps from a model's hidden state to its
next token.  No engine; device tensors in, device tensors out.

    w, w_scale = quantize_rows_int8(weights)                 # once: [n, k] -> int8 rows and their scales
    logits = linear_int8(hidden, w, w_scale)                 # [m, k] -> [m, n]
    token, prob = sample_rows(logits, u, temperature=0.8, top_k=50, top_p=0.9)

Matrices are 2-D with neighbouring elements in a row and any row stride.  The
work is enqueued on `stream` (default: torch's current stream on the tensors'
device); tensors made here belong to that stream.  None of these has a gradient:
what they return never requires one, whatever the inputs do.
"""
import ctypes

from . import _lib
from ._lib import SampleSettings


class _Once:
    """torch, the library and what is looked up in them once, at the first call."""
    lib = None

    def load(self):
        import torch
        lib = _lib.load()
        self.torch = torch
        self.tensor = torch.Tensor
        self.empty = torch.empty
        self.fp32, self.int32, self.int8, self.uint8 = torch.float32, torch.int32, torch.int8, torch.uint8
        self.floats = {torch.float32: _lib.RT_DTYPE_FLOAT32, torch.bfloat16: _lib.RT_DTYPE_BFLOAT16,
                       torch.float16: _lib.RT_DTYPE_FLOAT16}
        self.int8s = {torch.int8: None}
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # a tenth of current_stream()'s time
        self.stream = raw or (lambda device: torch.cuda.current_stream(device).cuda_stream)
        self.device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        self.lib = lib
        return self


_once = _Once()


def _elsewhere(o, x, name, stream):
    """None where x is on the current device and no stream is named; else the context to
    call again in: x's device current and, with a stream, torch's allocations that stream's."""
    if not isinstance(x, o.tensor):
        raise TypeError(f"{name} must be a torch tensor")
    device = x.get_device()
    if device < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if stream is not None:
        if stream.device_index != device:
            raise ValueError(f"the stream is on cuda:{stream.device_index}, {name} on cuda:{device}")
        return o.torch.cuda.stream(stream)
    return None if o.device() == device else o.torch.cuda.device(device)


def _matrix(o, t, name, dtypes, device):
    """Rows, columns and row stride of a 2-D CUDA tensor whose rows are dense and do not overlap."""
    if not isinstance(t, o.tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {t.dim()}-D")
    if t.get_device() != device:
        _wrong_device(t, name, device)
    rows, cols = t.shape
    ld, step = t.stride()
    if rows <= 1 or cols == 0:
        ld = cols
    if (step != 1 and cols > 1) or ld < cols:
        raise TypeError(f"{name} must have neighbouring elements in its rows and rows that do not overlap")
    return rows, cols, ld


def _wrong_device(t, name, device):
    if t.get_device() < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} is on {t.device}, the call on cuda:{device}")


def _vector(o, t, name, dtype, n, device):
    """Address of a contiguous CUDA tensor [n]."""
    if not isinstance(t, o.tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        _wrong_device(t, name, device)
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must have shape [{n}], got {list(t.shape)}")
    if n > 1 and t.stride(0) != 1:
        raise TypeError(f"{name} must be contiguous")
    return t.data_ptr()


def _output(o, out, dtype, default, m, n, like, device):
    """(out, its type's code, its row stride), made here where none is given, of type
    `dtype` (None: out's own, or `default`)."""
    if out is None:
        dtype = default if dtype is None else dtype
        code = o.floats.get(dtype)
        if code is None:
            raise TypeError(f"out_dtype must be torch.float32, torch.bfloat16 or torch.float16, got {dtype}")
        return o.empty(m, n, dtype=dtype, device=like.device), code, n
    rows, cols, ld = _matrix(o, out, "out", o.floats, device)
    if rows != m or cols != n:
        raise ValueError(f"out must have shape [{m}, {n}], got {list(out.shape)}")
    if dtype is not None and dtype != out.dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {dtype}")
    return out, o.floats[out.dtype], ld


def _workspace(o, t, device):
    if not isinstance(t, o.tensor) or t.dtype != o.uint8 or not t.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor")
    if t.get_device() != device:
        _wrong_device(t, "workspace", device)
    return t.data_ptr(), t.numel()


def quantize_rows_int8(x, out=None, out_scale=None, stream=None):
    """Each row of x ([m, k] fp32, bf16 or fp16) as int8 codes and an fp32 scale:
    scale = max|x| / 127, codes = x / scale rounded to the nearest whole number,
    ties to even.  Returns (codes int8 [m, k], scale fp32 [m]).  The codes made here
    have a row stride that is a multiple of 16 with zeros behind each row, the
    layout the products read fastest.  A row with an infinity or NaN gets scale
    NaN and zero codes."""
    o = _once if _once.lib else _once.load()
    context = _elsewhere(o, x, "x", stream)
    if context is not None:
        with context:
            return quantize_rows_int8(x, out, out_scale)
    device = x.get_device()
    m, k, ld = _matrix(o, x, "x", o.floats, device)
    if out is None:
        ldq = (k + 15) // 16 * 16
        out = o.empty(m, ldq, dtype=o.int8, device=x.device)
        if ldq != k:
            out[:, k:].zero_()
            out = out[:, :k]
    else:
        rows, cols, ldq = _matrix(o, out, "out", o.int8s, device)
        if (rows, cols) != (m, k):
            raise ValueError(f"out must have shape [{m}, {k}], got {list(out.shape)}")
    if out_scale is None:
        out_scale = o.empty(m, dtype=o.fp32, device=x.device)
    st = o.lib.rt_quantize_rows_int8(x.data_ptr(), o.floats[x.dtype], m, k, ld, out.data_ptr(), ldq,
                                     _vector(o, out_scale, "out_scale", o.fp32, m, device), o.stream(device))
    if st:
        raise _lib.ResidentTopKError(st, "quantize_rows_int8")
    return out, out_scale


def matmul_int8(a, a_scale, b, b_scale, bias=None, out=None, out_dtype=None, stream=None):
    """out[i, j] = sum(a[i] * b[j]) * a_scale[i] * b_scale[j] (+ bias[j]) for int8
    rows a [m, k] and b [n, k] with fp32 scales [m] and [n] and an fp32 bias [n].
    The sums are exact; what follows them rounds in fp32 step by step, the result once
    more to out_dtype (fp32, bf16 or fp16; default: out's type, or fp32).  Returns out [m, n]."""
    o = _once if _once.lib else _once.load()
    context = _elsewhere(o, a, "a", stream)
    if context is not None:
        with context:
            return matmul_int8(a, a_scale, b, b_scale, bias, out, out_dtype)
    device = a.get_device()
    m, k, lda = _matrix(o, a, "a", o.int8s, device)
    n, kb, ldb = _matrix(o, b, "b", o.int8s, device)
    if kb != k:
        raise ValueError(f"a has rows of {k}, b rows of {kb}")
    sa = _vector(o, a_scale, "a_scale", o.fp32, m, device)
    sb = _vector(o, b_scale, "b_scale", o.fp32, n, device)
    pbias = None if bias is None else _vector(o, bias, "bias", o.fp32, n, device)
    out, code, ldo = _output(o, out, out_dtype, o.fp32, m, n, a, device)
    st = o.lib.rt_matmul_int8(a.data_ptr(), lda, sa, b.data_ptr(), ldb, sb, pbias, out.data_ptr(), code, ldo, m, n, k,
                              o.stream(device))
    if st:
        raise _lib.ResidentTopKError(st, "matmul_int8")
    return out


def linear_int8(x, w, w_scale, bias=None, out=None, out_dtype=None, workspace=None, stream=None):
    """matmul_int8(*quantize_rows_int8(x), w, w_scale, bias): activations x [m, k]
    (fp32, bf16 or fp16), quantised row by row, times int8 rows w [n, k].  Returns
    out [m, n] in out_dtype (default: out's type, or x's).  `workspace`: a uint8 CUDA tensor
    of at least linear_int8_workspace(m, n, k) bytes, 16-byte aligned, for callers
    that keep one (one for each call that may run at the same time); by default
    one is taken from torch's allocator for the call."""
    o = _once if _once.lib else _once.load()
    context = _elsewhere(o, x, "x", stream)
    if context is not None:
        with context:
            return linear_int8(x, w, w_scale, bias, out, out_dtype, workspace)
    device = x.get_device()
    m, k, ldx = _matrix(o, x, "x", o.floats, device)
    n, kw, ldw = _matrix(o, w, "w", o.int8s, device)
    if kw != k:
        raise ValueError(f"x has rows of {k}, w rows of {kw}")
    sw = _vector(o, w_scale, "w_scale", o.fp32, n, device)
    pbias = None if bias is None else _vector(o, bias, "bias", o.fp32, n, device)
    out, code, ldo = _output(o, out, out_dtype, x.dtype, m, n, x, device)
    lib = o.lib
    if workspace is not None:
        ws, have = _workspace(o, workspace, device)
    else:
        ws, have = None, lib.rt_linear_int8_workspace(m, n, k)
        if have > 0:
            workspace = o.empty(have, dtype=o.uint8, device=x.device)
            ws = workspace.data_ptr()
    st = lib.rt_linear_int8(x.data_ptr(), o.floats[x.dtype], ldx, w.data_ptr(), ldw, sw, pbias, out.data_ptr(), code,
                            ldo, m, n, k, ws, have, o.stream(device))
    if st:
        raise _lib.ResidentTopKError(st, "linear_int8")
    return out


def linear_int8_workspace(m, n, k):
    """Bytes of workspace linear_int8 needs for m activations of depth k and n rows
    (outputs m n above 2^37 have a size here, too, but linear_int8 refuses them)."""
    need = _lib.load().rt_linear_int8_workspace(int(m), int(n), int(k))
    if need < 0:
        raise _lib.ResidentTopKError(_lib.RT_EINVAL, "linear_int8_workspace")
    return need


def sample_rows_workspace(r, v):
    """Bytes of workspace sample_rows needs for r rows of v logits."""
    need = _lib.load().rt_sample_rows_workspace(int(r), int(v))
    if need < 0:
        raise _lib.ResidentTopKError(_lib.RT_EINVAL, "sample_rows_workspace")
    return need


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
    o = _once if _once.lib else _once.load()
    context = _elsewhere(o, logits, "logits", stream)
    if context is not None:
        with context:
            return sample_rows(logits, u, temperature, top_k, top_p, min_p, out_token, out_prob, workspace)
    device = logits.get_device()
    r, v, ld = _matrix(o, logits, "logits", o.floats, device)
    pu = _vector(o, u, "u", o.fp32, r, device)
    s, tensor = SampleSettings(), o.tensor
    if isinstance(temperature, tensor):
        s.temperatures = _vector(o, temperature, "temperature", o.fp32, r, device)
    else:
        s.temperature = temperature
    if isinstance(top_k, tensor):
        s.top_ks = _vector(o, top_k, "top_k", o.int32, r, device)
    else:
        s.top_k = min(max(int(top_k), 0), 2147483647)
    if isinstance(top_p, tensor):
        s.top_ps = _vector(o, top_p, "top_p", o.fp32, r, device)
    else:
        s.top_p = top_p
    if isinstance(min_p, tensor):
        s.min_ps = _vector(o, min_p, "min_p", o.fp32, r, device)
    else:
        s.min_p = min_p
    if out_token is None:
        out_token = o.empty(r, dtype=o.int32, device=logits.device)
        ptoken = out_token.data_ptr()
    else:
        ptoken = _vector(o, out_token, "out_token", o.int32, r, device)
    if out_prob is None:
        out_prob = o.empty(r, dtype=o.fp32, device=logits.device)
        pprob = out_prob.data_ptr()
    else:
        pprob = _vector(o, out_prob, "out_prob", o.fp32, r, device)
    lib = o.lib
    if workspace is not None:
        ws, have = _workspace(o, workspace, device)
    else:
        ws, have = None, lib.rt_sample_rows_workspace(r, v)
        if have > 0:
            workspace = o.empty(have, dtype=o.uint8, device=logits.device)
            ws = workspace.data_ptr()
    st = lib.rt_sample_rows(logits.data_ptr(), o.floats[logits.dtype], r, v, ld, pu, ctypes.byref(s), ptoken, pprob,
                            ws, have, o.stream(device))
    if st:
        raise _lib.ResidentTopKError(st, "sample_rows")
    return out_token, out_prob
