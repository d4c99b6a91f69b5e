"""Operators of the language models that the optimizers of this library train.

Forward and gradient operators over the C ABI (device memory and streams only,
as in okls.py):

`embedding`, `embedding_grad`            rows of a token table, scaled; gradient by sorted tokens
`rms_norm`, `rms_norm_grad`              norm with the residual's addition, output in 32, 16 or 8 bits
`fp8_quantize`, `fp8_matmul`             e4m3 values with a scale for each 128, and their product
`token_logprobs`, `token_logprobs_grad`  log probabilities of given tokens, entropy, best alternatives

and the same as differentiable functions of torch.autograd:

`embed`, `norm`, `linear`, `logprobs`

Tensors are CUDA tensors on one device whose last dimension is contiguous;
rows may have any pitch.  fp32 and bf16 are taken, ids are int32 or int64.
Negative ids are padding: zeros out, no loss, no gradient.  An id at or past
the vocabulary is treated as padding and recorded in the device's status
word, which `query_status` reads.

Every function runs on the current stream, or on `stream`.  Outputs and
scratch come from torch's allocator on that stream.  No call synchronises,
apart from `query_status`.
"""

from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass

import torch

from . import _lib as L

FP8_GROUP = 128
_FLOATS = {torch.float32: L.OKLS_F32, torch.bfloat16: L.OKLS_BF16}
_BLOCKS = {"row": L.FP8_ROW, "square": L.FP8_SQUARE}
_STATUS: dict[int, torch.Tensor] = {}


# ------------------------------------------------------------------ helpers
def _fail(msg: str):
    raise ValueError("okls.lm: " + msg)


def _dtype(t: torch.Tensor, name: str) -> int:
    code = _FLOATS.get(t.dtype)
    if code is None:
        _fail(f"{name} must be fp32 or bf16, not {t.dtype}")
    return code


def _out_dtype(dtype: torch.dtype) -> int:
    code = _FLOATS.get(dtype)
    if code is None:
        _fail(f"the output type must be fp32 or bf16, not {dtype}")
    return code


def _matrix(t: torch.Tensor, name: str) -> torch.Tensor:
    """`t` as rows x columns without a copy."""
    if t.dim() == 2:
        if t.stride(1) == 1 or t.shape[1] <= 1 or t.numel() == 0:
            return t
        _fail(f"the last dimension of {name} must be contiguous")
    if t.dim() == 0:
        _fail(f"{name} needs at least one dimension")
    try:
        t = t.view(-1, t.shape[-1]) if t.numel() else t.reshape(t.shape[:-1].numel(), t.shape[-1])
    except RuntimeError:
        _fail(f"the leading dimensions of {name} do not fold into rows without a copy")
    if t.numel() and t.shape[1] > 1 and t.stride(1) != 1:
        _fail(f"the last dimension of {name} must be contiguous")
    return t


def _vector(t: torch.Tensor, name: str, dtype=None, count: int | None = None) -> torch.Tensor:
    if not t.is_contiguous():
        _fail(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        _fail(f"{name} must be {dtype}, not {t.dtype}")
    if count is not None and t.numel() != count:
        _fail(f"{name} must hold {count} values, not {t.numel()}")
    return t


def _ids(t: torch.Tensor, count: int) -> int:
    if t.dtype not in (torch.int32, torch.int64):
        _fail(f"ids must be int32 or int64, not {t.dtype}")
    _vector(t, "ids", count=count)
    return int(t.dtype == torch.int64)


def _ld(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _same(t: torch.Tensor, like: torch.Tensor, name: str):
    if t.shape != like.shape:
        _fail(f"{name} has shape {tuple(t.shape)}, not {tuple(like.shape)}")
    if t.dtype != like.dtype:
        _fail(f"{name} is {t.dtype}, not {like.dtype}")


@contextlib.contextmanager
def _other(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


_HERE = contextlib.nullcontext()


def _on(stream, *tensors):
    """The device and stream that a call runs on; its allocations belong to them."""
    device = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            _fail("tensors must be on a CUDA device")
        if device is None:
            device = t.device
        elif t.device != device:
            _fail(f"tensors on {device} and {t.device}")
    if stream is None and device.index == torch.cuda.current_device():
        return _HERE
    return _other(device, stream)


def _stream(t: torch.Tensor) -> int:
    """Handle of the current stream of t's device (the current device)."""
    # the same handle as torch.cuda.current_stream().cuda_stream, without building a Stream object, which
    # costs more than a launch
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _ptr(t: torch.Tensor | None) -> int:
    return 0 if t is None else t.data_ptr()


def _status_word(device: torch.device) -> torch.Tensor:
    w = _STATUS.get(device.index)
    if w is None:
        # zeroed and waited for, so that any stream may use it from now on
        w = torch.zeros(64, dtype=torch.int32, device=device)
        torch.cuda.current_stream().synchronize()
        _STATUS[device.index] = w
    return w


def query_status(device=None, stream=None) -> int:
    """Synchronise the stream and return (and clear) the device's status word;
    raises OklsError for a token id past the vocabulary or an expired wait."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    with _other(dev, stream):
        w = _status_word(dev)
        v = ctypes.c_uint32(0)
        L.check(L.lib().okls_status_word_read(w.data_ptr(), _stream(w), ctypes.byref(v)))
    return v.value


def _workspace(need: int, device) -> torch.Tensor | None:
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


# ---------------------------------------------------------------- embedding
def embedding(weight: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0, out_dtype: torch.dtype | None = None,
              stream=None) -> torch.Tensor:
    """scale * weight[ids], of shape ids.shape + (dim,); zeros for padding."""
    if weight.dim() != 2:
        _fail("weight must be vocab x dim")
    w = _matrix(weight, "weight")
    dt, i64 = _dtype(w, "weight"), _ids(ids, ids.numel())
    od = dt if out_dtype is None else _out_dtype(out_dtype)
    with _on(stream, weight, ids):
        out = torch.empty(*ids.shape, w.shape[1], dtype=out_dtype or w.dtype, device=w.device)
        L.check(L.lib().okls_embedding(_ptr(w), dt, _ld(w), w.shape[0], w.shape[1], _ptr(ids), i64, ids.numel(),
                                       scale, _ptr(out), od, w.shape[1], _ptr(_status_word(w.device)), _stream(w)))
    return out


def embedding_grad(dy: torch.Tensor, ids: torch.Tensor, vocab: int, *, scale: float = 1.0,
                   base: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """base + scale * (sum of dy's rows by token), vocab x dim.

    `base` None stands for zeros.  With `out` the result goes there; out=base
    adds in place and touches only the rows of tokens that occur."""
    d = _matrix(dy, "dy")
    dt, i64 = _dtype(d, "dy"), _ids(ids, d.shape[0])
    shape = (vocab, d.shape[1])
    for t, name in ((base, "base"), (out, "out")):
        if t is not None and (tuple(t.shape) != shape or _matrix(t, name) is not t):
            _fail(f"{name} must be a matrix of shape {shape}")
    if base is not None and out is not None and base.dtype != out.dtype:
        _fail("base and out must have one type")
    with _on(stream, dy, ids, base, out):
        if out is None:
            out = torch.empty(shape, dtype=dtype if base is None else base.dtype, device=d.device)
        od = _out_dtype(out.dtype)
        need = ctypes.c_size_t()
        lib = L.lib()
        L.check(lib.okls_embedding_grad_workspace_bytes(d.shape[0], vocab, d.shape[1], ctypes.byref(need)))
        ws = _workspace(need.value, d.device)
        L.check(lib.okls_embedding_grad(_ptr(d), dt, _ld(d), _ptr(ids), i64, d.shape[0], vocab, d.shape[1], scale,
                                        _ptr(base), 0 if base is None else _ld(base), _ptr(out), od, _ld(out),
                                        _ptr(ws), need.value, _ptr(_status_word(d.device)), _stream(d)))
    return out


# --------------------------------------------------------------------- norm
@dataclass
class NormOutput:
    """y (a tensor, or an Fp8Tensor), the sum that was normed, and 1 / rms."""
    y: object
    residual: torch.Tensor
    rstd: torch.Tensor


def rms_norm(x: torch.Tensor, weight: torch.Tensor, *, residual: torch.Tensor | None = None, eps: float = 1e-6,
             out_dtype: torch.dtype | None = None, inplace: bool = False, stream=None) -> NormOutput:
    """s = x + residual; y = s / sqrt(mean(s^2) + eps) * weight.

    `out_dtype` may be fp32, bf16 (default: x's type) or float8_e4m3fn; an
    8-bit y is an Fp8Tensor with row groups.  `inplace` writes s over
    `residual`.  Without a residual, s is x itself."""
    m = _matrix(x, "x")
    dt = _dtype(m, "x")
    wd = _dtype(_vector(weight, "weight", count=m.shape[1]), "weight")
    out_dtype = out_dtype or m.dtype
    fp8 = out_dtype == torch.float8_e4m3fn
    od = L.OKLS_E4M3 if fp8 else _out_dtype(out_dtype)
    r = None
    if residual is not None:
        r = _matrix(residual, "residual")
        _same(residual, x, "residual")
    rows, dim = m.shape
    with _on(stream, x, weight, residual):
        dev = m.device
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        r_ptr = ldr = s_ptr = lds = sc_ptr = sc_row = sc_group = 0
        total = x
        if r is not None:
            r_ptr, ldr = r.data_ptr(), _ld(r)
            total = residual if inplace else torch.empty(x.shape, dtype=x.dtype, device=dev)
            s_ptr, lds = (r_ptr, ldr) if inplace else (total.data_ptr(), dim)
        if fp8:
            y = _fp8_empty(rows, dim, "row", dev)
            y_ptr, ldy, sc_ptr = y.data.data_ptr(), y.data.stride(0), y.scale.data_ptr()
            sc_row, sc_group = y.scale.stride()
        else:
            y = torch.empty(x.shape, dtype=out_dtype, device=dev)
            y_ptr, ldy = y.data_ptr(), dim
        L.check(L.lib().okls_rms_norm(m.data_ptr(), dt, _ld(m), r_ptr, ldr, weight.data_ptr(), wd, rows, dim, eps,
                                      y_ptr, od, ldy, sc_ptr, sc_row, sc_group, s_ptr, lds, rstd.data_ptr(),
                                      _stream(m)))
    return NormOutput(y, total, rstd)


def rms_norm_grad(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, *,
                  dresidual: torch.Tensor | None = None, need_dweight: bool = True, stream=None):
    """(ds, dweight): the gradient of x and residual alike, of s's type, and of
    the weight in fp32 (None unless `need_dweight`).  `s` and `rstd` are what
    rms_norm returned; `dresidual` is the gradient that reaches s from elsewhere."""
    g, m = _matrix(dy, "dy"), _matrix(s, "s")
    if g.shape != m.shape:
        _fail(f"dy has shape {tuple(dy.shape)}, not {tuple(s.shape)}")
    gd, sd = _dtype(g, "dy"), _dtype(m, "s")
    rows, dim = m.shape
    wd = _dtype(_vector(weight, "weight", count=dim), "weight")
    _vector(rstd, "rstd", torch.float32, rows)
    e = None
    if dresidual is not None:
        e = _matrix(dresidual, "dresidual")
        _same(dresidual, s, "dresidual")
    with _on(stream, dy, s, weight, rstd, dresidual):
        ds = torch.empty(s.shape, dtype=m.dtype, device=m.device)
        dw = torch.empty(dim, dtype=torch.float32, device=m.device) if need_dweight else None
        need = ctypes.c_size_t()
        lib = L.lib()
        if need_dweight:
            L.check(lib.okls_rms_norm_grad_workspace_bytes(rows, dim, ctypes.byref(need)))
        ws = _workspace(need.value, m.device)
        L.check(lib.okls_rms_norm_grad(_ptr(g), gd, _ld(g), _ptr(m), sd, _ld(m), _ptr(weight), wd, _ptr(rstd), _ptr(e),
                                       0 if e is None else _ld(e), rows, dim, _ptr(ds), dim, _ptr(dw), _ptr(ws),
                                       need.value, _stream(m)))
    return ds, dw


# -------------------------------------------------------------------- 8 bits
@dataclass
class Fp8Tensor:
    """A matrix in e4m3 with a scale for each 128: data[i, j] * scale[i or
    i // 128, j // 128] stands for the value.  block "row" has a scale for
    each 128 columns of a row, "square" for each 128 x 128 block."""
    data: torch.Tensor
    scale: torch.Tensor
    block: str = "row"

    def __post_init__(self):
        if self.block not in _BLOCKS:
            _fail(f"block must be one of {sorted(_BLOCKS)}")
        if self.data.dim() != 2 or self.data.dtype != torch.float8_e4m3fn:
            _fail("data must be a matrix of float8_e4m3fn")
        rows, cols = self.data.shape
        want = (rows if self.block == "row" else -(-rows // FP8_GROUP), -(-cols // FP8_GROUP))
        if tuple(self.scale.shape) != want or self.scale.dtype != torch.float32:
            _fail(f"scale must be fp32 of shape {want}")
        if self.data.numel() and cols > 1 and self.data.stride(1) != 1:
            _fail("the last dimension of data must be contiguous")

    @property
    def shape(self):
        return self.data.shape

    def float(self) -> torch.Tensor:
        """The values in fp32."""
        s = self.scale
        if self.block == "square":
            s = s.repeat_interleave(FP8_GROUP, 0)[: self.data.shape[0]]
        return self.data.float() * s.repeat_interleave(FP8_GROUP, 1)[:, : self.data.shape[1]]


def _fp8_empty(rows: int, cols: int, block: str, device) -> Fp8Tensor:
    """Rows start at multiples of 128 bytes (the product's copies need 16); the
    scales lie group by group, so that neighbouring rows' scales are neighbours."""
    groups = -(-cols // FP8_GROUP)
    data = torch.empty_strided((rows, cols), (max(groups, 1) * FP8_GROUP, 1), dtype=torch.float8_e4m3fn, device=device)
    lines = rows if block == "row" else -(-rows // FP8_GROUP)
    scale = torch.empty_strided((lines, groups), (1, max(-(-lines // 4) * 4, 1)), dtype=torch.float32, device=device)
    q = object.__new__(Fp8Tensor)  # right by construction: __post_init__ has nothing to check
    q.data, q.scale, q.block = data, scale, block
    return q


def fp8_quantize(x: torch.Tensor, *, block: str = "row", transpose: bool = False, both: bool = False, stream=None):
    """An Fp8Tensor of x (rows x columns), of its transpose, or the pair of
    them from one read.  The groups of the transpose lie along its own rows."""
    if block not in _BLOCKS:
        _fail(f"block must be one of {sorted(_BLOCKS)}")
    m = _matrix(x, "x")
    dt = _dtype(m, "x")
    rows, cols = m.shape
    with _on(stream, x):
        q = _fp8_empty(rows, cols, block, m.device) if both or not transpose else None
        t = _fp8_empty(cols, rows, block, m.device) if both or transpose else None
        args = []
        for f in (q, t):
            args += (0, 0, 0, 0, 0) if f is None else (f.data.data_ptr(), f.data.stride(0), f.scale.data_ptr(),
                                                       *f.scale.stride())
        L.check(L.lib().okls_fp8_quantize(m.data_ptr(), dt, _ld(m), rows, cols, _BLOCKS[block], *args, _stream(m)))
    return (q, t) if both else t if transpose else q


def fp8_matmul(a: Fp8Tensor, b: Fp8Tensor, *, out_dtype: torch.dtype = torch.bfloat16,
               out: torch.Tensor | None = None, accumulate: bool = False, stream=None) -> torch.Tensor:
    """a b^T for a (m x k, row groups) and b (n x k, row groups or square
    blocks): m x n in bf16 or fp32.  With `accumulate` it is added to `out`."""
    if a.block != "row":
        _fail("the first factor needs row groups")
    (m, k), (n, k2) = a.shape, b.shape
    if k != k2:
        _fail(f"sums of length {k} and {k2}")
    if out is None and accumulate:
        _fail("accumulate needs out")
    if out is not None:
        if tuple(out.shape) != (m, n) or _matrix(out, "out") is not out:
            _fail(f"out must be a matrix of shape {(m, n)}")
        out_dtype = out.dtype
    od = _out_dtype(out_dtype)
    with _on(stream, a.data, a.scale, b.data, b.scale, out):
        dev = a.data.device
        if out is None:
            out = torch.empty((m, n), dtype=out_dtype, device=dev)
        lib = L.lib()
        need = ctypes.c_size_t()
        L.check(lib.okls_fp8_matmul_workspace_bytes(m, n, k, ctypes.byref(need)))
        ws = _workspace(need.value, dev)
        L.check(lib.okls_fp8_matmul(a.data.data_ptr(), a.data.stride(0), a.scale.data_ptr(), *a.scale.stride(),
                                    b.data.data_ptr(), b.data.stride(0), b.scale.data_ptr(), *b.scale.stride(),
                                    _BLOCKS[b.block], m, n, k, out.data_ptr(), od, _ld(out), int(accumulate), _ptr(ws),
                                    need.value, _status_word(dev).data_ptr(), _stream(out)))
    return out


# --------------------------------------------------------- log probabilities
@dataclass
class TokenLogprobs:
    """Per row: log probability of the given token, entropy, log of the sum of
    exponentials; with top_k, the best tokens and their log probabilities."""
    logp: torch.Tensor
    entropy: torch.Tensor
    lse: torch.Tensor
    top_ids: torch.Tensor | None = None
    top_logp: torch.Tensor | None = None


def token_logprobs(logits: torch.Tensor, ids: torch.Tensor, *, top_k: int = 0, scale: float = 1.0,
                   stream=None) -> TokenLogprobs:
    """Log probabilities of `ids` under softmax(scale * logits), shaped like
    ids; `top_k` <= 32 best alternatives, equal logits in the order of their ids."""
    z = _matrix(logits, "logits")
    rows, vocab = z.shape
    dt, i64 = _dtype(z, "logits"), _ids(ids, rows)
    lead = logits.shape[:-1]
    with _on(stream, logits, ids):
        dev = z.device
        logp = torch.empty(lead, dtype=torch.float32, device=dev)
        entropy = torch.empty(lead, dtype=torch.float32, device=dev)
        lse = torch.empty(lead, dtype=torch.float32, device=dev)
        top_ids = top_logp = None
        if top_k > 0:
            top_ids = torch.empty((*lead, top_k), dtype=torch.int32, device=dev)
            top_logp = torch.empty((*lead, top_k), dtype=torch.float32, device=dev)
        L.check(L.lib().okls_token_logprobs(z.data_ptr(), dt, _ld(z), ids.data_ptr(), i64, rows, vocab, scale, top_k,
                                            logp.data_ptr(), entropy.data_ptr(), lse.data_ptr(), _ptr(top_ids),
                                            _ptr(top_logp), _status_word(dev).data_ptr(), _stream(z)))
    return TokenLogprobs(logp, entropy, lse, top_ids, top_logp)


def token_logprobs_grad(logits: torch.Tensor, ids: torch.Tensor, result: TokenLogprobs, dlogp: torch.Tensor, *,
                        dentropy: torch.Tensor | None = None, scale: float = 1.0, inplace: bool = False,
                        stream=None) -> torch.Tensor:
    """Gradient of sum(dlogp * logp) + sum(dentropy * entropy) with respect to
    the logits, of their type; `inplace` writes it over the logits."""
    z = _matrix(logits, "logits")
    rows, vocab = z.shape
    dt, i64 = _dtype(z, "logits"), _ids(ids, rows)
    _vector(dlogp, "dlogp", torch.float32, rows)
    _vector(result.lse, "lse", torch.float32, rows)
    if dentropy is not None:
        _vector(dentropy, "dentropy", torch.float32, rows)
        _vector(result.entropy, "entropy", torch.float32, rows)
    with _on(stream, logits, ids, result.lse, dlogp, dentropy):
        d = z if inplace else torch.empty(logits.shape, dtype=z.dtype, device=z.device)
        L.check(L.lib().okls_token_logprobs_grad(_ptr(z), dt, _ld(z), _ptr(ids), i64, rows, vocab, scale,
                                                 _ptr(result.lse), _ptr(result.entropy if dentropy is not None else None),
                                                 _ptr(dlogp), _ptr(dentropy), _ptr(d),
                                                 _ld(d) if inplace else vocab, _stream(z)))
    return logits if inplace else d


# ------------------------------------------------------------------ autograd
class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale, out_dtype):
        ctx.save_for_backward(ids)
        ctx.meta = (weight.shape[0], scale, weight.dtype)
        return embedding(weight, ids, scale=scale, out_dtype=out_dtype)

    @staticmethod
    def backward(ctx, dy):
        (ids,) = ctx.saved_tensors
        vocab, scale, dtype = ctx.meta
        return embedding_grad(dy.contiguous(), ids, vocab, scale=scale, dtype=dtype), None, None, None


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps, out_dtype):
        r = rms_norm(x, weight, residual=residual, eps=eps, out_dtype=out_dtype)
        ctx.save_for_backward(r.residual, weight, r.rstd)
        ctx.has_residual = residual is not None
        if residual is None:
            return r.y
        return r.y, r.residual

    @staticmethod
    def backward(ctx, dy, ds=None):
        s, weight, rstd = ctx.saved_tensors
        dx, dw = rms_norm_grad(dy.contiguous(), s, weight, rstd,
                               dresidual=None if ds is None else ds.contiguous(),
                               need_dweight=ctx.needs_input_grad[1])
        return (dx, None if dw is None else dw.to(weight.dtype).view(weight.shape), dx if ctx.has_residual else None,
                None, None)


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, out_dtype):
        m = _matrix(x, "x")
        need_x, need_w = ctx.needs_input_grad[:2]
        xq, xt = fp8_quantize(m, both=True) if need_w else (fp8_quantize(m), None)
        wq, wt = fp8_quantize(weight, block="square", both=True) if need_x else (
            fp8_quantize(weight, block="square"), None)
        ctx.save_for_backward(*[t for f in (xt, wt) if f is not None for t in (f.data, f.scale)])
        ctx.meta = (xt is not None, wt is not None, x.shape, x.dtype, weight.dtype)
        return fp8_matmul(xq, wq, out_dtype=out_dtype or x.dtype).view(*x.shape[:-1], weight.shape[0])

    @staticmethod
    def backward(ctx, dy):
        has_xt, has_wt, shape, xd, wd = ctx.meta
        saved = list(ctx.saved_tensors)
        xt = Fp8Tensor(saved.pop(0), saved.pop(0), "row") if has_xt else None
        wt = Fp8Tensor(saved.pop(0), saved.pop(0), "square") if has_wt else None
        g = _matrix(dy.contiguous(), "dy")
        dx = dw = None
        if has_xt and has_wt:
            gq, gt = fp8_quantize(g, both=True)
        else:
            gq, gt = (fp8_quantize(g), None) if has_wt else (None, fp8_quantize(g, transpose=True))
        if has_wt:
            dx = fp8_matmul(gq, wt, out_dtype=xd).view(shape)
        if has_xt:
            dw = fp8_matmul(gt, xt, out_dtype=wd)
        return dx, dw, None


class _Logprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, scale):
        r = token_logprobs(logits, ids, scale=scale)
        ctx.save_for_backward(logits, ids, r.entropy, r.lse)
        ctx.scale = scale
        return r.logp, r.entropy

    @staticmethod
    def backward(ctx, dlogp, dentropy):
        logits, ids, entropy, lse = ctx.saved_tensors
        r = TokenLogprobs(None, entropy, lse)
        return token_logprobs_grad(logits, ids, r, dlogp.contiguous(), dentropy=dentropy.contiguous(),
                                   scale=ctx.scale), None, None


def embed(weight: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0, out_dtype=None) -> torch.Tensor:
    """Differentiable `embedding`; the gradient has the weight's type."""
    return _Embed.apply(weight, ids, scale, out_dtype)


def norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *, eps: float = 1e-6,
         out_dtype=None):
    """Differentiable `rms_norm` in 16 or 32 bits: y, or (y, x + residual)."""
    return _Norm.apply(x, weight, residual, eps, out_dtype)


def linear(x: torch.Tensor, weight: torch.Tensor, *, out_dtype=None) -> torch.Tensor:
    """x weight^T with every product in 8 bits: the activations and the output's
    gradient in groups of 128 along each product's sum, the weight in 128 x 128
    blocks.  Gradients have the types of x and weight."""
    return _Linear.apply(x, weight, out_dtype)


def logprobs(logits: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0):
    """Differentiable (logp, entropy) of `token_logprobs`."""
    return _Logprobs.apply(logits, ids, scale)
