"""Operators of the language models that the optimizers of this library train.

Forward and gradient operators over the C ABI (device memory and streams only,
as in okls.py):

`embedding`, `embedding_grad`            rows of a token table, scaled; gradient by sorted tokens
`rms_norm`, `rms_norm_grad`              norm with the residual's addition, output in 32, 16 or 8 bits
`fp8_quantize`, `fp8_matmul`             e4m3 values with a scale for each 128, and their product
`token_logprobs`, `token_logprobs_grad`  log probabilities of given tokens, entropy, best alternatives
`int4_quantize`, `int4_matmul`           4-bit weights with a scale for each group, and their product with a few rows
`sample`                                 tokens drawn with temperature, top-k, top-p and min-p from given random numbers

and the same as differentiable functions of torch.autograd:

`embed`, `norm`, `linear`, `logprobs`

Their gradients are not differentiable: a second derivative through one of
them raises RuntimeError.

Calls that write over a tensor of the caller (`out`, `inplace`) raise its
version, so that a backward which saved it says so, and refuse a tensor that
requires a gradient.

Tensors are CUDA tensors on one device whose last dimension is contiguous;
rows may have any pitch.  fp32 and bf16 are taken, ids are int32 or int64.
Negative ids are padding: zeros out, log probability 0, and no gradient of
either (a row's entropy does not depend on its id, and keeps its gradient).  An
id at or past the vocabulary is treated as padding and recorded in the device's
status word, which only `query_status` reads.

Every function runs on the current stream, or on `stream`.  Outputs and
scratch come from torch's allocator on that stream.  A call on another
`stream` does not wait for the work that makes its inputs, nor does the
current stream wait for its outputs: order the two streams as for any torch
call.  The inputs' memory stays theirs until `stream` has passed the call;
outputs used on another stream are the caller's to record there.  No call
synchronises, apart from `query_status`.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib as L

FP8_GROUP = 128
_BLOCKS = ("row", "square")
_NATIVE = None


def _fail(msg: str):
    raise ValueError("okls.lm: " + msg)


def _n():
    """The compiled torch binding (checks, allocation, the call of the C entry)."""
    global _NATIVE
    if _NATIVE is None:
        L.lib()  # says how to build when the library is missing
        from . import _lm_native
        _NATIVE = _lm_native
    return _NATIVE


def _on(stream, *tensors):
    """The context of a call on `stream`.  The allocator is told that the inputs are used there, so that a caller who
    lets go of one does not have its memory handed out while the call still reads it."""
    for t in tensors:
        if t is not None and t.is_cuda:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def query_status(device=None, stream=None) -> int:
    """Synchronise the stream and return (and clear) the device's status word;
    raises OklsError for a token id past the vocabulary or an expired wait.

    One word serves all streams of the device.  The read covers the work
    ordered before it on the given stream; other streams' work may report to
    this read or to the next."""
    index = torch.device("cuda" if device is None else device).index
    if index is None:
        index = torch.cuda.current_device()
    with torch.cuda.device(index):
        word = _n().status_word(index)
        s = torch.cuda.current_stream() if stream is None else stream
        v = ctypes.c_uint32(0)
        L.check(L.lib().okls_status_word_read(word, s.cuda_stream, ctypes.byref(v)))
    return v.value


# ---------------------------------------------------------------- embedding
def embedding(weight: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0, out_dtype: torch.dtype | None = None,
              stream=None) -> torch.Tensor:
    """scale * weight[ids], of shape ids.shape + (dim,); zeros for padding."""
    if stream is not None:
        with _on(stream, weight, ids):
            return embedding(weight, ids, scale=scale, out_dtype=out_dtype)
    return _n().embedding(weight, ids, scale, out_dtype)


def embedding_grad(dy: torch.Tensor, ids: torch.Tensor, vocab: int, *, scale: float = 1.0,
                   base: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """base + scale * (sum of dy's rows by token), vocab x dim.

    `base` None stands for zeros.  With `out` the result goes there; out=base
    adds in place and touches only the rows of tokens that occur.  A new result
    has the type of `base`, or `dtype` without one."""
    if stream is not None:
        with _on(stream, dy, ids, base, out):
            return embedding_grad(dy, ids, vocab, scale=scale, base=base, out=out, dtype=dtype)
    got = _n().embedding_grad(dy, ids, vocab, scale, base, out, dtype)
    return got if out is None else out


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
    if stream is not None:
        with _on(stream, x, weight, residual):
            return rms_norm(x, weight, residual=residual, eps=eps, out_dtype=out_dtype, inplace=inplace)
    y, scale, total, rstd = _n().rms_norm(x, weight, residual, eps, out_dtype, inplace)
    if scale is not None:
        y = _fp8(y, scale, "row")
    return NormOutput(y, x if residual is None else residual if inplace else total, rstd)


def rms_norm_grad(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, *,
                  dresidual: torch.Tensor | None = None, need_dweight: bool = True, stream=None):
    """(ds, dweight): the gradient of x and residual alike, of s's type, and of
    the weight in fp32 (None unless `need_dweight`).  `s` and `rstd` are what
    rms_norm returned; `dresidual` is the gradient that reaches s from elsewhere."""
    if stream is not None:
        with _on(stream, dy, s, weight, rstd, dresidual):
            return rms_norm_grad(dy, s, weight, rstd, dresidual=dresidual, need_dweight=need_dweight)
    return _n().rms_norm_grad(dy, s, weight, rstd, dresidual, need_dweight)


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
            _fail(f"block must be one of {_BLOCKS}")
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


def _fp8(data: torch.Tensor, scale: torch.Tensor, block: str) -> Fp8Tensor:
    """An Fp8Tensor that is right by construction."""
    q = object.__new__(Fp8Tensor)
    q.data, q.scale, q.block = data, scale, block
    return q


def fp8_quantize(x: torch.Tensor, *, block: str = "row", transpose: bool = False, both: bool = False, stream=None):
    """An Fp8Tensor of x (rows x columns), of its transpose, or the pair of
    them from one read.  The groups of the transpose lie along its own rows."""
    if block not in _BLOCKS:
        _fail(f"block must be one of {_BLOCKS}")
    if stream is not None:
        with _on(stream, x):
            return fp8_quantize(x, block=block, transpose=transpose, both=both)
    q, s, qt, st = _n().fp8_quantize(x, block == "square", both or not transpose, both or transpose)
    if both:
        return _fp8(q, s, block), _fp8(qt, st, block)
    return _fp8(qt, st, block) if transpose else _fp8(q, s, block)


def fp8_matmul(a: Fp8Tensor, b: Fp8Tensor, *, out_dtype: torch.dtype = torch.bfloat16,
               out: torch.Tensor | None = None, accumulate: bool = False, stream=None) -> torch.Tensor:
    """a b^T for a (m x k, row groups) and b (n x k, row groups or square
    blocks): m x n in bf16 or fp32.  With `accumulate` it is added to `out`."""
    if a.block != "row":
        _fail("the first factor needs row groups")
    if stream is not None:
        with _on(stream, a.data, a.scale, b.data, b.scale, out):
            return fp8_matmul(a, b, out_dtype=out_dtype, out=out, accumulate=accumulate)
    got = _n().fp8_matmul(a.data, a.scale, b.data, b.scale, b.block == "square", out, out_dtype, accumulate)
    return got if out is None else out


# --------------------------------------------------------- log probabilities
@dataclass
class TokenLogprobs:
    """Per row: log probability of the given token, entropy, log of the sum of
    exponentials; with top_k, the best tokens and their log probabilities.
    lse + lse_rest is the logarithm before its rounding: the gradient needs the
    remainder where a row's logits share a large offset."""
    logp: torch.Tensor
    entropy: torch.Tensor
    lse: torch.Tensor
    top_ids: torch.Tensor | None = None
    top_logp: torch.Tensor | None = None
    lse_rest: torch.Tensor | None = None


def token_logprobs(logits: torch.Tensor, ids: torch.Tensor, *, top_k: int = 0, scale: float = 1.0,
                   stream=None) -> TokenLogprobs:
    """Log probabilities of `ids` under softmax(scale * logits), shaped like the
    logits' rows; `top_k` <= 32 best alternatives, equal logits in the order of their ids."""
    if stream is not None:
        with _on(stream, logits, ids):
            return token_logprobs(logits, ids, top_k=top_k, scale=scale)
    return TokenLogprobs(*_n().token_logprobs(logits, ids, top_k, scale))


def token_logprobs_grad(logits: torch.Tensor, ids: torch.Tensor, result: TokenLogprobs, dlogp: torch.Tensor, *,
                        dentropy: torch.Tensor | None = None, scale: float = 1.0, inplace: bool = False,
                        stream=None) -> torch.Tensor:
    """Gradient of sum(dlogp * logp) + sum(dentropy * entropy) with respect to
    the logits, of their type; `inplace` writes it over the logits."""
    if stream is not None:
        with _on(stream, logits, ids, result.lse, result.lse_rest, result.entropy, dlogp, dentropy):
            return token_logprobs_grad(logits, ids, result, dlogp, dentropy=dentropy, scale=scale, inplace=inplace)
    d = _n().token_logprobs_grad(logits, ids, result.lse, result.lse_rest, result.entropy, dlogp, dentropy, scale, inplace)
    return logits if inplace else d


# -------------------------------------------------------------------- 4 bits
@dataclass
class Int4Tensor:
    """A weight (rows x cols) in 4 bits: codes 0..15, two in a byte with the even column in the low half (`data`, uint8,
    rows x ceil(cols / 2)), and a bf16 scale for each `group` consecutive columns of a row (32, 64 or a multiple of 128).
    (code - zero) * scale stands for the value; `zero` is bf16 of scale's shape, or None for 8.  scale and zero may be
    laid in any way; group by group (scale.t() contiguous, rows a multiple of 8), as `int4_quantize` does, is read fastest.

    Codes from elsewhere are taken as they are; `int4_matmul` needs rows of data that start on 16-byte boundaries."""
    data: torch.Tensor
    scale: torch.Tensor
    cols: int
    group: int = 128
    zero: torch.Tensor | None = None

    def __post_init__(self):
        if self.group not in (32, 64) and (self.group < 128 or self.group % 128):
            _fail(f"group must be 32, 64 or a multiple of 128, not {self.group}")
        if self.data.dim() != 2 or self.data.dtype != torch.uint8 or self.data.shape[1] != -(-self.cols // 2):
            _fail(f"data must be a matrix of uint8 with {-(-self.cols // 2)} columns")
        if self.data.numel() and self.data.shape[1] > 1 and self.data.stride(1) != 1:
            _fail("the last dimension of data must be contiguous")
        want = (self.data.shape[0], -(-self.cols // self.group))
        for name, t in (("scale", self.scale), ("zero", self.zero)):
            if t is not None and (tuple(t.shape) != want or t.dtype != torch.bfloat16):
                _fail(f"{name} must be bf16 of shape {want}")

    @property
    def shape(self):
        return torch.Size((self.data.shape[0], self.cols))

    def float(self) -> torch.Tensor:
        """The values in fp32."""
        c = torch.stack((self.data & 15, self.data >> 4), 2).flatten(1)[:, : self.cols].float()

        def spread(t):
            return t.float().repeat_interleave(self.group, 1)[:, : self.cols]
        return (c - (8.0 if self.zero is None else spread(self.zero))) * spread(self.scale)


def int4_quantize(w: torch.Tensor, *, group: int = 128, symmetric: bool = True, stream=None) -> Int4Tensor:
    """An Int4Tensor of w (rows x columns).  `symmetric` codes are 1..15 around
    8; otherwise a group's range, 0 included, is spread over 0..15 with a zero point."""
    if stream is not None:
        with _on(stream, w):
            return int4_quantize(w, group=group, symmetric=symmetric)
    q, s, z = _n().int4_quantize(w, group, symmetric)
    return Int4Tensor(q, s, w.shape[1], group, z)


def int4_matmul(x: torch.Tensor, w: Int4Tensor, *, out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                accumulate: bool = False, stream=None) -> torch.Tensor:
    """x w^T in fp32 or bf16 (default: x's type) for the tokens of a generation
    step: x (..., columns of w) fp32 or bf16, up to some 64 rows of it.  More
    rows are right but not fast; a prompt is `fp8_matmul`'s.  With `accumulate`
    it is added to `out` (rows x rows of w), which has no element in common with x
    and w.  No gradient flows through it."""
    if stream is not None:
        with _on(stream, x, w.data, w.scale, w.zero, out):
            return int4_matmul(x, w, out_dtype=out_dtype, out=out, accumulate=accumulate)
    got = _n().int4_matmul(x, w.data, w.scale, w.zero, w.cols, w.group, out, out_dtype, accumulate)
    return got if out is None else out


# ------------------------------------------------------------------ sampling
@dataclass
class TokenSample:
    """Per row: the drawn token (int32), and its log probability among the tokens that were left to draw from."""
    ids: torch.Tensor
    logp: torch.Tensor


def sample(logits: torch.Tensor, u: torch.Tensor, *, temperature=1.0, top_k=None, top_p=None, min_p=None,
           stream=None) -> TokenSample:
    """A token from each row of logits, drawn with the row's `u` in [0, 1) (fp32).

    `temperature` divides the logits (0: the best token); `top_k` keeps the k
    best tokens, equal logits in the order of their ids; `top_p` of those the
    shortest prefix that has at least this share of their probability; `min_p`
    those with at least this share of the best token's probability.  The token
    is the first, in the order of ids, at which the running probability of what
    is kept is above u.  A setting is a number, None (off), or a tensor with a
    value for each row (fp32; top_k int32, 0 or less: off).  A row without a possible token
    (all -inf) gets id -1 and log probability -inf."""
    if stream is not None:
        with _on(stream, logits, u, *(t for t in (temperature, top_k, top_p, min_p) if isinstance(t, torch.Tensor))):
            return sample(logits, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    return TokenSample(*_n().sample(logits, u, temperature, top_k, top_p, min_p))


# ------------------------------------------------------------------ autograd
class _FirstOrder(torch.autograd.Function):
    """Gradients that depend on `sources`, as they are, but not to be differentiated."""

    @staticmethod
    def forward(ctx, name, count, *tensors):
        ctx.name = name
        return tuple(t.view_as(t) for t in tensors[:count])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"okls.lm: the gradient of {ctx.name} cannot be differentiated")


def _first_order(name, grads, *sources):
    """The gradients a backward returns.  The kernels leave no graph: where one is asked for (create_graph), a gradient
    is tied to the tensors that it is made of, so that a second derivative through it raises instead of being dropped."""
    if not torch.is_grad_enabled():
        return grads
    some = [g for g in grads if g is not None]
    tied = iter(_FirstOrder.apply(name, len(some), *some, *(s for s in sources if s is not None)))
    return tuple(None if g is None else next(tied) for g in grads)


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
        dw = embedding_grad(dy.contiguous(), ids, vocab, scale=scale, dtype=dtype)
        return *_first_order("embed", (dw,), dy), None, None, None


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
        grads = (dx, None if dw is None else dw.to(weight.dtype).view(weight.shape), dx if ctx.has_residual else None)
        return *_first_order("norm", grads, dy, ds, s, weight), None, None


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, out_dtype):
        need_x, need_w = ctx.needs_input_grad[:2]
        xq, xt = fp8_quantize(x, both=True) if need_w else (fp8_quantize(x), None)
        wq, wt = fp8_quantize(weight, block="square", both=True) if need_x else (
            fp8_quantize(weight, block="square"), None)
        # an empty output of this node: stands in the backward for x and weight, which are not kept
        tie = x.new_empty(0)
        ctx.set_materialize_grads(False)  # nothing flows back into it
        ctx.save_for_backward(*[t for f in (xt, wt) if f is not None for t in (f.data, f.scale)], tie)
        ctx.meta = (xt is not None, wt is not None, x.shape, x.dtype, weight.dtype)
        return fp8_matmul(xq, wq, out_dtype=out_dtype or x.dtype).view(*x.shape[:-1], weight.shape[0]), tie

    @staticmethod
    def backward(ctx, dy, _):
        has_xt, has_wt, shape, xd, wd = ctx.meta
        *saved, tie = ctx.saved_tensors
        xt = Fp8Tensor(saved.pop(0), saved.pop(0), "row") if has_xt else None
        wt = Fp8Tensor(saved.pop(0), saved.pop(0), "square") if has_wt else None
        g = dy.contiguous()
        dx = dw = None
        if has_xt and has_wt:
            gq, gt = fp8_quantize(g, both=True)
        else:
            gq, gt = (fp8_quantize(g), None) if has_wt else (None, fp8_quantize(g, transpose=True))
        if has_wt:
            dx = fp8_matmul(gq, wt, out_dtype=xd).view(shape)
        if has_xt:
            dw = fp8_matmul(gt, xt, out_dtype=wd)
        return *_first_order("linear", (dx, dw), dy, tie), None


class _Logprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, scale):
        r = token_logprobs(logits, ids, scale=scale)
        ctx.save_for_backward(logits, ids, r.entropy, r.lse, r.lse_rest)
        ctx.scale = scale
        return r.logp, r.entropy

    @staticmethod
    def backward(ctx, dlogp, dentropy):
        logits, ids, entropy, lse, rest = ctx.saved_tensors
        r = TokenLogprobs(None, entropy, lse, lse_rest=rest)
        dz = token_logprobs_grad(logits, ids, r, dlogp.contiguous(), dentropy=dentropy.contiguous(), scale=ctx.scale)
        return *_first_order("logprobs", (dz,), dlogp, dentropy, logits), None, None


def embed(weight: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0, out_dtype=None) -> torch.Tensor:
    """Differentiable `embedding`; the gradient has the weight's type."""
    return _Embed.apply(weight, ids, scale, out_dtype)


def norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *, eps: float = 1e-6,
         out_dtype=None):
    """Differentiable `rms_norm` in 16 or 32 bits: y, or (y, x + residual)."""
    if out_dtype not in (None, torch.float32, torch.bfloat16):
        _fail(f"norm gives fp32 or bf16, not {out_dtype} (rms_norm has the 8-bit output)")
    return _Norm.apply(x, weight, residual, eps, out_dtype)


def linear(x: torch.Tensor, weight: torch.Tensor, *, out_dtype=None) -> torch.Tensor:
    """x weight^T with every product in 8 bits: the activations and the output's
    gradient in groups of 128 along each product's sum, the weight in 128 x 128
    blocks.  Gradients have the types of x and weight."""
    return _Linear.apply(x, weight, out_dtype)[0]


def logprobs(logits: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0):
    """Differentiable (logp, entropy) of `token_logprobs`."""
    return _Logprobs.apply(logits, ids, scale)
