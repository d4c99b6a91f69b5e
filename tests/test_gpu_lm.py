"""Language-model operators on the GPU against their definitions in 64 bits.

Tolerances come from the arithmetic: u = 2^-24 is fp32's unit roundoff, bf16
rounds to 2^-8 of a value (7 fraction bits), an e4m3 code to 2^-4 of a value (2^-10 of the scale
below the smallest normal code).  A sum of n terms in fp32 is off by at most
about n u times the sum of their magnitudes, whatever its order."""

import math

import pytest
import torch

from kronecker_factored_second_gb300 import _lib as L
from kronecker_factored_second_gb300 import lm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
OUT_ULP = {BF16: 2.0 ** -8, F32: U}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L.lib()
    torch.cuda.set_device(0)
    lm.query_status()
    yield
    assert lm.query_status() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def pitched(t, pitch, offset=0):
    """The same matrix with another row pitch, its first element `offset` elements into the buffer."""
    buf = torch.full((t.shape[0] * pitch + offset,), 7.0, device=t.device).to(t.dtype)
    v = buf[offset:offset + t.shape[0] * pitch].view(t.shape[0], pitch)[:, :t.shape[1]]
    v.copy_(t)
    return v


def close(got, want, bound, what=""):
    """|got - want| <= bound everywhere, equal where want is not finite."""
    got, want = got.double(), want.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), what + ": finite in other places"
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN in other places"
    inf = ~fin & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf]), what + ": infinities differ"
    bound = torch.as_tensor(bound, device=got.device, dtype=torch.float64).expand_as(want)
    over = ((got - want).abs() - bound)[fin]
    if over.numel():
        assert over.max().item() <= 0, f"{what}: {over.max().item():.3g} past the bound"


# ---------------------------------------------------------------- embedding
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [1, 7, 8, 64, 1000, 1024, 2049, 4096])
def test_embedding(dtype, dim):
    g = gen(dim)
    for tokens, i64, out_dtype, pitch, off in [(1, True, None, dim, 0), (37, False, None, dim + 8, 0),
                                               (130, True, F32, dim + 3, 1), (5, False, BF16, dim, 8)]:
        vocab = 53
        w = pitched(randn(g, vocab, dim, dtype=dtype), pitch, off)
        ids = torch.randint(-1, vocab, (tokens,), generator=g, device="cuda")
        ids = ids if i64 else ids.int()
        y = lm.embedding(w, ids, scale=1.7, out_dtype=out_dtype)
        od = out_dtype or dtype
        assert y.shape == (tokens, dim) and y.dtype == od
        want = torch.where(ids[:, None] >= 0, w.double()[ids.clamp_min(0).long()] * float(torch.tensor(1.7)), 0.0)
        # the product in fp32, then the output's rounding (once when it is fp32)
        close(y, want, (U + OUT_ULP[od]) * want.abs(), "embedding")


def test_embedding_shapes_and_empty():
    w = randn(gen(0), 11, 24)
    ids = torch.tensor([[1, 2, -1], [0, 10, 3]], device="cuda")
    y = lm.embedding(w, ids)
    assert y.shape == (2, 3, 24)
    assert torch.equal(y[0, 0], w[1]) and torch.equal(y[0, 2], torch.zeros(24, device="cuda"))
    assert lm.embedding(w, ids[:0]).shape == (0, 3, 24)


def _grad_ref(dy, ids, vocab, scale, base):
    """(sum in 64 bits, sum of magnitudes, number of terms) by row."""
    keep = (ids >= 0) & (ids < vocab)
    out = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device="cuda")
    mag, n = torch.zeros_like(out), torch.zeros(vocab, 1, dtype=torch.float64, device="cuda")
    at = ids[keep].long()
    out.index_add_(0, at, dy[keep].double())
    mag.index_add_(0, at, dy[keep].double().abs())
    n.index_add_(0, at, torch.ones(len(at), 1, dtype=torch.float64, device="cuda"))
    s = float(torch.tensor(scale))
    if base is not None:
        return out * s + base.double(), mag * s + base.double().abs(), n + 1
    return out * s, mag * s, n


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, F32), (F32, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("tokens,vocab,dim", [
    (1, 1, 1), (1, 300, 40), (31, 7, 129), (33, 5, 2048), (64, 64, 8), (1000, 3, 65), (4097, 511, 72),
    (4096, 512, 64), (9001, 40000, 24), (20011, 513, 48), (70001, 1 << 18, 16), (3000, 1, 2056)])
def test_embedding_grad(dtype, out_dtype, tokens, vocab, dim):
    g = gen(tokens + vocab)
    dy = randn(g, tokens, dim, dtype=dtype)
    # frequencies that fall with the rank, and padding
    ids = (vocab ** torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)).long() - 1
    ids = ids.clamp(0, vocab - 1)
    ids[torch.rand(tokens, generator=g, device="cuda") < 0.1] = -1
    base = randn(g, vocab, dim, dtype=out_dtype)
    for b in (None, base):
        got = lm.embedding_grad(dy, ids, vocab, scale=0.3, base=b, dtype=out_dtype)
        want, mag, n = _grad_ref(dy, ids, vocab, 0.3, b)
        close(got, want, (n + 2) * U * mag + OUT_ULP[out_dtype] * want.abs(), "embedding gradient")
    again = lm.embedding_grad(dy, ids, vocab, scale=0.3, base=base, dtype=out_dtype)
    assert torch.equal(again, got), "the same inputs give the same bits"
    inplace = base.clone()
    assert lm.embedding_grad(dy, ids.int(), vocab, scale=0.3, base=inplace, out=inplace) is inplace
    assert torch.equal(inplace, got)


def test_embedding_grad_one_token_everywhere_and_none():
    g = gen(5)
    dy = randn(g, 40000, 33)
    ids = torch.full((40000,), 17, device="cuda")
    want, mag, n = _grad_ref(dy, ids, 64, 1.0, None)
    close(lm.embedding_grad(dy, ids, 64), want, (n + 2) * U * mag, "one token")
    ids[:] = -1
    assert lm.embedding_grad(dy, ids, 64).abs().max().item() == 0
    base = randn(g, 64, 33)
    assert torch.equal(lm.embedding_grad(dy, ids, 64, base=base), base)
    assert torch.equal(lm.embedding_grad(dy[:0], ids[:0], 64, base=base), base)


def test_embedding_grad_strides():
    g = gen(6)
    dy = randn(g, 500, 100, dtype=BF16)
    ids = torch.randint(0, 90, (500,), generator=g, device="cuda")
    want = lm.embedding_grad(dy, ids, 90)
    out = pitched(torch.zeros(90, 100, device="cuda"), 131, 3)
    base = pitched(torch.zeros(90, 100, device="cuda"), 107, 1)
    lm.embedding_grad(pitched(dy, 113, 5), ids, 90, base=base, out=out)
    assert torch.equal(out, want)


def test_bad_tokens_are_flagged():
    w = randn(gen(1), 10, 16)
    ids = torch.tensor([3, 10, -1, 9], device="cuda")
    y = lm.embedding(w, ids)
    assert y[1].abs().max().item() == 0 and torch.equal(y[3], w[9])
    with pytest.raises(L.OklsError) as e:
        lm.query_status()
    assert e.value.code == L.OKLS_ERR_INVALID_ARG
    assert lm.query_status() == 0
    dy = randn(gen(2), 4, 16)
    dw = lm.embedding_grad(dy, ids, 10)
    assert torch.equal(dw[9], dy[3]) and dw[:3].abs().max().item() == 0
    with pytest.raises(L.OklsError):
        lm.query_status()
    z = randn(gen(3), 4, 10)
    r = lm.token_logprobs(z, ids)
    assert r.logp[1].item() == 0 and r.logp[2].item() == 0
    with pytest.raises(L.OklsError):
        lm.query_status()
    d = lm.token_logprobs_grad(z, ids, r, torch.ones(4, device="cuda"))
    assert d[1].abs().max().item() == 0 and d[0].abs().max().item() > 0


# --------------------------------------------------------------------- norm
DIMS = [1, 2, 127, 128, 200, 256, 257, 1000, 2048, 4096, 5504, 8191, 16384, 32768]


def _norm_ref(x, r, w, eps):
    s = x.double() if r is None else (x.double() + r.double()).to(x.dtype).double()
    rstd = 1.0 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    return s, rstd, s * rstd * w.double()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", DIMS)
def test_rms_norm(dtype, dim):
    g = gen(dim)
    # the sum of squares is off by at most (terms a thread adds + tree) u of itself, halved by the root;
    # the three products and the root add a few u
    rel = (dim / 64 + 24) * U if dim > 4096 else 88 * U
    for rows, res, wd, od, pitch, off in [(1, False, dtype, dtype, dim, 0), (3, True, F32, F32, dim, 0),
                                          (401, True, BF16, BF16, dim + 8, 0), (17, True, dtype, BF16, dim + 1, 1)]:
        x = pitched(randn(g, rows, dim, dtype=dtype), pitch, off)
        r = pitched(randn(g, rows, dim, dtype=dtype, std=3.0), pitch, off) if res else None
        w = randn(g, dim, dtype=wd)
        out = lm.rms_norm(x, w, residual=r, eps=1e-5, out_dtype=od)
        s, rstd, y = _norm_ref(x, r, w, float(torch.tensor(1e-5)))
        assert torch.equal(out.residual.double(), s)
        close(out.rstd, rstd[:, 0], rel * rstd[:, 0], "rstd")
        close(out.y, y, (rel + OUT_ULP[od]) * y.abs(), "norm")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", DIMS)
def test_rms_norm_fp8(dtype, dim):
    g = gen(dim + 1)
    rel = (dim / 64 + 24) * U if dim > 4096 else 88 * U
    for rows, pitch, off in [(1, dim, 0), (333, dim, 0), (9, dim + 1, 1)]:
        x = pitched(randn(g, rows, dim, dtype=dtype), pitch, off)
        r = randn(g, rows, dim, dtype=dtype)
        w = randn(g, dim, dtype=dtype)
        out = lm.rms_norm(x, w, residual=r, out_dtype=torch.float8_e4m3fn)
        s, _, y = _norm_ref(x, r, w, float(torch.tensor(1e-6)))
        assert torch.equal(out.residual.double(), s)
        pad = torch.nn.functional.pad(y, (0, -dim % 128)).view(rows, -1, 128)
        scale = pad.abs().amax(-1).clamp_min(2.0 ** -100) / 448
        close(out.y.scale, scale, (rel + 2 * U) * scale, "scale")
        unit = scale.repeat_interleave(128, 1)[:, :dim]
        got = out.y.data.double() * out.y.scale.double().repeat_interleave(128, 1)[:, :dim]
        close(got, y, torch.maximum(y.abs() * 2.0 ** -4, unit * 2.0 ** -10) + 4 * rel * y.abs() + 8 * U * unit, "codes")


def test_rms_norm_inplace_and_zero_rows():
    g = gen(9)
    x, r, w = randn(g, 5, 640), randn(g, 5, 640), randn(g, 640)
    want = lm.rms_norm(x, w, residual=r)
    keep = r.clone()
    out = lm.rms_norm(x, w, residual=keep, inplace=True)
    assert out.residual is keep and torch.equal(keep, want.residual) and torch.equal(out.y, want.y)
    assert lm.rms_norm(x[:0], w).y.shape == (0, 640)
    z = lm.rms_norm(torch.zeros(3, 640, device="cuda"), w, out_dtype=torch.float8_e4m3fn)
    assert z.y.float().abs().max().item() == 0 and torch.isfinite(z.y.scale).all()
    ds, dw = lm.rms_norm_grad(x[:0], r[:0], w, torch.empty(0, device="cuda"))
    assert ds.shape == (0, 640) and dw.abs().max().item() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [1, 127, 256, 1000, 2048, 4096, 5504, 8191, 16384, 20000])
def test_rms_norm_grad(dtype, dim):
    g = gen(dim + 2)
    rel = (dim / 64 + 32) * U if dim > 4096 else 96 * U
    for rows, dyd, wd, dres, pitch, off in [(1, dtype, dtype, True, dim, 0), (700, dtype, F32, False, dim, 0),
                                            (1301, BF16, BF16, True, dim + 8, 0), (19, F32, dtype, True, dim + 1, 1)]:
        if rows * dim > 1 << 23:
            rows = 450
        s = pitched(randn(g, rows, dim, dtype=dtype), pitch, off)
        dy = pitched(randn(g, rows, dim, dtype=dyd), pitch, off)
        w = randn(g, dim, dtype=wd)
        e = randn(g, rows, dim, dtype=dtype) if dres else None
        rstd = lm.rms_norm(s, w).rstd
        ds, dw = lm.rms_norm_grad(dy, s, w, rstd, dresidual=e)
        r64 = rstd.double()[:, None]
        xh, gg = s.double() * r64, dy.double() * w.double()
        dot, mag = (gg * xh).mean(-1, keepdim=True), (gg * xh).abs().mean(-1, keepdim=True)
        want = r64 * (gg - xh * dot) + (0 if e is None else e.double())
        terms = r64 * (gg.abs() + xh.abs() * mag) + (0 if e is None else e.double().abs())
        close(ds, want, rel * terms + OUT_ULP[dtype] * want.abs(), "ds")
        p = dy.double() * xh
        close(dw, p.sum(0), (rows + 8) * U * p.abs().sum(0), "dw")
    none = lm.rms_norm_grad(dy, s, w, rstd, dresidual=e, need_dweight=False)
    assert none[1] is None and torch.equal(none[0], ds)
    assert torch.equal(lm.rms_norm_grad(dy, s, w, rstd, dresidual=e)[1], dw)


# --------------------------------------------------------------- quantising
def _codes(x, axes):
    """Codes and scales by the definition, in fp32 (every step is one rounding)."""
    a = x.abs().amax(axes, keepdim=True).clamp_min(2.0 ** -100)
    m = torch.full_like(a, 448.0)  # a quotient of two tensors is rounded once
    return (x * (m / a)).to(torch.float8_e4m3fn), a / m


def _rows_ref(x):
    rows, cols = x.shape
    p = torch.nn.functional.pad(x.float(), (0, -cols % 128)).view(rows, -1, 128)
    q, s = _codes(p, (2,))
    return q.view(torch.uint8).view(rows, -1)[:, :cols], s[..., 0]


def _square_ref(x):
    rows, cols = x.shape
    p = torch.nn.functional.pad(x.float(), (0, -cols % 128, 0, -rows % 128))
    q, s = _codes(p.view(p.shape[0] // 128, 128, p.shape[1] // 128, 128), (1, 3))
    return q.view(torch.uint8).view(p.shape)[:rows, :cols], s[:, 0, :, 0]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2048), (3, 130), (127, 129), (128, 128), (129, 127), (200, 1000),
                                       (2048, 512), (515, 2047), (1, 5504)])
def test_fp8_quantize(dtype, rows, cols):
    g = gen(rows * 31 + cols)
    x = randn(g, rows, cols, dtype=dtype) * torch.exp(3 * randn(g, rows, 1)).to(dtype)
    x[rows // 2] = 0
    for v in (x, pitched(x, cols + 8), pitched(x, cols + 3, 1)):
        for block, ref in (("row", _rows_ref), ("square", _square_ref)):
            q, t = lm.fp8_quantize(v, block=block, both=True)
            for f, src in ((q, x), (t, x.t()), (lm.fp8_quantize(v, block=block), x),
                           (lm.fp8_quantize(v, block=block, transpose=True), x.t())):
                code, scale = ref(src)
                assert torch.equal(f.scale, scale), block
                assert torch.equal(f.data.view(torch.uint8), code), block


def test_fp8_quantize_extremes():
    x = torch.zeros(4, 256, device="cuda")
    x[0, :128] = 1e-38
    x[0, 128:] = 3e38
    x[1, 5] = float("inf")
    x[1, 130] = float("nan")
    x[2] = torch.linspace(-1, 1, 256, device="cuda")
    q = lm.fp8_quantize(x)
    v = q.float()
    assert torch.isnan(v[1]).all()
    assert torch.isfinite(v[[0, 2, 3]]).all() and v[3].abs().max().item() == 0
    assert v[0, :128].abs().max().item() <= 2.0 ** -100 and (v[0, 128:] / 3e38 - 1).abs().max().item() < 1e-6
    assert (v[2] - x[2]).abs().max().item() <= 2.0 ** -4


# ----------------------------------------------------------------- products
def _check_product(a, b, got, out_dtype, old=None, extra=0.0):
    av, bv = a.float().double(), b.float().double()
    want, mag = av @ bv.t(), av.abs() @ bv.abs().t()
    if old is not None:
        want, mag = want + old.double(), mag + old.double().abs()
    groups = -(-a.shape[1] // 128)
    # inside a group the tensor core may cut each of 128 additions at 2^-23 of the running sum; scaling and
    # adding the groups costs a few u each
    close(got, want, (128 * 2 * U + (groups + 6) * U) * mag + OUT_ULP[out_dtype] * want.abs(), "product")


SIZES = [(1, 1, 1), (1, 5504, 2048), (2, 17, 130), (8, 64, 128), (9, 130, 1000), (16, 2048, 512), (31, 33, 257),
         (32, 100, 64), (33, 100, 64), (64, 64, 128), (100, 300, 200), (128, 256, 128), (129, 257, 129),
         (200, 1000, 1111), (515, 2048, 2047), (1024, 1023, 640), (2048, 5504, 256), (37, 11008, 384), (2000, 2600, 300), (5003, 1290, 130),
         (4096, 2304, 1152), (300, 19500, 128)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_fp8_matmul(m, n, k):
    g = gen(m + n + k)
    for block in ("row", "square"):
        for out_dtype in (BF16, F32):
            a = lm.fp8_quantize(randn(g, m, k) * torch.exp(randn(g, m, 1)))
            b = lm.fp8_quantize(randn(g, n, k) * torch.exp(randn(g, n, 1)), block=block)
            got = lm.fp8_matmul(a, b, out_dtype=out_dtype)
            _check_product(a, b, got, out_dtype)
            assert torch.equal(lm.fp8_matmul(a, b, out_dtype=out_dtype), got)
        old = randn(g, m, n + 5, dtype=out_dtype)[:, :n]
        acc = pitched(old, n + 5, 3)
        lm.fp8_matmul(a, b, out=acc, accumulate=True)
        _check_product(a, b, acc, out_dtype, old)


def test_fp8_matmul_given_layouts():
    """Codes and scales that the caller laid out: pitches of 16, plain scale matrices, whole-number values."""
    g = gen(3)
    for m in (5, 140):
        a8 = torch.randint(-8, 9, (m, 208), generator=g, device="cuda").float()
        b8 = torch.randint(-8, 9, (70, 208), generator=g, device="cuda").float()
        a = lm.Fp8Tensor(a8.to(torch.float8_e4m3fn), torch.ones(m, 2, device="cuda"), "row")
        b = lm.Fp8Tensor(b8.to(torch.float8_e4m3fn), torch.full((70, 2), 0.5, device="cuda"), "row")
        # whole numbers below 2^24: exact whatever the order
        assert torch.equal(lm.fp8_matmul(a, b, out_dtype=F32), (a8.double() @ b8.double().t()).float() * 0.5)
        # bytes between a row's end and the next row are not read as values
        dirty = torch.full((m, 224), 0x7F, dtype=torch.uint8, device="cuda")
        dirty[:, :200] = a.data.view(torch.uint8)[:, :200]
        cut = lm.Fp8Tensor(dirty.view(torch.float8_e4m3fn)[:, :200], a.scale, "row")
        cutb = lm.Fp8Tensor(b.data[:, :200], b.scale, "row")
        assert torch.equal(lm.fp8_matmul(cut, cutb, out_dtype=F32),
                           (a8[:, :200].double() @ b8[:, :200].double().t()).float() * 0.5)


def test_fp8_matmul_nan_stays_in_its_row_and_empty():
    g = gen(4)
    for m in (3, 150):
        x = randn(g, m, 300)
        x[1, 7] = float("nan")
        w = lm.fp8_quantize(randn(g, 40, 300), block="square")
        y = lm.fp8_matmul(lm.fp8_quantize(x), w, out_dtype=F32)
        assert torch.isnan(y[1]).all() and torch.isfinite(y[[0] + list(range(2, m))]).all()
    e = lm.fp8_quantize(torch.empty(0, 300, device="cuda"))
    assert lm.fp8_matmul(e, w).shape == (0, 40)
    a0, b0 = lm.fp8_quantize(torch.empty(4, 0, device="cuda")), lm.fp8_quantize(torch.empty(6, 0, device="cuda"))
    assert lm.fp8_matmul(a0, b0).abs().max().item() == 0


# --------------------------------------------------------- log probabilities
def _score_ref(z, scale):
    s = z.double() * scale
    lse = torch.logsumexp(s, -1)
    lp = s - lse[:, None]
    p = lp.exp()
    return s, lse, lp, p, -torch.xlogy(p, p).sum(-1)


def _check_scores(z, ids, k, scale, r):
    sc = float(torch.tensor(scale))
    s, lse, lp, p, ent = _score_ref(z, sc)
    rows, vocab = z.shape
    top = torch.where(torch.isfinite(s) & (s.abs() < 1e30), s.abs(), 0.0).amax(-1)
    # exponents are fp32 differences of magnitude up to 2 |z|, so a term is off by a few |z| u relative to itself, as
    # is each of the dozen joins of partial sums, which add a few u of their own; a thread adds vocab / 512 terms
    e = (64 + 16 * top + vocab / 256) * U
    close(r.lse, lse, e + 2 * U * lse.abs(), "lse")
    spread = torch.where(p > 0, (s - s.amax(-1, keepdim=True)).abs() * p, 0.0).sum(-1)
    close(r.entropy, ent, e * (2 + 2 * spread + torch.where(p > 0, p * (s - s.amax(-1, keepdim=True)) ** 2, 0.0).sum(-1)),
          "entropy")
    keep = ids >= 0
    want = torch.where(keep, lp.gather(1, ids.clamp_min(0).long()[:, None])[:, 0], 0.0)
    close(r.logp, want, e + 4 * U * (want.abs().nan_to_num(posinf=0.0) + lse.abs()), "logp")
    if k:
        v, i = torch.sort(z.float(), dim=-1, descending=True, stable=True)
        assert torch.equal(r.top_ids, i[:, :k].int())
        tl = v[:, :k].double() * sc - lse[:, None]
        close(r.top_logp, tl, e[:, None] + 4 * U * (tl.abs().nan_to_num(posinf=0.0) + lse.abs()[:, None]), "top_logp")
    return s, lse, lp, p, ent


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (1, 32000, 8), (2, 33, 32), (3, 40, 5), (700, 1000, 0), (5, 4099, 20),
                                          (64, 32000, 32), (1, 131072, 1), (7, 128257, 20), (1500, 257, 3),
                                          (40, 50021, 0)])
def test_token_logprobs(dtype, rows, vocab, k):
    g = gen(rows + vocab + k)
    for pitch, off, scale in [(vocab, 0, 1.0), (vocab + 7, 3, 0.7)]:
        z = randn(g, rows, vocab, dtype=dtype, std=3.0)
        ids = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        ids[rows // 2] = -1
        if vocab > 64:
            z[::3, ::2] = float("-inf")          # most of a row forbidden
            z[:, -3:] = torch.finfo(dtype).min   # the type's lowest value as a mask
        zz = pitched(z, pitch, off)
        r = lm.token_logprobs(zz, ids.int() if off else ids, top_k=k, scale=scale)
        s, lse, lp, p, ent = _check_scores(zz, ids, k, scale, r)
        dlogp, dent = randn(g, rows), randn(g, rows)
        sc = float(torch.tensor(scale))
        top = torch.where(torch.isfinite(s) & (s.abs() < 1e30), s.abs(), 0.0).amax(-1)
        gl = torch.where(ids >= 0, dlogp.double(), 0.0)
        want = -p * gl[:, None]
        want[torch.arange(rows, device="cuda"), ids.clamp_min(0)] += gl
        plp = torch.xlogy(p, p)
        terms = p * gl.abs()[:, None] + dent.double().abs()[:, None] * (plp.abs() + p * (ent[:, None] + 1))
        terms[torch.arange(rows, device="cuda"), ids.clamp_min(0)] += gl.abs()
        want = sc * (want - dent.double()[:, None] * (plp + p * ent[:, None]))
        # the error of lse (above) and of the exponent, twice over for the entropy's term
        rel = (64 + 32 * top + vocab / 256)[:, None] * U
        for d in (lm.token_logprobs_grad(zz, ids, r, dlogp, dentropy=dent, scale=scale),
                  lm.token_logprobs_grad(pitched(z, pitch, off), ids, r, dlogp, dentropy=dent, scale=scale,
                                         inplace=True)):
            close(d, want, rel * sc * terms * 2 + OUT_ULP[dtype] * want.abs() + 2.0 ** -140, "dlogits")
        only = lm.token_logprobs_grad(zz, ids, r, dlogp, scale=scale)
        w1 = -p * gl[:, None]
        w1[torch.arange(rows, device="cuda"), ids.clamp_min(0)] += gl
        close(only, sc * w1, rel * sc * terms * 2 + OUT_ULP[dtype] * (sc * w1).abs() + 2.0 ** -140, "dlogits of logp")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_token_logprobs_ties_and_order(dtype):
    """Equal logits rank by column, in rows that are hard for a running list."""
    vocab = 9000
    up = torch.arange(vocab, device="cuda", dtype=F32)
    rows = torch.stack([torch.zeros(vocab, device="cuda"), up, -up, up % 7, (up // 1000), -(up % 3) * 0.0]).to(dtype)
    ids = torch.zeros(len(rows), dtype=torch.long, device="cuda")
    for k in (1, 7, 32):
        r = lm.token_logprobs(rows, ids, top_k=k)
        i = torch.sort(rows.float(), dim=-1, descending=True, stable=True)[1]
        assert torch.equal(r.top_ids, i[:, :k].int())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_token_logprobs_rows_without_a_value(dtype):
    inf = float("inf")
    z = randn(gen(8), 5, 700, dtype=dtype)
    z[0] = -inf
    z[1, 3:] = -inf
    z[2, 5] = float("nan")
    z[3, 6] = inf
    ids = torch.tensor([4, 1, 0, 0, 2], device="cuda")
    r = lm.token_logprobs(z, ids, top_k=4)
    assert r.lse[0].item() == -inf and r.logp[0].item() == -inf and r.entropy[0].item() == 0
    assert r.top_ids[0].tolist() == [0, 1, 2, 3] and (r.top_logp[0] == -inf).all()
    assert sorted(r.top_ids[1, :3].tolist()) == [0, 1, 2] and r.top_ids[1, 3].item() == 3
    assert r.top_logp[1, 3].item() == -inf and math.isfinite(r.entropy[1].item())
    for i in (2, 3):
        assert all(math.isnan(t[i].item()) for t in (r.lse, r.logp, r.entropy))
    d = lm.token_logprobs_grad(z, ids, r, torch.ones(5, device="cuda"), dentropy=torch.ones(5, device="cuda"))
    assert d[0].abs().max().item() == 0
    assert torch.isfinite(d[1]).all() and d[1, 3:].abs().max().item() == 0 and torch.isfinite(d[4]).all()
    assert torch.isnan(d[2]).all()
    assert lm.token_logprobs(z[:0], ids[:0], top_k=2).top_ids.shape == (0, 2)


def test_token_logprobs_common_offset():
    """A large offset common to a row costs the digits that fp32 logits lost, no more."""
    z = (torch.randint(-40, 41, (3, 5000), generator=gen(1), device="cuda") / 8).float()
    ids = torch.tensor([1, 2, 3], device="cuda")
    a, b = lm.token_logprobs(z, ids), lm.token_logprobs(z + 4096.0, ids)
    assert torch.equal(a.entropy, b.entropy)
    assert (a.logp - b.logp).abs().max().item() <= 4096 * 2 * U * 2


# ----------------------------------------------------- streams and gradients
def test_other_stream_gives_the_same_bits():
    g = gen(12)
    x = randn(g, 300, 512, dtype=BF16)
    w = randn(g, 700, 512, dtype=BF16, std=0.05)
    nw = randn(g, 512, dtype=BF16)
    ids = torch.randint(0, 700, (300,), generator=g, device="cuda")

    def chain(stream):
        n = lm.rms_norm(x, nw, residual=x, out_dtype=torch.float8_e4m3fn, stream=stream)
        z = lm.fp8_matmul(n.y, lm.fp8_quantize(w, block="square", stream=stream), stream=stream)
        r = lm.token_logprobs(z, ids, top_k=3, stream=stream)
        return z, r.logp, r.top_ids, lm.embedding_grad(x, ids, 700, stream=stream)

    want = chain(None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = chain(s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_calls_can_be_captured():
    """A captured chain of all operators, replayed on new inputs, gives what the calls give."""
    g = gen(16)
    x, dy = randn(g, 400, 256, dtype=BF16), randn(g, 400, 256, dtype=BF16)
    w, nw = randn(g, 600, 256, dtype=BF16, std=0.05), randn(g, 256, dtype=BF16)
    ids = torch.randint(-1, 600, (400,), generator=g, device="cuda")
    gl = randn(g, 400)

    def chain():
        h = lm.embedding(w, ids, scale=2.0)
        n = lm.rms_norm(x, nw, residual=h)
        q, qt = lm.fp8_quantize(n.y, both=True)
        z = lm.fp8_matmul(q, lm.fp8_quantize(w, block="square"))
        r = lm.token_logprobs(z, ids, top_k=5)
        dz = lm.token_logprobs_grad(z, ids, r, gl, dentropy=gl)
        dw = lm.fp8_matmul(lm.fp8_quantize(dz, transpose=True), qt)
        ds, dn = lm.rms_norm_grad(dy, n.residual, nw, n.rstd, dresidual=x)
        return z, r.logp, r.top_ids, dz, dw, ds, dn, lm.embedding_grad(ds, ids, 600)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = chain()
    for seed in (1, 2):
        h = gen(seed)
        x.copy_(randn(h, 400, 256, dtype=BF16))
        ids.copy_(torch.randint(-1, 600, (400,), generator=h, device="cuda"))
        graph.replay()
        for a, b in zip(captured, chain()):
            assert torch.equal(a, b)


def test_autograd_against_differences():
    """Directional differences of the loss through embed, norm and logprobs in fp32."""
    g = gen(13)
    V, D, T = 60, 96, 50
    E = randn(g, V, D).requires_grad_()
    nw = (1 + 0.1 * randn(g, D)).requires_grad_()
    H = randn(g, V, D, std=0.1).requires_grad_()
    ids = torch.randint(-1, V, (T,), generator=g, device="cuda")
    tgt = torch.randint(-1, V, (T,), generator=g, device="cuda")

    def loss(E, nw, H):
        h = lm.embed(E, ids, scale=0.5)
        y, s = lm.norm(h, nw, h.detach() * 0.3)
        logp, ent = lm.logprobs(y @ H.t() + 0.01 * s.sum(-1, keepdim=True), tgt, scale=0.8)
        return -(logp.double().sum() + 0.3 * ent.double().sum()) / T

    loss(E, nw, H).backward()
    for p in (E, nw, H):
        d = randn(g, *p.shape)
        d /= d.norm()
        eps = 0.02
        args = [E.detach(), nw.detach(), H.detach()]
        i = next(j for j, q in enumerate((E, nw, H)) if q is p)

        def at(t):
            a = list(args)
            a[i] = a[i] + t * d
            # the residual is a constant of the point of expansion
            h0 = lm.embed(args[0], ids, scale=0.5)
            h = lm.embed(a[0], ids, scale=0.5)
            y, s = lm.norm(h, a[1], h0 * 0.3)
            logp, ent = lm.logprobs(y @ a[2].t() + 0.01 * s.sum(-1, keepdim=True), tgt, scale=0.8)
            return (-(logp.double().sum() + 0.3 * ent.double().sum()) / T).item()

        num = (8 * (at(eps) - at(-eps)) - (at(2 * eps) - at(-2 * eps))) / (12 * eps)
        ana = (p.grad.double() * d.double()).sum().item()
        # fourth-order differences: rounding of the loss (about 1e-6) over eps dominates
        assert abs(num - ana) <= 5e-4 * max(1.0, abs(ana)), (num, ana)


def test_linear_autograd_is_the_product_of_the_codes():
    g = gen(14)
    x = randn(g, 3, 50, 300, dtype=BF16).requires_grad_()
    w = randn(g, 200, 300, dtype=BF16, std=0.05).requires_grad_()
    y = lm.linear(x, w)
    dy = randn(g, 3, 50, 200, dtype=BF16)
    y.backward(dy)
    X, W, G = x.detach().view(150, 300), w.detach(), dy.view(150, 200)
    _check_product(lm.fp8_quantize(X), lm.fp8_quantize(W, block="square"), y.detach().view(150, 200), BF16)
    _check_product(lm.fp8_quantize(G), lm.fp8_quantize(W, block="square", transpose=True), x.grad.view(150, 300), BF16)
    _check_product(lm.fp8_quantize(G, transpose=True), lm.fp8_quantize(X, transpose=True), w.grad, BF16)


def test_leading_dimensions_fold():
    """Leading dimensions that step over one another are rows; others are refused, never copied."""
    g = gen(15)
    x = randn(g, 6, 5, 64, dtype=BF16)
    w = randn(g, 64, dtype=BF16)
    wide = torch.zeros(6, 5, 80, dtype=BF16, device="cuda")
    wide[..., :64] = x
    want = lm.rms_norm(x.view(30, 64), w)
    for v in (x, wide[..., :64]):
        out = lm.rms_norm(v, w)
        assert out.y.shape == v.shape and torch.equal(out.y.reshape(30, 64), want.y)
    assert torch.equal(lm.rms_norm(x[2], w).y, want.y[10:15])
    assert torch.equal(lm.rms_norm(x[:, 3:4], w).y.reshape(6, 64), want.y[3::5])
    ids = torch.randint(0, 64, (6, 5), generator=g, device="cuda")
    assert torch.equal(lm.token_logprobs(wide[..., :64], ids).logp, lm.token_logprobs(x.view(30, 64), ids.view(30)).logp.view(6, 5))
    for v in (x.transpose(0, 1), x[:, :4], torch.zeros((), device="cuda")):
        with pytest.raises(ValueError):
            lm.rms_norm(v, w)
            pytest.fail("a layout that does not fold was taken")


# ---------------------------------------------------------------- refusals
def test_refusals():
    f = torch.float16
    x = torch.zeros(4, 256, device="cuda")
    w = torch.zeros(256, device="cuda")
    ids = torch.zeros(4, dtype=torch.long, device="cuda")
    bad = [
        lambda: lm.embedding(x.to(f), ids), lambda: lm.embedding(x, ids.short()), lambda: lm.embedding(x.t(), ids),
        lambda: lm.embedding(x.cpu(), ids), lambda: lm.embedding(x[0], ids),
        lambda: lm.embedding_grad(x, ids[:3], 9), lambda: lm.embedding_grad(x, ids, 9, base=x),
        lambda: lm.embedding_grad(x, ids, 4, base=x, out=x.bfloat16()),
        lambda: lm.rms_norm(x, w[:100]), lambda: lm.rms_norm(x, w, residual=x[:2]),
        lambda: lm.rms_norm(x, w, residual=x.bfloat16()), lambda: lm.rms_norm(x, w, out_dtype=f),
        lambda: lm.rms_norm_grad(x, x, w, w), lambda: lm.fp8_quantize(x, block="column"),
        lambda: lm.fp8_matmul(lm.fp8_quantize(x, block="square"), lm.fp8_quantize(x)),
        lambda: lm.fp8_matmul(lm.fp8_quantize(x), lm.fp8_quantize(x[:, :100])),
        lambda: lm.fp8_matmul(lm.fp8_quantize(x), lm.fp8_quantize(x), accumulate=True),
        lambda: lm.Fp8Tensor(x, x), lambda: lm.Fp8Tensor(lm.fp8_quantize(x).data, x),
        lambda: lm.token_logprobs(x, ids[:2]), lambda: lm.token_logprobs(x.to(f), ids),
        lambda: lm.token_logprobs_grad(x, ids, lm.token_logprobs(x, ids), w),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    refused = [
        lambda: lm.embedding_grad(x[:, :0], ids, 9), lambda: lm.token_logprobs(x, ids, top_k=33),
        lambda: lm.token_logprobs(x, ids, scale=0.0), lambda: lm.rms_norm(x, w, eps=-1.0),
        lambda: lm.rms_norm(torch.zeros(1, 40000, device="cuda"), torch.zeros(40000, device="cuda")),
        lambda: lm.fp8_matmul(lm.Fp8Tensor(lm.fp8_quantize(x).data.view(-1)[:4 * 200].view(4, 200),
                                           torch.ones(4, 2, device="cuda")), lm.fp8_quantize(x[:, :200])),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(L.OklsError):
            call()
            pytest.fail(f"call {i} was taken")
