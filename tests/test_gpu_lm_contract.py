"""What the language-model operators promise beyond their formulas, on the GPU: equal results whatever warps run first,
arguments that outlive a call, gradients that refuse what they cannot give, in-place writes that autograd sees."""

import pytest
import torch

from kronecker_factored_second_gb300 import _lib as L
from kronecker_factored_second_gb300 import lm

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24


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


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab", [(3, 131072), (600, 20000), (40, 300000)])
def test_alternatives_among_many_equal_logits(dtype, rows, vocab):
    """Rows in which thousands of columns share the best values, so that every warp inserts into its list and raises the
    bound that the CTA's warps share: the alternatives are the same, call after call."""
    g = gen(vocab)
    z = torch.randint(0, 3, (rows, vocab), generator=g, device="cuda").to(dtype)
    z[1::3] = torch.arange(vocab, device="cuda").to(dtype) % 128  # a new best value with every column up to 127
    ids = torch.zeros(rows, dtype=torch.long, device="cuda")
    for k in (1, 9, 32):
        want = torch.sort(z.float(), dim=-1, descending=True, stable=True)[1][:, :k].int()
        for _ in range(5):
            assert torch.equal(lm.token_logprobs(z, ids, top_k=k).top_ids, want)


def test_reassigned_fields_of_8_bit_tensors_are_checked():
    """An Fp8Tensor's fields can be assigned; scales that do not cover the codes are refused, not read past their end."""
    x = randn(gen(1), 300, 520)
    good = lm.fp8_quantize(x)
    want = lm.fp8_matmul(good, lm.fp8_quantize(x, block="square"))
    changes = [dict(scale=good.scale[:299]), dict(scale=good.scale[:, :4]), dict(scale=good.scale.double()),
               dict(scale=good.scale.cpu()), dict(scale=good.scale[0]), dict(data=x), dict(data=good.data.t()),
               dict(data=torch.cat([good.data.view(torch.uint8)] * 2).view(E4M3)), dict(data=good.data.cpu())]
    for i, change in enumerate(changes):
        for first in (True, False):
            f = lm.fp8_quantize(x)
            for name, v in change.items():
                setattr(f, name, v)
            with pytest.raises(ValueError):
                lm.fp8_matmul(*((f, good) if first else (good, f)))
                pytest.fail(f"change {i} was taken")
    f = lm.fp8_quantize(x)
    f.block = "square"
    with pytest.raises(ValueError):
        lm.fp8_matmul(good, f)
    assert torch.equal(lm.fp8_matmul(good, lm.fp8_quantize(x, block="square")), want)


def test_inputs_outlive_a_call_on_another_stream():
    """Temporaries handed to a call on a busy stream are not overwritten by what the current stream allocates next."""
    g = gen(2)
    keep = randn(g, 2048, 1024)
    w = randn(g, 1024)
    side = torch.cuda.Stream()
    for call, value in ((lambda x, s: lm.rms_norm(x, w, stream=s).y, lambda y: y),
                        (lambda x, s: lm.fp8_quantize(x, stream=s), lambda q: q.float())):
        want = value(call(keep, None))
        x = keep.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)  # some 25 ms
        got = call(x, side)
        del x
        later = [torch.full_like(keep, float("nan")) for _ in range(3)]  # takes x's memory if it is free
        torch.cuda.synchronize()
        assert torch.equal(value(got), want)
        del later


def _probabilities(z, ids, r, k):
    """logp, entropy, alternatives and gradients of rows whose logits share an offset, against 64 bits.  Differences to the
    row's maximum are exact, so the bounds hold the spread of the possible logits and not their size: an exponent is off by
    a few u of the spread, a sum of V terms on 128 threads and more by V / 256 + 64 u of itself, the logarithm by the same."""
    rows, vocab = z.shape
    s = z.double()
    m = s.amax(-1, keepdim=True)
    d = torch.where(s == -float("inf"), s, s - m)
    logs = torch.logsumexp(d, -1, keepdim=True)
    lp = d - logs
    p = lp.exp()
    plp = torch.xlogy(p, p)
    ent = -plp.sum(-1)
    spread = torch.where(p > 1e-40, d.abs(), 0.0).amax(-1)
    e = (64 + 16 * spread + vocab / 256) * U
    keep = ids >= 0
    at = ids.clamp_min(0)[:, None]
    want = torch.where(keep, lp.gather(1, at)[:, 0], 0.0)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(r.logp), fin)
    assert ((r.logp - want).abs() - e - 4 * U * want.abs())[fin].max().item() <= 0
    # the entropy's terms p log p are off by e (|log p| + 1) relative to p
    assert ((r.entropy - ent).abs() - e * (2 + 4 * spread + 2 * logs[:, 0])).max().item() <= 0
    if k:
        v, i = torch.sort(z.float(), dim=-1, descending=True, stable=True)
        assert torch.equal(r.top_ids, i[:, :k].int())
        tl = torch.gather(lp, 1, i[:, :k])
        fin = torch.isfinite(tl.float())  # lowest - largest is below every fp32 value: -inf
        assert torch.equal(torch.isfinite(r.top_logp), fin)
        assert ((r.top_logp - tl).abs() - e[:, None] - 4 * U * tl.abs())[fin].max().item() <= 0
    g, h = randn(gen(1), rows).abs() + 0.5, randn(gen(2), rows)
    gl = torch.where(keep, g.double(), 0.0)[:, None]
    own = torch.zeros_like(p).scatter_(1, at, 1.0) * gl
    hd = h.double()[:, None]
    out = 2.0 ** -8 if z.dtype == BF16 else U
    for dent in (None, h):
        d = lm.token_logprobs_grad(z, ids, r, g, dentropy=dent)
        want, mag = own - p * gl, own + p * gl
        if dent is not None:
            want = want - hd * (plp + p * ent[:, None])
            mag = mag + hd.abs() * (plp.abs() + p * (ent[:, None] + 1 + logs.abs()))
        bound = 4 * e[:, None] * mag + out * want.abs() + 2.0 ** -140
        assert ((d.double() - want).abs() - bound).max().item() <= 0


@pytest.mark.parametrize("dtype,offsets", [(F32, (0.0, 4096.0, -65536.0, 2.0 ** 20)), (BF16, (0.0, 64.0, -64.0))])
@pytest.mark.parametrize("rows,vocab,k", [(3, 5000, 0), (40, 777, 5), (1, 40000, 20), (5, 131072, 3)])
def test_a_common_offset_costs_no_digits(dtype, offsets, rows, vocab, k):
    g = gen(vocab)
    # whole steps that are exact at every offset
    z = torch.randint(-16, 17, (rows, vocab), generator=g, device="cuda").float() * (0.125 if dtype == F32 else 0.5)
    ids = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    ids[rows // 2] = -1 if rows > 1 else ids[0]
    first = None
    for o in offsets:
        zz = (z + o).to(dtype)
        assert torch.equal(zz.float(), z + o)
        r = lm.token_logprobs(zz, ids, top_k=k)
        _probabilities(zz, ids, r, k)
        if first is None:
            first = r
        # the same differences to the maximum: the same bits
        assert torch.equal(r.logp, first.logp) and torch.equal(r.entropy, first.entropy)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [7, 1000, 4097, 50000])
def test_rows_of_the_lowest_value(dtype, vocab):
    """A mask of the type's lowest value that leaves nothing, or one token, and the same where the rest is -inf."""
    low = torch.finfo(dtype).min
    z = torch.full((5, vocab), low, device="cuda", dtype=dtype)
    z[1, 3] = 1.5
    z[2, 2:] = -float("inf")
    z[3, 5:] = torch.finfo(dtype).max
    ids = torch.tensor([3, 3, 1, vocab - 1, -1], device="cuda")
    r = lm.token_logprobs(z, ids, top_k=3)
    _probabilities(z, ids, r, 3)
    d = lm.token_logprobs_grad(z, ids, r, torch.ones(5, device="cuda"))
    assert d[4].abs().max().item() == 0


def test_second_derivatives_are_refused():
    """With the kernels: gradients in a graph of gradients are the same, and differentiating them raises."""
    g = gen(3)
    ids = torch.tensor([1, 3, 3, 0], device="cuda")
    x, w, r = (randn(g, *s).requires_grad_() for s in ((4, 256), (256,), (4, 256)))
    a, b, z, t = (randn(g, *s).requires_grad_() for s in ((4, 256), (200, 256), (4, 99), (5, 64)))
    cases = [("norm", x, lambda: lm.norm(x, w)[:, :5].sum()), ("norm", w, lambda: lm.norm(x, w, r)[0].pow(2).sum()),
             ("norm", r, lambda: sum(y.pow(2).sum() for y in lm.norm(x, w, r))),
             ("linear", a, lambda: lm.linear(a, b).sum()), ("linear", b, lambda: lm.linear(a, b).sum()),
             ("logprobs", z, lambda: lm.logprobs(z, ids)[0].sum()), ("logprobs", z, lambda: lm.logprobs(z, ids)[1].sum()),
             ("embed", t, lambda: lm.embed(t, ids).pow(2).sum())]
    for name, v, fn in cases:
        plain, = torch.autograd.grad(fn(), v)
        loss = fn() + v.pow(3).sum()
        first, = torch.autograd.grad(loss, v, create_graph=True)
        assert torch.equal(first, plain + 3 * v.detach() ** 2)
        for second in (lambda: torch.autograd.grad(first.sum(), v, retain_graph=True),
                       lambda: (loss + first.pow(2).sum()).backward()):
            with pytest.raises(RuntimeError, match=name):
                second()
                pytest.fail(f"a second derivative through {name} was lost")


def test_backward_with_an_output_that_nobody_uses():
    """A loss that uses one of two outputs has the gradient of that output alone."""
    g = gen(4)
    x, w, r = (randn(g, *s).requires_grad_() for s in ((40, 300), (300,), (40, 300)))
    s = (x + r).detach()
    rstd = lm.rms_norm(s, w.detach()).rstd
    y, _ = lm.norm(x, w, r)
    c = randn(g, 40, 300)
    want = lm.rms_norm_grad(c, s, w.detach(), rstd)
    for got, v in zip(torch.autograd.grad(y, (x, r, w), c), (want[0], want[0], want[1])):
        assert torch.equal(got, v)
    _, t = lm.norm(x, w, r)
    dx, dr, dw = torch.autograd.grad(t, (x, r, w), c)
    assert torch.equal(dx, c) and torch.equal(dr, c) and dw.abs().max().item() == 0
    z = randn(g, 30, 500).requires_grad_()
    ids = torch.randint(-1, 500, (30,), generator=g, device="cuda")
    c = randn(g, 30)
    q = lm.token_logprobs(z.detach(), ids)
    zero = torch.zeros_like(c)
    got, = torch.autograd.grad(lm.logprobs(z, ids)[0], z, c)
    want = lm.token_logprobs_grad(z.detach(), ids, q, c)
    assert (got - want).abs().max().item() <= 4 * U * want.abs().max().item()
    got, = torch.autograd.grad(lm.logprobs(z, ids)[1], z, c)
    assert torch.equal(got, lm.token_logprobs_grad(z.detach(), ids, q, zero, dentropy=c))


def _writes(g):
    """(tensor that is written, call that writes it) of every call that writes over a tensor of the caller."""
    x, w, ids = randn(g, 6, 256), randn(g, 256), torch.tensor([1, 2, 0, 3, 3, -1], device="cuda")
    q, wq = lm.fp8_quantize(x), lm.fp8_quantize(randn(g, 40, 256), block="square")
    r, z, t, o = randn(g, 6, 256), randn(g, 6, 50), randn(g, 9, 256), randn(g, 6, 40)
    s = lm.token_logprobs(z, ids)
    one = torch.ones(6, device="cuda")
    return [(r, lambda v: lm.rms_norm(x, w, residual=v, inplace=True)),
            (z, lambda v: lm.token_logprobs_grad(v, ids, s, one, inplace=True)),
            (t, lambda v: lm.embedding_grad(x, ids, 9, out=v)), (t, lambda v: lm.embedding_grad(x, ids, 9, base=v, out=v)),
            (o, lambda v: lm.fp8_matmul(q, wq, out=v)), (o, lambda v: lm.fp8_matmul(q, wq, out=v, accumulate=True))]


def test_in_place_writes_are_known_to_autograd():
    for i, (v, call) in enumerate(_writes(gen(5))):
        leaf = torch.ones_like(v).requires_grad_()
        saved = leaf * v  # keeps v for its backward
        before, old = v._version, v.clone()
        call(v)
        assert v._version > before and not torch.equal(v, old), i
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved.sum().backward()
            pytest.fail(f"write {i} went unnoticed")
        # a tensor that requires a gradient: a leaf, and the result of a step that autograd knows
        for grad in (v.clone().requires_grad_(), v.clone().requires_grad_() * 1.0):
            with pytest.raises(ValueError, match="requires a gradient"):
                call(grad)
                pytest.fail(f"write {i} took a tensor that requires a gradient")
            with torch.no_grad():
                before = grad._version
                call(grad)
                assert grad._version > before, i
    with torch.inference_mode():
        inside = _writes(gen(5))
        for v, call in inside:
            call(v)
    for i, (v, call) in enumerate(inside):
        with pytest.raises(ValueError, match="inference"):
            call(v)
            pytest.fail(f"write {i} took an inference tensor")


def test_saved_stream_and_logits_are_guarded():
    """The norm's backward keeps the stream and the loss' keeps the logits: later writes in place are found out."""
    g = gen(6)
    x, w, r = (randn(g, *s).requires_grad_() for s in ((6, 256), (256,), (6, 256)))
    y, s = lm.norm(x, w, r)
    with torch.no_grad():
        lm.rms_norm(x, w, residual=s, inplace=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    z = randn(g, 6, 50).requires_grad_() * 1.0
    ids = torch.tensor([1, 2, 0, 3, 3, -1], device="cuda")
    logp, _ = lm.logprobs(z, ids)
    with torch.no_grad():
        lm.token_logprobs_grad(z, ids, lm.token_logprobs(z, ids), torch.ones(6, device="cuda"), inplace=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        logp.sum().backward()


@pytest.mark.parametrize("m,n,k", [(300, 19500, 128), (2048, 5504, 1024), (200, 1000, 4096)])
def test_an_old_timeout_does_not_stop_a_product(m, n, k):
    """A timeout that another call left in the status word stays to be read, and changes no later product."""
    g = gen(m)
    a, b = lm.fp8_quantize(randn(g, m, k)), lm.fp8_quantize(randn(g, n, k), block="square")
    want = lm.fp8_matmul(a, b)
    out = torch.empty_like(want)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    word[0] = L.DEV_TIMEOUT | L.DEV_BAD_TOKEN
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(3):
        out.fill_(float("nan"))
        assert L.lib().okls_fp8_matmul(
            a.data.data_ptr(), a.data.stride(0), a.scale.data_ptr(), a.scale.stride(0), a.scale.stride(1),
            b.data.data_ptr(), b.data.stride(0), b.scale.data_ptr(), b.scale.stride(0), b.scale.stride(1), L.FP8_SQUARE,
            m, n, k, out.data_ptr(), L.OKLS_BF16, n, 0, word.data_ptr(), stream) == L.OKLS_OK
        assert torch.equal(out, want)
    assert word.item() == L.DEV_TIMEOUT | L.DEV_BAD_TOKEN


def test_status_bits_of_other_streams_are_not_lost():
    """Bad tokens on one stream while another reads and clears the word: each is reported once they are both done."""
    w = randn(gen(7), 10, 16)
    bad, good = torch.tensor([11], device="cuda"), torch.tensor([1], device="cuda")
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()

    def read(stream=None):
        try:
            return lm.query_status(stream=stream)
        except L.OklsError as e:
            assert e.code == L.OKLS_ERR_INVALID_ARG
            return L.DEV_BAD_TOKEN

    for i in range(300):
        with torch.cuda.stream(one):
            for _ in range(i % 7):
                lm.embedding(w, good)
            lm.embedding(w, bad)
        seen = read(two)
        one.synchronize()
        assert seen | read(two) == L.DEV_BAD_TOKEN, i
        assert read(one) == 0


FIRST = """
import torch
from kronecker_factored_second_gb300 import lm
g = torch.Generator(device="cuda"); g.manual_seed(0)
W = torch.randn(300, 256, generator=g, device="cuda"); nw = torch.ones(256, device="cuda")
ids = torch.randint(-1, 300, (200,), generator=g, device="cuda"); gl = torch.ones(200, device="cuda")
def chain():
    x = lm.embedding(W, ids)
    n = lm.rms_norm(x, nw, residual=x)
    z = lm.fp8_matmul(lm.fp8_quantize(n.y), lm.fp8_quantize(W, block="square"), out_dtype=torch.float32)
    r = lm.token_logprobs(z, ids, top_k=3)
    dz = lm.token_logprobs_grad(z, ids, r, gl, dentropy=gl)
    ds, dw = lm.rms_norm_grad(x, n.residual, nw, n.rstd)
    return z, r.logp, r.top_ids, dz, ds, dw, lm.embedding_grad(ds, ids, 300)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    first = chain()
graph.replay()
for a, b in zip(first, chain()):
    assert torch.equal(a, b)
assert lm.query_status() == 0
print("captured")
"""


def test_first_calls_of_a_process_can_be_captured():
    """No call synchronises or sets anything up that a capture forbids, the first of a process included."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("dim", [1, 153, 257, 1001, 1028, 2044, 2049, 3001, 4102])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, F32), (F32, F32), (F32, BF16)])
def test_embedding_gradient_of_rows_that_are_not_aligned(dtype, out_dtype, dim):
    """Rows that start off 16-byte boundaries in any of dy, base and out: new, added, in place, and with few tokens."""
    g = gen(dim)
    vocab = 700
    for tokens, pd, pb, po in ((5, 0, 0, 0), (900, 0, 0, 0), (900, 3, 1, 8), (900, 1, 8, 5), (2500, 8, 0, 1)):
        def rows(n, pitch, dt):
            return randn(g, n, dim + pitch, dtype=dt)[:, :dim]
        dy, base, out = rows(tokens, pd, dtype), rows(vocab, pb, out_dtype), rows(vocab, po, out_dtype)
        ids = torch.randint(-20, vocab, (tokens,), generator=g, device="cuda").clamp_min(-1)
        ids[tokens // 3:tokens // 2] = 17  # a token of many chunks
        keep = ids >= 0
        zero = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda")
        total = zero.index_add(0, ids[keep], dy[keep].double())
        mag = zero.index_add(0, ids[keep], dy[keep].double().abs())
        n = torch.bincount(ids[keep], minlength=vocab).double()[:, None]
        for b in (None, base):
            want = total * 0.5 + (0 if b is None else b.double())
            # n additions, the scaling and the base: one rounding each, then the output's
            bound = (n + 2) * U * (mag * 0.5 + (0 if b is None else b.double().abs()))
            bound = bound + (2.0 ** -8 if out_dtype == BF16 else U) * want.abs()
            fresh = lm.embedding_grad(dy, ids, vocab, scale=0.5, base=b, dtype=out_dtype)
            assert ((fresh.double() - want).abs() - bound).max().item() <= 0
            lm.embedding_grad(dy, ids, vocab, scale=0.5, base=b, out=out)
            assert torch.equal(out, fresh)
        lm.embedding_grad(dy, ids, vocab, scale=0.5, base=base, out=base)
        assert torch.equal(base, fresh)


@pytest.mark.parametrize("tokens,vocab,dim", [(79, 37178, 3435), (9, 55846, 1662), (2112, 33216, 5217), (100, 65536, 1001)])
def test_embedding_gradient_is_no_slower_than_a_plain_one(tokens, vocab, dim):
    """Rows off 16-byte boundaries: the new and the added gradient against torch's fill or copy and index_add_."""
    g = gen(tokens)
    dy, base = randn(g, tokens, dim), randn(g, vocab, dim)
    ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")

    def us(f):
        times = []
        for i in range(13):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            f()
            b.record()
            b.synchronize()
            if i >= 3:
                times.append(a.elapsed_time(b) * 1e3)
        return sorted(times)[len(times) // 2]

    for own, plain in ((lambda: lm.embedding_grad(dy, ids, vocab),
                        lambda: torch.zeros(vocab, dim, device="cuda").index_add_(0, ids, dy)),
                       (lambda: lm.embedding_grad(dy, ids, vocab, base=base), lambda: base.clone().index_add_(0, ids, dy))):
        a, b = us(own), us(plain)
        assert a <= 1.5 * b, f"{a:.0f} us, plain {b:.0f}"


@pytest.mark.parametrize("m,n,k", [(7, 300, 520), (300, 19500, 130), (2048, 5504, 256), (515, 700, 2047)])
def test_scales_laid_out_by_the_caller(m, n, k):
    """Scale matrices with contiguous rows, and cut out of wider ones: the products of the quantiser's own layout."""
    g = gen(m + n)
    x, w = randn(g, m, k) * torch.exp(randn(g, m, 1)), randn(g, n, k)
    a = lm.fp8_quantize(x)

    def laid_out(f):
        wide = torch.full((f.scale.shape[0], f.scale.shape[1] + 3), float("nan"), device="cuda")
        wide[:, 1:1 + f.scale.shape[1]] = f.scale
        tall = torch.full((f.scale.shape[1], f.scale.shape[0] + 5), float("nan"), device="cuda")
        tall[:, 2:2 + f.scale.shape[0]] = f.scale.t()
        return [lm.Fp8Tensor(f.data, s, f.block) for s in
                (f.scale.contiguous(), wide[:, 1:1 + f.scale.shape[1]], tall[:, 2:2 + f.scale.shape[0]].t())]

    for block in ("row", "square"):
        b = lm.fp8_quantize(w, block=block)
        for out_dtype in (BF16, F32):
            want = lm.fp8_matmul(a, b, out_dtype=out_dtype)
            for f, h in zip(laid_out(a), laid_out(b)):
                assert torch.equal(lm.fp8_matmul(f, h, out_dtype=out_dtype), want)
                assert torch.equal(lm.fp8_matmul(a, h, out_dtype=out_dtype), want)


def test_two_streams_at_once():
    """Two chains of all operators that run at the same time give what they give one after the other."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    data = []
    for seed in (1, 2):
        g = gen(seed)
        rows = 1500 + 700 * seed
        data.append((randn(g, rows, 1024, dtype=BF16), randn(g, 2304, 1024, dtype=BF16, std=0.03), randn(g, 1024, dtype=BF16),
                     torch.randint(-1, 2304, (rows,), generator=g, device="cuda")))

    def chain(x, w, nw, ids):
        h = lm.embedding(w, ids, scale=2.0)
        n = lm.rms_norm(x, nw, residual=h)
        q, qt = lm.fp8_quantize(n.y, both=True)
        z = lm.fp8_matmul(q, lm.fp8_quantize(w, block="square"))
        r = lm.token_logprobs(z, ids, top_k=9)
        one = torch.ones(x.shape[0], device="cuda")
        dz = lm.token_logprobs_grad(z, ids, r, one, dentropy=one)
        dw = lm.fp8_matmul(lm.fp8_quantize(dz, transpose=True), qt)
        ds, dn = lm.rms_norm_grad(x, n.residual, nw, n.rstd)
        return z, r.logp, r.top_ids, dz, dw, ds, dn, lm.embedding_grad(ds, ids, 2304)

    want = [chain(*d) for d in data]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [[], []]
        for _ in range(3):
            for i, (s, d) in enumerate(zip(streams, data)):
                with torch.cuda.stream(s):
                    got[i].append(chain(*d))
        torch.cuda.synchronize()
        for i in range(2):
            for each in got[i]:
                for a, b in zip(each, want[i]):
                    assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last rows are those of the same rows alone."""
    g = gen(8)
    rows, cols, tail = 66000, 32768, 200
    x = torch.empty(rows, cols, device="cuda", dtype=BF16)
    x[:-tail] = 0.25
    x[-tail:] = randn(g, tail, cols, dtype=BF16)
    assert x.numel() > 1 << 31
    end = x[-tail:].clone()
    ids = torch.randint(0, cols, (rows,), generator=g, device="cuda")
    # norm and its gradient, and the 8-bit output
    w = randn(g, cols, dtype=BF16)
    n, m = lm.rms_norm(x, w), lm.rms_norm(end, w)
    assert torch.equal(n.y[-tail:], m.y) and torch.equal(n.rstd[-tail:], m.rstd)
    del n
    n = lm.rms_norm(x, w, out_dtype=E4M3)
    e8 = lm.rms_norm(end, w, out_dtype=E4M3).y
    assert torch.equal(n.y.data[-tail:].view(torch.uint8), e8.data.view(torch.uint8))
    assert torch.equal(n.y.scale[-tail:], e8.scale)
    del n
    ds, _ = lm.rms_norm_grad(x, x, w, torch.ones(rows, device="cuda"), need_dweight=False)
    assert torch.equal(ds[-tail:], lm.rms_norm_grad(end, end, w, torch.ones(tail, device="cuda"), need_dweight=False)[0])
    del ds
    # log probabilities and their gradient in place, over the same memory
    r, s = lm.token_logprobs(x, ids, top_k=4), lm.token_logprobs(end, ids[-tail:], top_k=4)
    assert torch.equal(r.top_ids[-tail:], s.top_ids)
    # few rows are split between CTAs, so the sums have another order: each is off by (64 + 16 spread + vocab / 256) u
    for a, b in ((r.logp, s.logp), (r.entropy, s.entropy), (r.lse, s.lse)):
        assert ((a[-tail:] - b).abs() - 2 * (64 + 16 * 12 + cols / 256) * U - 4 * U * b.abs()).max().item() <= 0
    s = lm.TokenLogprobs(None, r.entropy[-tail:], r.lse[-tail:], lse_rest=r.lse_rest[-tail:])
    one = torch.ones(rows, device="cuda")
    d = lm.token_logprobs_grad(x, ids, r, one)
    assert torch.equal(d[-tail:], lm.token_logprobs_grad(end, ids[-tail:], s, one[-tail:]))
    del d
    # codes of both orientations, and a product whose output passes 2^31
    q, qt = lm.fp8_quantize(x, both=True)
    e = lm.fp8_quantize(end)
    assert torch.equal(q.data[-tail:].view(torch.uint8), e.data.view(torch.uint8)) and torch.equal(q.scale[-tail:], e.scale)
    assert torch.equal(lm.fp8_quantize(x[rows // 128 * 128:], transpose=True).data.view(torch.uint8),
                       qt.data[:, rows // 128 * 128:].view(torch.uint8))
    del q, qt
    # the table, its rows and its gradient
    at = torch.cat([torch.arange(rows - tail, rows, device="cuda"), torch.tensor([-1], device="cuda")])
    y = lm.embedding(x, at)
    assert torch.equal(y[:-1], end) and y[-1].abs().max().item() == 0
    dw = lm.embedding_grad(y, at, rows, dtype=BF16)
    assert torch.equal(dw[-tail:], end) and dw[:-tail].abs().max().item() == 0
    del dw, y, x
    a, b = lm.fp8_quantize(randn(g, rows, 128)), lm.fp8_quantize(randn(g, cols, 128), block="square")
    c = lm.fp8_matmul(a, b)
    last = lm.Fp8Tensor(a.data[-512:], a.scale[-512:], "row")
    want = last.float() @ b.float().t()
    # bf16's rounding, and the order of 128 additions
    assert ((c[-512:].float() - want).abs() - 2.0 ** -8 * want.abs() - 1e-3).max().item() <= 0


def test_alternatives_of_a_very_long_row():
    """Rows longer than the maxima that a cluster keeps (131072 columns a CTA, 8 CTAs)."""
    g = gen(9)
    z = randn(g, 2, 1_100_003, dtype=BF16)
    ids = torch.tensor([1_100_002, 5], device="cuda")
    r = lm.token_logprobs(z, ids, top_k=7)
    i = torch.sort(z.float(), dim=-1, descending=True, stable=True)[1][:, :7]
    assert torch.equal(r.top_ids, i.int())
    lp = torch.log_softmax(z.double(), -1)
    assert (r.logp - lp.gather(1, ids[:, None])[:, 0]).abs().max().item() < 1e-4
