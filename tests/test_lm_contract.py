"""What the language-model operators refuse, and how their gradients behave, without a GPU."""

import ctypes

import pytest

from kronecker_factored_second_gb300 import _lib as L

P = 4096  # stands for a device address; never followed
BAD = L.OKLS_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(L.LIB_PATH):
        from kronecker_factored_second_gb300.build import build_library
        build_library()
    return L.lib()


def test_misaligned_vectors_are_refused(lib):
    """Every vector of 4-byte elements that a kernel follows is refused off a 4-byte boundary."""
    need = ctypes.c_size_t()
    assert lib.okls_embedding_grad_workspace_bytes(10, 100, 64, ctypes.byref(need)) == L.OKLS_OK
    calls = [
        (lib.okls_embedding, [P, 0, 64, 100, 64, P, 1, 10, 1.0, P, 0, 64, P, None], (12,)),
        (lib.okls_embedding_grad, [P, 0, 64, P, 1, 10, 100, 64, 1.0, None, 0, P, 0, 64, P, need.value, P, None], (16,)),
        (lib.okls_rms_norm, [P, 0, 64, None, 0, P, 0, 10, 64, 1e-6, P, 2, 64, P, 1, 12, None, 0, P, None], (13, 18)),
        (lib.okls_rms_norm_grad, [P, 0, 64, P, 0, 64, P, 0, P, None, 0, 10, 64, P, 64, P, P, 1 << 30, None], (8, 15)),
        (lib.okls_fp8_quantize, [P, 0, 64, 10, 64, 0, P, 128, P, 1, 12, P, 128, P, 1, 64, None], (8, 13)),
        (lib.okls_fp8_matmul, [P, 128, P, 1, 12, P, 128, P, 1, 12, 1, 10, 20, 64, P, 1, 20, 0, P, None], (2, 7, 18)),
        (lib.okls_token_logprobs, [P, 0, 64, P, 1, 10, 64, 1.0, 4, P, P, P, P, P, P, None], (9, 10, 11, 12, 13, 14)),
        (lib.okls_token_logprobs_grad, [P, 0, 64, P, 1, 10, 64, 1.0, P, P, P, P, P, 64, None], (8, 9, 10, 11)),
        (lib.okls_status_word_read, [P, None, None], (0,)),
    ]
    for fn, ok, where in calls:
        for i in where:
            a = list(ok)
            a[i] = P + 2
            assert fn(*a) == BAD, (fn.__name__, i, L.last_error())
            assert "aligned" in L.last_error(), (fn.__name__, i, L.last_error())


class _Lent:
    """Stands for a CUDA tensor: remembers the streams that were told of it."""
    is_cuda = True

    def __init__(self):
        self.streams = []

    def record_stream(self, s):
        self.streams.append(s)


def test_inputs_of_a_call_on_another_stream_are_recorded(monkeypatch):
    """The allocator learns that `stream` uses the inputs, so their memory is not handed out again too early."""
    import contextlib
    import dataclasses
    import types

    import torch

    from kronecker_factored_second_gb300 import lm
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(lm, "_n", lambda: types.SimpleNamespace(
        embedding=lambda *a: None, embedding_grad=lambda *a: None, rms_norm=lambda *a: (None,) * 4,
        rms_norm_grad=lambda *a: None, fp8_quantize=lambda *a: (None,) * 4, fp8_matmul=lambda *a: None,
        token_logprobs=lambda *a: (None,) * len(dataclasses.fields(lm.TokenLogprobs)), token_logprobs_grad=lambda *a: None))
    t = [_Lent() for _ in range(6)]
    f = [lm._fp8(t[0], t[1], "row"), lm._fp8(t[2], t[3], "square")]
    r = lm.TokenLogprobs(None, t[2], t[3])
    calls = [
        (lambda s: lm.embedding(t[0], t[1], stream=s), 2),
        (lambda s: lm.embedding_grad(t[0], t[1], 9, base=t[2], out=t[3], stream=s), 4),
        (lambda s: lm.rms_norm(t[0], t[1], residual=t[2], stream=s), 3),
        (lambda s: lm.rms_norm(t[0], t[1], stream=s), 2),
        (lambda s: lm.rms_norm_grad(t[0], t[1], t[2], t[3], dresidual=t[4], stream=s), 5),
        (lambda s: lm.fp8_quantize(t[0], stream=s), 1),
        (lambda s: lm.fp8_matmul(*f, out=t[4], stream=s), 5),
        (lambda s: lm.token_logprobs(t[0], t[1], stream=s), 2),
        (lambda s: lm.token_logprobs_grad(t[0], t[1], r, t[4], dentropy=t[5], stream=s), 6),
    ]
    for i, (call, count) in enumerate(calls):
        for stream in (None, f"stream {i}"):
            for x in t:
                x.streams.clear()
            call(stream)
            told = [] if stream is None else [stream]
            assert [x.streams for x in t] == [told] * count + [[]] * (6 - count), (i, stream)


@pytest.fixture
def on_cpu(monkeypatch):
    """The calls under the differentiable functions, computed on the CPU by torch."""
    import torch

    from kronecker_factored_second_gb300 import lm

    def embedding(weight, ids, *, scale=1.0, out_dtype=None):
        return weight.detach()[ids] * scale

    def embedding_grad(dy, ids, vocab, *, scale=1.0, dtype=torch.float32):
        return torch.zeros(vocab, dy.shape[-1]).index_add_(0, ids, dy.detach() * scale)

    def rms_norm(x, weight, *, residual=None, eps=1e-6, out_dtype=None):
        s = x.detach() if residual is None else x.detach() + residual.detach()
        rstd = torch.rsqrt((s * s).mean(-1) + eps)
        return lm.NormOutput(s * rstd[:, None] * weight.detach(), x if residual is None else s, rstd)

    def rms_norm_grad(dy, s, weight, rstd, *, dresidual=None, need_dweight=True):
        dy, s, weight = dy.detach(), s.detach(), weight.detach()
        xh, g = s * rstd[:, None], dy * weight
        ds = rstd[:, None] * (g - xh * (g * xh).mean(-1, keepdim=True))
        return ds if dresidual is None else ds + dresidual.detach(), (dy * xh).sum(0)

    def fp8_quantize(x, *, block="row", transpose=False, both=False):
        def q(m):
            lines = m.shape[0] if block == "row" else -(-m.shape[0] // 128)
            return lm._fp8(m.to(torch.float8_e4m3fn), torch.ones(lines, -(-m.shape[1] // 128)), block)
        x = x.detach()
        return (q(x), q(x.t().contiguous())) if both else q(x.t().contiguous() if transpose else x)

    def fp8_matmul(a, b, *, out_dtype=torch.bfloat16):
        return (a.data.float() @ b.data.float().t()).to(out_dtype)

    def token_logprobs(logits, ids, *, scale=1.0):
        lp = torch.log_softmax(logits.detach() * scale, -1)
        ent = -(lp.exp() * lp).sum(-1)
        lse = torch.logsumexp(logits.detach() * scale, -1)
        return lm.TokenLogprobs(lp.gather(1, ids[:, None])[:, 0], ent, lse, lse_rest=torch.zeros_like(lse))

    def token_logprobs_grad(logits, ids, result, dlogp, *, dentropy=None, scale=1.0):
        lp = logits.detach() * scale - result.lse[:, None]
        p, g = lp.exp(), dlogp.detach()[:, None]
        d = torch.zeros_like(p).scatter_(1, ids[:, None], 1.0) * g - p * g
        return scale * (d - dentropy.detach()[:, None] * p * (lp + result.entropy[:, None]))

    for f in (embedding, embedding_grad, rms_norm, rms_norm_grad, fp8_quantize, fp8_matmul, token_logprobs,
              token_logprobs_grad):
        monkeypatch.setattr(lm, f.__name__, f)
    return lm


def _second_order_cases(lm):
    import torch
    g = torch.Generator().manual_seed(0)
    ids = torch.tensor([1, 3, 3, 0])

    def leaf(*shape):
        return torch.randn(*shape, generator=g).requires_grad_()
    # each output is summed, so that the gradient that comes back is a constant, and squared, so that it is not
    x, w, r = leaf(4, 8), leaf(8), leaf(4, 8)
    yield "norm", x, lambda: lm.norm(x, w)[:, :5].sum()
    yield "norm", w, lambda: lm.norm(x, w)[:, :5].sum()
    yield "norm", r, lambda: lm.norm(x, w, r)[0][:, :5].sum()
    yield "norm", x, lambda: lm.norm(x.detach().requires_grad_(), w, r)[1].sum() + lm.norm(x * 1.0, w, r)[0].pow(2).sum()
    a, b = leaf(4, 8), leaf(6, 8)
    yield "linear", a, lambda: lm.linear(a, b).sum()
    yield "linear", b, lambda: lm.linear(a, b).sum()
    yield "linear", b, lambda: lm.linear(a.detach(), b).pow(2).sum()
    z = leaf(4, 9)
    yield "logprobs", z, lambda: lm.logprobs(z, ids)[0].sum()
    yield "logprobs", z, lambda: lm.logprobs(z, ids)[1].sum()
    t = leaf(5, 6)
    yield "embed", t, lambda: lm.embed(t, ids).pow(2).sum()


def test_second_derivatives_are_refused(on_cpu):
    """A gradient of a gradient through these functions is not computed: it has to raise, also where another path to the
    same input is differentiable twice, and only where it is asked for."""
    import torch
    for i, (name, x, fn) in enumerate(_second_order_cases(on_cpu)):
        plain, = torch.autograd.grad(fn(), x)
        loss = fn() + x.pow(3).sum()
        first, = torch.autograd.grad(loss, x, create_graph=True)
        assert torch.allclose(first, plain + 3 * x.detach() ** 2), (i, name)
        for second in (lambda: torch.autograd.grad(first.sum(), x, retain_graph=True),
                       lambda: (loss + first.pow(2).sum()).backward()):
            with pytest.raises(RuntimeError, match=name):
                second()
                pytest.fail(f"case {i} lost a second derivative")


def test_first_derivatives_in_a_graph_of_gradients(on_cpu):
    """What does not go through the refused part is differentiable twice: the embedding is linear in its table."""
    import torch
    t = torch.randn(5, 6).requires_grad_()
    ids = torch.tensor([1, 3, 3, 0])
    loss = on_cpu.embed(t, ids).sum() + t.pow(3).sum()
    first, = torch.autograd.grad(loss, t, create_graph=True)
    second, = torch.autograd.grad(first.sum(), t)
    assert torch.allclose(second, 6 * t.detach())
    # and gradients in a graph that nobody differentiates are plain gradients
    x, w = torch.randn(4, 8).requires_grad_(), torch.randn(8).requires_grad_()
    on_cpu.norm(x, w).sum().backward(create_graph=True)
    assert x.grad is not None and w.grad is not None


def test_norm_refuses_outputs_without_a_gradient(on_cpu):
    """An 8-bit output is not a tensor of autograd: the differentiable norm does not offer it."""
    import torch
    x, w = torch.randn(4, 8).requires_grad_(), torch.randn(8).requires_grad_()
    for dtype in (torch.float8_e4m3fn, torch.float16, torch.int8):
        for res in (None, torch.randn(4, 8)):
            with pytest.raises(ValueError, match="norm"):
                on_cpu.norm(x, w, res, out_dtype=dtype)
                pytest.fail(f"{dtype} was taken")
    for dtype in (None, torch.float32, torch.bfloat16):
        assert on_cpu.norm(x, w, out_dtype=dtype).requires_grad


def test_library_status_word_needs_a_place(lib):
    assert lib.okls_status_word(None) == BAD


def test_c_library_is_built_without_the_torch_binding(monkeypatch, tmp_path):
    """A C client needs nvcc alone: whatever fails in the torch binding, the C library is in place and the error says so."""
    from kronecker_factored_second_gb300 import build
    for name in ("BUILD", "LIB", "BINDING_LIB"):
        monkeypatch.setattr(build, name, str(tmp_path / name))

    def run_without(broken):
        def run(cmd):
            if broken in " ".join(cmd):
                raise RuntimeError("command failed")
            if "-o" in cmd:
                open(cmd[cmd.index("-o") + 1], "w").close()
        return run

    def no_torch():
        raise ImportError("no torch here")

    import os
    for broken in ("torch", build.BINDING, "-lokls"):
        for f in ("LIB", "BINDING_LIB"):
            if os.path.exists(tmp_path / f):
                os.remove(tmp_path / f)
        with monkeypatch.context() as m:
            m.setattr(build, "_run", run_without(broken if broken != "torch" else "nothing"))
            m.setattr(build, "_torch_flags", no_torch if broken == "torch" else lambda: ([], []))
            with pytest.raises((RuntimeError, ImportError), match="libokls.so is built"):
                build.build_library()
        assert os.path.exists(tmp_path / "LIB") and not os.path.exists(tmp_path / "BINDING_LIB"), broken
    with monkeypatch.context() as m:
        m.setattr(build, "_run", run_without("nothing"))
        m.setattr(build, "_torch_flags", lambda: ([], []))
        assert build.build_library() == str(tmp_path / "LIB")
    assert os.path.exists(tmp_path / "BINDING_LIB")
