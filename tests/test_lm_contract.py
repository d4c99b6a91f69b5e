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
