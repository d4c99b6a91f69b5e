"""Argument checks of the language-model operators' C entries (no GPU needed):
a bad argument is refused before anything reaches the device."""

import ctypes

import pytest
import torch

from kronecker_factored_second_gb300 import _lib as L
from kronecker_factored_second_gb300 import lm

P = 4096  # stands for a device address; never followed
BAD, UNSUP = L.OKLS_ERR_INVALID_ARG, L.OKLS_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(L.LIB_PATH):
        from kronecker_factored_second_gb300.build import build_library
        build_library()
    return L.lib()


def refused(args, changes, fn):
    """Every (index, value) change of a valid argument list returns its code and a message."""
    for change, code in changes:
        a = list(args)
        for i, v in change.items():
            a[i] = v
        assert fn(*a) == code, (change, L.last_error())
        assert L.last_error()


def test_embedding_arguments(lib):
    ok = [P, 0, 64, 100, 64, P, 1, 10, 1.0, P, 0, 64, P, None]
    refused(ok, [({0: None}, BAD), ({1: 2}, BAD), ({2: 63}, BAD), ({3: 0}, BAD), ({4: 0}, BAD), ({5: None}, BAD),
                 ({5: P + 4}, BAD), ({6: 2}, BAD), ({7: -1}, BAD), ({9: None}, BAD), ({9: P + 2}, BAD), ({10: 5}, BAD),
                 ({11: 60}, BAD), ({12: None}, BAD), ({3: 1 << 31}, BAD)], lib.okls_embedding)


def test_embedding_grad_arguments(lib):
    need = ctypes.c_size_t()
    assert lib.okls_embedding_grad_workspace_bytes(10, 100, 64, ctypes.byref(need)) == L.OKLS_OK and need.value > 0
    assert lib.okls_embedding_grad_workspace_bytes(10, 100, 64, None) == BAD
    assert lib.okls_embedding_grad_workspace_bytes(-1, 100, 64, ctypes.byref(need)) == BAD
    ok = [P, 0, 64, P, 1, 10, 100, 64, 1.0, None, 0, P, 0, 64, P, need.value, P, None]
    refused(ok, [({0: None}, BAD), ({1: 2}, BAD), ({2: 8}, BAD), ({3: None}, BAD), ({4: 3}, BAD), ({6: 0}, BAD),
                 ({9: P, 10: 3}, BAD), ({9: P, 10: 128}, BAD), ({11: None}, BAD), ({12: 2}, BAD), ({14: None}, BAD),
                 ({14: P + 8}, BAD), ({15: need.value - 1}, BAD), ({16: None}, BAD),
                 ({6: (1 << 31) - 2, 7: 4096, 2: 4096, 13: 4096}, UNSUP)], lib.okls_embedding_grad)


def test_rms_norm_arguments(lib):
    ok = [P, 0, 64, None, 0, P, 0, 10, 64, 1e-6, P, 0, 64, None, 0, 0, None, 0, P, None]
    refused(ok, [({0: None}, BAD), ({1: 2}, BAD), ({2: 3}, BAD), ({3: P, 4: 64}, BAD), ({16: P, 17: 64}, BAD),
                 ({5: None}, BAD), ({6: 2}, BAD), ({7: -1}, BAD), ({8: 0}, BAD),
                 ({8: 40000, 2: 40000, 12: 40000}, UNSUP), ({9: -1.0}, BAD), ({9: float("nan")}, BAD),
                 ({10: None}, BAD), ({11: 3}, BAD), ({11: 2}, BAD), ({13: P}, BAD),
                 ({11: 2, 13: P, 14: -1}, BAD)], lib.okls_rms_norm)
    ok = [P, 0, 64, P, 0, 64, P, 0, P, None, 0, 10, 64, P, 64, None, None, 0, None]
    refused(ok, [({0: None}, BAD), ({1: 2}, BAD), ({3: None}, BAD), ({4: 2}, BAD), ({6: None}, BAD), ({8: None}, BAD),
                 ({9: P, 10: 1}, BAD), ({11: -1}, BAD), ({12: 0}, BAD), ({13: None}, BAD), ({14: 2}, BAD)],
            lib.okls_rms_norm_grad)


def test_fp8_arguments(lib):
    ok = [P, 0, 64, 10, 64, 0, P, 128, P, 1, 12, None, 0, None, 0, 0, None]
    refused(ok, [({0: None}, BAD), ({1: 2}, BAD), ({2: 1}, BAD), ({3: -1}, BAD), ({5: 2}, BAD), ({6: None, 8: None}, BAD),
                 ({8: None}, BAD), ({6: None}, BAD), ({7: 32}, BAD), ({11: P, 12: 2, 13: P}, BAD), ({11: P}, BAD),
                 ({9: -1}, BAD), ({3: 1 << 25}, UNSUP)], lib.okls_fp8_quantize)
    ok = [P, 128, P, 1, 12, P, 128, P, 1, 12, 1, 10, 20, 64, P, 1, 20, 0, P, None]
    refused(ok, [({0: None}, BAD), ({1: 32}, BAD), ({1: 136}, UNSUP), ({0: P + 8}, UNSUP), ({5: P + 8}, UNSUP),
                 ({2: None}, BAD), ({7: None}, BAD), ({3: -1}, BAD), ({10: 2}, BAD), ({11: -1}, BAD), ({14: None}, BAD),
                 ({14: P + 1}, BAD), ({15: 2}, BAD), ({16: 10}, BAD), ({17: 2}, BAD), ({18: None}, BAD)],
            lib.okls_fp8_matmul)
    # nothing to compute: taken without a device
    assert lib.okls_fp8_matmul(*[0 if i in (11,) else v for i, v in enumerate(ok)]) == L.OKLS_OK


def test_token_logprobs_arguments(lib):
    ok = [P, 0, 64, P, 1, 10, 64, 1.0, 4, P, P, P, P, P, P, None]
    refused(ok, [({0: None}, BAD), ({1: 2}, BAD), ({2: 63}, BAD), ({3: None}, BAD), ({4: 2}, BAD), ({5: -1}, BAD),
                 ({6: 0}, BAD), ({7: 0.0}, BAD), ({7: float("inf")}, BAD), ({8: 33}, BAD), ({8: -1}, BAD),
                 ({6: 3, 8: 4}, BAD), ({12: None}, BAD), ({13: None}, BAD), ({14: None}, BAD)], lib.okls_token_logprobs)
    ok = [P, 0, 64, P, 1, 10, 64, 1.0, P, P, P, None, P, 64, None]
    refused(ok, [({0: None}, BAD), ({1: 2}, BAD), ({3: None}, BAD), ({7: -1.0}, BAD), ({8: None}, BAD), ({10: None}, BAD),
                 ({9: None, 11: P}, BAD), ({12: None}, BAD), ({13: 2}, BAD)], lib.okls_token_logprobs_grad)
    assert lib.okls_status_word_read(None, None, None) == BAD


def test_python_refuses_host_tensors():
    x, ids = torch.zeros(4, 64), torch.zeros(4, dtype=torch.long)
    for call in (lambda: lm.embedding(x, ids), lambda: lm.embedding_grad(x, ids, 9),
                 lambda: lm.rms_norm(x, torch.zeros(64)), lambda: lm.fp8_quantize(x),
                 lambda: lm.token_logprobs(x, ids)):
        with pytest.raises(ValueError):
            call()
