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
