"""The example trains: every operator with its gradient, the optimizer, and the served model."""

import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("train_lm", os.path.join(ROOT, "examples", "train_lm.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_learns_and_serves(example):
    vocab = 512
    model, losses, successor = example.train(60, vocab=vocab)
    # an untrained model is near log(vocab) = 6.2; the data's own entropy is about 0.9
    assert abs(losses[0] - math.log(vocab)) < 1.0
    assert all(math.isfinite(x) for x in losses)
    assert losses[-1] < 3.0, losses[::10]
    # the served model, 16 tokens at a time and one alone, names the successor
    ids = torch.arange(vocab, device="cuda")
    server = example.Server(model)
    many = torch.cat([server.next_tokens(c).top_ids[:, 0] for c in ids.split(16)])
    assert (many == successor).float().mean().item() > 0.8
    one = server.next_tokens(ids[5:6])
    assert one.top_ids.shape == (1, 5) and one.top_ids[0, 0].item() == many[5].item()
    assert (one.top_logp.diff() <= 0).all()


def test_training_step_matches_plain_gradients(example):
    """The model's gradients against the same model in fp32 without 8-bit products."""
    m = example.TokenModel(vocab=300, dim=128, hidden=192, blocks=1, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    ids = torch.randint(-1, 300, (500,), generator=g, device="cuda")
    tgt = torch.randint(-1, 300, (500,), generator=g, device="cuda")
    loss, _ = m.loss(ids, tgt)
    loss.backward()
    own = [p.grad.clone() for p in m.matrices() + m.others()]
    for p in m.matrices() + m.others():
        p.grad = None

    def norm(x, w):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w

    keep = (ids >= 0)[:, None]
    h = m.table[ids.clamp_min(0)] * m.scale * keep
    x = torch.nn.functional.silu(norm(h, m.norms[0]) @ m.up[0].t()) @ m.down[0].t()
    z = norm(x + h, m.norms[1]) @ m.out.t()
    lp = torch.log_softmax(z, -1).gather(1, tgt.clamp_min(0)[:, None])[:, 0]
    plain = -(lp * (tgt >= 0)).sum() / (tgt >= 0).sum()
    plain.backward()
    assert abs(loss.item() - plain.item()) < 0.05
    # e4m3 keeps 4 significant bits: a product of two rounded operands is off by about 4% of its size, less in sums;
    # two or three such products lie on the way of each gradient
    for p, o in zip(m.matrices() + m.others(), own):
        assert ((o - p.grad).norm() / p.grad.norm()).item() < 0.2, p.shape
