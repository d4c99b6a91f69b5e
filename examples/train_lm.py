"""A small token model trained and served with the library's operators.

Training: embedding, RMS norms with the residual's addition, 8-bit linear layers (the weights' and activations'
quantisations and all three products of each), log probabilities and their gradients, and the weight matrices stepped by
Online KL Shampoo (AdamW for the tables and the norms' weights).  Serving: weights quantised once, the norms write the 8-bit
inputs of the products, and the best next tokens come back with their log probabilities.

    python examples/train_lm.py [--steps 80]

The data is synthetic: each token is followed by a fixed successor nine times out of ten, and by any token otherwise, so the
loss can fall from log(vocab) to about 0.9.
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from kronecker_factored_second_gb300 import lm  # noqa: E402
from kronecker_factored_second_gb300.okls import OnlineKLShampoo  # noqa: E402


class TokenModel:
    """Token table, feed-forward blocks on a residual stream, output layer (no attention: the data is a chain)."""

    def __init__(self, vocab=512, dim=256, hidden=512, blocks=2, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def mat(rows, cols, std):
            return (torch.randn(rows, cols, generator=g, device="cuda") * std).requires_grad_()

        self.scale = math.sqrt(dim)
        self.table = mat(vocab, dim, 1.0 / self.scale)
        self.norms = [torch.ones(dim, device="cuda", requires_grad=True) for _ in range(blocks + 1)]
        self.up = [mat(hidden, dim, 1.0 / math.sqrt(dim)) for _ in range(blocks)]
        self.down = [mat(dim, hidden, 0.5 / math.sqrt(hidden)) for _ in range(blocks)]
        self.out = mat(vocab, dim, 0.5 / math.sqrt(dim))

    def matrices(self):
        return self.up + self.down

    def others(self):
        return [self.table, self.out] + self.norms

    def logits(self, ids):
        x, res = lm.embed(self.table, ids, scale=self.scale, out_dtype=torch.bfloat16), None
        for norm, up, down in zip(self.norms, self.up, self.down):
            if res is None:
                y, res = lm.norm(x, norm), x
            else:
                y, res = lm.norm(x, norm, res)
            x = lm.linear(torch.nn.functional.silu(lm.linear(y, up)), down)
        y, _ = lm.norm(x, self.norms[-1], res)
        return lm.linear(y, self.out)

    def loss(self, ids, targets):
        logp, entropy = lm.logprobs(self.logits(ids), targets)
        n = (targets >= 0).sum()
        return -logp.sum() / n, entropy.detach().mean()


class Server:
    """The trained model with its weights in 8 bits, for a few tokens at a time."""

    def __init__(self, model):
        self.m = model
        q = lambda ws: [lm.fp8_quantize(w.detach(), block="square") for w in ws]  # noqa: E731
        self.up, self.down, self.out = q(model.up), q(model.down), q([model.out])[0]
        self.table = model.table.detach().bfloat16()
        self.norms = [n.detach() for n in model.norms]

    def next_tokens(self, ids, top_k=5):
        e4m3 = torch.float8_e4m3fn
        x, res = lm.embedding(self.table, ids, scale=self.m.scale), None
        for norm, up, down in zip(self.norms, self.up, self.down):
            r = lm.rms_norm(x, norm, residual=res, out_dtype=e4m3)
            res = r.residual
            x = lm.fp8_matmul(lm.fp8_quantize(torch.nn.functional.silu(lm.fp8_matmul(r.y, up))), down)
        r = lm.rms_norm(x, self.norms[-1], residual=res, out_dtype=e4m3)
        return lm.token_logprobs(lm.fp8_matmul(r.y, self.out), ids, top_k=top_k)


def batches(vocab, tokens, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    successor = torch.randperm(vocab, generator=g, device="cuda")
    while True:
        ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        noise = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        follow = torch.rand(tokens, generator=g, device="cuda") < 0.9
        targets = torch.where(follow, successor[ids], noise)
        pad = torch.rand(tokens, generator=g, device="cuda") < 0.05
        yield torch.where(pad, -1, ids), torch.where(pad, -1, targets), successor


def train(steps=80, vocab=512, tokens=4096, log=None):
    model = TokenModel(vocab)
    shampoo = OnlineKLShampoo(model.matrices(), lr=0.05, weight_decay=0.0)
    adam = torch.optim.AdamW(model.others(), lr=1e-2, weight_decay=0.0)
    data, losses, successor = batches(vocab, tokens), [], None
    for step in range(steps):
        ids, targets, successor = next(data)
        loss, entropy = model.loss(ids, targets)
        loss.backward()
        shampoo.step()
        adam.step()
        for p in model.matrices() + model.others():
            p.grad = None
        losses.append(loss.item())
        if log and step % 10 == 0:
            log(f"step {step:4d}  loss {losses[-1]:.4f}  entropy {entropy.item():.4f}")
    lm.query_status()
    return model, losses, successor


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=80)
    a = ap.parse_args()
    model, losses, successor = train(a.steps, log=print)
    print(f"last loss {losses[-1]:.4f}")
    ids = torch.arange(4, device="cuda")
    r = Server(model).next_tokens(ids)
    for i in range(4):
        best = ", ".join(f"{t} ({p:.2f})" for t, p in zip(r.top_ids[i].tolist(), r.top_logp[i].tolist()))
        print(f"after {i} (successor {successor[i].item()}): {best}")


if __name__ == "__main__":
    main()
