"""Cases of the language-model operators: what is run, in which sizes, and what a pass cannot do without.

The operators are the ends and the linear layers of a transformer that is trained with this library's optimizers:
the token embedding (with its gradient by sorted tokens), the root-mean-square norm with the residual's addition
(output in 16 or 8 bits, and its gradient), the 8-bit linear layer with a scale for each block of 128 (forward, and
the three products of a training step), and the log probabilities of given tokens with entropy and top alternatives
(and their gradient).

`run` has two forms.  With `own` false the operators are computed in their plain form, from elementary torch operations
in 32 bits.  With `own` true they are the calls of `kronecker_factored_second_gb300.lm`.
"""

import math

import torch

own = False

FP8_MAX = 448.0          # largest e4m3 value
AMAX_FLOOR = 2.0 ** -100  # a group's largest magnitude is taken as at least this
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a generation step looks up the tokens of a few sequences: latency counts
        dict(name="embed_few", op="embed", tokens=5, vocab=32000, dim=2048, dtype="bf16", grad="none", pad=0.0),
        # a training micro-batch of 8 x 2048 tokens less a ragged end, hidden size 2048: rows out, fp32 gradient back
        dict(name="embed_train", op="embed", tokens=16363, vocab=32000, dim=2048, dtype="bf16", grad="new", pad=0.05),
        # a large vocabulary and a long batch with a quarter of padding, gradient added to the output layer's (tied)
        dict(name="embed_tied", op="embed", tokens=32768, vocab=131072, dim=2048, dtype="bf16", grad="add", pad=0.25),
        # one token through a norm: latency
        dict(name="norm_token", op="norm", rows=1, dim=4096, dtype="bf16", out="bf16", residual=True, grad=False),
        # 8-bit input of a linear layer, training batch, feed-forward width of the 1.2B layer set
        dict(name="norm_fp8", op="norm", rows=16384, dim=5504, dtype="bf16", out="fp8", residual=True, grad=False),
        # forward and gradient of a training batch, ragged rows
        dict(name="norm_train", op="norm", rows=8191, dim=4096, dtype="bf16", out="bf16", residual=True, grad=True),
        # generation, one token, 8-bit weights: the weight's bytes bound it
        dict(name="linear_token", op="linear", rows=1, n=5504, k=2048, kind="infer"),
        # a prompt through the 1.2B set's feed-forward layer with stored 8-bit weights
        dict(name="linear_prompt", op="linear", rows=8192, n=5504, k=2048, kind="infer"),
        # a training step's three products with all their quantisations, feed-forward layer of the 7B slice
        dict(name="linear_train", op="linear", rows=8192, n=11008, k=4096, kind="train"),
        # scoring one next token with its best alternatives: latency
        dict(name="score_token", op="score", rows=1, vocab=32000, dtype="bf16", top=8, grad=False),
        # loss of a training batch: log probabilities, entropy, gradient of both
        dict(name="score_train", op="score", rows=8192, vocab=32000, dtype="bf16", top=0, grad=True),
        # scoring a batch against a large odd vocabulary with 20 alternatives, fp32 logits
        dict(name="score_top", op="score", rows=1024, vocab=128257, dtype="fp32", top=20, grad=False),
    ]


def _log_int(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def _size(rng, lo, hi):
    """Half of the sizes are multiples of 64, the rest as they fall, odd ones among them."""
    v = _log_int(rng, lo, hi)
    if rng.random() < 0.5 and v >= 64:
        v = v // 64 * 64
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["embed", "norm", "linear", "score"])
    if op == "embed":
        vocab = _size(rng, 500, 131072)
        dim = _size(rng, 32, min(8192, (1 << 28) // vocab))
        tokens = _size(rng, 1, min(65536, (1 << 27) // dim))
        return dict(op=op, tokens=tokens, vocab=vocab, dim=dim, dtype=rng.choice(["bf16", "fp32"]),
                    grad=rng.choice(["none", "new", "add"]), pad=rng.choice([0.0, 0.1, 0.6]))
    if op == "norm":
        dim = _size(rng, 32, 16384)
        rows = _size(rng, 1, min(32768, (1 << 26) // dim))
        grad = rng.random() < 0.5
        return dict(op=op, rows=rows, dim=dim, dtype=rng.choice(["bf16", "fp32"]),
                    out="bf16" if grad else rng.choice(["bf16", "fp8"]), residual=rng.random() < 0.7, grad=grad)
    if op == "linear":
        return dict(op=op, rows=_size(rng, 1, 8192), n=_size(rng, 32, 11008), k=_size(rng, 32, 4096),
                    kind=rng.choice(["infer", "train"]))
    vocab = _size(rng, 40, 131072)
    rows = _size(rng, 1, min(8192, (1 << 27) // vocab))
    return dict(op=op, rows=rows, vocab=vocab, dtype=rng.choice(["bf16", "fp32"]),
                top=rng.choice([0, 1, 5, 20, 32]), grad=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _tokens(gen, count, vocab, pad):
    """Token ids with frequencies that fall as 1/rank over a shuffled vocabulary; a share `pad` is the padding id -1."""
    u = torch.rand(count, generator=gen, device="cuda", dtype=torch.float64)
    rank = torch.clamp((float(vocab) ** u).long() - 1, 0, vocab - 1)
    step = next(p for p in (7919, 104729, 1299709) if math.gcd(p, vocab) == 1)
    ids = rank * step % vocab
    drop = torch.rand(count, generator=gen, device="cuda") < pad
    return torch.where(drop, torch.full_like(ids, -1), ids)


def _pitched(t, multiple):
    """The same matrix with rows that start at a multiple of `multiple` elements (as a padded buffer has them)."""
    rows, cols = t.shape
    pitch = -(-cols // multiple) * multiple
    buf = torch.zeros(rows, pitch, device=t.device, dtype=t.dtype)
    buf[:, :cols] = t
    return buf[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "embed":
        dt = DTYPES[case["dtype"]]
        st["weight"] = _normal(gen, case["vocab"], case["dim"], std=0.02, dtype=dt)
        st["ids"] = _tokens(gen, case["tokens"], case["vocab"], case["pad"])
        st["scale"] = math.sqrt(case["dim"])
        if case["grad"] != "none":
            st["dy"] = _normal(gen, case["tokens"], case["dim"], std=1e-2, dtype=dt)
        if case["grad"] == "add":
            st["dw"] = _normal(gen, case["vocab"], case["dim"], std=1e-2)
    elif case["op"] == "norm":
        dt = DTYPES[case["dtype"]]
        st["x"] = _normal(gen, case["rows"], case["dim"], dtype=dt)
        st["residual"] = _normal(gen, case["rows"], case["dim"], std=3.0, dtype=dt) if case["residual"] else None
        st["weight"] = (1.0 + _normal(gen, case["dim"], std=0.1)).to(dt)
        st["eps"] = 1e-6
        if case["grad"]:
            st["dy"] = _normal(gen, case["rows"], case["dim"], std=1e-2, dtype=dt)
            st["dres"] = _normal(gen, case["rows"], case["dim"], std=1e-2, dtype=dt) if case["residual"] else None
    elif case["op"] == "linear":
        rows, n, k = case["rows"], case["n"], case["k"]
        st["x"] = _normal(gen, rows, k, dtype=torch.bfloat16)
        w = _normal(gen, n, k, std=1.0 / math.sqrt(k), dtype=torch.bfloat16)
        if case["kind"] == "infer":
            q, s = _quantize_square(w)
            st["wq"], st["ws"] = _pitched(q.view(torch.uint8), 128).view(torch.float8_e4m3fn), s
        else:
            st["w"] = w
            # gradients of a loss averaged over the batch: small, and of another size in each token
            g = _normal(gen, rows, n, std=1e-3) * torch.exp(_normal(gen, rows, 1))
            st["dy"] = g.to(torch.bfloat16)
    else:
        rows, vocab = case["rows"], case["vocab"]
        dt = DTYPES[case["dtype"]]
        z = _normal(gen, rows, vocab, std=2.5, dtype=dt)
        # every fourth row has a grammar's mask that forbids most of the vocabulary
        banned = torch.rand(vocab, generator=gen, device="cuda") < 0.9
        banned[: max(1, vocab // 16)] = False
        z[3::4].masked_fill_(banned, float("-inf"))
        st["logits"] = _pitched(z, 64)
        ids = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
        ids[3::4] = ids[3::4] % max(1, vocab // 16)
        ids[5::16] = -1  # padding
        st["ids"] = ids
        if case["grad"]:
            st["dlogp"] = _normal(gen, rows, std=1.0 / rows) - 1.0 / rows
            st["dent"] = _normal(gen, rows, std=1e-2 / rows)
    return st


# ------------------------------------------------------------------ plain forms
def _plain_embed(st):
    case, ids = st["case"], st["ids"]
    keep = (ids >= 0)
    safe = torch.where(keep, ids, torch.zeros_like(ids))
    rows = st["weight"][safe].float() * st["scale"] * keep[:, None]
    out = [rows.to(st["weight"].dtype)]
    if case["grad"] != "none":
        g = st["dy"].float() * st["scale"] * keep[:, None]
        dw = torch.zeros(case["vocab"], case["dim"], device="cuda") if case["grad"] == "new" else st["dw"].clone()
        out.append(dw.index_add_(0, safe, g))
    return out


def _groups(y, dim):
    """The last axis in groups of 128 (zeros after the end)."""
    pad = -dim % 128
    if pad:
        y = torch.nn.functional.pad(y, (0, pad))
    return y.view(*y.shape[:-1], -1, 128)


def _quantize_rows(y):
    """e4m3 values and a scale for each 128 of a row: q = y * (448 / amax), scale = amax / 448."""
    rows, dim = y.shape
    g = _groups(y.float(), dim)
    amax = g.abs().amax(-1, keepdim=True).clamp_min(AMAX_FLOOR)
    q = (g * (FP8_MAX / amax)).to(torch.float8_e4m3fn).view(rows, -1)[:, :dim]
    return q, (amax / FP8_MAX)[..., 0]


def _quantize_square(w):
    """e4m3 values and a scale for each 128 x 128 block."""
    n, k = w.shape
    p = torch.nn.functional.pad(w.float(), (0, -k % 128, 0, -n % 128))
    b = p.view(p.shape[0] // 128, 128, p.shape[1] // 128, 128)
    amax = b.abs().amax((1, 3), keepdim=True).clamp_min(AMAX_FLOOR)
    q = (b * (FP8_MAX / amax)).to(torch.float8_e4m3fn).view(p.shape)[:n, :k]
    return q, (amax / FP8_MAX)[:, 0, :, 0]


def _value_rows(q, s):
    return q.float() * s.repeat_interleave(128, 1)[:, : q.shape[1]]


def _value_square(q, s):
    return q.float() * s.repeat_interleave(128, 0)[: q.shape[0]].repeat_interleave(128, 1)[:, : q.shape[1]]


def _plain_norm(st):
    case = st["case"]
    dt = st["x"].dtype
    s = st["x"].float()
    if st["residual"] is not None:
        s = (s + st["residual"].float()).to(dt).float()  # the residual stream is held in its own type
    w = st["weight"].float()
    rstd = torch.rsqrt((s * s).mean(-1, keepdim=True) + st["eps"])
    xhat = s * rstd
    y = xhat * w
    out = list(_quantize_rows(y)) if case["out"] == "fp8" else [y.to(torch.bfloat16)]
    if st["residual"] is not None:
        out.append(s.to(dt))
    if case["grad"]:
        dy = st["dy"].float()
        g = dy * w
        ds = rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))
        if st["dres"] is not None:
            ds = ds + st["dres"].float()
        out += [ds.to(dt), (dy * xhat).sum(0)]
    return out


def _plain_linear(st):
    x = st["x"]
    xv = _value_rows(*_quantize_rows(x))
    if st["case"]["kind"] == "infer":
        return [(xv @ _value_square(st["wq"], st["ws"]).t()).to(torch.bfloat16)]
    dy = st["dy"]
    wv = _value_square(*_quantize_square(st["w"]))
    dyv = _value_rows(*_quantize_rows(dy))
    # the weight's gradient sums over the tokens: both operands have their groups along the tokens
    xt, dyt = _value_rows(*_quantize_rows(x.t())), _value_rows(*_quantize_rows(dy.t()))
    return [(xv @ wv.t()).to(torch.bfloat16), (dyv @ wv).to(torch.bfloat16), (dyt @ xt.t()).to(torch.bfloat16)]


def _plain_score(st):
    case, ids = st["case"], st["ids"]
    z = st["logits"].float()
    m = z.amax(-1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    total = e.sum(-1, keepdim=True)
    lse = m + torch.log(total)
    ent = (torch.log(total) - torch.where(e > 0, e * d, torch.zeros_like(e)).sum(-1, keepdim=True) / total)[:, 0]
    keep = ids >= 0
    safe = torch.where(keep, ids, torch.zeros_like(ids))
    logp = torch.where(keep, z.gather(1, safe[:, None])[:, 0] - lse[:, 0], torch.zeros_like(ent))
    out = [logp, ent]
    if case["top"]:
        top_z, top = torch.sort(z, dim=-1, descending=True, stable=True)
        out += [top[:, : case["top"]].to(torch.int32), top_z[:, : case["top"]] - lse]
    if case["grad"]:
        p = e / total
        lp = torch.where(p > 0, z - lse, torch.zeros_like(z))
        dz = st["dlogp"][:, None] * -p
        dz.scatter_add_(1, safe[:, None], st["dlogp"][:, None])
        dz = dz * keep[:, None] - st["dent"][:, None] * p * (lp + ent[:, None])
        out.append(dz.to(st["logits"].dtype))
    return out


# ------------------------------------------------------------------ the framework's operators
def _own_embed(st):
    from kronecker_factored_second_gb300 import lm
    case = st["case"]
    out = [lm.embedding(st["weight"], st["ids"], scale=st["scale"])]
    if case["grad"] != "none":
        out.append(lm.embedding_grad(st["dy"], st["ids"], case["vocab"], scale=st["scale"], base=st.get("dw")))
    return out


def _own_norm(st):
    from kronecker_factored_second_gb300 import lm
    case = st["case"]
    r = lm.rms_norm(st["x"], st["weight"], residual=st["residual"], eps=st["eps"],
                    out_dtype=torch.float8_e4m3fn if case["out"] == "fp8" else torch.bfloat16)
    out = [r.y.data, r.y.scale] if case["out"] == "fp8" else [r.y]
    if st["residual"] is not None:
        out.append(r.residual)
    if case["grad"]:
        out += lm.rms_norm_grad(st["dy"], r.residual, st["weight"], r.rstd, dresidual=st["dres"])
    return out


def _own_linear(st):
    from kronecker_factored_second_gb300 import lm
    x = st["x"]
    if st["case"]["kind"] == "infer":
        return [lm.fp8_matmul(lm.fp8_quantize(x), lm.Fp8Tensor(st["wq"], st["ws"], "square"))]
    dy = st["dy"]
    xq, xqt = lm.fp8_quantize(x, both=True)
    dyq, dyqt = lm.fp8_quantize(dy, both=True)
    wq, wqt = lm.fp8_quantize(st["w"], block="square", both=True)
    return [lm.fp8_matmul(xq, wq), lm.fp8_matmul(dyq, wqt), lm.fp8_matmul(dyqt, xqt)]


def _own_score(st):
    from kronecker_factored_second_gb300 import lm
    case = st["case"]
    r = lm.token_logprobs(st["logits"], st["ids"], top_k=case["top"])
    out = [r.logp, r.entropy]
    if case["top"]:
        out += [r.top_ids, r.top_logp]
    if case["grad"]:
        out.append(lm.token_logprobs_grad(st["logits"], st["ids"], r, st["dlogp"], dentropy=st["dent"]))
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"embed": _own_embed, "norm": _own_norm, "linear": _own_linear, "score": _own_score}[op](state)
    return {"embed": _plain_embed, "norm": _plain_norm, "linear": _plain_linear, "score": _plain_score}[op](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "embed":
        e = 2 if case["dtype"] == "bf16" else 4
        t, v, d = case["tokens"], case["vocab"], case["dim"]
        moved = 8 * t + 2 * t * d * e
        flops = t * d
        if case["grad"] != "none":
            moved += 8 * t + t * d * e + v * d * 4 * (2 if case["grad"] == "add" else 1)
            flops += 2 * t * d
        return {"bytes": moved, "flops": flops}
    if op == "norm":
        e = 2 if case["dtype"] == "bf16" else 4
        n, d = case["rows"] * case["dim"], case["dim"]
        moved = n * e + d * e + (n * 2 if case["out"] == "bf16" else n + 4 * case["rows"] * -(-d // 128))
        if case["residual"]:
            moved += 2 * n * e
        flops = 5 * n
        if case["grad"]:
            moved += n * e * (4 if case["residual"] else 3) + d * e + 4 * d
            flops += 10 * n
        return {"bytes": moved, "flops": flops}
    if op == "linear":
        m, n, k = case["rows"], case["n"], case["k"]
        if case["kind"] == "infer":
            return {"bytes": 2 * m * k + n * k + 2 * m * n, "flops": 2 * m * n * k}
        # x, w and dy in 16 bits in; y, dx and dw in 16 bits out
        return {"bytes": 2 * (2 * m * k + 2 * m * n + 2 * n * k), "flops": 6 * m * n * k}
    e = 2 if case["dtype"] == "bf16" else 4
    n = case["rows"] * case["vocab"]
    moved = n * e + case["rows"] * (16 + 8 * case["top"])
    if case["grad"]:
        moved += 2 * n * e + case["rows"] * 24
    return {"bytes": moved, "flops": (10 if case["grad"] else 5) * n}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_codes(v64, axes):
    """Scales and the values of the e4m3 codes of an array whose groups lie along `axes`."""
    top = torch.clamp(torch.amax(torch.abs(v64), dim=axes, keepdim=True), min=AMAX_FLOOR)
    unit = top / FP8_MAX
    return (v64 / unit).float().to(torch.float8_e4m3fn).double(), unit


def _exact_rows(v):
    r, c = v.shape
    blocks = (c + 127) // 128
    full = torch.zeros(r, blocks * 128, dtype=torch.float64, device=v.device)
    full[:, :c] = v
    code, unit = _exact_codes(full.reshape(r, blocks, 128), (2,))
    return code.reshape(r, -1)[:, :c], unit.reshape(r, blocks), (code * unit).reshape(r, -1)[:, :c]


def _exact_blocks(v):
    r, c = v.shape
    br, bc = (r + 127) // 128, (c + 127) // 128
    full = torch.zeros(br * 128, bc * 128, dtype=torch.float64, device=v.device)
    full[:r, :c] = v
    code, unit = _exact_codes(full.reshape(br, 128, bc, 128), (1, 3))
    return (code * unit).reshape(br * 128, bc * 128)[:r, :c]


def _exact_embed(st, case):
    ids = st["ids"]
    at = torch.nonzero(ids >= 0)[:, 0]
    y = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
    y[at] = st["weight"].double()[ids[at]] * st["scale"]
    out = [y]
    if case["grad"] != "none":
        dw = st["dw"].double() if case["grad"] == "add" else torch.zeros(case["vocab"], case["dim"],
                                                                        dtype=torch.float64, device="cuda")
        dw.index_put_((ids[at],), st["dy"].double()[at] * st["scale"], accumulate=True)
        out.append(dw)
    return out


def _exact_norm(st, case):
    dt = st["x"].dtype
    s = st["x"].double()
    if st["residual"] is not None:
        s = (s + st["residual"].double()).to(dt).double()
    w = st["weight"].double()
    d = case["dim"]
    r = 1.0 / torch.sqrt(torch.einsum("rd,rd->r", s, s) / d + st["eps"])
    y = s * r[:, None] * w
    if case["out"] == "fp8":
        code, unit, _ = _exact_rows(y)
        out = [code, unit]
    else:
        out = [y]
    if st["residual"] is not None:
        out.append(s)
    if case["grad"]:
        g = st["dy"].double() * w
        dot = torch.einsum("rd,rd->r", g, s)
        ds = g * r[:, None] - s * (r ** 3 * dot / d)[:, None]
        if st["dres"] is not None:
            ds = ds + st["dres"].double()
        out += [ds, torch.einsum("rd,rd,r->d", st["dy"].double(), s, r)]
    return out


def _exact_linear(st, case):
    x = st["x"].double()
    xq = _exact_rows(x)[2]
    if case["kind"] == "infer":
        n, k = case["n"], case["k"]
        i = torch.arange(n, device="cuda") // 128
        j = torch.arange(k, device="cuda") // 128
        return [xq @ (st["wq"].double() * st["ws"].double()[i][:, j]).T]
    dy = st["dy"].double()
    w = _exact_blocks(st["w"].double())
    return [xq @ w.T, _exact_rows(dy)[2] @ w, _exact_rows(dy.T)[2] @ _exact_rows(x.T)[2].T]


def _exact_score(st, case):
    z = st["logits"].double()
    ids = st["ids"]
    lse = torch.logsumexp(z, -1)
    lp = z - lse[:, None]
    p = torch.exp(lp)
    plp = torch.xlogy(p, p)
    ent = -plp.sum(-1)
    rows = torch.arange(case["rows"], device="cuda")
    at = rows[ids >= 0]
    logp = torch.zeros(case["rows"], dtype=torch.float64, device="cuda")
    logp[at] = lp[at, ids[at]]
    out = [logp, ent]
    if case["top"]:
        best = torch.topk(z, case["top"], dim=-1, sorted=True).values
        out += [None, best - lse[:, None]]
    if case["grad"]:
        gl = st["dlogp"].double() * (ids >= 0)
        dz = -p * gl[:, None]
        dz[at, ids[at]] += gl[at]
        dz -= st["dent"].double()[:, None] * (plp + p * ent[:, None])
        out.append(dz)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"embed": _exact_embed, "norm": _exact_norm, "linear": _exact_linear,
            "score": _exact_score}[case["op"]](st, case)
