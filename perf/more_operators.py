"""Cases of the optimizer step and the serving operators around the matrix optimizers: what is run, in which sizes, and what
a pass cannot do without.

The operators are what a model trained with this library needs besides the matrix optimizers' steps and the operators of
`perf/operators.py`: the AdamW step of everything that is no matrix (or of whole layers), over many tensors at once, with
states in 32 or in 8 bits; and a generation step's products with 4-bit weights and the sampling of the next token from its
logits with temperature, top-k, top-p and min-p.

`run` has two forms.  With `own` false the operators are computed in their plain form, from elementary torch operations in
32 bits (in 64 where a value lies next to a border).  With `own` true they are the calls of
`kronecker_factored_second_gb300.okls` and `.lm`.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
GROUP = 128               # elements of an 8-bit state that share a scale
FP8_MAX = 448.0           # largest e4m3 value
AMAX_FLOOR = 2.0 ** -100  # a group's largest magnitude is taken as at least this
LR, BETA1, BETA2, EPS, DECAY = 2e-3, 0.9, 0.999, 1e-8, 0.01
SEED = 1234               # of the rounding of 8-bit states


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the norms of the 1.2B layer set beside the matrix optimizers: many short vectors, latency counts
        dict(name="adamw_norms", op="adamw", big=0, big_n=0, small=49, small_n=2048, param="fp32", grad="fp32", bits=32),
        # token table and output layer with the norms, fp32 with 32-bit states
        dict(name="adamw_tables", op="adamw", big=2, big_n=32000 * 2048, small=49, small_n=2048, param="fp32", grad="fp32",
             bits=32),
        # the same in bf16 with odd sizes and 8-bit states
        dict(name="adamw_tables8", op="adamw", big=2, big_n=32003 * 2049, small=49, small_n=2049, param="bf16", grad="bf16",
             bits=8),
        # feed-forward matrices of nine layers of the 1.2B set, bf16 with 32-bit states
        dict(name="adamw_layers", op="adamw", big=27, big_n=5504 * 2048, small=18, small_n=2048, param="bf16", grad="bf16",
             bits=32),
        # generation, one token, feed-forward layer of the 1.2B set: latency and the weight's bytes
        dict(name="four_token", op="four", rows=1, n=5504, k=2048, group=128, zero=False, dtype="bf16"),
        # the output layer of a large vocabulary for one token, zero points
        dict(name="four_head", op="four", rows=1, n=131072, k=2048, group=64, zero=True, dtype="bf16"),
        # a batch of sequences through the feed-forward layer of the 7B slice
        dict(name="four_batch", op="four", rows=16, n=11008, k=4096, group=128, zero=False, dtype="bf16"),
        # a few fp32 rows, odd sizes, short groups with zero points
        dict(name="four_odd", op="four", rows=5, n=8193, k=2047, group=32, zero=True, dtype="fp32"),
        # the next token of one sequence with every filter: latency
        dict(name="sample_token", op="sample", rows=1, vocab=32000, dtype="bf16", kind="all"),
        # a serving batch whose requests carry settings of their own, some of them with masked logits
        dict(name="sample_batch", op="sample", rows=256, vocab=32000, dtype="bf16", kind="mixed"),
        # nucleus sampling of a large odd vocabulary, fp32 logits
        dict(name="sample_nucleus", op="sample", rows=512, vocab=128257, dtype="fp32", kind="nucleus"),
        # samples of the whole distribution (rollouts for training)
        dict(name="sample_free", op="sample", rows=1024, vocab=131072, dtype="bf16", kind="free"),
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
    return v


def draw(rng):
    op = rng.choice(["adamw", "four", "sample"])
    if op == "adamw":
        big = rng.choice([0, 1, 2, 5, 12])
        return dict(op=op, big=big, big_n=_size(rng, 10000, (1 << 27) // big) if big else 0, small=_log_int(rng, 1, 400),
                    small_n=_size(rng, 1, 20000), param=rng.choice(["bf16", "fp32"]), grad=rng.choice(["bf16", "fp32"]),
                    bits=rng.choice([8, 32]))
    if op == "four":
        n = _size(rng, 48, 65536)
        return dict(op=op, rows=_log_int(rng, 1, 64), n=n, k=_size(rng, 48, min(8192, (1 << 27) // n)),
                    group=rng.choice([32, 64, 128]), zero=rng.random() < 0.4, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    vocab = _size(rng, 100, 131072)
    return dict(op=op, rows=_size(rng, 1, min(1024, (1 << 26) // vocab)), vocab=vocab, dtype=rng.choice(["bf16", "fp32"]),
                kind=rng.choice(["all", "mixed", "nucleus", "free"]))


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _counts(case):
    """Elements of each tensor of an optimizer case."""
    return [case["big_n"]] * case["big"] + [case["small_n"]] * case["small"]


def _padded(n):
    return -(-n // GROUP) * GROUP


def _views(flat, counts, unit=1):
    """The tensors that lie one after the other in a flat buffer, each at a multiple of 128 elements; with `unit` 128 the
    groups of each of them."""
    out, at = [], 0
    for n in counts:
        size = _padded(n) // unit
        out.append(flat[at:at + (n if unit == 1 else size)])
        at += size
    return out


def _inside(counts):
    """Which elements of the flat buffer belong to a tensor."""
    keep = torch.ones(sum(_padded(n) for n in counts), device="cuda", dtype=torch.bool)
    at = 0
    for n in counts:
        keep[at + n:at + _padded(n)] = False
        at += _padded(n)
    return keep


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "adamw":
        counts = _counts(case)
        keep = _inside(counts)
        total = keep.numel()
        # gradients whose size differs from group to group; states as some steps left them
        size = torch.exp(_normal(gen, total // GROUP, 1)) * 1e-3
        spread = lambda std: (_normal(gen, total // GROUP, GROUP, std=std) * size).view(-1) * keep  # noqa: E731
        st["p"] = (_normal(gen, total, std=0.02) * keep).to(DTYPES[case["param"]])
        st["g"] = spread(1.0).to(DTYPES[case["grad"]])
        m, r = spread(0.3), spread(1.0).abs_().add_(size.mul(0.1).expand(-1, GROUP).reshape(-1) * keep)
        if case["bits"] == 32:
            st["m"], st["v"] = m, r * r
        else:
            for name, x in (("m", m), ("v", r)):  # the second holds the root of the second moment
                x = x.view(-1, GROUP)
                a = x.abs().amax(1, keepdim=True).clamp_min(AMAX_FLOOR)
                st[name] = (x * (FP8_MAX / a)).to(torch.float8_e4m3fn).view(-1)
                st[name + "s"] = (a / FP8_MAX).view(-1)
        st["step"] = 100
        st["counts"] = counts
        # what a program holds of the flat buffers: a tensor for each parameter
        st["tensors"] = [_views(st[name], counts) for name in ("p", "g", "m", "v")]
        st["scales"] = [_views(st[name], counts, GROUP) for name in ("ms", "vs")] if case["bits"] == 8 else [None, None]
    elif case["op"] == "four":
        rows, n, k, group = case["rows"], case["n"], case["k"], case["group"]
        groups, pitch = -(-k // group), -(-k // 128) * 64
        st["x"] = _normal(gen, rows, k, dtype=DTYPES[case["dtype"]])
        st["codes"] = torch.randint(0, 256, (n, pitch), generator=gen, device="cuda", dtype=torch.uint8)[:, :-(-k // 2)]
        # neighbouring rows' scales are neighbours
        lay = lambda t: t.to(torch.bfloat16).t()  # noqa: E731
        st["scale"] = lay((1.0 + torch.rand(groups, n, generator=gen, device="cuda")) / (8 * math.sqrt(k)))
        st["zero"] = lay(7.5 + _normal(gen, groups, n)) if case["zero"] else None
    else:
        rows, vocab = case["rows"], case["vocab"]
        z = _normal(gen, rows, vocab, std=2.5, dtype=DTYPES[case["dtype"]])
        if case["kind"] == "mixed":  # every fourth row has a grammar's mask that forbids most of the vocabulary
            banned = torch.rand(vocab, generator=gen, device="cuda") < 0.9
            banned[: max(1, vocab // 16)] = False
            z[3::4].masked_fill_(banned, float("-inf"))
        st["logits"] = z
        st["u"] = torch.rand(rows, generator=gen, device="cuda")
        pick = lambda values, dtype: torch.tensor(values, device="cuda", dtype=dtype)[  # noqa: E731
            torch.randint(0, len(values), (rows,), generator=gen, device="cuda")]
        f, i = torch.float32, torch.int32
        mixed = case["kind"] == "mixed"
        st["temperature"] = {"all": lambda: 0.8, "nucleus": lambda: 1.0, "free": lambda: 1.0,
                             "mixed": lambda: pick([0.0, 0.3, 0.7, 1.0, 1.3], f)}[case["kind"]]()
        st["top_k"] = pick([0, 1, 20, 50, 1000], i) if mixed else 50 if case["kind"] == "all" else None
        st["top_p"] = pick([0.5, 0.9, 0.95, 1.0], f) if mixed else {"all": 0.95, "nucleus": 0.9}.get(case["kind"])
        st["min_p"] = pick([0.0, 0.0, 0.02, 0.1], f) if mixed else 0.02 if case["kind"] == "all" else None
    return st


# ------------------------------------------------------------------ plain forms
def _product(a, b):
    """Upper and lower word of the products of 32-bit words (held in 64-bit integers)."""
    p, q = (a & 0xFFFF) * b, (a >> 16) * b
    return (q + (p >> 16)) >> 16, (((q & 0xFFFF) << 16) + p) & 0xFFFFFFFF


def _dither(counts, step):
    """Two 16-bit random numbers for each element of the flat buffer: Philox-2x32 of five rounds; the counter is the pair of
    elements and the tensor, the key the seed and the step."""
    s = (SEED + step * 0x9E3779B97F4A7C15) % (1 << 64)
    key, low = s >> 32, s & 0xFFFFFFFF
    sizes = torch.tensor([_padded(n) // 2 for n in counts], device="cuda")
    which = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), sizes)
    x = torch.arange(which.numel(), device="cuda") - (torch.cumsum(sizes, 0) - sizes)[which]
    y = (which + low) & 0xFFFFFFFF
    for i in range(5):
        hi, lo = _product(x, 0xD256D193)
        x, y = hi ^ ((key + i * 0x9E3779B9) & 0xFFFFFFFF) ^ y, lo
    words = torch.stack((x, y), 1).view(-1)
    return words & 0xFFFF, words >> 16


def _round_state(x, random, root):
    """e4m3 codes and scales of groups of 128, rounded up or down by chance so that the mean is right; a root that is not
    zero keeps a code that is not."""
    y = x.double().view(-1, GROUP)
    a = y.abs().amax(1, keepdim=True).clamp_min(AMAX_FLOOR)
    y = y * (FP8_MAX / a)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    q = (torch.floor(y.abs() / step + (random.view(-1, GROUP) + 0.5) / 65536) * step).clamp_max(FP8_MAX)
    if root:
        q = torch.where((y > 0) & (q == 0), torch.full_like(q, 2.0 ** -9), q)
    return (q * torch.sign(y)).float().to(torch.float8_e4m3fn).view(-1), (a / FP8_MAX).float().view(-1)


def _plain_adamw(st):
    case = st["case"]
    st["step"] += 1
    t = st["step"]
    p, g = st["p"].float(), st["g"].float()
    if case["bits"] == 32:
        m, v = st["m"], st["v"]
    else:
        value = lambda q, s: (q.float().view(-1, GROUP) * s[:, None]).view(-1)  # noqa: E731
        m, v = value(st["m"], st["ms"]), value(st["v"], st["vs"]).square()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    update = (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    st["p"].copy_(p - LR * DECAY * p - LR * update)
    if case["bits"] == 32:
        st["m"].copy_(m)
        st["v"].copy_(v)
        return [st["p"], st["m"], st["v"]]
    rm, rv = _dither(st["counts"], t)
    for name, x, r in (("m", m, rm), ("v", torch.sqrt(v), rv)):
        q, s = _round_state(x, r, name == "v")
        st[name].copy_(q)
        st[name + "s"].copy_(s)
    return [st["p"], st["m"], st["ms"], st["v"], st["vs"]]


def _plain_four(st):
    case = st["case"]
    k, group = case["k"], case["group"]
    both = torch.stack((st["codes"] & 15, st["codes"] >> 4), 2).view(case["n"], -1)[:, :k].float()
    spread = lambda t: t.float().repeat_interleave(group, 1)[:, :k]  # noqa: E731
    w = (both - (spread(st["zero"]) if case["zero"] else 8.0)) * spread(st["scale"])
    return [(st["x"].float() @ w.t()).to(st["x"].dtype)]


def _column(value, rows, off):
    """A setting for each row, in 64 bits."""
    if value is None:
        value = off
    t = value if isinstance(value, torch.Tensor) else torch.full((rows,), value, device="cuda", dtype=torch.float32)
    return t.double()[:, None]


def _plain_sample(st):
    rows, vocab = st["logits"].shape
    temperature, u = _column(st["temperature"], rows, 1.0), st["u"].double()[:, None]
    top_k, top_p, min_p = (_column(st[n], rows, off) for n, off in (("top_k", 0), ("top_p", 1.0), ("min_p", 0.0)))
    z, order = torch.sort(st["logits"].float(), dim=-1, descending=True, stable=True)
    z = z.double()
    best = z[:, :1]
    heat = torch.where(temperature > 0, temperature, torch.ones_like(temperature))
    w = torch.exp((z - best) / heat)
    rank = torch.arange(vocab, device="cuda")[None]
    w = w * ((top_k <= 0) | (rank < top_k)) * ((temperature > 0) | (rank < 1))
    mass = torch.cumsum(w, -1)
    keep = ((top_p >= 1) | (mass - w < top_p * mass[:, -1:])) & ((min_p <= 0) | (z >= best + heat * torch.log(min_p)))
    w = w * keep
    cum = torch.cumsum(torch.zeros_like(w).scatter_(1, order, w), -1)
    ids = (cum <= u * cum[:, -1:]).sum(-1)
    chosen = st["logits"].double().gather(1, ids[:, None])
    logp = (chosen - best) / heat - torch.log(w.sum(-1, keepdim=True))
    return [ids.to(torch.int32), logp[:, 0].float()]


# ------------------------------------------------------------------ the framework's operators
def _own_adamw(st):
    from kronecker_factored_second_gb300 import okls
    st["step"] += 1
    okls.adamw_step(*st["tensors"], step=st["step"], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY,
                    avg_scales=st["scales"][0], sq_scales=st["scales"][1], seed=SEED)
    return [st[n] for n in (("p", "m", "v") if st["case"]["bits"] == 32 else ("p", "m", "ms", "v", "vs"))]


def _own_four(st):
    from kronecker_factored_second_gb300 import lm
    if "weight" not in st:  # the program's handle of the weight
        st["weight"] = lm.Int4Tensor(st["codes"], st["scale"], st["case"]["k"], st["case"]["group"], st["zero"])
    return [lm.int4_matmul(st["x"], st["weight"])]


def _own_sample(st):
    from kronecker_factored_second_gb300 import lm
    r = lm.sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                  min_p=st["min_p"])
    return [r.ids, r.logp]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"adamw": _own_adamw, "four": _own_four, "sample": _own_sample}[op](state)
    return {"adamw": _plain_adamw, "four": _plain_four, "sample": _plain_sample}[op](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "adamw":
        n = sum(_counts(case))
        states = 16 * n if case["bits"] == 32 else 4 * n + 16 * sum(-(-c // GROUP) for c in _counts(case))
        return {"bytes": (2 * size[case["param"]] + size[case["grad"]]) * n + states, "flops": 16 * n}
    if case["op"] == "four":
        r, n, k = case["rows"], case["n"], case["k"]
        scales = 2 * n * -(-k // case["group"]) * (2 if case["zero"] else 1)
        return {"bytes": n * -(-k // 2) + scales + size[case["dtype"]] * r * (k + n), "flops": 2 * r * n * k}
    n = case["rows"] * case["vocab"]
    return {"bytes": size[case["dtype"]] * n + (12 + (16 if case["kind"] == "mixed" else 0)) * case["rows"], "flops": 4 * n}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_words(counts, step):
    """The random words of each pair of elements, from products of whole 64-bit integers (b split instead of a)."""
    mask = (1 << 32) - 1
    s = (SEED + step * 0x9E3779B97F4A7C15) & ((1 << 64) - 1)
    parts = []
    for which, n in enumerate(counts):
        a = torch.arange(_padded(n) // 2, device="cuda", dtype=torch.int64)
        b = torch.full_like(a, ((s & mask) + which) & mask)
        for i in range(5):
            up, down = a * 0xD256, a * 0xD193  # a * 0xD256D193 = up * 2^16 + down
            high = (up + (down >> 16)) >> 16
            low = (up * 65536 + down) & mask
            a, b = high ^ (((s >> 32) + i * 0x9E3779B9) & mask) ^ b, low
        parts.append(torch.stack((a, b), -1).reshape(-1))
    return torch.cat(parts)


def _exact_codes(x, random, root):
    """Values of the codes and units of groups: the value is one of its two neighbours on the e4m3 grid, the upper one
    where the part between them is past 1 - (random + 1/2) / 65536."""
    y = x.reshape(-1, GROUP)
    unit = torch.clamp(y.abs().max(1, keepdim=True).values, min=AMAX_FLOOR) / FP8_MAX
    mag = (y / unit).abs()
    _, e = torch.frexp(mag)  # mag = f 2^e, f in [1/2, 1)
    gap = torch.ldexp(torch.ones_like(mag), torch.clamp(e - 1, min=-6) - 3)
    below = torch.floor(mag / gap)
    up = (mag / gap - below) + (random.reshape(-1, GROUP).double() + 0.5) / 65536 >= 1
    q = torch.clamp((below + up) * gap, max=FP8_MAX)
    if root:
        q = torch.where((mag > 0) & (q == 0), 2.0 ** -9, q)
    return torch.copysign(q, y).reshape(-1), unit.reshape(-1)


def _exact_adamw(st, case):
    t = st["step"] + 1
    p, g = st["p"].double(), st["g"].double()
    m, v = st["m"].double(), st["v"].double()
    if case["bits"] == 8:
        m = (m.reshape(-1, GROUP) * st["ms"].double()[:, None]).reshape(-1)
        v = (v.reshape(-1, GROUP) * st["vs"].double()[:, None]).reshape(-1) ** 2
    m = m + (1 - BETA1) * (g - m)
    v = v + (1 - BETA2) * (g ** 2 - v)
    p = p * (1 - LR * DECAY) - LR / (1 - BETA1 ** t) * m / (v.sqrt() / math.sqrt(1 - BETA2 ** t) + EPS)
    if case["bits"] == 32:
        return [p, m, v]
    words = _exact_words(st["counts"], t)
    return [p, *_exact_codes(m, words % 65536, False), *_exact_codes(v.sqrt(), words // 65536, True)]


def _exact_four(st, case):
    n, k, group = case["n"], case["k"], case["group"]
    at = torch.arange(k, device="cuda")
    codes = (st["codes"][:, at // 2].int() >> (4 * (at % 2)).int()[None]) % 16
    y = torch.zeros(case["rows"], n, device="cuda", dtype=torch.float64)
    x = st["x"].double()
    for j in range(-(-k // group)):
        cols = slice(j * group, min(k, (j + 1) * group))
        c, xs = codes[:, cols].double(), x[:, cols]
        z = st["zero"][:, j].double() if case["zero"] else torch.full((n,), 8.0, device="cuda", dtype=torch.float64)
        y += (xs @ c.T - xs.sum(1, keepdim=True) * z) * st["scale"][:, j].double()
    return [y]


def _exact_sample(st, case):
    """Log probability of the drawn token: the kept set from its least value and the ids that share it."""
    z = st["logits"].double()
    rows, vocab = z.shape
    t, k, p, lo = (_column(st[n], rows, off) for n, off in (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0),
                                                           ("min_p", 0.0)))
    greedy = t <= 0
    t = torch.where(greedy, 1.0, t)
    k = torch.where(greedy, 1.0, torch.where(k <= 0, float(vocab), k))
    lp = torch.log_softmax(z / t, -1)
    falling, ids = torch.sort(lp, dim=-1, descending=True, stable=True)
    del z
    q = torch.exp(falling)
    place = torch.arange(vocab, device="cuda")[None]
    q = torch.where(place < k, q, 0.0)
    share = torch.cumsum(q, -1) / q.sum(-1, keepdim=True)
    count = torch.where(p >= 1, float(vocab), (share < p).sum(-1, keepdim=True) + 1.0)
    count = torch.minimum(torch.minimum(count, k),
                          torch.where(lo <= 0, float(vocab), (falling >= falling[:, :1] + lo.log()).sum(-1, keepdim=True)))
    q = torch.where(place < count, q, 0.0)
    del share, falling
    total = q.sum(-1, keepdim=True)
    run_up = torch.empty_like(q).scatter_(1, ids, q / total).cumsum(-1)
    at = torch.searchsorted(run_up, st["u"].double()[:, None] * run_up[:, -1:], right=True)
    return [None, (lp.gather(1, at) - total.log())[:, 0]]


def exact(case, seed):
    st = prepare(case, seed)
    return {"adamw": _exact_adamw, "four": _exact_four, "sample": _exact_sample}[case["op"]](st, case)
