"""AdamW over many tensors, the product with 4-bit weights and the sampling of tokens on the GPU, against their definitions
in 64 bits.

Tolerances come from the arithmetic: u = 2^-24 is fp32's unit roundoff, bf16 rounds to 2^-8 of a value.  A sum of n terms
in fp32 is off by at most about n u times the sum of their magnitudes, whatever its order."""

import math

import pytest
import torch

from kronecker_factored_second_gb300 import _lib as L
from kronecker_factored_second_gb300 import lm, okls

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
OUT = {BF16: 2.0 ** -8, F32: U}
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L.lib()
    torch.cuda.set_device(0)
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


# -------------------------------------------------------------------- AdamW
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


def _moments(g, m, v, h):
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    return m, h["beta2"] * v + (1 - h["beta2"]) * g * g


def _check_update(got, p, g, m, v, t, h, fast=False):
    """p against the step's formula from the moments m, v before it, in 64 bits.

    m is off by 4 u of its two terms, v by 5 u of itself; the root halves that and adds 1 u (2 fast), the product with its
    factor (rounded) 2 u, the sum 1 u, the quotient 1 u (4 fast), the rate 1 u, the last two products and sums 2 u of their
    terms: 16 u of the update taken with the terms' magnitudes, twice that with the fast root and quotient."""
    g64, p64 = g.double(), p.double()
    mag = h["beta1"] * m.abs() + (1 - h["beta1"]) * g64.abs()
    m, v = _moments(g64, m, v, h)
    rate = h["lr"] / (1 - h["beta1"] ** t)
    den = torch.sqrt(v / (1 - h["beta2"] ** t)) + h["eps"]
    want = p64 - h["lr"] * h["weight_decay"] * p64 - rate * m / den
    bound = (32 if fast else 16) * U * rate * mag / den + 4 * U * p64.abs() + OUT[got.dtype] * want.abs()
    close(got, want, bound, "parameter")
    return m, v, mag


@pytest.mark.parametrize("pd,gd", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("sizes,off", [((1,), 0), ((7, 8, 9), 0), ((2048,) * 5, 0), ((8191, 1, 8193, 0, 16385), 0), ((100003,), 1),
                                       ((33, 260), 3), (tuple(range(1, 60)), 0), (tuple(range(1, 900, 2)), 0)])
def test_adamw_32(pd, gd, sizes, off):
    g = gen(len(sizes) + off)
    place = lambda n, dt, std: randn(g, n + off + 5, dtype=dt, std=std)[off:off + n]  # noqa: E731
    ps, gs = [place(n, pd, 1.0) for n in sizes], [place(n, gd, 1e-2) for n in sizes]
    ms, vs = [place(n, F32, 1e-2) for n in sizes], [place(n, F32, 1e-2).square_() for n in sizes]
    for t in (1, 2, 1000):
        old = [(p.clone(), m.double(), v.double()) for p, m, v in zip(ps, ms, vs)]
        okls.adamw_step(ps, gs, ms, vs, step=t, **HYPER)
        for i, n in enumerate(sizes):
            m, v, mag = _check_update(ps[i], old[i][0], gs[i], old[i][1], old[i][2], t, HYPER)
            close(ms[i], m, 4 * U * mag, "first moment")
            close(vs[i], v, 5 * U * v, "second moment")


def test_adamw_touches_nothing_else():
    for bits in (32, 8):
        flat = [torch.full((5000,), 3.0, device="cuda") for _ in range(4)]
        scales = [torch.full((40,), 3.0, device="cuda") for _ in range(2)]
        if bits == 8:
            flat[2:] = [x.to(E4M3) for x in flat[2:]]
        before = [x.clone() for x in flat + scales]
        part = [[x[16:1017], x[2000:2001], x[2004:2004 + 300]] for x in flat]
        sc = [[x[1:9], x[10:11], x[12:15]] for x in scales] if bits == 8 else (None, None)
        okls.adamw_step(*part, step=1, avg_scales=sc[0], sq_scales=sc[1], **HYPER)
        keep = torch.ones(5000, dtype=torch.bool, device="cuda")
        keep[16:1017], keep[2000], keep[2004:2304] = False, False, False
        for x, y in zip(flat, before):
            assert torch.equal(x.float()[keep], y.float()[keep])
        assert not (flat[0] == before[0])[~keep].any()
        left = torch.ones(40, dtype=torch.bool, device="cuda")
        left[1:9], left[10], left[12:15] = False, False, False
        for x, y in zip(scales, before[4:]):
            assert torch.equal(x[left], y[left])


def _philox(n, ident, t, seed, first=0):
    """The two 16-bit numbers of each of n elements, by the published rounds in whole numbers (`first` is even)."""
    s = (seed + t * 0x9E3779B97F4A7C15) % (1 << 64)
    x = torch.arange((n + 1) // 2, device="cuda") + first // 2
    y = torch.full_like(x, (ident + s) % (1 << 32))
    for i in range(5):
        p, q = (x & 0xFFFF) * 0xD256D193, (x >> 16) * 0xD256D193
        hi, lo = (q + (p >> 16)) >> 16, (((q & 0xFFFF) << 16) + p) & 0xFFFFFFFF
        x, y = hi ^ (((s >> 32) + i * 0x9E3779B9) & 0xFFFFFFFF) ^ y, lo
    w = torch.stack((x, y), 1).view(-1)[:n]
    return w & 0xFFFF, w >> 16


def _groups(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % 128)).view(-1, 128)


def _check_codes(codes, scale, x, off, random, root):
    """Codes and scales of x (64 bits), which the kernel knows to `off`: the scale to off and 2 u of itself, the code exactly
    unless x, moved by off and 4 u, crosses the border that the random number sets."""
    n = x.numel()
    amax = _groups(x).abs().amax(1).clamp_min(2.0 ** -100)
    close(scale, amax / 448, (_groups(off).amax(1) + 3 * U * amax) / 448, "scale")
    unit = (amax / 448).repeat_interleave(128)[:n]
    y, e = (x / unit).abs(), off / unit + 4 * U * (x / unit).abs()

    def rounded(y):
        step = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
        q = (torch.floor(y / step + (random + 0.5) / 65536) * step).clamp(max=448)
        return torch.where((y > 0) & (q == 0), torch.full_like(q, 2.0 ** -9), q) if root else q
    # (the group's largest value moves with its own scale)
    e = e + y * (3 * U + (_groups(off).amax(1) / amax).repeat_interleave(128)[:n])
    # a sum of 2^-6 and a value below it is rounded to 2^-30
    e = e + 2.0 ** -30
    lo, hi = rounded((y - e).clamp_min(0)), rounded(y + e)
    got = codes.double().abs()
    assert ((got == lo) | (got == hi) | (got == rounded(y))).all()
    assert (got != rounded(y)).double().mean().item() < 1e-3
    at = got > 0
    assert torch.equal(codes.double().sign()[at], x.sign()[at])


@pytest.mark.parametrize("pd,gd", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("sizes,off", [((1,), 0), ((127, 128, 129), 0), ((4096, 0, 4097, 16), 0), ((50001,), 1), ((130, 77, 2050), 5),
                                       (tuple(range(1, 900, 15)), 0)])
def test_adamw_8(pd, gd, sizes, off):
    g = gen(len(sizes) + off)
    place = lambda n, dt, std: randn(g, n + off + 5, dtype=dt, std=std)[off:off + n]  # noqa: E731
    ps = [place(n, pd, 1.0) for n in sizes]
    state = [[torch.zeros(n + off + 5, device="cuda").to(E4M3)[off:off + n] for n in sizes] for _ in range(2)]
    scales = [[torch.zeros(-(-n // 128), device="cuda") for n in sizes] for _ in range(2)]
    value = lambda k, i: state[k][i].double() * scales[k][i].double().repeat_interleave(128)[:sizes[i]]  # noqa: E731
    for t in (1, 2, 3):
        gs = [place(n, gd, 1e-2) * torch.exp(2 * place(n, gd, 1.0)) for n in sizes]
        old = [(ps[i].clone(), value(0, i), value(1, i).square()) for i in range(len(sizes))]
        okls.adamw_step(ps, gs, *state, step=t, avg_scales=scales[0], sq_scales=scales[1], seed=5, **HYPER)
        for i, n in enumerate(sizes):
            if n == 0:
                continue
            m, v, mag = _check_update(ps[i], old[i][0], gs[i], old[i][1], old[i][2], t, HYPER, fast=True)
            dm, dv = _philox(n, i, t, 5)
            _check_codes(state[0][i], scales[0][i], m, 5 * U * mag, dm, False)
            _check_codes(state[1][i], scales[1][i], v.sqrt(), 8 * U * v.sqrt(), dv, True)


def test_adamw_8_keeps_means_and_changes_below_a_code():
    """The second moment follows gradients of one size although a step changes it by 0.1%: rounding to nearest would leave
    it where the first steps put it, some thirtieth."""
    n = 1 << 16
    p, gr = torch.zeros(n, device="cuda"), torch.full((n,), 0.01, device="cuda")
    m, r = (torch.zeros(n, device="cuda").to(E4M3) for _ in range(2))
    ms, rs = (torch.zeros(n // 128, device="cuda") for _ in range(2))
    h = {**HYPER, "beta2": 0.999}
    steps = 400
    for t in range(1, steps + 1):
        okls.adamw_step([p], [gr], [m], [r], step=t, avg_scales=[ms], sq_scales=[rs], **h)
    want = 0.01 * math.sqrt(1 - 0.999 ** steps)
    got = (r.float().view(-1, 128) * rs[:, None]).mean().item()
    # the variance of the rounded roots adds to v: at most a step of 1/8 squared over 4, for each of some 1 / (1 - beta2)
    # steps by beta2^t: an upper shift, which the mean of the roots sees as below 10%
    assert 0.9 * want < got < 1.1 * want


def test_adamw_8_groups_that_are_not_finite():
    n = 1024
    p, gr = torch.ones(n, device="cuda"), torch.full((n,), 0.01, device="cuda")
    gr[130], gr[300] = NAN, INF
    m, r = (torch.zeros(n, device="cuda").to(E4M3) for _ in range(2))
    ms, rs = (torch.zeros(n // 128, device="cuda") for _ in range(2))
    okls.adamw_step([p], [gr], [m], [r], step=1, avg_scales=[ms], sq_scales=[rs], **HYPER)
    bad = torch.zeros(8, dtype=torch.bool, device="cuda")
    bad[1], bad[2] = True, True
    assert torch.equal(ms.isnan(), bad) and torch.equal(rs.isnan(), bad)
    only = torch.zeros(n, dtype=torch.bool, device="cuda")
    only[130], only[300] = True, True
    assert torch.equal(p.isnan(), only)


@pytest.mark.parametrize("pd,gd", [(F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("eps", [0.0, 1e-8])
@pytest.mark.parametrize("low,high", [(-21, -17), (-28, -17), (-29, -1), (18, 24), (30, 38), (-20, 38)])
def test_adamw_8_moments_whose_squares_leave_fp32(pd, gd, eps, low, high):
    """Gradients of 10^low to 10^high, each group's and each element's in a place of its own: the moments lie in fp32 where
    their squares do not.  A root formed in fp32's middle is off by as much as any other: 8 u of itself, as above."""
    g = gen(30 + high - low)
    h, n = {**HYPER, "eps": eps}, 1000
    ps, state = [randn(g, n, dtype=pd)], [[torch.zeros(n, device="cuda").to(E4M3)] for _ in range(2)]
    scales = [[torch.zeros(-(-n // 128), device="cuda")] for _ in range(2)]
    value = lambda k: state[k][0].double() * scales[k][0].double().repeat_interleave(128)[:n]  # noqa: E731
    for t in (1, 2, 3):
        at = torch.rand(n, generator=g, device="cuda")
        at[:256] = at[:256].view(2, 128)[:, :1].expand(2, 128).reshape(-1)  # (two groups of one size each)
        gr = (torch.pow(10.0, (low + (high - low) * at).double()) * torch.sign(randn(g, n)).double()).to(gd)
        gr[500:520] = 0 if eps and t == 1 else gr[500:520]
        old = (ps[0].clone(), value(0), value(1).square())
        okls.adamw_step(ps, [gr], state[0], state[1], step=t, avg_scales=scales[0], sq_scales=scales[1], seed=5, **h)
        m, v, mag = _check_update(ps[0], *old[:1], gr, *old[1:], t, h, fast=True)
        dm, dv = _philox(n, 0, t, 5)
        _check_codes(state[0][0], scales[0][0], m, 5 * U * mag, dm, False)
        _check_codes(state[1][0], scales[1][0], v.sqrt(), 8 * U * v.sqrt(), dv, True)
        zero = v == 0
        assert torch.equal(state[1][0].float() == 0, zero), "a root that is not zero became zero"
        assert torch.isfinite(ps[0]).all() and torch.isfinite(scales[1][0]).all()


def test_adamw_8_ordinary_values_beside_far_ones():
    """Tensors with and without a far value in the same warp: the others' parameters and codes keep their bits."""
    g = gen(31)
    n = 4096
    p, gr = randn(g, n), randn(g, n, std=1e-2)
    runs = []
    for far in (False, True):
        q, d = p.clone(), gr.clone()
        if far:
            d[1030], d[3000] = 1e-21, 1e21
        state = [torch.zeros(n, device="cuda").to(E4M3) for _ in range(2)]
        scales = [torch.zeros(n // 128, device="cuda") for _ in range(2)]
        for t in (1, 2):
            okls.adamw_step([q], [d], state[:1], state[1:], step=t, avg_scales=scales[:1], sq_scales=scales[1:], **HYPER)
        runs.append([q, state[0].float(), state[1].float(), *scales])
    same = torch.ones(n, dtype=torch.bool, device="cuda")
    same[1030] = False
    same[3000 // 128 * 128:][:128] = False  # (its group's scale is another)
    for x, y in zip(*(r[:3] for r in runs)):
        assert torch.equal(x[same], y[same])
    assert torch.isfinite(runs[1][0]).all() and runs[1][0][3000] != runs[0][0][3000]


def _adamw_set(seed, n=6, bits=32, pd=F32):
    g = gen(seed)
    sizes = [300 + 77 * i for i in range(n)]
    ps = [randn(g, s, dtype=pd) for s in sizes]
    dt = F32 if bits == 32 else E4M3
    st = [[torch.zeros(s, device="cuda", dtype=F32).to(dt) for s in sizes] for _ in range(2)]
    sc = [[torch.zeros(-(-s // 128), device="cuda") for s in sizes] for _ in range(2)] if bits == 8 else [None, None]
    return ps, [randn(g, s, dtype=pd, std=1e-2) for s in sizes], st, sc


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_is_the_same_each_time_in_any_company(bits):
    """The same bits from one call as from two runs, and (32 bits) as from a call for each tensor."""
    runs = []
    for _ in range(2):
        ps, gs, st, sc = _adamw_set(1, bits=bits)
        for t in (1, 2):
            okls.adamw_step(ps, gs, *st, step=t, avg_scales=sc[0], sq_scales=sc[1], **HYPER)
        runs.append(ps + st[0] + st[1])
    assert all(torch.equal(a.float(), b.float()) for a, b in zip(*runs))
    if bits == 32:
        ps, gs, st, _ = _adamw_set(1)
        for t in (1, 2):
            for i in range(len(ps)):
                okls.adamw_step(ps[i:i + 1], gs[i:i + 1], st[0][i:i + 1], st[1][i:i + 1], step=t, **HYPER)
        assert all(torch.equal(a, b) for a, b in zip(ps, runs[0]))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_mixed_types_in_one_call(bits):
    a = _adamw_set(2, bits=bits)
    b = _adamw_set(3, bits=bits, pd=BF16)
    alone = []
    for s in (a, b):
        c = [x.clone() for x in s[0]]
        st = [[x.clone() for x in y] for y in s[2]]
        sc = [[x.clone() for x in y] if y else None for y in s[3]]
        okls.adamw_step(c, s[1], *st, step=1, avg_scales=sc[0], sq_scales=sc[1], **HYPER)
        alone.append(c)
    both = [a[0] + b[0], a[1] + b[1], a[2][0] + b[2][0], a[2][1] + b[2][1]]
    sc = [a[3][0] + b[3][0], a[3][1] + b[3][1]] if bits == 8 else [None, None]
    okls.adamw_step(*both, step=1, avg_scales=sc[0], sq_scales=sc[1], **HYPER)
    # (the first step's update comes from the gradients alone, not from the rounding of 8-bit moments)
    assert all(torch.equal(x, y) for x, y in zip(both[0], alone[0] + alone[1]))


def test_adamw_refusals():
    ps, gs, st, _ = _adamw_set(4)
    call = lambda a=ps, b=gs, c=st[0], d=st[1], **kw: okls.adamw_step(a, b, c, d, **{**dict(step=1, lr=0.1), **kw})  # noqa: E731
    flat = torch.zeros(1000, device="cuda")
    sc = [torch.zeros(-(-p.numel() // 128), device="cuda") for p in ps]
    wrong = [
        lambda: call(ps[:-1]), lambda: call(ps[:1] * 2, gs[:1] * 2, st[0][:2], st[1][:2]), lambda: call(c=st[1]),
        lambda: call([p.half() for p in ps]), lambda: call(b=[p.double() for p in gs]), lambda: call(c=[p.bfloat16() for p in ps]),
        lambda: call(b=gs[1:] + gs[:1]), lambda: call(b=[p.cpu() for p in gs]), lambda: call(step=0), lambda: call(lr=-1.0),
        lambda: call([flat[:100], flat[99:200]], [flat[300:400], flat[300:401]], [flat[400:500], flat[500:601]],
                     [flat[700:800], flat[800:901]]),
        lambda: call([flat.view(10, 100).t()], [flat.clone()], [flat.clone()], [flat.clone()]),
        lambda: call(avg_scales=sc), lambda: call(avg_scales=sc, sq_scales=[s.clone() for s in sc]),
        lambda: call(c=[m.to(E4M3) for m in st[0]], d=[m.to(E4M3) for m in st[1]]),
        lambda: call(c=[m.to(E4M3) for m in st[0]], d=[m.to(E4M3) for m in st[1]], avg_scales=sc, sq_scales=[s[1:] for s in sc]),
        lambda: call(lr=torch.tensor(0.1, device="cuda")), lambda: call(step=torch.zeros(1, device="cuda")),
        lambda: call(step=torch.zeros(1, dtype=torch.int64)), lambda: call(beta1=1.0), lambda: call(a=[1.0] * 6), lambda: call(a=None),
    ]
    before = [x.clone() for x in ps + st[0] + st[1]]
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    wrong.append(lambda: call(step=step, beta2=1.5))
    for i, f in enumerate(wrong):
        with pytest.raises((ValueError, L.OklsError, TypeError)):
            f()
            pytest.fail(f"call {i} was taken")
    assert step.item() == 0 and all(torch.equal(x, y) for x, y in zip(ps + st[0] + st[1], before))
    # (the functional step writes under no_grad, as optimizers do: leaves are taken)
    leaf = [p.clone().requires_grad_() for p in ps]
    version = leaf[0]._version
    call(leaf)
    assert leaf[0]._version > version


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_refuses_a_gradient_over_what_it_writes(bits):
    """Gradients that share memory with a parameter or a state of any tensor of the call, in separate buffers and in one;
    gradients may be one and the same tensor."""
    n, dt = 300, F32 if bits == 32 else E4M3
    for together in (False, True):
        flat = torch.zeros(40 * n, device="cuda")
        at = [0]

        def place(count):
            if not together:
                return torch.zeros(count, device="cuda")
            at[0] += count + 20
            return flat[at[0] - count - 20:at[0] - 20]
        ps, gs, ms, vs = ([place(n) for _ in range(3)] for _ in range(4))
        sc = [[place(3) for _ in range(3)] for _ in range(2)] if bits == 8 else [None, None]
        if bits == 8:
            ms, vs = ([x.view(E4M3)[:n] for x in y] for y in (ms, vs))
        kw = dict(step=1, lr=0.1, avg_scales=sc[0], sq_scales=sc[1])
        written = [ps[0], ps[2], ms[1].view(torch.uint8), vs[0].view(torch.uint8)] + (sc[0][1:2] + sc[1][:1] if bits == 8 else [])
        for t in written:
            storage = torch.empty(0, device="cuda").set_(t.untyped_storage())
            first = t.data_ptr() // 4 * 4 - t.untyped_storage().data_ptr()
            for off in (0, 4, -4):
                begin = (first + off) // 4
                if begin < 0 or begin + n > storage.numel():
                    continue
                bad = list(gs)
                bad[1] = storage[begin:begin + n]
                with pytest.raises(ValueError, match="gradient overlaps"):
                    okls.adamw_step(ps, bad, ms, vs, **kw)
        assert all((x.float() == 0).all() for x in ps + ms + vs)
        okls.adamw_step(ps, [gs[0], gs[0], gs[0][:n]], ms, vs, **kw)
        assert dt == ms[0].dtype


def test_adamw_refuses_too_long_a_tensor_before_it_counts():
    """A tensor past 2^33 elements, of other types than the first: neither the counter nor the first tensor moves."""
    n = (1 << 33) + 1
    ps, gs, st, sc = _adamw_set(10, n=1, bits=8)
    before = ps[0].clone()
    big = [torch.empty(n, device="cuda", dtype=BF16) for _ in range(2)]
    states = [torch.empty(n, device="cuda", dtype=torch.uint8).view(E4M3) for _ in range(2)]
    scales = [torch.empty(-(-n // 128), device="cuda") for _ in range(2)]
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    with pytest.raises((ValueError, L.OklsError), match="2\\^33"):
        okls.adamw_step(ps + big[:1], gs + big[1:], st[0] + states[:1], st[1] + states[1:], step=step, lr=0.1,
                        avg_scales=sc[0] + scales[:1], sq_scales=sc[1] + scales[1:])
    assert step.item() == 0 and torch.equal(ps[0], before)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_captured_step_counts(bits):
    """Replays of a captured step are the steps that follow each other; a captured step with a number of the host is refused."""
    ps, gs, st, sc = _adamw_set(5, bits=bits)
    want, _, st2, sc2 = _adamw_set(5, bits=bits)
    step, lr = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.full((1,), 1e-2, device="cuda")
    h = {k: v for k, v in HYPER.items() if k != "lr"}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        okls.adamw_step(ps, gs, *st, step=step, lr=lr, avg_scales=sc[0], sq_scales=sc[1], seed=9, **h)
    for t in range(1, 5):
        if t == 3:
            lr.fill_(2e-2)
            for g in gs:
                g.mul_(-0.5)
        graph.replay()
        okls.adamw_step(want, gs, *st2, step=t, lr=lr.item(), avg_scales=sc2[0], sq_scales=sc2[1], seed=9, **h)
        assert step.item() == t
        assert all(torch.equal(a.float(), b.float()) for a, b in zip(ps + st[0] + st[1], want + st2[0] + st2[1]))
    side = torch.cuda.CUDAGraph()
    with pytest.raises(ValueError, match="captured"):
        with torch.cuda.graph(side):
            okls.adamw_step(ps, gs, *st, step=5, lr=1e-2, avg_scales=sc[0], sq_scales=sc[1])
    torch.cuda.synchronize()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_optimizer(bits):
    """The class over parameters of both types against torch's on fp32 (32 bits: to the sums of the steps' roundings)."""
    def params():
        g = gen(6)
        return [randn(g, 64, 33).requires_grad_(), randn(g, 100).requires_grad_(), randn(g, 3, 5, 7).requires_grad_()]
    a, b = params(), params()
    own = okls.AdamW(a, lr=1e-2, weight_decay=0.1, state_bits=bits)
    ref = torch.optim.AdamW(b, lr=1e-2, weight_decay=0.1)
    g = gen(7)
    for _ in range(10):
        for p, q in zip(a, b):
            p.grad = randn(g, *p.shape)
            q.grad = p.grad.clone()
        own.step(), ref.step()
    for p, q in zip(a, b):
        if bits == 32:
            # ten updates of at most some 1e-2 (3 of it in the first ones), each to 32 u, and 10 roundings of p
            assert ((p - q).abs() <= 10 * (64 * U * 3e-2 + 4 * U * q.abs())).all()
        else:
            # codes are off by at most 1/8 of a value: an update by less than 1/2 of itself
            assert ((p - q).abs().max().item()) < 10 * 0.5 * 1e-2 and not torch.equal(p, q)


def test_adamw_optimizer_captured():
    g = gen(8)
    a = [randn(g, 300).requires_grad_(), randn(g, 40, 9).requires_grad_()]
    b = [p.detach().clone().requires_grad_() for p in a]
    grads = [[randn(g, *p.shape) for p in a] for _ in range(4)]
    lr = torch.full((1,), 1e-2, device="cuda")
    own, ref = okls.AdamW(a, lr=lr, capturable=True), okls.AdamW(b, lr=1e-2)
    for p, x in zip(a, grads[0]):
        p.grad = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        own.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        own.step()
    for t in range(4):
        for p, q, x in zip(a, b, grads[t]):
            p.grad.copy_(x)
            q.grad = x.clone()
        if t:
            graph.replay()
        ref.step()
    assert own.state[a[0]]["step"].item() == 4
    for p, q in zip(a, b):
        close(p, q, 8 * U * (q.abs() + 1e-2), "captured")


def test_adamw_optimizer_refuses_a_capture_that_would_not_count():
    g = gen(9)
    p = randn(g, 200).requires_grad_()
    p.grad = randn(g, 200)
    host, new = okls.AdamW([p], lr=1e-2), okls.AdamW([p], lr=1e-2, capturable=True)
    before = p.detach().clone()
    host.step()
    moved = p.detach().clone()
    other, graph = torch.zeros(4, device="cuda"), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.add_(1)
        with pytest.raises(RuntimeError, match="capturable=True"):
            host.step()  # each replay would be the same step
        with pytest.raises(RuntimeError, match="before one is captured"):
            new.step()  # each replay would clear the states
    graph.replay()
    assert torch.equal(other, torch.ones(4, device="cuda"))
    assert torch.equal(p.detach(), moved) and not torch.equal(moved, before)
    new.step()  # and takes part once they are there
    assert new.state[p]["step"].item() == 1 and host.state[p]["step"] == 1


# -------------------------------------------------------------------- 4 bits
def _int4_ref(x, group, sym):
    """Codes, scale and zero point by the definition; every step in fp32 is one rounding."""
    rows, cols = x.shape
    groups = -(-cols // group)
    p = torch.nn.functional.pad(x.float(), (0, groups * group - cols)).view(rows, groups, group)
    lo, hi = p.amin(2).clamp_max(0), p.amax(2).clamp_min(0)
    div = lambda a, b: a / torch.full_like(a, b)  # noqa: E731
    s = div(torch.maximum(-lo, hi), 7.0) if sym else 2 * div(0.5 * hi - 0.5 * lo, 15.0)
    s = s.clamp_min(2.0 ** -100).bfloat16().float()
    z = torch.full_like(s, 8.0) if sym else (-lo / s).bfloat16().float()
    c = (torch.round(p / s[..., None] + z[..., None])).clamp(1 if sym else 0, 15)
    return c.view(rows, -1)[:, :cols], s, z


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (5, 33), (64, 64), (3, 127), (17, 129), (200, 1000), (33, 2047)])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
def test_int4_quantize(dtype, rows, cols, group):
    g = gen(rows * 31 + cols)
    x = randn(g, rows, cols, dtype=dtype) * torch.exp(2 * randn(g, rows, 1)).to(dtype)
    x[rows // 2, : cols // 2] = 0
    for sym in (True, False):
        c, s, z = _int4_ref(x, group, sym)
        for v in (x, pitched(x, cols + 3, 1)):
            q = lm.int4_quantize(v, group=group, symmetric=sym)
            assert q.shape == x.shape and (q.zero is None) == sym
            assert torch.equal(q.scale.float(), s)
            assert sym or torch.equal(q.zero.float(), z)
            got = torch.stack((q.data & 15, q.data >> 4), 2).view(rows, -1)
            assert torch.equal(got[:, :cols].float(), c) and got[:, cols:].sum() == 0
    # what the codes stand for: half a step away at most, and what the scale's and zero point's rounding moves (2^-9 of
    # 7 or 15 steps, and of a zero point of 15), which can clamp the last code
    v = q.float().double()
    step = s.double().repeat_interleave(group, 1)[:, :cols]
    assert ((v - x.double()).abs() <= step * (0.5 + 15 * 2.0 ** -8 + 15 * 2.0 ** -8)).all()


def test_int4_quantize_extremes():
    x = torch.zeros(5, 128, device="cuda")
    x[0, 3], x[1, 70] = NAN, -INF
    x[2] = torch.linspace(-1, 1, 128, device="cuda") * 3.4e38
    x[3] = 5.0
    for sym in (True, False):
        q = lm.int4_quantize(x, group=64, symmetric=sym)
        bad = torch.zeros(5, 2, dtype=torch.bool, device="cuda")
        bad[0, 0], bad[1, 1] = True, True
        assert torch.equal(q.scale.isnan(), bad)
        v = q.float()
        assert torch.isfinite(v[3:]).all() and v[4].abs().max().item() == 0
        assert (v[3] - 5.0).abs().max().item() <= 5.0 * 2.0 ** -8
        assert torch.isfinite(q.scale[2]).all()


def _weight(g, n, k, group, zero, rowwise=False):
    pitch = max(1, -(-k // 128)) * 64
    data = torch.randint(0, 256, (n, pitch), generator=g, device="cuda", dtype=torch.uint8)[:, : -(-k // 2)]
    groups = -(-k // group)
    s = (torch.rand(groups, n, generator=g, device="cuda") + 0.5).bfloat16()
    z = (torch.rand(groups, n, generator=g, device="cuda") * 15).bfloat16()
    lay = (lambda t: t.t().contiguous()) if rowwise else (lambda t: t.t())
    return lm.Int4Tensor(data, lay(s), k, group, lay(z) if zero else None)


def _check_int4(x, w, got, od, old=None):
    """Products are exact; a group's sum is fp32, of 16 + c and of -(16 + zero) times x apart; the groups' sums are joined in
    fp32.  Every addition of a sum of k terms, on the tensor core (which may cut off instead of rounding: 2 u) or off it, is
    off by 2 u of at most the sum of magnitudes; of k terms, no chain is longer than k / 4 + 16."""
    x64, k, gr = x.double(), w.cols, w.group
    s = w.scale.double().repeat_interleave(gr, 1)[:, :k]
    z = torch.full_like(s, 8.0) if w.zero is None else w.zero.double().repeat_interleave(gr, 1)[:, :k]
    c = torch.stack((w.data & 15, w.data >> 4), 2).view(w.data.shape[0], -1)[:, :k].double()
    v = (c - z) * s
    mag = x64.abs() @ ((32 + c + z) * s).t()
    want = x64 @ v.t()
    if old is not None:
        want, mag = want + old.double(), mag + old.double().abs()
    close(got, want, (w.cols / 4 + 32) * 2 * U * mag + OUT[od] * want.abs(), "4-bit product")


@pytest.mark.parametrize("group,zero", [(32, True), (32, False), (64, True), (64, False), (128, True), (128, False), (256, True)])
@pytest.mark.parametrize("rows,n,k", [(1, 1, 1), (1, 16, 128), (2, 17, 129), (3, 100, 31), (5, 33, 1000), (8, 48, 2048), (9, 16, 640),
                                      (16, 130, 257), (17, 20, 384), (33, 47, 4097), (70, 31, 96), (1, 2000, 5504)])
def test_int4_matmul(group, zero, rows, n, k):
    g = gen(rows + n + k)
    for dtype, od, pitch, off, rowwise in ((BF16, None, k, 0, False), (F32, None, k + 8, 0, True), (BF16, F32, k + 3, 1, True),
                                           (F32, BF16, k, 3, False)):
        w = _weight(g, n, k, group, zero, rowwise)
        x = pitched(randn(g, rows, k, dtype=dtype), pitch, off)
        y = lm.int4_matmul(x, w, out_dtype=od)
        od = od or dtype
        assert y.shape == (rows, n) and y.dtype == od
        _check_int4(x, w, y, od)
        assert torch.equal(y, lm.int4_matmul(x, w, out_dtype=od))
    # added to an output with a pitch of its own, neighbours left as they are
    old = randn(g, rows, n, dtype=BF16)
    out = pitched(old, n + 5, 3)
    around = out.as_strided((rows, n + 5), (n + 5, 1))
    assert lm.int4_matmul(x, w, out=out, accumulate=True) is out
    _check_int4(x, w, out, BF16, old)
    assert (around[:-1, n:] == 7).all()
    lm.int4_matmul(x, w, out=out)
    _check_int4(x, w, out, BF16)


@pytest.mark.parametrize("rows", [31, 33, 48, 49, 64, 65])
@pytest.mark.parametrize("n,k,group,zero", [(4099, 2055, 32, True), (2051, 4104, 128, False), (1040, 8111, 64, True)])
def test_int4_matmul_of_large_weights_by_several_passes(rows, n, k, group, zero):
    g = gen(rows + n)
    w = _weight(g, n, k, group, zero)
    for dtype in (BF16, F32):
        x = pitched(randn(g, rows, k, dtype=dtype), k + 1, 1)
        out = torch.full((rows + 1, n), 7.0, device="cuda")
        lm.int4_matmul(x, w, out=out[:rows])
        _check_int4(x, w, out[:rows], F32)
        assert (out[rows] == 7).all()


def test_int4_matmul_many_and_no_rows():
    g = gen(1)
    w = _weight(g, 100, 256, 64, True)
    x = randn(g, 500, 256, dtype=BF16)
    _check_int4(x, w, lm.int4_matmul(x, w), BF16)
    assert lm.int4_matmul(x.view(5, 100, 256), w).shape == (5, 100, 100)
    assert lm.int4_matmul(x[:0], w).shape == (0, 100)
    e = lm.Int4Tensor(w.data[:, :0], w.scale[:, :0], 0, 64)
    assert lm.int4_matmul(x[:, :0], e).abs().max().item() == 0
    none = lm.Int4Tensor(w.data[:0], w.scale[:0], 256, 64)
    assert lm.int4_matmul(x, none).shape == (500, 0)


def test_int4_matmul_refuses_an_output_over_its_input():
    g = gen(9)
    w = _weight(g, 64, 64, 32, False)
    buf = randn(g, 6, 64)
    for x, out in ((buf[:4], buf[:4]), (buf[:4], buf[2:]), (buf[1:5, :], buf[1:5])):
        with pytest.raises((ValueError, L.OklsError), match="share"):
            lm.int4_matmul(x, w, out=out)
    halves = randn(g, 4, 128)  # side by side: no element is shared
    x = halves[:, :64]
    _check_int4(x, w, lm.int4_matmul(x, w, out=halves[:, 64:]), F32)
    _check_int4(buf[:2], w, lm.int4_matmul(buf[:2], w, out=buf[2:4]), F32)


def test_int4_matmul_refuses_an_output_among_its_input():
    """Views of one buffer with columns in common, and outputs in the weight; columns beside each other are taken."""
    g = gen(10)
    w = _weight(g, 64, 64, 32, True)
    buf = randn(g, 4, 256)
    x = buf[:, :64]
    for out in (buf[:, 32:96], buf[:, 63:127], buf.view(-1)[60:60 + 4 * 128].view(4, 128)[:, :64], buf.view(BF16)[:, 127:191]):
        with pytest.raises((ValueError, L.OklsError), match="share"):
            lm.int4_matmul(x, w, out=out)
    scale = torch.zeros(64 * 64, device="cuda", dtype=BF16)
    inside = lm.Int4Tensor(w.data, scale.view(64, 64)[:2].t(), 64, 32)
    with pytest.raises((ValueError, L.OklsError), match="share"):
        lm.int4_matmul(x, inside, out=scale.view(F32)[32:32 + 256].view(4, 64))
    left = x.clone()
    for out in (buf[:, 64:128], buf[:, 192:]):
        _check_int4(left, w, lm.int4_matmul(x, w, out=out), F32)
        assert torch.equal(x, left)
    _check_int4(left, w, lm.int4_matmul(x, w, out=buf.view(BF16)[:, 128:192]), BF16)


def test_int4_matmul_of_its_own_quantisation():
    """fp32 activations reach the products with all their digits, also next to each other's extremes."""
    g = gen(2)
    wt = randn(g, 300, 512)
    x = randn(g, 4, 512) * torch.exp(8 * randn(g, 4, 512))
    x[1, 7], x[2, 9] = 3.4e38, 1e-42
    x[1] *= 1e-3
    for sym in (True, False):
        w = lm.int4_quantize(wt, symmetric=sym)
        _check_int4(x, w, lm.int4_matmul(x, w), F32)


def _whole_weight(g, n, k, group, zero):
    """Scales are powers of two, zero points whole: (code - zero) * scale has no rounding anywhere."""
    w = _weight(g, n, k, group, zero)
    w.scale.copy_(torch.exp2(torch.randint(0, 3, w.scale.shape, generator=g, device="cuda").float()))
    if zero:
        w.zero.copy_(torch.randint(0, 16, w.zero.shape, generator=g, device="cuda"))
    return w


@pytest.mark.parametrize("group,zero", [(32, True), (32, False), (64, True), (64, False), (128, True), (128, False), (256, True)])
@pytest.mark.parametrize("rows,n,k", [(1, 40, 31), (1, 2003, 2048), (3, 33, 32768), (8, 100, 4097), (16, 4100, 2055), (16, 48, 8192),
                                      (33, 47, 4097), (64, 1040, 8111), (70, 31, 1000), (130, 64, 16384)])
def test_int4_matmul_of_whole_numbers(group, zero, rows, n, k):
    """Whole x of at most 2: the sums of 31 * 2 * 4 for each of k terms stay below 2^24, so that every order of the additions
    is exact and a term that is missing or counted twice shows."""
    assert 31 * 2 * 4 * k < 1 << 24
    g = gen(rows * 7 + k)
    w = _whole_weight(g, n, k, group, zero)
    x = torch.randint(1, 3, (rows, k), generator=g, device="cuda") * (2 * torch.randint(0, 2, (rows, k), generator=g, device="cuda") - 1)
    want = x.double() @ w.float().double().t()
    for dtype in (BF16, F32):
        got = lm.int4_matmul(x.to(dtype), w, out_dtype=F32)
        assert torch.equal(got.double(), want)
        assert torch.equal(lm.int4_matmul(x.to(dtype), w, out=got, accumulate=True).double(), 2 * want)


@pytest.mark.parametrize("group,zero", [(32, True), (64, False), (128, True), (256, False)])
@pytest.mark.parametrize("rows", [8, 16, 70])
def test_int4_matmul_of_one_column_at_a_time(group, zero, rows):
    """Each row of x has one value, in every column in turn: three bf16 terms of fp32 x (1, 2^-9 and 2^-19 of it) times a code
    less a zero point fill 24 bits, so the output is the weight's column times that value, exactly."""
    g = gen(40 + rows)
    n, k = 37, 600
    w = _whole_weight(g, n, k, group, zero)
    v = w.float().double().t()
    for dtype, value in ((F32, 1 + 2.0 ** -9 + 2.0 ** -19), (BF16, 1 + 2.0 ** -7)):
        for first in range(0, k, rows):
            at = torch.arange(first, min(first + rows, k), device="cuda")
            x = torch.zeros(rows, k, device="cuda", dtype=dtype)
            x[torch.arange(at.numel(), device="cuda"), at] = value
            got = lm.int4_matmul(x, w, out_dtype=F32)
            assert torch.equal(got[:at.numel()].double(), v[at] * value) and (got[at.numel():] == 0).all()


def test_int4_matmul_not_finite():
    g = gen(3)
    for dtype in (BF16, F32):
        for zero in (False, True):
            w = _weight(g, 40, 256, 128, zero)
            x = randn(g, 6, 256, dtype=dtype)
            clean = lm.int4_matmul(x, w)
            bad = x.clone()
            bad[1, 100], bad[4, 3] = NAN, INF
            y = lm.int4_matmul(bad, w)
            assert y[1].isnan().all() and not torch.isfinite(y[4]).any()
            rest = [0, 2, 3, 5]
            assert torch.equal(y[rest], clean[rest])
            w.scale[7, 1] = NAN
            y = lm.int4_matmul(x, w)
            assert y[:, 7].isnan().all() and torch.equal(y[:, 8:], clean[:, 8:]) and torch.equal(y[:, :7], clean[:, :7])


def test_int4_refusals():
    g = gen(4)
    x, w = randn(g, 3, 256), _weight(g, 40, 256, 64, True)
    wrong = [lambda: lm.int4_matmul(x[:, :255], w), lambda: lm.int4_matmul(x.half(), w), lambda: lm.int4_matmul(x.cpu(), w),
             lambda: lm.int4_matmul(x, w, accumulate=True), lambda: lm.int4_matmul(x, w, out=torch.empty(3, 41, device="cuda")),
             lambda: lm.int4_matmul(x, w, out_dtype=torch.float16), lambda: lm.int4_matmul(x.t(), w),
             lambda: lm.int4_matmul(x, w, out=torch.empty(3, 40, device="cuda", requires_grad=True)),
             lambda: lm.int4_quantize(x, group=16), lambda: lm.int4_quantize(x.half()), lambda: lm.int4_quantize(x[0])]
    for field, v in (("data", w.data[:, :-1]), ("data", w.data.cpu()), ("scale", w.scale[:, :2]), ("scale", w.scale.float()),
                     ("zero", w.zero[:5]), ("group", 128), ("cols", 254), ("cols", -1)):
        bad = lm.Int4Tensor(w.data, w.scale, w.cols, w.group, w.zero)
        setattr(bad, field, v)
        wrong.append(lambda bad=bad: lm.int4_matmul(x, bad))
    odd = lm.Int4Tensor(torch.zeros(40, 131, dtype=torch.uint8, device="cuda")[:, 1:129], w.scale, 256, 64)
    wrong.append(lambda: lm.int4_matmul(x, odd))
    for i, f in enumerate(wrong):
        with pytest.raises((ValueError, L.OklsError)):
            f()
            pytest.fail(f"call {i} was taken")


# ------------------------------------------------------------------ sampling
def _column(v, rows, off):
    t = v if isinstance(v, torch.Tensor) else torch.full((rows,), off if v is None else v, device="cuda", dtype=F32)
    return t.double()[:, None]


def _kept(logits, temperature=1.0, top_k=None, top_p=None, min_p=None):
    """Weights (0 where a token is not kept) by the definition in 64 bits, in the order of ids."""
    z = torch.where(logits.isnan(), -INF, logits.float())
    rows, vocab = z.shape
    t, k, p, lo = (_column(v, rows, off) for v, off in ((temperature, 1.0), (top_k, 0), (top_p, 1.0), (min_p, 0.0)))
    v, order = torch.sort(z, dim=-1, descending=True, stable=True)
    v = v.double()
    best = v[:, :1]
    infinite = best == INF
    v = torch.where(infinite, torch.where(v == INF, 0.0, -INF), v)
    best = torch.where(infinite, 0.0, best)
    cold = ~(t >= 2.0 ** -20)
    t = torch.where(cold, 1.0, t)
    k = torch.where(cold | (p <= 0), 1.0, torch.where(k <= 0, vocab, k))
    w = torch.where(v == -INF, 0.0, torch.exp((v - torch.where(best == -INF, 0.0, best)) / t))
    place = torch.arange(vocab, device="cuda")[None]
    w = torch.where(place < k, w, 0.0)
    mass = torch.cumsum(w, -1)
    keep = (p >= 1) | (p <= 0) | (mass - w < p * mass[:, -1:])
    keep &= (lo <= 0) | (v >= best + t * torch.log(lo.clamp(max=1.0)))
    return torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))


def _check_sample(logits, u, r, **kw):
    """The drawn token is kept and u lies where it was drawn from.  A weight is known to 2^-32.5 of itself (its exponent to
    2^-35, the factor's rounding 2^-33) and rounded to a multiple of 2^-(62 - log2 vocab) of the largest, so a running sum
    of n weights is off by 2^-32.5 of the sum and n halves of that unit, and its share of the sum by twice that."""
    shape = logits.shape[:-1]
    assert r.ids.shape == shape and r.logp.shape == shape and r.ids.dtype == torch.int32 and r.logp.dtype == F32
    z, u = logits.reshape(-1, logits.shape[-1]), u.reshape(-1)
    w = _kept(z, **kw)
    total = w.sum(-1)
    ids, logp = r.ids.reshape(-1).long(), r.logp.reshape(-1)
    assert ((ids >= -1) & (ids < z.shape[1])).all(), "an id outside the vocabulary"
    none = total == 0
    assert torch.equal(ids == -1, none) and (logp[none] == -INF).all()
    some = ~none
    w, total, ids, logp = w[some], total[some], ids[some], logp[some]
    u = torch.where(u.isnan(), 0.0, u)[some].double().clamp(0, 1 - 2.0 ** -24)
    share = torch.cumsum(w, -1) / total[:, None]
    own = w.gather(1, ids[:, None])[:, 0]
    assert (own > 0).all(), "a token that is not kept"
    end = share.gather(1, ids[:, None])[:, 0]
    unit = 2.0 ** (max(1, math.ceil(math.log2(z.shape[1]))) - 62)
    off = 2.0 ** -32.5 + (w > 0).sum(-1) * (unit / 2) / (total / w.amax(-1))
    assert (u < end + 2 * off).all() and (u >= end - own / total - 2 * off).all()
    want = torch.log(own / total)
    # two fp32 terms of one sign and their sum: a difference and a quotient (2 u); the logarithm of 1 + a quotient of two
    # rounded sums (3 u of the quotient, which is no more of the logarithm, and 2 u of its own); the sum's rounding
    close(logp, want, 2 * off + 6 * U * want.abs(), "log probability")
    return w, total


SETTINGS = [dict(), dict(temperature=0.3), dict(temperature=2.5), dict(temperature=0.0), dict(top_k=1), dict(top_k=7),
            dict(top_k=600), dict(top_p=0.9), dict(top_p=0.2), dict(top_p=0.9999), dict(min_p=0.05), dict(min_p=1.0),
            dict(top_k=40, top_p=0.9), dict(top_k=700, top_p=0.95, temperature=3.0), dict(top_p=0.8, min_p=0.1),
            dict(top_k=20, min_p=0.02), dict(top_k=50, top_p=0.95, min_p=0.02, temperature=0.8), dict(top_p=0.0), dict(top_k=-1)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,vocab,pitch,off", [(1, 1, 1, 0), (3, 2, 2, 0), (4, 7, 9, 1), (1, 255, 255, 0), (5, 257, 260, 3),
                                                  (33, 1000, 1000, 0), (2, 4099, 4101, 5), (1, 32000, 32000, 0),
                                                  (300, 5000, 5001, 1), (3, 131072, 131072, 0), (160, 33001, 33001, 0),
                                                  (2, 300007, 300009, 7), (1, 1 << 20, 1 << 20, 0)])
def test_sample(dtype, rows, vocab, pitch, off):
    g = gen(vocab)
    z = pitched(randn(g, rows, vocab, dtype=dtype, std=2.5), pitch, off)
    for kw in SETTINGS:
        if rows * vocab > 3e6 and kw in SETTINGS[4:10:2]:
            continue
        u = torch.rand(rows, generator=g, device="cuda")
        _check_sample(z, u, lm.sample(z, u, **kw), **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [9, 1000, 70000])
def test_sample_equal_logits(dtype, vocab):
    """Rows with a few values each, all equal ones, and masks of the type's lowest value: cuts inside runs of equals."""
    g = gen(vocab)
    rows = 12
    z = torch.randint(0, 3, (rows, vocab), generator=g, device="cuda").to(dtype)
    z[1] = 0.25
    z[2] = torch.finfo(dtype).min
    z[3, : vocab // 2] = torch.finfo(dtype).min
    z[4] = torch.finfo(dtype).max
    z[5, ::2] = -INF
    z[6] = -0.0
    z[6, 1::3] = 0.0
    for kw in SETTINGS + [dict(top_k=vocab - 1), dict(top_k=vocab), dict(top_k=max(2, vocab // 3)), dict(top_p=0.5)]:
        for u in (torch.rand(rows, generator=g, device="cuda"), torch.zeros(rows, device="cuda"),
                  torch.full((rows,), 1 - 2.0 ** -24, device="cuda")):
            _check_sample(z, u, lm.sample(z, u, **kw), **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_first_k_end_with_a_run_of_equals(dtype):
    """The first k are all tokens of the best value, or of the best two: what lies below has no share in the mass."""
    g = gen(18)
    rows, vocab = 6, 50000
    z = randn(g, rows, vocab, std=0.5).clamp(-2, 0.9)
    z[:3, 7:2007] = 1.0
    z[3:, 7:1507] = 1.0
    z[3:, 20000:21000] = 0.95
    z = z.to(dtype)
    for k, some in ((2000, slice(0, 3)), (2500, slice(3, 6)), (1500, slice(3, 6)), (1999, slice(0, 3)), (2501, slice(3, 6))):
        for p in (0.3, 0.9, 1.0):
            kw = dict(top_k=k, top_p=p, min_p=0.01)
            u = torch.rand(3, generator=g, device="cuda")
            _check_sample(z[some], u, lm.sample(z[some], u, **kw), **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [5, 3000, 40000])
def test_sample_rows_that_are_not_finite(dtype, vocab):
    g = gen(vocab + 1)
    z = randn(g, 8, vocab, dtype=dtype)
    z[0] = -INF
    z[1] = NAN
    z[2, 1:] = -INF
    z[3, ::2] = NAN
    z[4, 3] = INF
    z[5, 2:5] = INF
    z[6, :4] = -INF
    z[6, 4] = NAN
    for kw in SETTINGS:
        u = torch.rand(8, generator=g, device="cuda")
        r = lm.sample(z, u, **kw)
        _check_sample(z, u, r, **kw)
        assert r.ids[:2].tolist() == [-1, -1] and r.ids[2].item() == 0 and r.ids[4].item() == 3


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_values_of_all_sizes(dtype):
    """Values over many powers of ten, offsets, temperatures at both ends."""
    g = gen(11)
    rows, vocab = 10, 20000
    z = randn(g, rows, vocab)
    z[0] *= 1e30
    z[1] *= 1e-30
    z[2] = torch.exp(60 * z[2]) * torch.where(z[2] > 0, 1.0, -1.0)
    z[3] += 65536
    z[4] -= 1e9
    z[5] *= 1e-3
    z[6] *= 3e5
    z[7, ::3] = -INF  # (with temperatures past 1e36 as well)
    z = z.to(dtype)
    for kw in SETTINGS + [dict(temperature=t, **f) for t in (2.0 ** -20, 1e-4, 50.0, 1e10, 1e38, INF)
                          for f in (dict(), dict(top_p=0.7), dict(top_k=500, min_p=0.3))]:
        u = torch.rand(rows, generator=g, device="cuda")
        _check_sample(z, u, lm.sample(z, u, **kw), **kw)


def test_sample_settings_of_rows():
    """Settings as vectors are the settings as numbers, row by row; NaN turns a filter off, a cold row is greedy."""
    g = gen(12)
    rows, vocab = 64, 9000
    z = randn(g, rows, vocab, std=3.0)
    u = torch.rand(rows, generator=g, device="cuda")
    pick = lambda v, dt=F32: torch.tensor(v, device="cuda", dtype=dt)[torch.randint(0, len(v), (rows,), generator=g, device="cuda")]  # noqa: E731
    kw = dict(temperature=pick([0.0, 0.5, 1.0, 2.0]), top_k=pick([-5, 0, 1, 30, 2000, 1 << 30], torch.int32),
              top_p=pick([0.0, 0.3, 0.9, 1.0, 2.0]), min_p=pick([-1.0, 0.0, 0.1, 0.5, 3.0]))
    r = lm.sample(z, u, **kw)
    _check_sample(z, u, r, **kw)
    for i in range(0, rows, 5):
        one = lm.sample(z[i:i + 1], u[i:i + 1], **{k: v[i].item() for k, v in kw.items()})
        assert one.ids.item() == r.ids[i].item() and one.logp.item() == r.logp[i].item()
    off = torch.full((rows,), NAN, device="cuda")
    a, b = lm.sample(z, u, top_p=off, min_p=off), lm.sample(z, u)
    assert torch.equal(a.ids, b.ids)
    assert torch.equal(lm.sample(z, u, temperature=off).ids.long(), z.argmax(-1))
    assert torch.equal(lm.sample(z, off).ids, lm.sample(z, torch.zeros_like(u)).ids)
    assert torch.equal(lm.sample(z, off.fill_(5.0)).ids, lm.sample(z, torch.full_like(u, 1 - 2.0 ** -24)).ids)
    assert torch.equal(lm.sample(z, off.fill_(-5.0)).ids, lm.sample(z, torch.zeros_like(u)).ids)


def test_sample_shapes_and_scores():
    g = gen(13)
    z = randn(g, 3, 5, 700, dtype=BF16)
    u = torch.rand(3, 5, generator=g, device="cuda")
    r = lm.sample(z, u)
    assert r.ids.shape == (3, 5)
    # with every token kept the log probability is the score of the drawn token: both to a few u and a sum's error
    s = lm.token_logprobs(z, r.ids)
    assert (s.logp - r.logp).abs().max().item() < 64 * U * 10
    assert lm.sample(z[:0], u[:0]).ids.shape == (0, 5)
    many = lm.sample(z.view(15, 700), u.view(15), stream=torch.cuda.current_stream())
    assert torch.equal(many.ids.view(3, 5), r.ids)


def test_sample_counts_follow_the_distribution():
    """A grid of u draws each token as often as its probability says, to one grid step at each end of its interval."""
    n, vocab = 4096, 50
    z = randn(gen(14), 1, vocab).repeat(n, 1)
    u = (torch.arange(n, device="cuda") + 0.5) / n
    r = lm.sample(z, u, temperature=0.7, top_k=20)
    w = _kept(z[:1], temperature=0.7, top_k=20)[0]
    count = torch.bincount(r.ids.long(), minlength=vocab)
    assert ((count - n * w / w.sum()).abs() <= 1).all()


def test_sample_refusals():
    z, u = torch.zeros(4, 100, device="cuda"), torch.zeros(4, device="cuda")
    for f in (lambda: lm.sample(z, u[:3]), lambda: lm.sample(z, u.double()), lambda: lm.sample(z.half(), u),
              lambda: lm.sample(z, u.cpu()), lambda: lm.sample(z, u, temperature=-1.0), lambda: lm.sample(z, u, temperature=NAN),
              lambda: lm.sample(z, u, top_p=NAN), lambda: lm.sample(z, u, top_k=2.5), lambda: lm.sample(z, u, top_k=u),
              lambda: lm.sample(z, u, temperature=u[:2]), lambda: lm.sample(z, u, min_p=u.cpu()), lambda: lm.sample(z[:, :0], u),
              lambda: lm.sample(z.t(), u), lambda: lm.sample(torch.zeros(1, (1 << 20) + 1, device="cuda"), u[:1])):
        with pytest.raises((ValueError, L.OklsError)):
            f()


# ------------------------------------------------------------------ sizes past 32 bits
def test_adamw_past_32_bits():
    """A tensor of more than 2^31 elements, both kinds of states: the last elements against the formula."""
    n, tail = (1 << 31) + 1029, 3000
    p = torch.ones(n, device="cuda", dtype=BF16)
    gr = torch.full((n,), 1e-2, device="cuda", dtype=BF16)
    g = gen(20)
    for x in (p, gr):
        x[-tail:] = randn(g, tail, dtype=BF16)
    old, cut = p[-tail:].clone(), slice(n - tail, n)
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    okls.adamw_step([p], [gr], [m], [v], step=1, **HYPER)
    zero = torch.zeros(tail, dtype=torch.float64, device="cuda")
    want = _check_update(p[cut], old, gr[cut], zero, zero, 1, HYPER)
    close(m[cut], want[0], 4 * U * want[2], "first moment")
    close(v[cut], want[1], 5 * U * want[1], "second moment")
    assert (p[1 << 20] == p[0]).item() and (m[: 1 << 20] == m[0]).all()
    del m, v
    p[cut] = old
    m, r = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    ms, rs = (torch.zeros(-(-n // 128), device="cuda") for _ in range(2))
    okls.adamw_step([p], [gr], [m], [r], step=1, avg_scales=[ms], sq_scales=[rs], seed=3, **HYPER)
    wm, wv, mag = _check_update(p[cut], old, gr[cut], zero, zero, 1, HYPER, fast=True)
    # whole groups at the end
    at = (n - tail + 127) // 128 * 128
    skip = at - (n - tail)
    dm, dv = _philox(n - at, 0, 1, 3, first=at)
    _check_codes(m[at:], ms[at // 128:], wm[skip:], 5 * U * mag[skip:], dm, False)
    _check_codes(r[at:], rs[at // 128:], wv[skip:].sqrt(), 8 * U * wv[skip:].sqrt(), dv, True)


def test_int4_matmul_past_32_bits():
    n, k = 140003, 32768  # 2.3 GB of codes
    g = gen(21)
    data = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(k // 128, 140008, generator=g, device="cuda") + 0.5).bfloat16()[:, :n].t()
    w = lm.Int4Tensor(data, s, k)
    x = randn(g, 1, k, dtype=BF16)
    y = lm.int4_matmul(x, w)
    for rows in (slice(0, 50), slice(n - 50, n), slice(131000, 131100)):
        _check_int4(x, lm.Int4Tensor(data[rows], s[rows], k), y[:, rows], BF16)


@pytest.mark.parametrize("zero", [False, True])
def test_int4_matmul_of_the_most_rows(zero):
    """2^30 rows of weights, the most that the kernel for generated tokens takes, with sums that end inside a chunk."""
    n, k = 1 << 30, 31  # 17 GB of codes
    data = torch.zeros(n, 16, device="cuda", dtype=torch.uint8)
    scale, z = (torch.ones(1, n, device="cuda", dtype=BF16).t() for _ in range(2))
    g = gen(23)
    for rows in (slice(0, 64), slice(n - 64, n)):
        data[rows] = torch.randint(0, 256, (64, 16), generator=g, device="cuda", dtype=torch.uint8)
        scale[rows] = torch.rand(64, 1, generator=g, device="cuda").bfloat16() + 0.5
    w = lm.Int4Tensor(data, scale, k, 32, z if zero else None)
    x = randn(g, 1, k, dtype=BF16)
    y = lm.int4_matmul(x, w, out_dtype=F32)
    for rows in (slice(0, 64), slice(n - 64, n), slice(1 << 29, (1 << 29) + 64)):
        part = lm.Int4Tensor(data[rows], scale[rows], k, 32, w.zero[rows] if zero else None)
        _check_int4(x, part, y[:, rows], F32)
        assert (y[:, rows] != 0).all()
    assert (y[:, 64:n - 64] == y[0, 64]).all()


def test_sample_past_32_bits():
    rows, vocab = 20000, 131072  # 5.2 GB of logits
    z = torch.zeros(rows, vocab, device="cuda", dtype=BF16)
    g = gen(22)
    some = [0, 1, 16383, 16384, 16385, rows - 1]
    z[some] = randn(g, len(some), vocab, dtype=BF16, std=3.0)
    u = torch.rand(rows, generator=g, device="cuda")
    for kw in (dict(), dict(top_p=0.7), dict(top_k=30)):
        r = lm.sample(z, u, **kw)
        one = lm.sample(z[some].contiguous(), u[some], **kw)
        assert torch.equal(r.ids[some], one.ids) and torch.equal(r.logp[some], one.logp)
        # rows of equal logits: the id says where u lies (the shortest prefix of at least p of them, or the first k)
        left = torch.ones(rows, dtype=torch.bool, device="cuda")
        left[some] = False
        count = 30 if "top_k" in kw else math.ceil(vocab * float(torch.tensor(kw.get("top_p", 1.0))))
        want = torch.floor(u.double() * count).int()
        assert torch.equal(r.ids[left], want[left])


@pytest.mark.parametrize("vocab", [1 << 20, 1040001])
def test_sample_of_more_equals_than_a_bin_counts(vocab):
    """Rows of so many equal logits, each in one or two blocks, that a bin's 32-bit sum of their weights wraps around (2^18
    tokens of the largest weight): all equal, two values, and a run of equals below a few better ones."""
    g = gen(24)
    rows = 96  # (more would give a row more blocks)
    z = torch.zeros(rows, vocab, device="cuda", dtype=BF16)
    z[1, ::2] = -1.0
    z[2] = -2.0
    z[2, 1000:1040] = 1.0
    z[3, : 1 << 18] = 0.5
    z[4, : (1 << 18) + 1] = 0.5
    z[5] = randn(g, vocab, dtype=BF16).clamp(max=0.0)  # half of them are the best
    some = list(range(6)) + [rows - 1]
    for kw in (dict(top_p=0.3), dict(top_p=0.9), dict(top_p=0.5, temperature=0.7), dict(top_k=400000), dict(top_k=700001, top_p=0.6),
               dict(top_p=0.95, min_p=0.2), dict()):
        u = torch.rand(rows, generator=g, device="cuda")
        r = lm.sample(z, u, **kw)
        _check_sample(z[some], u[some], lm.TokenSample(r.ids[some], r.logp[some]), **kw)


# ------------------------------------------------------------------ together
def test_generation_step_captured_and_on_two_streams():
    """A 4-bit output layer and the sampling of its logits: captured and replayed with new inputs, two graphs of it, and two
    streams at once, give the bits of eager calls."""
    g = gen(15)
    w = lm.int4_quantize(randn(g, 4000, 512, std=0.1), symmetric=False)
    kw = dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.01)

    def step(x, u):
        z = lm.int4_matmul(x, w, out_dtype=F32)
        return lm.sample(z, u, **kw)
    xs, us = [randn(g, 6, 512, dtype=BF16) for _ in range(4)], [torch.rand(6, generator=g, device="cuda") for _ in range(4)]
    want = [step(x, u) for x, u in zip(xs, us)]
    graphs = []
    for _ in range(2):
        x, u = xs[0].clone(), us[0].clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(x, u)
        graphs.append((graph, x, u, out))
    for i in range(4):
        for k, (graph, x, u, out) in enumerate(graphs):
            x.copy_(xs[(i + k) % 4]), u.copy_(us[(i + k) % 4])
            graph.replay()
        for k, (_, _, _, out) in enumerate(graphs):
            r = want[(i + k) % 4]
            assert torch.equal(out.ids, r.ids) and torch.equal(out.logp, r.logp)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            got.append(step(xs[i % 4], us[i % 4]))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert torch.equal(r.ids, want[i % 4].ids) and torch.equal(r.logp, want[i % 4].logp)


@pytest.mark.parametrize("state_bits", [32, 8])
def test_example_trains_and_generates(state_bits):
    """The example with AdamW's states in both sizes, and generation from its weights in 4 bits: it runs, and its logits are
    those of the same weights in fp32."""
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("train_lm_serving", os.path.join(root, "examples", "train_lm.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    model, losses, _ = example.train(4, vocab=300, tokens=256, state_bits=state_bits)
    assert all(math.isfinite(x) for x in losses)
    maker = example.Generator(model)
    ids = torch.arange(5, device="cuda")
    z = maker.logits(ids)

    def norm(x, w):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    res = model.table.detach()[ids] * model.scale
    x = None
    for n, up, down in zip(maker.norms, maker.up, maker.down):
        res = res if x is None else res + x
        x = torch.nn.functional.silu(norm(res, n) @ up.float().t()) @ down.float().t()
    want = norm(res + x, maker.norms[-1]) @ maker.out.float().t()
    # some ten roundings to bf16 (2^-8 each) lie between the table and a logit, in sums whose terms they hit at random
    assert ((z - want).norm() / want.norm()).item() < 10 * 2.0 ** -8
    tokens, scores = maker.generate(ids, 6, temperature=0.9, top_k=40, top_p=0.9, min_p=0.01)
    assert tokens.shape == scores.shape == (5, 6) and ((tokens >= 0) & (tokens < 300)).all() and (scores <= 0).all()
    again, _ = example.Generator(model).generate(ids, 6, temperature=0.9, top_k=40, top_p=0.9, min_p=0.01)
    assert torch.equal(tokens, again)
    best, _ = maker.generate(ids, 1, temperature=0.0)
    assert torch.equal(best[:, 0].long(), z.argmax(-1))
