"""AdamW over many tensors, 4-bit weights and sampling: what their C entries and Python functions refuse, and how the
optimizer keeps its states, without a GPU."""

import copy
import ctypes
import math

import pytest
import torch

from kronecker_factored_second_gb300 import _lib as L
from kronecker_factored_second_gb300 import lm, okls

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


def test_adamw_arguments(lib):
    def config(**kw):
        return ctypes.byref(L.okls_adamw_config(**{**dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1), **kw}))

    def tensors(**kw):
        good = dict(param=P, grad=P, exp_avg=P, exp_avg_sq=P, avg_scale=P, sq_scale=P, count=5)
        return (L.okls_adamw_tensor * 2)(L.okls_adamw_tensor(**good), L.okls_adamw_tensor(**{**good, **kw}))

    ok = [tensors(), 2, 0, 0, 0, config(), 1, None, None]
    changes = [({0: None}, BAD), ({1: -1}, BAD), ({2: 2}, BAD), ({3: 3}, BAD), ({4: 1}, BAD), ({5: None}, BAD), ({6: 0}, BAD),
               ({7: P + 8}, BAD)]
    changes += [({5: config(**kw)}, BAD) for kw in (
        dict(lr=-1.0), dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(eps=-1.0),
        dict(eps=math.nan), dict(weight_decay=-1.0), dict(weight_decay=math.inf))]
    changes += [({0: tensors(**kw)}, BAD) for kw in (
        dict(param=None), dict(grad=None), dict(exp_avg=None), dict(exp_avg_sq=None), dict(param=P + 2), dict(grad=P + 1),
        dict(exp_avg=P + 2), dict(count=-1), dict(count=(1 << 33) + 1))]
    changes += [({0: tensors(**kw), 4: 2}, BAD) for kw in (dict(avg_scale=None), dict(sq_scale=None), dict(sq_scale=P + 2))]
    refused(ok, changes, lib.okls_adamw_step)
    assert lib.okls_adamw_step(None, 0, 0, 0, 0, config(), 1, None, None) == L.OKLS_OK  # nothing to step
    ok = [config(), None, P, P, None]
    refused(ok, [({0: None}, BAD), ({1: P + 2}, BAD), ({2: None}, BAD), ({2: P + 4}, BAD), ({3: None}, BAD), ({3: P + 8}, BAD)],
            lib.okls_adamw_clock)


def test_adamw_checks_every_tensor_before_the_first_launch(lib):
    """A wrong tensor behind those of the first launch is refused before the device is asked for anything."""
    config = ctypes.byref(L.okls_adamw_config(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1))
    for num in (2, 401, 1000):
        for wrong in (dict(count=(1 << 33) + 1), dict(param=None), dict(grad=P + 1)):
            good = dict(param=P, grad=P, exp_avg=P, exp_avg_sq=P, count=5)
            if torch.cuda.is_available():
                good["count"] = 0  # (they would be stepped if the last one were not looked at)
            t = (L.okls_adamw_tensor * num)(*[L.okls_adamw_tensor(**good)] * (num - 1), L.okls_adamw_tensor(**{**good, "count": 5, **wrong}))
            assert lib.okls_adamw_step(t, num, 0, 0, 0, config, 1, None, None) == BAD, (num, wrong, L.last_error())


def test_int4_arguments(lib):
    ok = [P, 0, 64, 10, 64, 32, P, 32, P, 1, 16, None, 0, 0, None]
    refused(ok, [({0: None}, BAD), ({1: 2}, BAD), ({2: 63}, BAD), ({3: -1}, BAD), ({4: 1 << 31}, BAD), ({5: 16}, BAD),
                 ({5: 96}, BAD), ({5: 0}, BAD), ({6: None}, BAD), ({7: 31}, BAD), ({8: None}, BAD), ({8: P + 1}, BAD),
                 ({9: -1}, BAD), ({11: P + 1}, BAD), ({11: P, 12: -1}, BAD), ({3: 1 << 30, 4: 1 << 10, 2: 1 << 10, 7: 1 << 9}, UNSUP)],
            lib.okls_int4_quantize)
    ok = [P, 0, 64, P, 32, P, 1, 16, None, 0, 0, 64, 10, 20, 64, P, 0, 20, 0, None]
    refused(ok, [({0: None}, BAD), ({1: 2}, BAD), ({2: 10}, BAD), ({3: None}, BAD), ({3: P + 8}, UNSUP), ({4: 31}, BAD),
                 ({4: 40}, UNSUP), ({5: None}, BAD), ({5: P + 1}, BAD), ({7: -1}, BAD), ({8: P + 1}, BAD), ({11: 48}, BAD),
                 ({12: -1}, BAD), ({13: -1}, BAD), ({14: -1}, BAD), ({15: None}, BAD), ({15: P + 2}, BAD), ({16: 2}, BAD),
                 ({17: 19}, BAD), ({18: 2}, BAD), ({12: 524281}, UNSUP)], lib.okls_int4_matmul)
    for i in (12, 13):  # nothing to compute: taken without a device
        assert lib.okls_int4_matmul(*[0 if j == i else v for j, v in enumerate(ok)]) == L.OKLS_OK


def _bytes(p, rows, cols, ld, size):
    return {p + (i * ld + j) * size + b for i in range(rows) for j in range(cols) for b in range(size)}


def test_int4_refuses_an_output_over_what_it_reads(lib):
    """Refused exactly where a byte is shared, for pitches alike and not: an output between the rows of x is none of them."""
    rows, n, k = 3, 6, 32
    far = [1 << 20, 2 << 20, 3 << 20]  # codes, scale, zero

    def call(x, ldx, out, ldo, od=0, codes=far[0], scale=far[1], ls=(1, 8), zero=far[2], lz=(1, 8), r=rows):
        return lib.okls_int4_matmul(x, 0, ldx, codes, 16, scale, *ls, zero, *lz, 32, r, n, k, out, od, ldo, 0, None)
    seen = {True: 0, False: 0}
    for od in (0, 1):
        size = 2 if od else 4
        for ldx in (32, 37, 64):
            read = _bytes(P, rows, k, ldx, 4)
            for ldo in (6, 13, 32 * 4 // size, 37 * 4 // size, 64 * 4 // size):
                for at in list(range(-80, 80, 4)) + list(range(80, 1024, 44)):
                    shared = bool(read & _bytes(P + at, rows, n, ldo, size))
                    if not shared and torch.cuda.is_available():
                        continue  # it would run
                    seen[shared] += 1
                    code = call(P, ldx, P + at, ldo, od)
                    assert (code == BAD and "share" in L.last_error()) == shared, (od, ldx, ldo, at)
    assert seen[True] > 500 and (seen[False] > 200 or torch.cuda.is_available())
    for at in (far[0] + 90, far[0] - 68, far[1] + 8, far[2]):  # 6 rows of 16 bytes of codes, 6 scales, 6 zero points
        assert call(P, 64, at // 4 * 4, 6) == BAD and "weight" in L.last_error()
    assert call(P, 64, far[1] + 100, 6, ls=(40, 1)) == BAD and call(P, 64, far[2] + 80, 6, lz=(9, 7)) == BAD
    if not torch.cuda.is_available():
        for at in (far[0] + 96, far[0] - 72, far[1] + 12):
            assert call(P, 64, at, 6, r=3) != BAD
        assert call(P, 64, far[1] + 8, 6, ls=(40, 1), r=1) != BAD and call(P, 64, far[2] + 12, 6, zero=None) != BAD


def test_sample_arguments(lib):
    def settings(**kw):
        return ctypes.byref(L.okls_sample_settings(**{**dict(temperature=1.0, top_p=1.0), **kw}))
    ok = [P, 0, 64, 10, 64, P, settings(), P, P, None]
    refused(ok, [({0: None}, BAD), ({1: 2}, BAD), ({2: 63}, BAD), ({3: -1}, BAD), ({4: 0}, BAD), ({4: (1 << 20) + 1, 2: 1 << 21}, UNSUP),
                 ({5: None}, BAD), ({5: P + 2}, BAD), ({6: None}, BAD), ({7: None}, BAD), ({8: None}, BAD), ({8: P + 2}, BAD)]
            + [({6: settings(**{n: P + 2})}, BAD) for n in ("temperature_dev", "top_k_dev", "top_p_dev", "min_p_dev")],
            lib.okls_sample)
    assert lib.okls_sample(*[0 if i == 3 else v for i, v in enumerate(ok)]) == L.OKLS_OK


def test_python_refuses_host_tensors():
    x = torch.zeros(4, 64)
    w = lm.Int4Tensor(torch.zeros(8, 32, dtype=torch.uint8), torch.ones(8, 1, dtype=torch.bfloat16), 64)
    for call in (lambda: lm.int4_quantize(x), lambda: lm.int4_matmul(x, w), lambda: lm.sample(x, torch.zeros(4)),
                 lambda: okls.adamw_step([x], [x], [x], [x], step=1, lr=0.1)):
        with pytest.raises(ValueError):
            call()


def test_int4_tensor_checks_and_values():
    codes = torch.randint(0, 256, (5, 50), dtype=torch.uint8)
    s, z = torch.rand(5, 4).bfloat16(), torch.rand(5, 4).bfloat16() * 15
    for cols in (99, 100):
        w = lm.Int4Tensor(codes, s, cols, 32, z)
        assert w.shape == (5, cols)
        v = w.float()
        for i, j in ((0, 0), (1, 31), (2, 32), (4, 98), (3, cols - 1)):
            c = (codes[i, j // 2].item() >> (4 * (j % 2))) & 15
            assert v[i, j].item() == pytest.approx((c - z[i, j // 32].item()) * s[i, j // 32].item(), rel=1e-6)
    assert lm.Int4Tensor(codes, s, 100, 32).float()[0, 1].item() == ((codes[0, 0] >> 4).item() - 8) * s[0, 0].item()
    for bad in (dict(group=48), dict(group=0), dict(cols=101), dict(data=codes.int()), dict(data=codes[0]),
                dict(data=torch.cat([codes, codes], 1)[:, ::2]), dict(scale=s.float()), dict(scale=s[:, :3]), dict(zero=z[:4])):
        with pytest.raises(ValueError):
            lm.Int4Tensor(**{**dict(data=codes, scale=s, cols=100, group=32, zero=z), **bad})


def test_int4_tensor_without_rows_or_columns():
    for rows, cols in ((0, 100), (0, 0), (5, 0)):
        groups = -(-cols // 32)
        w = lm.Int4Tensor(torch.zeros(rows, -(-cols // 2), dtype=torch.uint8), torch.ones(rows, groups).bfloat16(), cols, 32,
                          torch.ones(rows, groups).bfloat16())
        assert w.float().shape == w.shape == (rows, cols)


class _Lent:
    """Stands for a CUDA tensor: remembers the streams that were told of it."""
    is_cuda = True
    shape = (4, 8)

    def __init__(self):
        self.streams = []

    def record_stream(self, s):
        self.streams.append(s)


def test_inputs_of_a_call_on_another_stream_are_recorded(monkeypatch):
    import contextlib
    import types
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(lm, "_n", lambda: types.SimpleNamespace(
        int4_quantize=lambda *a: (torch.zeros(4, 4, dtype=torch.uint8), torch.zeros(4, 1).bfloat16(), None),
        int4_matmul=lambda *a: None, sample=lambda *a: (None, None), adamw_step=lambda *a: None))
    t = [_Lent() for _ in range(6)]
    w = object.__new__(lm.Int4Tensor)
    w.data, w.scale, w.zero, w.cols, w.group = t[1], t[2], t[3], 8, 128
    for fn, told in ((lambda s: lm.int4_quantize(t[0], stream=s), 1), (lambda s: lm.int4_matmul(t[0], w, out=t[4], stream=s), 5),
                     (lambda s: lm.sample(t[0], t[1], top_k=5, stream=s), 2)):
        for x in t:
            x.streams.clear()
        fn("side")
        assert [x.streams for x in t] == [["side"]] * told + [[]] * (6 - told)
    seen = []
    monkeypatch.setattr(lm, "_on", lambda s, *ts: seen.extend(ts) or contextlib.nullcontext())
    a = [torch.zeros(2) for _ in range(8)]
    lm.sample(a[0], a[1], temperature=a[2], top_k=a[3], top_p=a[4], min_p=a[5], stream="side")
    assert [id(x) for x in seen] == [id(x) for x in a[:6]]
    seen.clear()
    okls.adamw_step(a[:1], a[1:2], a[2:3], a[3:4], step=a[4], lr=a[5], avg_scales=a[6:7], sq_scales=a[7:], stream="side")
    assert {id(x) for x in seen} == {id(x) for x in a}


@pytest.fixture
def on_cpu(monkeypatch):
    """AdamW's step on the CPU: 32-bit moments by torch, 8-bit ones without rounding by chance."""
    calls = []

    def step(params, grads, ms, vs, mscales, vscales, step, lr, b1, b2, eps, wd, seed):
        calls.append(len(params))
        for i, (p, g) in enumerate(zip(params, grads)):
            if g.isnan().any():
                raise ValueError("stands for a refusal")
        if isinstance(step, torch.Tensor):
            step += 1
            t = step.item()
        else:
            t = step
        for i, (p, g) in enumerate(zip(params, grads)):
            m, v = ms[i].float(), vs[i].float()
            if mscales is not None:
                m, v = m * mscales[i][0], (v * vscales[i][0]).square()
            m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
            p -= lr * wd * p + lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + eps)
            if mscales is not None:
                v = v.sqrt()
                mscales[i].fill_(m.abs().max().clamp_min(2.0 ** -100) / 448)
                vscales[i].fill_(v.max().clamp_min(2.0 ** -100) / 448)
                m, v = m / mscales[i][0], v / vscales[i][0]
            ms[i].copy_(m)
            vs[i].copy_(v)

    import types
    monkeypatch.setattr(lm, "_n", lambda: types.SimpleNamespace(adamw_step=step))
    return calls


def _params(n=4):
    g = torch.Generator().manual_seed(0)
    return [torch.randn(5 + i, generator=g).requires_grad_() for i in range(n)]


def _set_grads(params, seed, skip=()):
    g = torch.Generator().manual_seed(seed)
    for i, p in enumerate(params):
        d = torch.randn(p.shape, generator=g)
        p.grad = None if i in skip else d.to(p.dtype)


@pytest.mark.parametrize("capturable", [False, True])
def test_optimizer_steps_like_torch(on_cpu, capturable):
    a, b = _params(), _params()
    own = okls.AdamW(a, lr=0.1, betas=(0.8, 0.95), weight_decay=0.2, capturable=capturable)
    ref = torch.optim.AdamW(b, lr=0.1, betas=(0.8, 0.95), weight_decay=0.2)
    for t in range(4):
        skip = (2,) if t == 0 or (t == 2 and not capturable) else ()
        for ps in (a, b):
            _set_grads(ps, t, skip)
        own.step(), ref.step()
    for x, y in zip(a, b):
        assert torch.allclose(x, y, rtol=1e-5, atol=1e-6)
    # tensors of one number of steps go together
    assert on_cpu == ([3, 3, 1, 3, 1, 3, 1] if capturable else [3, 3, 1, 3, 3, 1])
    if capturable:
        _set_grads(a, 9, (1,))
        with pytest.raises(RuntimeError, match="gradient"):
            own.step()


@pytest.mark.parametrize("capturable", [False, True])
def test_tensors_of_a_step_have_chances_of_their_own(monkeypatch, capturable):
    """The counter's second word and the key of the random numbers differ between any two tensors of a step, whatever groups
    and numbers of steps they are in; a single group's are those of adamw_step with the optimizer's seed."""
    import types
    seen = []

    def step(params, grads, ms, vs, mscales, vscales, step, lr, b1, b2, eps, wd, seed):
        if isinstance(step, torch.Tensor):
            step += 1
            step = step.item()
        s = (seed + step * 0x9E3779B97F4A7C15) % (1 << 64)
        seen.extend((s >> 32, (i + s) % (1 << 32)) for i in range(len(params)))
    monkeypatch.setattr(lm, "_n", lambda: types.SimpleNamespace(adamw_step=step))
    for seed in (0, 7, (1 << 64) - 1, -1):
        p = _params(9)
        opt = okls.AdamW([dict(params=p[:4]), dict(params=p[4:6]), dict(params=p[6:], lr=0.5)], state_bits=8, seed=seed,
                         capturable=capturable)
        for t, skip in enumerate([(1, 5), (), (1, 4) if not capturable else ()]):
            _set_grads(p, t, skip)
            seen.clear()
            opt.step()
            assert len(set(seen)) == len(seen) == 9 - len(skip)
        alone = okls.AdamW(_params(3), state_bits=8, seed=seed)
        _set_grads(alone.param_groups[0]["params"], 0)
        seen.clear()
        alone.step()
        s = (seed + 0x9E3779B97F4A7C15) % (1 << 64)
        assert seen == [(s >> 32, (i + s) % (1 << 32)) for i in range(3)]


def test_a_refused_step_is_not_counted(on_cpu):
    p = _params(1)
    opt = okls.AdamW(p)
    _set_grads(p, 0)
    opt.step()
    p[0].grad.fill_(math.nan)
    with pytest.raises(ValueError):
        opt.step()
    assert opt.state[p[0]]["step"] == 1


@pytest.mark.parametrize("bits,capturable", [(32, False), (8, False), (32, True)])
def test_optimizer_state_round_trip(on_cpu, bits, capturable):
    """Saved and loaded states continue with the same bits, in their own types."""
    a = [p.detach().bfloat16().requires_grad_() if i == 1 else p for i, p in enumerate(_params())]
    opt = okls.AdamW(a, state_bits=bits, capturable=capturable)
    for t in range(2):
        _set_grads(a, t)
        opt.step()
    b = copy.deepcopy(a)
    again = okls.AdamW(b, state_bits=bits, capturable=capturable)
    again.load_state_dict(copy.deepcopy(opt.state_dict()))
    for p, q in zip(a, b):
        for k, x in opt.state[p].items():
            y = again.state[q][k]
            assert type(x) is type(y)
            if isinstance(x, torch.Tensor):
                assert x.dtype == y.dtype and torch.equal(x.float(), y.float()) and x.data_ptr() != y.data_ptr()
            else:
                assert x == y
    for t in range(2, 4):
        for o, ps in ((opt, a), (again, b)):
            _set_grads(ps, t)
            on_cpu.clear()
            o.step()
            assert on_cpu == [4]
    for p, q in zip(a, b):
        assert torch.equal(p, q)


@pytest.mark.parametrize("first", [False, True])
def test_steps_are_counted_on_when_capturable_changes(on_cpu, first):
    """A group that is made capturable after some steps (or no longer is) goes on with its next number, its tensors together."""
    a, b = _params(), _params()
    own, ref = okls.AdamW(a, lr=0.1, capturable=first), torch.optim.AdamW(b, lr=0.1, weight_decay=0.01)
    for t in range(6):
        for ps in (a, b):
            _set_grads(ps, t)
        on_cpu.clear()
        own.step(), ref.step()
        assert on_cpu == [4]
        for p in a:
            n = own.state[p]["step"]
            assert int(n) == t + 1 and isinstance(n, torch.Tensor) == own.param_groups[0]["capturable"]
        if t in (1, 3):
            own.param_groups[0]["capturable"] = not own.param_groups[0]["capturable"]
    for x, y in zip(a, b):
        assert torch.allclose(x, y, rtol=1e-5, atol=1e-6)


def test_a_group_that_is_refused_keeps_the_others_from_stepping(on_cpu):
    p = _params()
    opt = okls.AdamW([dict(params=p[:2]), dict(params=p[2:], capturable=True)])
    _set_grads(p, 0)
    opt.step()
    _set_grads(p, 1, (3,))
    before = [x.detach().clone() for x in p]
    with pytest.raises(RuntimeError, match="gradient"):
        opt.step()
    assert all(torch.equal(x, y) for x, y in zip(p, before)) and opt.state[p[0]]["step"] == 1


def test_optimizer_refuses_settings():
    p = _params(1)
    for kw in (dict(state_bits=16), dict(betas=(1.0, 0.9)), dict(eps=-1.0), dict(weight_decay=-0.1), dict(lr=torch.tensor(0.1))):
        with pytest.raises(ValueError):
            okls.AdamW(p, **kw)
