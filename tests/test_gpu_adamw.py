"""GPU checks of sa_adamw_step against the fp64 oracle.

Tolerances, in half steps of fp32 (2^-24 of a value): m and v are two products, their sum and the
factors' own rounding (<= 4 each, of the absolute terms); the update is then a square root, a
product, a sum, a quotient, a product, a difference and the rounding of lr, eps and the bias
corrections (<= 16, of the step's absolute value) beside p's own (<= 4).  8-bit states: half a step
of e4m3 (2^-4 of the value, at least 2^-10 of the scale), the second moment's root never below
2^-9 of the scale."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)


def _tensor(n, bits, grad=torch.float32, copy=False, decay=0.01, seed=0):
    g = torch.Generator().manual_seed(seed + n)
    r = lambda s: torch.randn(n, generator=g) * s
    t = {"param": r(0.02).cuda(), "grad": r(1e-3).to(grad).cuda(), "weight_decay": decay,
         "param_bf16": torch.zeros(n, dtype=torch.bfloat16, device="cuda") if copy else None}
    m, v = r(1e-3), r(1e-3).square()
    if bits == 32:
        return {**t, "m": m.cuda(), "v": v.cuda()}
    blocks = -(-n // 128)
    for name, x in (("m", m), ("v", v.sqrt())):
        y = torch.cat([x, torch.zeros(blocks * 128 - n)]).view(blocks, 128)
        scale = y.abs().amax(1) / 448
        t[name] = (y / scale[:, None]).to(torch.float8_e4m3fn).view(-1)[:n].cuda()
        t[name + "_scale"] = scale.cuda()
    return t


def _moments(t):
    """m, v in 64 bits, as the state stands for them."""
    if t["m"].dtype == torch.float32:
        return t["m"].double().cpu().numpy(), t["v"].double().cpu().numpy()
    each = lambda n: t[n].float().double().cpu().numpy() * np.repeat(t[n + "_scale"].double().cpu().numpy(), 128)[:t[n].numel()]  # noqa: E731
    return each("m"), each("v") ** 2


def _snapshot(ts):
    return [{k: x.clone() if isinstance(x, torch.Tensor) else x for k, x in t.items()} for t in ts]


def _check(before, after, step, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0):
    for b, a in zip(before, after):
        p0, g = b["param"].double().cpu().numpy(), b["grad"].double().cpu().numpy()
        m0, v0 = _moments(b)
        p, m, v = oracle.adamw_step(p0, g, m0, v0, lr, beta1, beta2, eps, b["weight_decay"], step, grad_scale)
        gs = np.abs(g * grad_scale)
        m_err = 4 * U * (beta1 * np.abs(m0) + (1 - beta1) * gs)
        v_err = 4 * U * v
        root = np.sqrt(v / (1 - beta2 ** step)) + eps
        size = abs(lr) / (1 - beta1 ** step) * (np.abs(m) + m_err / U / 16) / root
        got = a["param"].double().cpu().numpy()
        assert (np.abs(got - p) <= 16 * U * size + 4 * U * np.abs(p0)).all()
        if a.get("param_bf16") is not None:
            assert torch.equal(a["param_bf16"], a["param"].bfloat16())
        gm, gv = _moments(a)
        if b["m"].dtype == torch.float32:
            assert (np.abs(gm - m) <= m_err).all() and (np.abs(gv - v) <= v_err).all()
            continue
        n = len(m)
        for name, x, y, err in (("m", m, gm, m_err), ("v", np.sqrt(v), np.sqrt(gv), 4 * U * np.sqrt(v))):
            pad = np.zeros(-(-n // 128) * 128)
            pad[:n] = np.abs(x)
            top = pad.reshape(-1, 128).max(1)
            top[top < 2.0 ** -100] = 0             # held as zeros
            s = a[name + "_scale"].double().cpu().numpy()
            np.testing.assert_allclose(s, top / 448, rtol=8 * U + 1e-6, atol=0)
            sc = np.repeat(s, 128)[:n]
            # half a step of the code, and the fp32 value's own error; a root may be lifted to 2^-9
            room = np.where(sc > 0, np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * sc) * (1 + 1e-5) + err, 2.0 ** -100)
            if name == "v":
                room = np.maximum(room, np.where(x < 2.0 ** -9 * sc, 2.0 ** -9 * sc - x, 0) * (1 + 1e-5))
                assert ((y > 0) | (x == 0) | (sc == 0)).all()
            assert (np.abs(y - x) <= room).all(), name


SIZES = (1, 7, 8, 127, 128, 129, 2047, 2048, 2049, 5000, 70_001)


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16], ids=["gf32", "gbf16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_sizes(lib, bits, grad):
    ts = [_tensor(n, bits, grad, copy=n % 2 == 1, decay=0.01 if n > 128 else 0.0) for n in SIZES]
    before = _snapshot(ts)
    lib.sa_adamw_step(ts, **HYPER, step=3)
    torch.cuda.synchronize()
    _check(before, ts, 3)


def test_long_lists_of_both_kinds(lib):
    """More tensors than one launch takes, both kinds of state and gradient mixed, some empty."""
    ts = [_tensor(1 + 37 * i % 900, 8 if i % 3 else 32, torch.bfloat16 if i % 5 == 0 else torch.float32, seed=i)
          for i in range(430)]
    ts.insert(100, {k: torch.empty(0, device="cuda") for k in ("param", "grad", "m", "v")})
    before = _snapshot(ts)
    lib.sa_adamw_step(lib.AdamWTensors(ts), **HYPER, step=10)
    torch.cuda.synchronize()
    keep = [i for i in range(len(ts)) if i != 100]
    _check([before[i] for i in keep], [ts[i] for i in keep], 10)


@pytest.mark.parametrize("hyper", [
    dict(lr=1e-2, beta1=0.0, beta2=0.0, eps=1e-3), dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8),
    dict(lr=-1e-3, beta1=0.5, beta2=0.9, eps=1e-6), dict(lr=0.0, beta1=0.9, beta2=0.95, eps=1e-8)], ids=str)
@pytest.mark.parametrize("bits", [32, 8])
def test_hyperparameters_and_the_first_step(lib, bits, hyper):
    ts = [_tensor(3000, bits)]
    for name in ("m", "v", "m_scale", "v_scale"):
        if name in ts[0]:
            ts[0][name].zero_()                   # the fresh state
    for step in (1, 2):
        before = _snapshot(ts)
        lib.sa_adamw_step(ts, **hyper, step=step)
        torch.cuda.synchronize()
        _check(before, ts, step, **hyper)


@pytest.mark.parametrize("bits", [32, 8])
def test_device_scalars_in_a_captured_step(lib, bits):
    ts = [_tensor(4000, bits, copy=True), _tensor(77, bits)]
    same = _snapshot(ts)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    lr, scale = torch.tensor([1e-3], device="cuda"), torch.tensor([0.5], device="cuda")
    held = lib.AdamWTensors(ts)
    lib.sa_adamw_step(lib.AdamWTensors(_snapshot(ts)), 0.0, step=1)           # loads the kernel before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        lib.sa_adamw_step(held, 123.0, step_dev=step, lr_dev=lr, grad_scale=scale)
    for t, rate in ((1, 1e-3), (2, 2e-3), (3, 5e-4)):
        lr.fill_(rate)
        before = _snapshot(ts)
        graph.replay()
        torch.cuda.synchronize()
        _check(before, ts, t, lr=float(np.float32(rate)), grad_scale=0.5)
    # the host's scalars give the same up to the rounding of the bias corrections
    for t, rate in ((1, 1e-3), (2, 2e-3), (3, 5e-4)):
        lib.sa_adamw_step(same, float(np.float32(rate)), step=t, grad_scale=scale)
    torch.cuda.synchronize()
    if bits == 32:
        for a, b in zip(ts, same):
            torch.testing.assert_close(a["param"], b["param"], rtol=0, atol=1e-6 * 3.5e-3 * 30)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_grad_scale_that_is_not_finite_leaves_everything(lib, bits, value):
    ts = [_tensor(1000, bits, copy=True)]
    ts[0]["grad"][5] = float("inf")
    before = _snapshot(ts)
    lib.sa_adamw_step(ts, **HYPER, step=2, grad_scale=torch.tensor([value], device="cuda"))
    torch.cuda.synchronize()
    for k, x in before[0].items():
        if isinstance(x, torch.Tensor):
            assert torch.equal(x.view(torch.uint8), ts[0][k].view(torch.uint8)), k


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_gradient_that_is_not_finite_stays_in_its_block(lib, bits, value):
    ts = [_tensor(1000, bits)]
    clean = _snapshot(ts)
    ts[0]["grad"][300] = value
    for s, t in ((2, ts), (2, clean)):
        lib.sa_adamw_step(t, **HYPER, step=s)
    for t in (ts, clean):
        lib.sa_adamw_step(t, **HYPER, step=3)
    torch.cuda.synchronize()
    hit = np.zeros(1000, bool)
    hit[300:301] = True
    if bits == 8:
        hit[256:384] = True                       # its block of 128 values
    got, want = ts[0]["param"].cpu().numpy(), clean[0]["param"].cpu().numpy()
    assert np.array_equal(got[~hit], want[~hit])
    assert np.isnan(got[hit]).all()


def test_zero_blocks_and_tiny_ones(lib):
    """A block of zeros stays zero without dividing by it; one below 2^-100 is held as zeros."""
    t = _tensor(384, 8)
    for name in ("param", "grad", "m", "v", "m_scale", "v_scale"):
        t[name].zero_()
    t["grad"][128:256] = 1e-36                     # m = 1e-37 < 2^-100, v = 0
    t["grad"][256:384] = torch.linspace(1e-9, 1.0, 128, device="cuda")
    lib.sa_adamw_step([t], **HYPER, step=1)
    torch.cuda.synchronize()
    assert bool(t["param"].isfinite().all()) and torch.count_nonzero(t["param"][:128]) == 0
    assert t["m_scale"][1] == 0 and torch.count_nonzero(t["m"].float()[:256]) == 0
    assert bool((t["v"].float()[256:] > 0).all())  # no positive second moment is lost
    before = _snapshot([t])
    lib.sa_adamw_step([t], **HYPER, step=2)
    torch.cuda.synchronize()
    _check(before, [t], 2)


@pytest.mark.parametrize("bits", [32, 8])
def test_only_the_tensors_are_written(lib, bits):
    n, guard = 1001, 135                           # the tensors' ends fall inside a thread's 8 values
    t = _tensor(n, bits, copy=True)
    room = {}
    for k, x in t.items():
        if isinstance(x, torch.Tensor):
            raw = torch.full(((x.numel() + guard) * x.element_size(),), 0x5A, dtype=torch.uint8, device="cuda")
            room[k] = raw.view(x.dtype)
            room[k][:x.numel()] = x
            t[k] = room[k][:x.numel()]
    before = _snapshot([t])
    lib.sa_adamw_step([t], **HYPER, step=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mid = _snapshot([t])
    torch.cuda.synchronize()
    _check(before, mid, 1)
    lib.sa_adamw_step([t], **HYPER, step=2, stream=side)
    torch.cuda.synchronize()
    _check(mid, [t], 2)
    for k, x in room.items():
        tail = x[t[k].numel():].view(torch.uint8)
        assert bool((tail == 0x5A).all()), k


def test_binding_refuses_wrong_states(lib):
    t = _tensor(300, 8)
    for bad in ({"m_scale": t["m_scale"][:2]}, {"v": t["v"].float()}, {"grad": t["grad"][:299]},
                {"param": t["param"].double()}, {"grad": t["grad"].cpu()}):
        with pytest.raises((TypeError, ValueError)):
            lib.AdamWTensors([{**t, **bad}])


def test_codes_are_the_rounded_quotients(lib):
    """The 8-bit codes are those of the IEEE quotient value / scale, over many exponents: the kernel
    divides by a reciprocal and a residual step."""
    n = 128 * 4000
    g = torch.Generator().manual_seed(3)
    t = _tensor(n, 8)
    for name in ("m", "v", "m_scale", "v_scale"):
        t[name].zero_()
    size = torch.exp2(torch.randint(-60, 20, (n // 128,), generator=g).float()).repeat_interleave(128)
    t["grad"] = (torch.randn(n, generator=g) * size * torch.exp2(torch.randn(n, generator=g) * 4)).cuda()
    lib.sa_adamw_step([t], 1e-3, 0.5, 0.75, 1e-8, step=1)
    m, v = t["grad"] * 0.5, (t["grad"] * t["grad"]) * 0.25      # exact scalings of fp32 values
    for name, x, floor in (("m", m, False), ("v", v.sqrt(), True)):
        x = x.view(-1, 128)
        top = x.abs().amax(1, keepdim=True)
        scale = torch.where(top >= 2.0 ** -100, top * (torch.ones((), device="cuda") / 448), 0.0)
        assert torch.equal(scale.view(-1), t[name + "_scale"])
        y = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0)
        if floor:
            y = torch.where((x > 0) & (scale > 0), y.clamp_min(2.0 ** -9), y)
        want = y.to(torch.float8_e4m3fn).view(torch.uint8).view(-1)
        assert torch.equal(want & 0x7F, t[name].view(torch.uint8) & 0x7F)   # but for the sign of zero


def test_an_array_twice_in_the_list_is_refused(lib):
    a, b = _tensor(300, 8), _tensor(300, 8, seed=1)
    for name in ("param", "m", "v", "m_scale"):
        with pytest.raises(ValueError):
            lib.AdamWTensors([a, {**b, name: a[name]}])
    lib.AdamWTensors([a, {**b, "grad": a["grad"]}, _tensor(0, 32), _tensor(0, 32)])


def test_gradients_dropped_while_a_step_on_another_stream_runs(lib):
    """Their memory is not handed out again before the step has read it."""
    want, got = [_tensor(8_000_000, 32, seed=2)], [_tensor(8_000_000, 32, seed=2)]
    lib.sa_adamw_step(want, step=1, **HYPER)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    held = dict(got[0])
    del got[0]["grad"]
    step = [held]
    lib.sa_adamw_step([_tensor(30_000_000, 32, seed=3)], step=1, stream=stream, **HYPER)   # keeps the stream busy
    lib.sa_adamw_step(step, step=1, stream=stream, **HYPER)
    del step, held
    for _ in range(3):
        torch.full((8_000_000,), float("nan"), device="cuda")
    torch.cuda.synchronize()
    for name in ("param", "m", "v"):
        assert torch.equal(got[0][name], want[0][name])
