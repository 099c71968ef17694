"""GPU checks of sa_backward_tokenwise against the fp64 oracle, through the C ABI.

Tolerances, from the roundings (half a step: bf16 2^-8, fp32 2^-24 of a value), element by
element against the sums of absolute terms that the oracle's values give:
* Z, G = [U; dH] X^T take U and dH as hi + lo bf16 (the rest is <= 2^-8 2^-8 of the operand) and X
  exactly; 16 tensor-core steps of K = 16 that truncate (<= 2^-23 of the sum of terms each).  So
  |dz| <= KZ z_abs with z_abs = |U| |x| and KZ = 2^-16 + 16 2^-23, and A = exp(z - lse) is off by
  <= A (dz_i + max dz + 2^-20) (lse is a weighted mean of z; 2^-20 for exp, lse's sum and the
  subtraction of values up to 16).
* dZ = A (G - c): |err| <= A_err |G - c| + A (KZ g_abs + c_err), c = dH . H in fp32
  (c_err <= 130 2^-24 |dH| |H|), then hi + lo of dZ for E: <= 2^-16 |dZ|.
* E: sums of those over events, + at most 2 8 (kDrain = 8 tiles) steps a tile kept in TMEM
  truncating 2^-23, + fp32 sums of the drained parts (n / 1024 + 150 terms, 2^-24 each).
* dP, dW_Q, dW_K: |E_err| through the fp32 projections (three of K <= max(k, 128) terms).
* dX is one bf16 rounding (2^-8) of A^T dH + dZ^T U, whose operands A, dH, dZ, U are bf16 (2^-8
  each); G and c there take a bf16 dH (2^-8 (g_abs + |dH| |H|)).  E's take dH as hi + lo, c too
  (2^-16 |dH| |H|)."""
import math

import numpy as np
import pytest
import torch

import oracle
from helpers import dev_f32, sa_device_inputs
from sa_inputs import make_sa_problem

pytestmark = pytest.mark.gpu

BF, F32 = 2.0 ** -8, 2.0 ** -24
KZ = 2.0 ** -16 + 16 * 2.0 ** -23
NAMES = ("dX", "dP", "dW_Q", "dW_K", "dW_V")


def _run(lib, p, dS, dv=None, H=None, **kw):
    dv = dv or sa_device_inputs(p)
    if H is None:
        H = lib.sa_forward_tokenwise(dv["X"], p.offsets, dv["P"], dv["W_Q"], dv["W_K"], dv["W_V"], p.eps,
                                     want_H=True)["H"]
    g = lib.sa_backward_tokenwise(dv["X"], p.offsets, dv["P"], dv["W_Q"], dv["W_K"], dv["W_V"], p.eps, H, dS, **kw)
    return g, H


def _check(lib, p, got, H, dS):
    """Every gradient within the bounds above; returns the worst share of a bound that is used."""
    x, H, dS = p.x_f64(), H.double().cpu().numpy(), dS.double().cpu().numpy()
    P, WQ, WK, WV = (a.astype(np.float64) for a in (p.P, p.W_Q, p.W_K, p.W_V))
    k, d = P.shape
    root = math.sqrt(d)
    U = P @ WQ @ WK.T / root
    U_err = 300 * F32 * (np.abs(P) @ np.abs(WQ) @ np.abs(WK.T) / root)       # two fp32 products of 128 terms
    E_err, dX_err = np.zeros_like(P), np.zeros_like(x)
    dWV_err = np.zeros_like(WV)
    for u in range(p.B):
        lo, hi = int(p.offsets[u]), int(p.offsets[u + 1])
        n = hi - lo
        if n == 0:
            continue
        xu, ax = x[lo:hi], np.abs(x[lo:hi])
        A = oracle._softmax_rows(U @ xu.T)
        dH = dS[u] @ WV.T / (1 + p.eps)
        dH_err = 150 * F32 * (np.abs(dS[u]) @ np.abs(WV.T))
        c = (dH * H[u]).sum(1, keepdims=True)
        c_abs = (np.abs(dH) * np.abs(H[u])).sum(1, keepdims=True)
        c_err = (130 * F32 + 2.0 ** -16) * c_abs + (dH_err * np.abs(H[u])).sum(1, keepdims=True)
        dz = KZ * (np.abs(U) @ ax.T) + U_err @ ax.T
        A_err = A * np.minimum(dz + dz.max(1, keepdims=True) + 2.0 ** -20, 1)
        g, g_abs = dH @ xu.T, np.abs(dH) @ ax.T
        one = n == 1                                                          # dZ is zero exactly
        dZ = np.zeros_like(A) if one else A * (g - c)
        dZ_err = np.zeros_like(A) if one else A_err * np.abs(g - c) + A * (KZ * g_abs + dH_err @ ax.T + c_err)
        s = 2.0 ** -16 + 128 * 2.0 ** -23 + (n / 1024 + 150) * F32
        E_err += (dZ_err + s * np.abs(dZ)) @ ax
        low = BF + 2.0 ** -12                                                 # bf16, and the fp32 sums' own
        dZ_low = A * BF * (g_abs + c_abs) + dZ_err + low * np.abs(A * (g - c))
        dX_err[lo:hi] = (A_err + 2 * low * A).T @ np.abs(dH) + dZ_low.T @ np.abs(U) + low * np.abs(dZ).T @ np.abs(U)
        dWV_err += (p.B * k + 40) * F32 * (np.abs(H[u]).T @ np.abs(dS[u]))
    ref = oracle.sa_backward_tokenwise(x, p.offsets, P, WQ, WK, WV, p.eps, dS, H=H)
    f = 1.01 + 3 * max(k, d) * F32                                            # the last fp32 products
    E_abs = E_err + 3 * max(k, d) * F32 * np.abs(_E(x, p.offsets, U, WV, p.eps, dS, H))
    bounds = (dX_err * (1 + BF) + BF * np.abs(ref[0]), f * E_abs @ np.abs(WK) @ np.abs(WQ.T) / root,
              f * np.abs(P.T) @ E_abs @ np.abs(WK) / root, f * E_abs.T @ np.abs(P) @ np.abs(WQ) / root, dWV_err)
    worst = {}
    for name, r, b in zip(NAMES, ref, bounds):
        e = np.abs(got[name].double().cpu().numpy() - r)
        assert e.shape == r.shape and np.isfinite(e).all(), name
        tiny = 1e-30
        worst[name] = float((e / (b + tiny)).max(initial=0.0))
        assert worst[name] <= 1.0, (name, worst[name], float(e.max()))
        if name != "dX" and np.abs(r).max() > 0:
            # and as a whole: fp32-grade (every term's bound met at random signs is far below this)
            assert np.linalg.norm(e) <= 2e-5 * max(np.linalg.norm(r), np.linalg.norm(b) * 1e-2), name
    return worst


def _E(x, off, U, WV, eps, dS, H):
    E = np.zeros_like(U)
    for u in range(len(off) - 1):
        xu = x[int(off[u]):int(off[u + 1])]
        if len(xu) > 1:
            A = oracle._softmax_rows(U @ xu.T)
            dH = dS[u] @ WV.T / (1 + eps)
            E += np.abs(A * (dH @ xu.T - (dH * H[u]).sum(1, keepdims=True))) @ np.abs(xu)
    return E


def _problem(lengths, k, ps=1.0, seed=60):
    p = make_sa_problem(lengths, k, 128, "bf16", seed=seed + k, x_kind="gauss", p_scale=ps)
    dS = dev_f32(np.random.default_rng(seed).standard_normal((p.B, k, 128)))
    return p, dS


CASES = [
    ((1,), 1, 1.0), ((2,), 3, 1.0), ((128,), 128, 1.0), ((129,), 129, 2.0), ((256, 257), 64, 1.0),
    ((130, 0, 700, 5, 1), 100, 1.0), ((0, 0, 3), 65, 1.0), ((1, 2000), 200, 4.0), ((5000,), 300, 0.25),
    ((300,) * 7, 384, 1.0), ((37000, 20), 40, 1.0), ((1100, 1024, 1023), 1024, 2.0), ((700, 257), 4096, 1.0),
    ((2,) * 40, 600, 2.0), ((9, 0, 300, 1) * 10, 130, 1.0), ((17,) * 170, 128, 1.0), ((4, 3) * 100, 500, 1.0),
]


@pytest.mark.parametrize("lengths,k,ps", CASES, ids=[f"n{'-'.join(map(str, c[0][:4]))}_k{c[1]}" for c in CASES])
def test_against_the_oracle(lib, lengths, k, ps):
    p, dS = _problem(lengths, k, ps)
    got, H = _run(lib, p, dS)
    torch.cuda.synchronize()
    lib.poll_device_status()
    _check(lib, p, got, H, dS)


def test_many_short_users(lib):
    """More users than CTAs, most of them without events or with one to five: every chunk holds
    many pieces."""
    rng = np.random.default_rng(8)
    p, dS = _problem(tuple(int(n) for n in rng.integers(0, 6, 700)), 130)
    got, H = _run(lib, p, dS)
    torch.cuda.synchronize()
    lib.poll_device_status()
    _check(lib, p, got, H, dS)


def test_no_events_at_all(lib):
    p, dS = _problem((0, 0), 64)
    got, H = _run(lib, p, dS)
    torch.cuda.synchronize()
    assert got["dX"].numel() == 0
    for name in NAMES[1:]:
        assert torch.count_nonzero(got[name]) == 0


def test_against_differences_of_the_forward(lib):
    """<gradient, way> against the central difference of the oracle's loss along that way."""
    p, dS = _problem((90, 200), 96)
    got, _ = _run(lib, p, dS)
    args = [p.x_f64(), *(a.astype(np.float64) for a in (p.P, p.W_Q, p.W_K, p.W_V))]
    w = dS.double().cpu().numpy()
    rng = np.random.default_rng(9)
    for i, name in enumerate(NAMES):
        way, at, h = rng.standard_normal(args[i].shape), args[i], 1e-5
        loss = []
        for s in (h, -h):
            args[i] = at + s * way
            loss.append((oracle.sa_forward_tokenwise(args[0], p.offsets, *args[1:], p.eps)[0] * w).sum())
        args[i] = at
        want = (loss[0] - loss[1]) / (2 * h)
        g = got[name].double().cpu().numpy()
        # the forward's H is a bf16 product (3e-3 of its values); a random way averages the errors,
        # so a share of |g| |way| bounds them
        assert abs((g * way).sum() - want) <= 1e-2 * np.linalg.norm(g) * np.linalg.norm(way)


def test_the_same_bits_twice_and_only_the_outputs_written(lib):
    p, dS = _problem((700, 33, 0, 1500), 200)
    dv = sa_device_inputs(p)
    first, H = _run(lib, p, dS, dv)
    kept = {k: t.clone() for k, t in dv.items()}
    n, guard = int(p.offsets[-1]), 512
    buf = {"dX": torch.full((n * 128 + guard,), 7.0, dtype=torch.bfloat16, device="cuda")}
    for name, size in (("dP", 200 * 128), ("dW_Q", 16384), ("dW_K", 16384), ("dW_V", 16384)):
        buf[name] = torch.full((size + guard,), 7.0, device="cuda")
    size = lib.sa_backward_tokenwise_workspace(p.B, n, 200, 128, lib.SA_BF16)
    ws = torch.full((size + guard,), 0x5A, dtype=torch.uint8, device="cuda")
    out = {name: t[:-guard].view(first[name].shape) for name, t in buf.items()}
    again, _ = _run(lib, p, dS, dv, H=H, out=out, workspace=ws[:size])
    torch.cuda.synchronize()
    for name in NAMES:
        assert again[name].data_ptr() == out[name].data_ptr()
        assert torch.equal(first[name], again[name]), name
        assert bool((buf[name][-guard:] == 7.0).all()), name
    assert bool((ws[size:] == 0x5A).all())
    assert all(torch.equal(kept[k], dv[k]) for k in kept)


def test_captured_and_on_another_stream(lib):
    p, dS = _problem((400, 0, 77), 256)
    dv = sa_device_inputs(p)
    eager, H = _run(lib, p, dS, dv)
    offd = torch.from_numpy(p.offsets).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other, _ = _run(lib, p, dS, dv, H=H, offsets_dev=offd, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held, _ = _run(lib, p, dS, dv, H=H, offsets_dev=offd)
    dS2 = dS.clone()
    dS.mul_(2)                                   # the replay reads the buffers as they are then
    graph.replay()
    torch.cuda.synchronize()
    want, _ = _run(lib, p, dS2 * 2, dv, H=H)
    torch.cuda.synchronize()
    for name in NAMES:
        assert torch.equal(eager[name], other[name]), name
        assert torch.equal(want[name], held[name]), name
    lib.poll_device_status()


def test_two_calls_at_once(lib):
    """Calls on two streams, each with its own buffers, do not disturb one another, nor does it matter
    that a call's offsets are dropped (and their memory handed out again) while its kernels run."""
    problems = [_problem((3000, 500), 256, seed=70), _problem((200, 0, 4100), 512, seed=71)]
    inputs = [(p, dS, sa_device_inputs(p)) for p, dS in problems]
    alone = [_run(lib, p, dS, dv) for p, dS, dv in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in problems]
    got = []
    for _ in range(3):
        for s, (p, dS, dv), (_, H) in zip(streams, inputs, alone):
            got.append(_run(lib, p, dS, dv, H=H, stream=s, offsets_dev=torch.from_numpy(p.offsets).cuda())[0])
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for name in NAMES:
            assert torch.equal(g[name], alone[i % 2][0][name]), name


@pytest.mark.parametrize("users", [1, 60])
def test_h_of_users_without_events_is_not_read(lib, users):
    p, dS = _problem((50, 0, 30) * users, 100)
    clean, H = _run(lib, p, dS)
    H = H.clone()
    H[1::3] = float("nan")
    dS[1::3] = float("nan")
    got, _ = _run(lib, p, dS, H=H)
    torch.cuda.synchronize()
    for name in NAMES:
        assert torch.equal(clean[name], got[name]), name


@pytest.mark.parametrize("users", [1, 60])
def test_a_gradient_that_is_not_finite_stays_with_its_user(lib, users):
    """In dX; the weights' gradients are sums over the users."""
    p, dS = _problem((50, 20, 30) * users, 100)
    clean, H = _run(lib, p, dS)
    dS[1, 7, 3] = float("inf")
    got, _ = _run(lib, p, dS, H=H)
    torch.cuda.synchronize()
    lo, hi = int(p.offsets[1]), int(p.offsets[2])
    assert not bool(got["dX"][lo:hi].isfinite().any())
    assert torch.equal(got["dX"][:lo], clean["dX"][:lo]) and torch.equal(got["dX"][hi:], clean["dX"][hi:])
    for name in ("dP", "dW_Q", "dW_K", "dW_V"):
        assert not bool(got[name].isfinite().all())


def test_the_range_of_gradients(lib):
    """Powers of two times dS scale every gradient, to the bit where nothing is lost below the range."""
    for lengths in ((40, 9), (5, 6) * 80):
        p, dS = _problem(lengths, 128)
        one, H = _run(lib, p, dS)
        for scale in (2.0 ** -40, 2.0 ** 30):
            got, _ = _run(lib, p, dS * scale, H=H)
            torch.cuda.synchronize()
            for name in NAMES:
                assert torch.equal(got[name].double(), one[name].double() * scale), (name, scale)
