"""sa_backward_tokenwise where the softmax is sharp (logits of a standard deviation from 1/4 to 8), with
an H of fp32 accuracy and with the one that sa_forward_tokenwise gives.

Tolerances, as norms over a gradient.  A rounding to nearest is off by at most half a step (bf16 2^-8
relative); over many values its root mean square is at most 2^-8 / sqrt(3).
* dP, dW_Q, dW_K: U, dH and dZ are bf16 pairs, 2^-17 relative at most, so 2^-17 / sqrt(3) = 4.4e-6 each
  as a norm, three of them 7.6e-6; an error of a logit of a standard deviation s is a relative error of
  its A, s 4.4e-6, and the same of the row's sum, 6.2e-6 s; the tensor core's truncation adds 1e-6.
  1e-5 (1 + s) is above that sum for every s.
* dW_V is an fp32 product over the rows: 40 2^-24.
* dX: its own rounding; in A^T dH and dZ^T U both operands bf16, and dH hi in G - c.  The mean
  squares of those add up, value by value; 1.5 times their root covers the scatter.
An H that is off by e changes c by dH . e, hence E by -(dH . e) A X per user and prototype, and dW_V
by the sum of i e^T dS: that is exact, and the test adds it to the oracle's gradients."""
import math

import numpy as np
import pytest
import torch

import oracle
from helpers import dev_f32, sa_device_inputs
from sa_inputs import make_sa_problem

NAMES = ("dX", "dP", "dW_Q", "dW_K", "dW_V")
STDS = (0.25, 1.0, 2.0, 4.0, 8.0)


def _problem(lengths, k, std, seed=90):
    """Logits of that standard deviation (the inputs' own scale gives 1/128)."""
    p = make_sa_problem(lengths, k, 128, "bf16", seed=seed + k, x_kind="gauss", p_scale=128 * std)
    dS = np.random.default_rng(seed).standard_normal((p.B, k, 128)).astype(np.float32)
    return p, dS


def _weights(p):
    return [a.astype(np.float64) for a in (p.P, p.W_Q, p.W_K, p.W_V)]


def _off_by(p, dS, e):
    """What an H off by e [B, k, d] adds to (dP, dW_Q, dW_K, dW_V)."""
    P, WQ, WK, WV = _weights(p)
    x, root = p.x_f64(), math.sqrt(p.d)
    H = oracle.sa_forward_tokenwise(x, p.offsets, P, WQ, WK, WV, p.eps)[2]
    dE, dWV = np.zeros_like(P), np.zeros_like(WV)
    for u in range(p.B):
        if p.offsets[u + 1] - p.offsets[u] == 0:
            continue
        if p.offsets[u + 1] - p.offsets[u] > 1:
            dE -= ((dS[u] @ WV.T / (1 + p.eps)) * e[u]).sum(1, keepdims=True) * H[u]
        dWV += e[u].T @ dS[u] / (1 + p.eps)
    return dE @ WK @ WQ.T / root, P.T @ dE @ WK / root, dE.T @ P @ WQ / root, dWV


def test_the_effect_of_h_on_the_oracle():
    p, dS = _problem((40, 1, 0, 7), 9, 2.0)
    args = (p.x_f64(), p.offsets, *_weights(p), p.eps)
    H = oracle.sa_forward_tokenwise(*args)[2]
    e = 1e-2 * np.random.default_rng(1).standard_normal(H.shape)
    e[2] = 0
    true, off = oracle.sa_backward_tokenwise(*args, dS), oracle.sa_backward_tokenwise(*args, dS, H=H + e)
    for a, b, more in zip(off[1:], true[1:], _off_by(p, dS, e)):
        np.testing.assert_allclose(a, b + more, rtol=1e-9, atol=1e-9 * np.abs(b).max())


def _dx_error(p, dS, H):
    """The root mean square bound of dX's roundings, as a norm."""
    P, WQ, WK, WV = _weights(p)
    x, one = p.x_f64(), 2.0 ** -16 / 3                   # the mean square of one bf16 rounding
    U = P @ WQ @ WK.T / math.sqrt(p.d)
    total = 0.0
    for u in range(p.B):
        xu = x[int(p.offsets[u]):int(p.offsets[u + 1])]
        if len(xu) == 0:
            continue
        A, dH = oracle._softmax_rows(U @ xu.T), dS[u] @ WV.T / (1 + p.eps)
        dZ = A * (dH @ xu.T - (dH * H[u]).sum(1, keepdims=True))
        # sum_c dH_c^2 (x - H)_c^2 of every (prototype, event): G - c of a rounded dH
        rest = (dH ** 2) @ (xu ** 2).T - 2 * (dH ** 2 * H[u]) @ xu.T + (dH ** 2 * H[u] ** 2).sum(1, keepdims=True)
        total += one * ((A.T @ dH + dZ.T @ U) ** 2).sum()
        total += one * (2 * ((A ** 2).T @ dH ** 2).sum() + 2 * ((dZ ** 2).T @ U ** 2).sum())
        total += one * ((A ** 2 * np.maximum(rest, 0)).T @ U ** 2).sum()
    return 1.5 * math.sqrt(total)


def _far(a, b):
    return float(np.linalg.norm(a - b))


CASES = [((2500, 777), 200), ((5000,), 64), ((300, 0, 1, 2, 129), 130), ((40,) * 30, 300), ((1024, 1500), 1024)]


@pytest.mark.gpu
@pytest.mark.parametrize("std", STDS)
@pytest.mark.parametrize("lengths,k", CASES, ids=[f"n{'-'.join(map(str, c[0][:4]))}_k{c[1]}" for c in CASES])
def test_sharp_softmaxes(lib, lengths, k, std):
    p, dS = _problem(lengths, k, std)
    dv, g = sa_device_inputs(p), dev_f32(dS)
    weights = (dv["P"], dv["W_Q"], dv["W_K"], dv["W_V"])
    args = (p.x_f64(), p.offsets, *_weights(p), p.eps)
    H = oracle.sa_forward_tokenwise(*args)[2]
    true = oracle.sa_backward_tokenwise(*args, dS)
    exact = lib.sa_backward_tokenwise(dv["X"], p.offsets, *weights, p.eps, dev_f32(H.astype(np.float32)), g)
    held = lib.sa_forward_tokenwise(dv["X"], p.offsets, *weights, p.eps, want_H=True)["H"]
    pair = lib.sa_backward_tokenwise(dv["X"], p.offsets, *weights, p.eps, held, g)
    torch.cuda.synchronize()
    lib.poll_device_status()
    e = held.double().cpu().numpy() - H
    e[np.diff(p.offsets) == 0] = 0
    more = _off_by(p, dS, e)
    of = lambda d, name: d[name].double().cpu().numpy()  # noqa: E731
    for i, name in enumerate(NAMES[1:]):
        tol = 1e-5 * (1 + std) if name != "dW_V" else 40 * 2.0 ** -24
        size = np.linalg.norm(true[i + 1])
        assert _far(of(exact, name), true[i + 1]) <= tol * size, name
        # the pair is off by what its H makes of it, and by no more
        assert _far(of(pair, name), true[i + 1] + more[i]) <= tol * (size + np.linalg.norm(more[i])), name
    assert _far(of(exact, "dX"), true[0]) <= _dx_error(p, dS, H)
    off = oracle.sa_backward_tokenwise(*args, dS, H=held.double().cpu().numpy())[0]
    assert _far(of(pair, "dX"), off) <= _dx_error(p, dS, H)
