"""The token-wise gradients against central differences of the oracle's forward, along ways that see
mistakes: each gradient itself, where <gradient, way> is its whole norm, and for dX its two terms
A^T dH and dZ^T U (along a random way of N values it would be about 1 / sqrt(N) of the norm).

Tolerances, as shares of the gradient's norm, which bounds an error's part along any way: 1e-5 (1 + std
of the logits) for dP, dW_Q and dW_K, 40 2^-24 for dW_V (see test_gpu_tokenwise_bwd_logits.py); dX has
its own rounding to bf16, two operands' in each of its two products and dH's in G, six of at most
2^-8 / sqrt(3) as norms: 1.5 sqrt(6) 2^-8 / sqrt(3) = 8.3e-3.  With the forward's H, 2e-3 to 5e-3 off:
1e-2.  The difference itself, over h = 1e-4 of a unit way: its third derivative and the losses'
rounding, 1e-6."""
import numpy as np
import pytest
import torch

import oracle
from helpers import dev_f32, sa_device_inputs
from sa_inputs import make_sa_problem

NAMES = ("dX", "dP", "dW_Q", "dW_K", "dW_V")
STD = 1.0
TOL = {"dX": 8.3e-3, "dP": 1e-5 * (1 + STD), "dW_Q": 1e-5 * (1 + STD), "dW_K": 1e-5 * (1 + STD), "dW_V": 40 * 2.0 ** -24}


def _problem():
    p = make_sa_problem((90, 0, 200, 1), 96, 128, "bf16", seed=77, x_kind="gauss", p_scale=128 * STD)
    return p, np.random.default_rng(78).standard_normal((p.B, 96, 128)).astype(np.float32)


def _args(p):
    return [p.x_f64(), *(a.astype(np.float64) for a in (p.P, p.W_Q, p.W_K, p.W_V))]


def _terms(p, dS):
    """A^T dH, and what the oracle's dX has beside it."""
    x, P, WQ, WK, WV = _args(p)
    U, values = P @ WQ @ WK.T / np.sqrt(p.d), np.zeros_like(x)
    for u in range(p.B):
        at = slice(int(p.offsets[u]), int(p.offsets[u + 1]))
        if at.stop > at.start:
            values[at] = oracle._softmax_rows(U @ x[at].T).T @ (dS[u] @ WV.T / (1 + p.eps))
    return values, oracle.sa_backward_tokenwise(x, p.offsets, P, WQ, WK, WV, p.eps, dS)[0] - values


def _gap(p, dS, i, g, way=None):
    """|<g, way> - d loss / d way| / |g|, way a unit vector (along g by default) in argument i."""
    args, h = _args(p), 1e-4
    way = g if way is None else way
    way, at = way / np.linalg.norm(way), args[i]
    loss = []
    for s in (h, -h):
        args[i] = at + s * way
        loss.append((oracle.sa_forward_tokenwise(args[0], p.offsets, *args[1:], p.eps)[0] * dS).sum())
    return abs((g * way).sum() - (loss[0] - loss[1]) / (2 * h)) / np.linalg.norm(g)


def test_what_the_comparison_sees():
    """The oracle's gradients agree; halved, negated, unrelated or incomplete ones do not."""
    p, dS = _problem()
    ref = oracle.sa_backward_tokenwise(_args(p)[0], p.offsets, *_args(p)[1:], p.eps, dS)
    rng = np.random.default_rng(1)
    for i, g in enumerate(ref):
        assert _gap(p, dS, i, g) <= 1e-6, NAMES[i]
        other = rng.standard_normal(g.shape)
        for wrong in (0.5 * g, -g, 1.03 * g, other * np.linalg.norm(g) / np.linalg.norm(other)):
            assert _gap(p, dS, i, wrong) > 2e-2, NAMES[i]
    values, logits = _terms(p, dS)
    for way, wrong in ((values, logits), (logits, values), (logits, values + 0.5 * logits), (logits, values - logits)):
        assert _gap(p, dS, 0, ref[0], way) <= 1e-6
        assert _gap(p, dS, 0, wrong, way) > 2e-2


@pytest.mark.gpu
@pytest.mark.parametrize("exact", [True, False], ids=["exact_H", "forward_H"])
def test_along_the_gradients(lib, exact):
    p, dS = _problem()
    dv = sa_device_inputs(p)
    W = (dv["P"], dv["W_Q"], dv["W_K"], dv["W_V"])
    if exact:
        H = dev_f32(oracle.sa_forward_tokenwise(_args(p)[0], p.offsets, *_args(p)[1:], p.eps)[2].astype(np.float32))
    else:
        H = lib.sa_forward_tokenwise(dv["X"], p.offsets, *W, p.eps, want_H=True)["H"]
    got = lib.sa_backward_tokenwise(dv["X"], p.offsets, *W, p.eps, H, dev_f32(dS))
    torch.cuda.synchronize()
    lib.poll_device_status()
    for i, name in enumerate(NAMES):
        g, tol = got[name].double().cpu().numpy(), (TOL[name] if exact else max(TOL[name], 1e-2)) + 1e-6
        for way in (g, *(_terms(p, dS) if name == "dX" else ())):
            assert _gap(p, dS, i, g, way) <= tol, name
