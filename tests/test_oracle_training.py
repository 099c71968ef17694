"""Pins of the oracle's training operators (no GPU): the token-wise backward against
central differences of the token-wise forward, the event tables' gradients as the
adjoint of the event rows, and AdamW against torch's own optimiser."""
import numpy as np
import pytest
import torch

import oracle


def _problem(seed, lengths=(4, 0, 1, 6), k=5, d=8):
    rng = np.random.default_rng(seed)
    off = np.concatenate([[0], np.cumsum(lengths)])
    w = lambda *s: rng.standard_normal(s) / np.sqrt(s[0])
    return (rng.standard_normal((off[-1], d)), off, rng.standard_normal((k, d)), w(d, d), w(d, d), w(d, d), 1e-3,
            rng.standard_normal((len(lengths), k, d)))


@pytest.mark.parametrize("which", range(5), ids=["X", "P", "W_Q", "W_K", "W_V"])
def test_tokenwise_backward_against_differences(which):
    X, off, P, WQ, WK, WV, eps, dS = _problem(3)
    args = [X, P, WQ, WK, WV]

    def loss():
        return (oracle.sa_forward_tokenwise(args[0], off, *args[1:], eps)[0] * dS).sum()

    grad = oracle.sa_backward_tokenwise(X, off, P, WQ, WK, WV, eps, dS)[which]
    rng = np.random.default_rng(4)
    for _ in range(3):
        way = rng.standard_normal(args[which].shape)
        h, at = 1e-5, args[which]
        args[which] = at + h * way
        up = loss()
        args[which] = at - h * way
        down = loss()
        args[which] = at
        # central differences: O(h^2) + the rounding of the losses, 1e-16 |L| / h
        np.testing.assert_allclose((grad * way).sum(), (up - down) / (2 * h), rtol=1e-6, atol=1e-7)


def test_tokenwise_backward_takes_the_forwards_h():
    X, off, P, WQ, WK, WV, eps, dS = _problem(5)
    H = oracle.sa_forward_tokenwise(X, off, P, WQ, WK, WV, eps)[2]
    for a, b in zip(oracle.sa_backward_tokenwise(X, off, P, WQ, WK, WV, eps, dS),
                    oracle.sa_backward_tokenwise(X, off, P, WQ, WK, WV, eps, dS, H=H)):
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-12)


def test_event_table_grads_are_the_adjoint_of_the_rows():
    """<rows(item, action), dX> = <item, d_item> + <action, d_action>, with repeated ids."""
    rng = np.random.default_rng(6)
    item, action = rng.standard_normal((9, 4)), rng.standard_normal((3, 4))
    ids, acts = rng.integers(0, 9, 40), rng.integers(0, 3, 40)
    dX = rng.standard_normal((40, 4))
    gi, ga = oracle.event_table_grads(ids, acts, dX, 9, 3)
    np.testing.assert_allclose((oracle.event_rows(item, action, ids, acts) * dX).sum(),
                               (item * gi).sum() + (action * ga).sum(), rtol=1e-12)


def test_event_table_grads_leave_out_events_outside_the_tables():
    gi, ga = oracle.event_table_grads([0, -1, 4, 2, 1], [0, 0, 0, 2, 1], np.ones((5, 2)), 4, 2)
    np.testing.assert_array_equal(gi[:, 0], [1, 1, 0, 0])
    np.testing.assert_array_equal(ga[:, 0], [1, 1])


def test_adamw_step_is_torchs():
    rng = np.random.default_rng(7)
    p0 = rng.standard_normal(50)
    t = torch.tensor(p0, requires_grad=True)
    opt = torch.optim.AdamW([t], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    p, m, v = p0, np.zeros(50), np.zeros(50)
    for step in range(1, 5):
        g = rng.standard_normal(50)
        t.grad = torch.tensor(g)
        opt.step()
        p, m, v = oracle.adamw_step(p, g, m, v, 1e-2, 0.8, 0.95, 1e-6, 0.1, step)
        np.testing.assert_allclose(p, t.detach().numpy(), rtol=1e-12, atol=1e-14)
