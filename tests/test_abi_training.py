"""Refusals and workspace queries of the training entry points (token-wise backward,
event-table gradients, AdamW): status codes before any GPU work, so these run without one."""
import ctypes

import numpy as np
import pytest
import torch

import sketch_attention_b200 as sab

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5


@pytest.fixture(scope="module")
def clib():
    from sketch_attention_b200 import build
    build.build()
    return sab.load()


def _at(addr):
    return ctypes.c_void_p(addr)


P = 0x10000          # a 16-byte aligned address that is never read


def _tokenwise(lib, offsets=(0, 5), k=64, d=128, dtype=sab.SA_BF16, eps=1e-6, X=P, H=P, dX=2 * P, dW=P, ws=P,
               ws_bytes=1 << 40):
    off = np.asarray(offsets, np.int64)
    return lib.sa_backward_tokenwise(_at(X), dtype, off.ctypes.data_as(ctypes.c_void_p), _at(P), len(off) - 1, k, d,
                                     _at(P), _at(P), _at(P), _at(P), eps, _at(H), _at(P), _at(dX), _at(P), _at(P),
                                     _at(P), _at(dW), _at(ws), ws_bytes, None)


@pytest.mark.parametrize("want,bad", [
    (INVALID, dict(offsets=(0, 5, 3))), (INVALID, dict(offsets=(1, 5))), (UNSUPPORTED, dict(k=0)),
    (UNSUPPORTED, dict(k=4097)), (UNSUPPORTED, dict(d=64)), (UNSUPPORTED, dict(dtype=sab.SA_F32)),
    (INVALID, dict(dtype=7)), (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))), (INVALID, dict(X=0)),
    (INVALID, dict(X=P + 4)), (INVALID, dict(H=0)), (INVALID, dict(dX=P + 8)), (INVALID, dict(dX=P)),
    (INVALID, dict(dW=0)), (WORKSPACE, dict(ws=0)), (WORKSPACE, dict(ws_bytes=64)), (INVALID, dict(ws=P + 4)),
    (UNSUPPORTED, dict(offsets=(0, (1 << 31) - 1))),
], ids=str)
def test_tokenwise_backward_refuses(clib, want, bad):
    assert _tokenwise(clib, **bad) == want
    assert clib.sa_last_error()


def test_tokenwise_backward_refuses_too_many_rows(clib):
    assert _tokenwise(clib, offsets=(0,) * (1 << 18), k=4096) == UNSUPPORTED
    assert b"2^30" in clib.sa_last_error()


def test_tokenwise_backward_workspace(clib):
    ws = sab.sa_backward_tokenwise_workspace
    assert ws(2, 1000, 200, 128, sab.SA_BF16) >= 2 * 256 * 128 * 2 * 2      # dH as two bf16 parts, k rounded up
    assert ws(4, 1000, 200, 128, sab.SA_BF16) > ws(2, 1000, 200, 128, sab.SA_BF16)
    for bad in ((0, 10, 64, 128, sab.SA_BF16), (1, -1, 64, 128, sab.SA_BF16), (1, 10, 4097, 128, sab.SA_BF16),
                (1, 10, 64, 64, sab.SA_BF16), (1, 10, 64, 128, sab.SA_F32)):
        assert ws(*bad) == 0


def _events(lib, n=10, vocab=100, actions=8, d=128, dtype=sab.SA_BF16, ids=P, acts=P, dX=P, item=P, action=P, ws=P,
            ws_bytes=1 << 40):
    return lib.sa_gather_events_backward(_at(ids), _at(acts), n, _at(dX), dtype, vocab, actions, d, _at(item),
                                         _at(action), _at(ws), ws_bytes, None)


@pytest.mark.parametrize("want,bad", [
    (INVALID, dict(n=-1)), (INVALID, dict(vocab=0)), (INVALID, dict(actions=0)), (INVALID, dict(actions=257)),
    (INVALID, dict(dtype=3)), (UNSUPPORTED, dict(d=12)), (UNSUPPORTED, dict(d=0)), (UNSUPPORTED, dict(n=1 << 31)),
    (UNSUPPORTED, dict(vocab=1 << 31)), (INVALID, dict(ids=0)), (INVALID, dict(ids=P + 2)), (INVALID, dict(acts=0)),
    (INVALID, dict(dX=0)), (INVALID, dict(dX=P + 4)), (INVALID, dict(item=P + 4)), (INVALID, dict(action=P + 4)),
    (WORKSPACE, dict(ws=0)), (WORKSPACE, dict(ws_bytes=16)), (INVALID, dict(ws=P + 4)),
], ids=str)
def test_event_gradients_refuse(clib, want, bad):
    assert _events(clib, **bad) == want
    assert clib.sa_last_error()


def test_event_gradients_workspace(clib):
    ws = sab.sa_gather_events_backward_workspace
    assert ws(1000, 100, 8, 128) >= 4 * 1000 * 4                             # two lists of (id, event)
    for bad in ((-1, 100, 8, 128), (10, 0, 8, 128), (10, 100, 300, 128), (10, 100, 8, 20)):
        assert ws(*bad) == 0


def _adamw(lib, n_tensors=1, config=True, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, step_dev=0, lr_dev=0,
           grad_scale=0, **tensor):
    t = sab.AdamWTensorC(param=P, grad=P, grad_dtype=sab.SA_F32, state=sab.SA_STATE_F32, m=P, v=P, n=8)
    for k, x in tensor.items():
        setattr(t, k, x)
    arr = (sab.AdamWTensorC * 1)(t)
    cfg = sab.AdamWConfigC(lr, beta1, beta2, eps, step, step_dev, lr_dev, grad_scale)
    return lib.sa_adamw_step(arr, n_tensors, ctypes.byref(cfg) if config else None, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad", [
    dict(n_tensors=-1), dict(config=False), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=NAN),
    dict(eps=-1.0), dict(eps=INF), dict(lr=NAN), dict(step=0), dict(step_dev=P + 4), dict(lr_dev=P + 2),
    dict(grad_scale=P + 1), dict(n=-1), dict(grad_dtype=9), dict(state=2), dict(weight_decay=NAN), dict(param=0),
    dict(param=P + 4), dict(grad=0), dict(grad=P + 2), dict(m=0), dict(v=P + 8), dict(param_bf16=P + 2),
    dict(state=sab.SA_STATE_8BIT), dict(state=sab.SA_STATE_8BIT, m_scale=P, v_scale=P + 2),
], ids=str)
def test_adamw_refuses(clib, bad):
    assert _adamw(clib, **bad) == INVALID
    assert clib.sa_last_error()


def test_adamw_without_values_does_nothing(clib):
    assert _adamw(clib, n_tensors=0) == OK
    assert _adamw(clib, n=0, param=0, grad=0, m=0, v=0) == OK


def test_binding_refuses_what_the_library_cannot_see():
    """Host tensors, wrong types and wrong sizes raise before the library is called."""
    f = torch.zeros
    x, p, w = f(4, 128, dtype=torch.bfloat16), f(3, 128), f(128, 128)
    with pytest.raises(ValueError):
        sab.sa_backward_tokenwise(x, [0, 4], p, w, w, w, 1e-6, f(1, 3, 128), f(1, 3, 128))
    with pytest.raises(ValueError):
        sab.sa_gather_events_backward(f(4, dtype=torch.int32), f(4, dtype=torch.uint8), x, 10, 8)
    with pytest.raises(ValueError):
        sab.AdamWTensors([dict(param=f(8), grad=f(8), m=f(8), v=f(8))])
