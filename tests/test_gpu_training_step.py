"""The training operators together: event ids to updated tables and weights, as a program that
trains the token-wise variant uses them, eagerly and as one captured graph."""
import numpy as np
import pytest
import torch

import oracle
from helpers import compare, tol_for

pytestmark = pytest.mark.gpu

LENS, K, VOCAB, ACTIONS, D, EPS = (700, 0, 1, 1300), 192, 3000, 8, 128, 1e-3


class Program:
    """Tables and weights, their moments, and one training step over a fixed batch."""

    def __init__(self, lib, bits):
        self.lib = lib
        g = torch.Generator().manual_seed(11)
        self.off = np.concatenate([[0], np.cumsum(LENS)]).astype(np.int64)
        self.off_dev = torch.from_numpy(self.off).cuda()
        n = int(self.off[-1])
        self.ids = torch.randint(0, VOCAB, (n,), generator=g).int().cuda()
        self.acts = torch.randint(0, ACTIONS, (n,), generator=g).to(torch.uint8).cuda()
        self.dS = torch.randn(len(LENS), K, D, generator=g).cuda()
        r = lambda *s, std: (torch.randn(*s, generator=g) * std).cuda()  # noqa: E731
        self.w = {"item": r(VOCAB, D, std=0.7), "action": r(ACTIONS, D, std=0.7), "P": r(K, D, std=1.0),
                  **{x: r(D, D, std=D ** -0.5) for x in ("W_Q", "W_K", "W_V")}}
        self.low = {x: self.w[x].bfloat16() for x in ("item", "action")}
        self.g = {x: torch.empty_like(t) for x, t in self.w.items()}
        self.dX = torch.empty(n, D, dtype=torch.bfloat16, device="cuda")
        self.step = torch.zeros(1, dtype=torch.int64, device="cuda")
        entries = []
        for x, t in self.w.items():
            e = {"param": t, "grad": self.g[x], "param_bf16": self.low.get(x), "weight_decay": 0.01}
            for s in ("m", "v"):
                if bits == 8 and x == "item":      # the large table's moments in 8 bits, the rest in 32
                    e[s] = torch.zeros(t.numel(), device="cuda").to(torch.float8_e4m3fn)
                    e[s + "_scale"] = torch.zeros(-(-t.numel() // 128), device="cuda")
                else:
                    e[s] = torch.zeros_like(t)
            entries.append(e)
        self.entries = entries
        self.tensors = lib.AdamWTensors(entries)

    def run(self):
        lib, w, g = self.lib, self.w, self.g
        self.X = lib.sa_gather_events(self.low["item"], self.low["action"], self.ids, self.acts)
        f = lib.sa_forward_tokenwise(self.X, self.off, w["P"], w["W_Q"], w["W_K"], w["W_V"], EPS, want_H=True,
                                     offsets_dev=self.off_dev)
        self.H = f["H"]
        lib.sa_backward_tokenwise(self.X, self.off, w["P"], w["W_Q"], w["W_K"], w["W_V"], EPS, self.H, self.dS,
                                  offsets_dev=self.off_dev,
                                  out={"dX": self.dX, "dP": g["P"], "dW_Q": g["W_Q"], "dW_K": g["W_K"], "dW_V": g["W_V"]})
        lib.sa_gather_events_backward(self.ids, self.acts, self.dX, VOCAB, ACTIONS,
                                      out={"d_item": g["item"], "d_action": g["action"]})
        self.step.add_(1)
        lib.sa_adamw_step(self.tensors, 1e-3, step_dev=self.step)


def test_one_step_against_the_oracle(lib):
    """The gradients of tables and weights against the oracle's chain from the ids; then each
    parameter against the oracle's AdamW on the gradients that the step used."""
    prog = Program(lib, 32)
    w0 = {x: t.double().cpu().numpy() for x, t in prog.w.items()}
    low0 = {x: t.double().cpu().numpy() for x, t in prog.low.items()}
    prog.run()
    torch.cuda.synchronize()
    lib.poll_device_status()
    ids, acts, dS = prog.ids.cpu().numpy(), prog.acts.cpu().numpy(), prog.dS.double().cpu().numpy()
    X = oracle.event_rows(low0["item"], low0["action"], ids, acts)
    ref = oracle.sa_backward_tokenwise(X, prog.off, w0["P"], w0["W_Q"], w0["W_K"], w0["W_V"], EPS, dS)
    tables = oracle.event_table_grads(ids, acts, ref[0], VOCAB, ACTIONS)
    tol = tol_for("bf16")                          # the rows and the forward's H are bf16
    for name, r in zip(("dX", "P", "W_Q", "W_K", "W_V", "item", "action"), (*ref, *tables)):
        compare(name, prog.dX if name == "dX" else prog.g[name], r, dict(max_rel=tol["max_rel"], mean_rel=1e-2))
    for x, t in prog.w.items():
        g = prog.g[x].double().cpu().numpy()
        p, _, _ = oracle.adamw_step(w0[x], g, 0 * g, 0 * g, 1e-3, 0.9, 0.999, 1e-8, 0.01, 1)
        # the first step is lr g / (|g| + eps'): 20 fp32 roundings of at most lr, and p's own
        np.testing.assert_allclose(t.double().cpu().numpy(), p, rtol=4 * 2.0 ** -24, atol=20 * 2.0 ** -24 * 1e-3 * 1.01)
        if x in prog.low:
            assert torch.equal(prog.low[x], t.bfloat16())


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_equal_eager_ones(lib, bits):
    eager, held = Program(lib, bits), Program(lib, bits)
    for _ in range(3):
        eager.run()
    warm = Program(lib, bits)                      # loads every kernel before the capture
    warm.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held.run()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    lib.poll_device_status()
    assert int(held.step) == 3
    for x in eager.w:
        assert torch.equal(eager.w[x], held.w[x]), x
    assert torch.equal(eager.low["item"], held.low["item"])
    moved = (eager.w["P"] - Program(lib, bits).w["P"]).abs().max().item()
    assert 0 < moved < 4e-3                        # three steps of at most about lr each
