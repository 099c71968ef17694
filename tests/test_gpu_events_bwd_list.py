"""The sums of sa_gather_events_backward over a list that its sort did not finish (a barrier that ran
out of time leaves any words in it): an error status, never an access outside a table.  The list
is given through the library's self-test entry; no wait is made to fail."""
import ctypes

import numpy as np
import pytest
import torch

import sketch_attention_b200 as sab

P = 0x10000          # a 16-byte aligned address that is never read


@pytest.mark.parametrize("want,bad", [
    (1, dict(n=0)), (1, dict(vocab=0)), (1, dict(actions=0)), (1, dict(actions=17)), (2, dict(d=12)),
    (2, dict(n=1 << 31)), (2, dict(vocab=1 << 31)), (1, dict(pairs=0)), (1, dict(pairs=P + 8)), (1, dict(dX=0)),
    (1, dict(acts=0)), (1, dict(item=0)), (1, dict(action=P + 4)), (5, dict(ws=0)), (5, dict(ws_bytes=16)),
], ids=str)
def test_the_self_test_refuses(want, bad):
    from sketch_attention_b200 import build
    build.build()
    a = {**dict(n=10, vocab=100, actions=8, d=128, pairs=P, dX=P, acts=P, item=P, action=P, ws=P, ws_bytes=1 << 40), **bad}
    at = ctypes.c_void_p
    got = sab.load().sa_selftest_unsorted_events(at(a["pairs"]), at(a["dX"]), at(a["acts"]), a["n"], a["vocab"], a["actions"],
                                                 a["d"], at(a["item"]), at(a["action"]), at(a["ws"]), a["ws_bytes"], None)
    assert got == want


def _sums(keys, events, acts, dX, vocab, actions):
    """What the header says of such a list, whose equal ids are neighbours."""
    rows = dX[np.where(events < len(dX), events, 0)]
    act = acts[np.where(events < len(dX), events, 0)]
    known = keys < vocab
    item, action = np.zeros((vocab, dX.shape[1])), np.zeros((actions, dX.shape[1]))
    np.add.at(item, keys[known], rows[known])
    there = known & (act < actions)
    np.add.at(action, act[there], rows[there])
    return item, action


# (n, vocab, actions, d): one position, parts of a window of 32, several CTAs, more than a warp's columns
@pytest.mark.gpu
@pytest.mark.parametrize("n,vocab,actions,d", [(1, 5, 1, 128), (33, 5, 3, 128), (5000, 40, 8, 128), (3001, 2000, 16, 200)])
def test_events_of_another_key_with_actions_outside_the_table(lib, n, vocab, actions, d):
    """Keys inside the table beside events whose action (any byte) or number is outside: the
    action sums leave them out.  c fp32 terms in any order: c 2^-24 of their absolute sum."""
    rng = np.random.default_rng(n)
    keys = np.sort(rng.integers(0, vocab + 2, n)).astype(np.int64)
    keys[keys == vocab + 1] = 2 ** 32 - 2
    events = rng.integers(0, 2 * n + 1, n).astype(np.int64)
    events[rng.random(n) < 0.1] = 2 ** 32 - 1
    acts = rng.integers(0, 256, n).astype(np.uint8)
    dX = rng.standard_normal((n, d)).astype(np.float32)
    pairs = torch.from_numpy(np.stack([keys, events], 1).astype(np.uint32).view(np.int32)).cuda()
    got = lib.selftest_unsorted_events(pairs, torch.from_numpy(dX).cuda(), torch.from_numpy(acts).cuda(), vocab, actions)
    torch.cuda.synchronize()
    wide = dX.astype(np.float64)
    for name, ref, size in zip(("d_item", "d_action"), _sums(keys, events, acts, wide, vocab, actions),
                               _sums(keys, events, acts, np.abs(wide), vocab, actions)):
        err = np.abs(got[name].double().cpu().numpy() - ref)
        assert (err <= n * 2.0 ** -24 * size).all(), name


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [3, 70_000, 2 ** 21])
def test_any_words_in_the_list(lib, vocab):
    n = 20_000
    g = torch.Generator().manual_seed(vocab)
    words = torch.randint(-2 ** 31, 2 ** 31, (n, 2), generator=g, dtype=torch.int64).int()
    words[::2, 0] = torch.randint(0, vocab, (n // 2,), generator=g).int()
    words[::3, 0] = words[3, 0]                     # a key in many places
    acts = torch.randint(0, 256, (n,), generator=g).to(torch.uint8).cuda()
    dX = torch.ones(n, 8, device="cuda")
    got = lib.selftest_unsorted_events(words.cuda(), dX, acts, vocab, 16)
    torch.cuda.synchronize()
    lib.poll_device_status()
    # every row counts one: whole numbers, at most as many as there are positions
    for t in got.values():
        assert bool(((t >= 0) & (t <= n) & (t == t.round())).all())
    # and the call itself is as before
    ids = torch.randint(0, vocab, (n,), generator=g).int().cuda()
    item = lib.sa_gather_events_backward(ids, (acts % 16).contiguous(), dX, vocab, 16)["d_item"]
    assert torch.equal(item[:, 0].long(), torch.bincount(ids.long(), minlength=vocab))
