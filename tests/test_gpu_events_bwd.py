"""GPU checks of sa_gather_events_backward against the fp64 oracle: the sum of c fp32 terms
in any order is off by at most c 2^-24 of the sum of their absolute values."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


def _inputs(n, vocab, actions, d, dtype, seed, ids=None):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, vocab, (n,), generator=g) if ids is None else ids
    acts = torch.randint(0, actions, (n,), generator=g)
    return ids.int().cuda(), acts.to(torch.uint8).cuda(), torch.randn(n, d, generator=g).to(dtype).cuda()


def _check(lib, ids, acts, dX, vocab, actions, **kw):
    got = lib.sa_gather_events_backward(ids, acts, dX, vocab, actions, **kw)
    torch.cuda.synchronize()
    i, a, x = ids.cpu().numpy(), acts.cpu().numpy(), dX.double().cpu().numpy()
    ones = np.ones((len(i), 1))
    for name, ref, size, cnt in zip(("d_item", "d_action"), oracle.event_table_grads(i, a, x, vocab, actions),
                                    oracle.event_table_grads(i, a, np.abs(x), vocab, actions),
                                    oracle.event_table_grads(i, a, ones, vocab, actions)):
        err = np.abs(got[name].double().cpu().numpy() - ref)
        assert err.shape == ref.shape
        assert (err <= cnt * 2.0 ** -24 * size).all(), (name, err.max())
    return got


# n, vocab, actions, d: one event; sizes around a warp, a list piece (256), a CTA's share, and what one CTA
# or 64 sort; one-row
# tables; more and fewer rows than a CTA takes; widths below, at and above a warp's 128 columns
CASES = [(1, 1, 1, 128), (31, 5, 2, 128), (257, 7, 8, 128), (1000, 1000, 3, 128), (1025, 200_000, 8, 128),
         (4097, 1023, 8, 128), (20_000, 1024, 16, 128), (50_001, 70_000, 8, 128), (3000, 300, 256, 128),
         (4096, 5000, 8, 128), (65_536, 9000, 4, 64), (65_537, 9000, 4, 64),
         (700, 90, 9, 8), (700, 90, 9, 64), (700, 90, 9, 200), (5000, 3, 2, 264)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,vocab,actions,d", CASES)
def test_against_the_oracle(lib, n, vocab, actions, d, dtype):
    _check(lib, *_inputs(n, vocab, actions, d, dtype, n + d), vocab, actions)
    lib.poll_device_status()


@pytest.mark.parametrize("n,shares", [(70_000, (1.0,)), (70_001, (0.5, 0.5)), (40_000, (0.9, 0.05)), (600, (0.5,)),
                                      (33, (1.0,)), (512, (1.0,)), (768, (0.33, 0.34))])
def test_popular_items(lib, n, shares):
    """Items with long runs (inside, at and across the 256-event pieces) beside rare ones."""
    vocab = 5000
    g = torch.Generator().manual_seed(n)
    ids = torch.randint(0, vocab, (n,), generator=g)
    at = 0
    for k, s in enumerate(shares):
        ids[at:at + int(n * s)] = 17 + 64 * k
        at += int(n * s)
    ids = ids[torch.randperm(n, generator=g)]
    _check(lib, *_inputs(n, vocab, 8, 128, torch.bfloat16, 3, ids=ids), vocab, 8)


def test_events_outside_the_tables_count_for_neither(lib):
    ids, acts, dX = _inputs(3000, 500, 8, 128, torch.bfloat16, 4)
    ids[7], ids[8], ids[9] = -1, 500, 2 ** 31 - 1
    ids[10] = -2 ** 31
    acts[11], acts[12] = 8, 255
    dX[7:13] = float("nan")                       # their gradient must not reach any sum
    _check_nan = lib.sa_gather_events_backward(ids, acts, dX, 500, 8)
    torch.cuda.synchronize()
    assert all(bool(t.isfinite().all()) for t in _check_nan.values())
    with pytest.raises(lib.SAError):
        lib.poll_device_status()
    lib.poll_device_status()
    dX[7:13] = 1.0
    _check(lib, ids, acts, dX, 500, 8)
    for only in ("want_item", "want_action"):     # each table alone reports them too
        lib.sa_gather_events_backward(ids, acts, dX, 500, 8, **{only: False})
        with pytest.raises(lib.SAError):
            lib.poll_device_status()


def test_no_events_and_one_table(lib):
    ids, acts, dX = _inputs(0, 40, 3, 128, torch.float32, 5)
    got = lib.sa_gather_events_backward(ids, acts, dX, 40, 3)
    assert all(torch.count_nonzero(t) == 0 for t in got.values())
    ids, acts, dX = _inputs(900, 40, 3, 128, torch.float32, 6)
    both = lib.sa_gather_events_backward(ids, acts, dX, 40, 3)
    item = lib.sa_gather_events_backward(ids, acts, dX, 40, 3, want_action=False)
    action = lib.sa_gather_events_backward(ids, acts, dX, 40, 3, want_item=False)
    assert set(item) == {"d_item"} and set(action) == {"d_action"}
    assert torch.equal(item["d_item"], both["d_item"])
    # alone, the action sums run in the events' order, not the items': 2 c 2^-24 of the absolute sums
    size = oracle.event_table_grads(ids.cpu().numpy(), acts.cpu().numpy(), dX.abs().cpu().numpy(), 40, 3)[1]
    err = (action["d_action"] - both["d_action"]).abs().double().cpu().numpy()
    assert (err <= 2 * 900 * 2.0 ** -24 * size).all()


def test_the_same_bits_twice_captured_and_only_the_outputs_written(lib):
    n, vocab = 30_000, 2000
    g = torch.Generator().manual_seed(1)
    hot = torch.where(torch.rand(n, generator=g) < 0.3, torch.full((n,), 5), torch.randint(0, vocab, (n,), generator=g))
    ids, acts, dX = _inputs(n, vocab, 8, 128, torch.bfloat16, 7, ids=hot)
    first = lib.sa_gather_events_backward(ids, acts, dX, vocab, 8)
    size, guard = lib.sa_gather_events_backward_workspace(n, vocab, 8, 128), 256
    ws = torch.full((size + guard,), 0x5A, dtype=torch.uint8, device="cuda")
    item = torch.full((vocab * 128 + guard,), 7.0, device="cuda")
    action = torch.full((8 * 128 + guard,), 7.0, device="cuda")
    out = {"d_item": item[:-guard].view(vocab, 128), "d_action": action[:-guard].view(8, 128)}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.sa_gather_events_backward(ids, acts, dX, vocab, 8, out=out, workspace=ws[:size])
    for _ in range(2):
        graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = lib.sa_gather_events_backward(ids, acts, dX, vocab, 8, stream=side)
    torch.cuda.synchronize()
    for name in first:
        assert torch.equal(first[name], out[name]) and torch.equal(first[name], other[name])
    assert bool((item[-guard:] == 7.0).all()) and bool((action[-guard:] == 7.0).all())
    assert bool((ws[size:] == 0x5A).all())


def test_two_calls_at_once(lib):
    a = _inputs(60_000, 5000, 8, 128, torch.bfloat16, 8)
    b = _inputs(90_000, 700, 16, 128, torch.float32, 9)
    alone = [lib.sa_gather_events_backward(*a, 5000, 8), lib.sa_gather_events_backward(*b, 700, 16)]
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        got.append(lib.sa_gather_events_backward(*a, 5000, 8, stream=s))
        got.append(lib.sa_gather_events_backward(*b, 700, 16, stream=t))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(g[k], alone[i % 2][k]) for k in g)


def test_a_gradient_that_is_not_finite_stays_in_its_rows(lib):
    ids, acts, dX = _inputs(5000, 300, 8, 128, torch.float32, 10)
    clean = lib.sa_gather_events_backward(ids, acts, dX, 300, 8)
    dX[1234] = float("nan")
    got = lib.sa_gather_events_backward(ids, acts, dX, 300, 8)
    torch.cuda.synchronize()
    for name, row in (("d_item", int(ids[1234])), ("d_action", int(acts[1234]))):
        assert bool(got[name][row].isnan().all())
        keep = torch.arange(len(got[name]), device="cuda") != row
        assert torch.equal(got[name][keep], clean[name][keep])


def test_the_default_dtype_does_not_matter(lib):
    x = _inputs(3000, 200, 4, 64, torch.bfloat16, 11)
    want = lib.sa_gather_events_backward(*x, 200, 4)
    torch.set_default_dtype(torch.float64)
    try:
        got = lib.sa_gather_events_backward(*x, 200, 4)
    finally:
        torch.set_default_dtype(torch.float32)
    assert all(got[k].dtype == torch.float32 and torch.equal(got[k], want[k]) for k in want)


def test_a_large_vocabulary(lib):
    """More zeros than the sort takes time for: rows without events are zero, the others their sums."""
    n, vocab = 150_000, 600_000
    ids, acts, dX = _inputs(n, vocab, 8, 128, torch.bfloat16, 12)
    out = {"d_item": torch.full((vocab, 128), 3.0, device="cuda")}
    got = lib.sa_gather_events_backward(ids, acts, dX, vocab, 8, out=out)
    ref = torch.zeros(vocab, 128, dtype=torch.float64, device="cuda").index_add_(0, ids.long(), dX.double())
    size = torch.zeros(vocab, 128, dtype=torch.float64, device="cuda").index_add_(0, ids.long(), dX.double().abs())
    count = torch.bincount(ids.long(), minlength=vocab)[:, None]
    assert bool(((got["d_item"].double() - ref).abs() <= count * 2.0 ** -24 * size).all())


def test_captured_on_an_explicit_stream(lib):
    x = _inputs(20_000, 900, 4, 128, torch.bfloat16, 13)
    want = lib.sa_gather_events_backward(*x, 900, 4)
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    temporary = [t.clone() for t in x]
    with torch.cuda.graph(graph, stream=stream):
        lib.sa_gather_events_backward(*temporary, 900, 4, stream=stream)   # dropped inside the capture
        got = lib.sa_gather_events_backward(*x, 900, 4, stream=stream)
    kept = temporary
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    del kept, temporary, graph
    torch.cuda.synchronize()
