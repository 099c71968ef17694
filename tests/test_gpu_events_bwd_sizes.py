"""sa_gather_events_backward where its sort takes other paths than at small sizes: three and four
passes (an id has more than 20 bits from 2^20 items on, more than 30 from 2^30), parts of a warp
that it reads again (more than 384 events each: from 909,313 events on 148 SMs), windows of more than 32
positions (from 113,665 events) and runs over many of them.  The sum of c fp32 terms in any order
is off by at most c 2^-24 of the sum of their absolute values."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _inputs(n, vocab, actions, d, dtype, seed, popular=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda high: torch.randint(0, high, (n,), generator=g, device="cuda")  # noqa: E731
    ids = r(vocab)
    ids[torch.rand(n, generator=g, device="cuda") < popular] = vocab // 3
    ids[:2] = torch.tensor([0, vocab - 1], device="cuda")[:n]          # the first and the last row
    return ids.int(), r(actions).to(torch.uint8), torch.randn(n, d, generator=g, device="cuda").to(dtype)


def _check_rows(rows, got, index, dX):
    """got[rows of index] against the sums of dX over index."""
    wide, one = dX.double(), torch.ones(len(dX), 1, dtype=torch.float64, device="cuda")
    add = lambda x: torch.zeros(rows, x.shape[1], dtype=torch.float64, device="cuda").index_add_(0, index, x)  # noqa: E731
    err = (got.double() - add(wide)).abs()
    assert bool((err <= add(one) * 2.0 ** -24 * add(wide.abs())).all()), float(err.max())


def _check(lib, n, vocab, actions, d, dtype, seed, popular=0.0):
    ids, acts, dX = _inputs(n, vocab, actions, d, dtype, seed, popular)
    got = lib.sa_gather_events_backward(ids, acts, dX, vocab, actions)
    again = lib.sa_gather_events_backward(ids, acts, dX, vocab, actions)
    torch.cuda.synchronize()
    lib.poll_device_status()
    _check_rows(vocab, got["d_item"], ids.long(), dX)
    _check_rows(actions, got["d_action"], acts.long(), dX)
    assert all(torch.equal(got[k], again[k]) for k in got)


# one CTA, up to 64 and more of them, for each number of items around the borders of two and three passes
@pytest.mark.parametrize("n", [1, 2, 700, 4096, 4097, 20_000, 70_000, 200_000])
@pytest.mark.parametrize("vocab", [2 ** 20 - 1, 2 ** 20, 2 ** 20 + 1, 2 ** 21 + 3])
def test_ids_of_more_than_20_bits(lib, n, vocab):
    _check(lib, n, vocab, 5, 8, torch.bfloat16, n)


@pytest.mark.parametrize("n", [113_664, 113_665, 909_312, 909_313, 1_000_001, 3_000_000])
@pytest.mark.parametrize("vocab,actions,popular", [(5000, 8, 0.3), (2 ** 20, 16, 0.01), (7, 40, 0.0)])
def test_long_parts_windows_and_runs(lib, n, vocab, actions, popular):
    _check(lib, n, vocab, actions, 8, torch.bfloat16, n, popular)


def test_long_parts_of_wide_fp32_rows(lib):
    _check(lib, 1_000_001, 30_000, 8, 136, torch.float32, 3, 0.1)


def test_one_item_of_many_events(lib):
    """A run over every window."""
    _check(lib, 1_500_000, 3, 2, 8, torch.float32, 4, 1.0)


def test_ids_of_more_than_30_bits(lib):
    """Four passes.  The table takes 34 GB; only the rows with events can be other than zero."""
    vocab, d, n = 2 ** 30, 8, 50_000
    if torch.cuda.mem_get_info()[0] < 3 * vocab * d * 4 // 2:
        pytest.skip("needs 52 GB of free memory")
    ids, acts, dX = _inputs(n, vocab, 3, d, torch.float32, 5, 0.01)
    ids[2:5] = torch.tensor([-1, 2 ** 30, 2 ** 31 - 1], device="cuda", dtype=torch.int32)
    dX[2:5] = float("nan")                             # outside the table: for neither sum
    got = lib.sa_gather_events_backward(ids, acts, dX, vocab, 3)
    torch.cuda.synchronize()
    with pytest.raises(lib.SAError):
        lib.poll_device_status()
    lib.poll_device_status()
    keep = torch.arange(n, device="cuda")
    keep = keep[(keep < 2) | (keep > 4)]
    rows, index = torch.unique(ids[keep].long(), return_inverse=True)
    _check_rows(len(rows), got["d_item"][rows], index, dX[keep])
    _check_rows(3, got["d_action"], acts[keep].long(), dX[keep])
    got["d_item"][rows] = 0
    assert all(float(part.abs().max()) == 0.0 for part in got["d_item"].split(2 ** 24))
    del got
    torch.cuda.empty_cache()
