"""AdamWTensors refuses arrays that share memory where a step writes them.  The list is only
described here: no step runs."""
import pytest
import torch

import sketch_attention_b200 as sab

N = 512


def _span(begin, end, written=True):
    return (begin, end, "param" if written else "grad")


def test_spans():
    """The rule alone, over intervals (no GPU)."""
    apart = [_span(0, 4), _span(4, 8), _span(20, 30), _span(8, 20, False)]
    sab._refuse_overlaps(apart)
    sab._refuse_overlaps([])
    sab._refuse_overlaps([_span(0, 9, False), _span(0, 9, False), _span(3, 30, False), _span(30, 31)])
    for more in (_span(0, 4), _span(3, 5), _span(29, 40), _span(0, 100), _span(21, 22), _span(21, 22, False),
                 _span(0, 100, False), _span(10, 11), _span(19, 20)):
        with pytest.raises(ValueError, match="share memory"):
            sab._refuse_overlaps(apart + [more])
    # one behind a shorter neighbour, covered by one that began long before
    with pytest.raises(ValueError, match="share memory"):
        sab._refuse_overlaps([_span(0, 100, False), _span(1, 2, False), _span(50, 60)])


def _entry(bits=32, n=N, **own):
    z = lambda size: torch.zeros(size, device="cuda")  # noqa: E731
    t = {"param": z(n), "grad": z(n)}
    for s in ("m", "v"):
        t[s] = z(n) if bits == 32 else z(n).to(torch.float8_e4m3fn)
        if bits == 8:
            t[s + "_scale"] = z(-(-n // sab.ADAMW_BLOCK))
    return {**t, **own}


def _refused(lib, *entries):
    try:
        lib.AdamWTensors(entries)
    except ValueError as e:
        assert "share memory" in str(e)
        return True
    return False


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 16, N - 4])
@pytest.mark.parametrize("first,second", [("param", "param"), ("m", "m"), ("param", "v"), ("m", "param"), ("v", "grad"),
                                          ("grad", "param")])
def test_shifted_views(lib, first, second, shift):
    room = torch.zeros(2 * N, device="cuda")
    a, b = _entry(**{first: room[:N]}), _entry(**{second: room[shift:shift + N]})
    assert _refused(lib, a, b) and _refused(lib, b, a)
    assert not _refused(lib, a, _entry(**{second: room[N:]}))        # neighbours are two arrays


@pytest.mark.gpu
def test_within_one_entry_and_of_other_types(lib):
    room = torch.zeros(2 * N, device="cuda")
    assert _refused(lib, _entry(m=room[:N], v=room[8:N + 8]))
    assert _refused(lib, _entry(grad=room[:N], param=room[4:N + 4]))
    low = room.view(torch.bfloat16)
    assert _refused(lib, _entry(param=room[:N], param_bf16=low[2 * N - 8:3 * N - 8]))
    assert _refused(lib, _entry(param=room[:N], grad=low[:N]))       # bf16: other places than the values it is for
    assert not _refused(lib, _entry(param=room[:N], param_bf16=low[2 * N:3 * N]))
    scales = torch.zeros(8, device="cuda")
    assert _refused(lib, _entry(8, m_scale=scales[:4], v_scale=scales[3:7]))
    assert not _refused(lib, _entry(8, m_scale=scales[:4], v_scale=scales[4:]))
    # scales that a 32-bit state does not use are not the step's
    assert not _refused(lib, _entry(m_scale=scales[:4]), _entry(m_scale=scales[:4]))


@pytest.mark.gpu
def test_gradients_may_be_shared_and_lie_in_their_own_entry(lib):
    g = torch.zeros(2 * N, device="cuda")
    assert not _refused(lib, _entry(grad=g[:N]), _entry(grad=g[:N]), _entry(grad=g[8:N + 8]))
    low = torch.zeros(N, dtype=torch.bfloat16, device="cuda")
    assert not _refused(lib, _entry(grad=low, param_bf16=low))       # read before it is written, value by value
    assert _refused(lib, _entry(grad=low), _entry(param_bf16=low))
    assert _refused(lib, _entry(grad=low, param_bf16=low), _entry(n=8, grad=low[:8]))
    assert not _refused(lib, _entry(n=0), _entry(n=0))
