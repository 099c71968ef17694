"""A rule of the sources (no GPU): a kernel launched by launch_after starts while the kernel before it
in the stream still runs.  `__restrict__` promises that nobody else touches the memory while the
kernel runs, so the compiler may move its accesses above wait_for_previous (as non-coherent loads,
too); in such a kernel only the caller's inputs, which no kernel of the call writes, may carry it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sketch_attention_b200", "csrc")
# arguments that are the caller's inputs, as the launches name them
INPUTS = {"dX", "acts", "ids", "a.off_dev", "a.X", "a.P", "a.W_Q", "a.W_K", "a.W_V", "a.H", "a.dS"}


def _closing(text, at):
    """Index of the parenthesis that closes the one at `at`."""
    depth = 0
    for i in range(at, len(text)):
        depth += {"(": 1, ")": -1}.get(text[i], 0)
        if depth == 0:
            return i
    raise AssertionError("unbalanced")


def _split(text):
    """The comma-separated parts of an argument or parameter list."""
    parts, depth, last = [], 0, 0
    for i, ch in enumerate(text + ","):
        depth += {"(": 1, "<": 1, ")": -1, ">": -1}.get(ch, 0)
        if ch == "," and depth == 0:
            parts.append(" ".join(text[last:i].split()))
            last = i + 1
    return parts


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def violations(code):
    """(function, parameter) of every `__restrict__` that the rule does not allow."""
    bad = []
    kernels = {}
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^)]*\)\s*)?(\w+)\s*\(", code):
        kernels[m.group(1)] = _split(code[m.end():_closing(code, m.end() - 1)])
    launched = set()
    for m in re.finditer(r"\blaunch_after\(", code):
        args = _split(code[m.end():_closing(code, m.end() - 1)])
        kernel = args[0].split("<")[0]
        if kernel not in kernels:                  # the definition of launch_after itself
            continue
        launched.add(kernel)
        params, given = kernels[kernel], args[5:]
        assert len(params) == len(given), kernel
        bad += [(kernel, p) for p, a in zip(params, given) if "__restrict__" in p and a not in INPUTS]
    if launched:
        # device functions see memory of both kinds: none of their parameters carries it
        for m in re.finditer(r"__device__[^;{(]*?(\w+)\s*\(", code):
            params = _split(code[m.end():_closing(code, m.end() - 1)])
            bad += [(m.group(1), p) for p in params if "__restrict__" in p]
    return bad, launched


SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


@pytest.mark.parametrize("name", SOURCES)
def test_restrict_is_on_inputs_only(name):
    assert violations(_code(name))[0] == []


def test_the_kernels_are_found():
    found = set().union(*(violations(_code(f))[1] for f in SOURCES))
    assert {"tw_lse_kernel", "tw_lse_combine_kernel", "tw_grads_kernel", "tw_weights_kernel", "tw_sum_kernel",
            "tw_values_kernel", "window_rows_kernel", "crossing_rows_kernel"} <= found


def test_the_rule_sees_a_mistake():
    code = """
__device__ float f(const float* __restrict__ part) { return *part; }
__global__ void __launch_bounds__(32) k(const float* __restrict__ dX, const float* __restrict__ part, float* out) {}
void go() { launch_after(k, 1, 32, 0, st, dX, w.part, out); }
"""
    assert violations(code)[0] == [("k", "const float* __restrict__ part"), ("f", "const float* __restrict__ part")]
