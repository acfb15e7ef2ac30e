"""What the sources of the train-step operators have to keep, checked on their text: a kernel that
may start while the one before it still runs waits, in every thread, before it touches memory that
other kernels write or read."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_moe_fine_gb300", "csrc")
SOURCES = ["router_aux.cu", "router_grad.cu", "router_grad_tc.cu", "act8.cu"]


def _text(name):
    t = open(os.path.join(CSRC, name)).read()
    t = re.sub(r"/\*.*?\*/", "", t, flags=re.S)
    return re.sub(r"//[^\n]*", "", t)


def _body(text, kernel):
    """The body of a __global__ function."""
    at = re.search(r"__global__[^{};]*?\b" + kernel + r"\s*\(", text)
    assert at, kernel
    start = text.index("{", at.end())
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start + 1:i]
    raise AssertionError(kernel)


def _dependent():
    """(source, kernel) of every kernel that launch_dep launches."""
    out = []
    for s in SOURCES:
        for k in re.findall(r"launch_dep\(\s*(\w+)", _text(s)):
            if k != "void":
                out.append((s, k))
    return sorted(set(out))


def test_dependent_kernels_are_found():
    assert {k for _, k in _dependent()} >= {"aux_final_kernel", "aux_bwd_kernel",
                                            "router_grad_w_tc_kernel", "router_grad_x_tc_kernel"}


@pytest.mark.parametrize("source,kernel", _dependent())
def test_dependent_kernels_wait_before_they_touch_global_memory(source, kernel):
    body = _body(_text(source), kernel)
    # the wait stands at the function's own level, whatever the arguments
    wait = re.search(r"^  dep_wait\(\);", body, flags=re.M)
    assert wait, "no unconditional dep_wait()"
    before = body[:wait.start()]
    for touch in (r"tma_load", r"__ldg", r"__ldcg", r"clamp_off\(", r"p\.off\b", r"\bload_row",
                  r"Groups \w+\(", r"load\(0\)", r"reduce_parts\("):
        # (a lambda or declaration before the wait is fine as long as it is not called)
        found = [m for m in re.finditer(touch, before) if not _in_lambda(before, m.start())]
        assert not found, touch


def _in_lambda(text, pos):
    """Whether pos lies within the braces of a lambda that text defines."""
    for m in re.finditer(r"\[&\]\([^)]*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth and i < len(text):
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        if m.start() < pos < i:
            return True
    return False


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC)
                                        if f in SOURCES + ["tc_ptx.cuh", "train.cuh",
                                                           "abi_train.cu"]))
def test_functions_keep_no_plain_static_variables(name):
    """Host threads may call at once, so what a function keeps is atomic (or made of atomics)."""
    for m in re.finditer(r"^\s+static (?!_|constexpr\b|const\b|assert)([^(;={]*)[;={]", _text(name),
                         flags=re.M):
        assert re.match(r"std::atomic<|OncePerDevice\b", m.group(1)), m.group(0)
