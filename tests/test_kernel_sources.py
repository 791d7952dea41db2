"""Kernels that start while the kernel before them still runs (those that call pdl_wait()): what that kernel wrote reaches
them only as Late<T>, whose loads stay behind the wait.  A plain load of constant memory (a const pointer, __ldg) may be
moved above it by the compiler, and then reads what was there before."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunk_wise_sparse_b200", "csrc")

# what the caller of a step hands in: complete before its first kernel starts
INPUTS = {"q", "kc", "vc", "kpg", "vpg", "table", "seqlens"}


def _strip(text):
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    return re.sub(r"//[^\n]*", " ", text)


def _balanced(text, at, pair):
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return text[at + 1:i], i
    raise AssertionError("unbalanced source")


def _kernels(text):
    """(name, parameters, body) of every kernel."""
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\s*)?", text):
        at = m.end()
        if text[at] == "(":                       # the launch bounds
            at = _balanced(text, at, "()")[1] + 1
        name = re.compile(r"\s*(\w+)\s*").match(text, at)
        params, end = _balanced(text, name.end(), "()")
        body = _balanced(text, text.index("{", end), "{}")[0]
        yield name.group(1), params, body


def _waiting():
    found = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            for name, params, body in _kernels(_strip(f.read())):
                if re.search(r"\bpdl_wait\s*\(", body):
                    found[name] = params, body
    return found


WAITING = _waiting()


def test_the_kernels_are_found():
    assert {"decode_topk_kernel", "decode_topk_reg_kernel", "decode_partial_union_kernel", "decode_combine_kernel",
            "quant_topk_kernel", "quant_attend_kernel"} <= set(WAITING)


@pytest.mark.parametrize("name", sorted(WAITING))
def test_results_of_the_kernel_before_are_loaded_late(name):
    params, body = WAITING[name]
    late = []
    for p in params.split(","):
        p = " ".join(p.split())
        arg = re.search(r"(\w+)$", p).group(1)
        if re.search(r"\bLate<", p):
            late.append(arg)
        elif "*" in p and re.search(r"\bconst\b", p.split("*")[0]):
            assert arg in INPUTS, f"{arg} of {name}: {p}"
    assert late, "a kernel that waits reads something"
    before = body[:re.search(r"\bpdl_wait\s*\(", body).start()]
    for arg in late:
        assert not re.search(rf"\b{arg}\b", before), f"{arg} is used before the wait"
        assert not re.search(rf"\b{arg}\.p\b", body), f"the address of {arg} is taken"
