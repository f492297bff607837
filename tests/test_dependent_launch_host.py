"""Kernels that may start while the previous kernel on the stream still runs
(programmatic dependent launch) read what that kernel writes only after their
wait. The wait orders plain loads. It does not order loads that are declared
read-only for the kernel's whole life: the compiler may move those in front of
it, and the non-coherent path may return an old line. So in every kernel that
waits no parameter that is read is __restrict__, and no load on the way from
such a kernel is __ldg or .nc. Read from the sources, without a GPU."""
import os
import re

import pytest

from linear_attention_recurrence_04_b200 import build as gdn_build

WAIT = re.compile(r"grid_dep_wait\(\)|griddepcontrol\.wait")
READ_ONLY = re.compile(r"const\s+\w+\s*\*\s*(const\s+)?__restrict__")
NON_COHERENT = re.compile(r"__ldg\s*\(|\.nc\b")


def code(path):
    """The file without comments (strings stay: they hold the inline PTX)."""
    with open(path) as f:
        s = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", s, flags=re.S)


def close(s, at, pair):
    """Index behind the bracket that closes the one at `at`."""
    depth = 0
    for i in range(at, len(s)):
        depth += (s[i] == pair[0]) - (s[i] == pair[1])
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced")


def functions(s):
    """(name, parameters, body) of every device function and kernel in `s`."""
    for m in re.finditer(r"(\w+)\s*\(", s):
        head = re.split(r"[;{}]", s[:m.start()])[-1]
        if m.group(1) == "__launch_bounds__" or not re.search(r"__(device|global)__", head):
            continue
        end = close(s, m.end() - 1, "()")
        tail = re.match(r"\s*(const\s*)?\{", s[end:])
        if tail:
            at = end + tail.end() - 1
            yield m.group(1), s[m.end():end - 1], s[at:close(s, at, "{}")]


def library():
    """name -> [(parameters, body)] over all sources."""
    out = {}
    for p in sorted(gdn_build.sources()) + [os.path.join(gdn_build.CSRC, n)
                                            for n in sorted(os.listdir(gdn_build.CSRC))
                                            if n.endswith((".cuh", ".h"))]:
        for name, params, body in functions(code(p)):
            out.setdefault(name, []).append((params, body))
    return out


LIB = library()
# Only a kernel itself waits; grid_dep_wait is the wait.
WAITING = sorted(n for n, defs in LIB.items()
                 if n != "grid_dep_wait" and any(WAIT.search(b) for _, b in defs))


def reached(name):
    """`name` and every function of the library that it can call."""
    seen, todo = set(), [name]
    while todo:
        n = todo.pop()
        if n in seen or n not in LIB:
            continue
        seen.add(n)
        for _, body in LIB[n]:
            todo += re.findall(r"\b(\w+)\s*(?:<[^;{}()]*>)?\s*\(", body)
    return seen


def test_the_scan_sees_the_kernels():
    assert {"linear_i8_vec_kernel", "linear_i8_split_kernel", "linear_i8_pair_kernel",
            "quantize_rows_kernel", "gated_norm_i8_kernel", "linear_bf16_kernel",
            "linear_bf16_splitk_kernel", "step_kernel", "short_conv_gate_kernel"} <= set(WAITING)
    assert "ld_stream_i4" in reached("linear_i8_vec_kernel")
    assert "scaled" in reached("linear_i8_pair_kernel")


@pytest.mark.parametrize("kernel", WAITING)
def test_reads_after_the_wait(kernel):
    for name in sorted(reached(kernel)):
        for params, body in LIB[name]:
            assert not READ_ONLY.search(params), f"{kernel}: {name}({params})"
            assert not NON_COHERENT.search(body), f"{kernel}: {name} loads past coherence"
