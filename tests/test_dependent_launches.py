"""Kernels launched as programmatic dependents start while the kernel before them still writes: each
waits before its first access to memory, and none uses the read-only path (__ldg, ld.global.nc),
whose loads need memory that nobody writes while the kernel runs and which the wait does not order.
Read from the sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_37_b200", "csrc")
WAIT, FIRST = "griddepcontrol.wait", r"\bp\.(n_new|kv_len|table|k|v|k_scale|v_scale|new_k|new_v|begin|Q|O|qbar|kbar)\b\s*[\[+)]|wk\.|find_run|next_piece|seq_lens"


def _code(name):
    src = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", src)


def _files():
    """Files whose kernels are launched dependently, and the headers that those share."""
    return sorted(f for f in os.listdir(CSRC) if re.search(r"launch_after|launch_dependent\b", _code(f))) + ["paged_sched.cuh"]


@pytest.mark.parametrize("name", _files())
def test_no_load_goes_through_the_read_only_path(name):
    """(Shared helpers take it as a template argument, which only kernels launched the plain way pass.)"""
    code = _code(name).replace("return READ_ONLY ? __ldg(a) : *a;", "")
    assert not re.search(r"__ldg|\.global\.nc|__ldcg|__ldcs|__restrict__|READ_ONLY = true", code)
    for kernel, body in _kernels(name):
        assert "kReadOnly" not in body, kernel


def _kernels(name):
    """(name, body) of the kernels that are launched dependently."""
    code = _code(name)
    launched = set(re.findall(r"launch_(?:after|dependent)\((\w+)", code))
    launched |= set(re.findall(r"auto fn = (\w+)<", code)) if "launch_after(fn" in code else set()
    for m in re.finditer(r"__global__[^;{]*?(\w+)\s*\(", code):
        kernel = [k for k in re.findall(r"\w+_kernel", code[m.start():m.start() + 400])][0]
        if kernel in launched:
            body = code[code.index("{", code.index(kernel, m.start())):]
            yield kernel, body[:body.find("__global__")]


@pytest.mark.parametrize("name", [f for f in _files() if f.endswith(".cu")])
def test_each_waits_before_its_first_access(name):
    seen = 0
    for kernel, body in _kernels(name):
        seen += 1
        first = re.search(FIRST, body)
        assert WAIT in body and first and body.index(WAIT) < first.start(), kernel
    assert seen
