"""Kernels launched while the one before them on the stream still runs (griddepcontrol)
must not read its results through the read-only path: such a load may be made before the
wait, and the wait does not make the cache behind it see new data.  Checked on the sources."""
import os
import re

import pytest

from block_sparse_attention_32_b200 import build as msa_build



def _source(name):
    with open(os.path.join(msa_build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def _kernels(text):
    """(name, parameters, body) of every __global__ function."""
    out = []
    for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\s*\(", text):
        at, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        params, start = text[m.end():at - 1], text.index("{", at)
        end, depth = start + 1, 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        out.append((m.group(1), params, text[start:end]))
    return out


def _waiting():
    return [(f, *k) for f in msa_build.SOURCES for k in _kernels(_source(f)) if "grid_wait()" in k[2]]


def test_the_dependent_kernels_are_found():
    names = {k[1] for k in _waiting()}
    assert {"norm_rope_dw_kernel", "paged_join_kernel", "window_attn_bwd_kernel",
            "window_bwd_join_kernel", "window_bwd_join_dq_kernel"} <= names


@pytest.mark.parametrize("kernel", _waiting(), ids=lambda k: k[1])
def test_results_of_the_kernel_before_are_read_coherently(kernel):
    _, name, params, body = kernel
    assert not re.search(r"const[^,]*\*\s*__restrict__", params), (name, params)
    for arg in re.findall(r"__ldg\(\s*(?:reinterpret_cast<[^>]*>\()?\s*([\w.]+)", body):
        assert arg in {"a.lse", "a.kv_len"}, (name, arg)


def test_what_a_work_item_is_decoded_from_is_read_coherently():
    """The work list and the partial sums' places, read by functions of the dependent kernel."""
    assert not re.findall(r"__ldg\(\s*p\.\w+", _source("window_attn_bwd.cu"))
