"""Kernels of the 8-bit cache begin while the launch before them ends. What that launch writes must not be read before
the kernel's wait, nor through a cache that is not coherent."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_tiered_gb300", "csrc")
SOURCES = {os.path.basename(p): re.sub(r"//[^\n]*", "", open(p).read()) for p in glob.glob(os.path.join(CSRC, "*.cu*"))}


def early():
    """(file, kernel) of every launch that may begin early."""
    return sorted({(f, m) for f, s in SOURCES.items() for m in re.findall(r"launch_early\((\w+)", s) if "kernel" in m and m != "kernel"})


def kernel_of(file, name):
    """(parameters, body) of a kernel."""
    s = SOURCES[file]
    m = re.search(r"__global__[^{;]*?\b%s\((.*?)\)\s*\{" % name, s, re.S)
    depth, at = 1, m.end()
    while depth:
        depth += {"{": 1, "}": -1}.get(s[at], 0)
        at += 1
    return m.group(1), s[m.end():at]


def test_they_are_found():
    assert {k for _, k in early()} == {"kv8_append_kernel", "kv8_decode_kernel", "kv8_prefill_kernel", "kv8_join_kernel"}


@pytest.mark.parametrize("file,name", early())
def test_no_pointer_promises_unchanged_memory(file, name):
    params, _ = kernel_of(file, name)
    assert "__restrict__" not in params


@pytest.mark.parametrize("file", sorted({f for f, _ in early()} | {"kv8.cuh", "kv8_dev.cuh"}))
def test_the_read_only_cache_has_constants_alone(file):
    """(g_ names the __device__ const tables)"""
    for m in re.findall(r"(?:__ldg|ld\.global\.nc)[^;]*", SOURCES[file]):
        assert "&g_" in m, m


@pytest.mark.parametrize("file,name", early())
def test_each_waits_before_it_reads(file, name):
    """Before the wait: barriers' and shared memory's beginnings, nothing through a pointer of the arguments."""
    params, body = kernel_of(file, name)
    assert body.count("griddepcontrol.wait") == 1
    before = body[: body.index("griddepcontrol.wait")]
    for p in re.findall(r"\*\s*(\w+)", params):
        assert not re.search(r"\b%s\s*(\[|\+|->)|\*\s*%s\b" % (p, p), before), p
    assert not re.search(r"\ba\.(cu|past|table|scales|tails|pages|summaries|err)\b", before)
