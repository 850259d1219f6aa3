"""The other kernels of the 8-bit cache that begin while the launch before them ends: nothing that they are given is touched
before the wait, and nothing is read through a cache that is not coherent."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_tiered_gb300", "csrc")
FILES = ["k_kv8_pool.cu", "k_kv8_select.cu", "k_kv8_rows.cu", "k_kv8_lists.cu"]
SOURCES = {os.path.basename(p): re.sub(r"//[^\n]*", "", open(p).read()) for p in glob.glob(os.path.join(CSRC, "*.cu*"))}
KERNELS = sorted((f, k) for f in FILES for k in re.findall(r"__global__ void[^;{]*?(kv8_\w+)\(", SOURCES[f]))


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
    assert {k for _, k in KERNELS} == {"kv8_pool_count", "kv8_pool_reserve", "kv8_pool_move", "kv8_pool_fork", "kv8_pool_lengths",
                                       "kv8_select_scores", "kv8_select_pick", "kv8_rows_blocks", "kv8_rows_single", "kv8_lists_attend"}


@pytest.mark.parametrize("file,name", KERNELS)
def test_all_are_launched_so(file, name):
    assert re.search(r"launch_early\(%s\b" % name, SOURCES[file]) and not re.search(r"%s\s*(<[^;()]*>)?\s*<<<" % name, SOURCES[file])


@pytest.mark.parametrize("file,name", KERNELS)
def test_no_pointer_promises_unchanged_memory(file, name):
    params, _ = kernel_of(file, name)
    assert "__restrict__" not in params


@pytest.mark.parametrize("file", FILES + ["kv8_rows.cuh", "kv8_tc.cuh"])
def test_nothing_is_read_through_the_read_only_cache(file):
    assert not re.search(r"__ldg|ld\.global\.nc", SOURCES[file])


@pytest.mark.parametrize("file,name", KERNELS)
def test_each_waits_before_it_touches_its_arguments(file, name):
    params, body = kernel_of(file, name)
    assert body.count("griddepcontrol.wait") == 1 and body.count("griddepcontrol.launch_dependents") == 1
    before = body[: body.index("griddepcontrol.wait")]
    for p in re.findall(r"(\w+)\s*(?:,|$)", params):
        assert p == "a" or not re.search(r"\b%s\s*(\.|\[|->)" % p, before), p
    assert not re.search(r"\ba\.(?!B\b|G\b|Hkv\b|max_pages\b|n_pages\b|total_new\b|max_new\b)", before)  # (its numbers are the call's own)
    assert "return" not in before  # every thread waits: what comes after this launch counts on what came before it
