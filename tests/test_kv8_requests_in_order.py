"""Requests whose cu_new descends, without a GPU: what the calls lay out for a step's rows has room for them, whatever cu_new holds.

The launch knows total_new alone. A block or tile of R rows of a head is made for every R rows of a request, and room for
total_new * G / R + min(batch, total_new) of them: enough as long as no two requests have a row in common."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_tiered_gb300", "csrc")
KERNELS = [("k_kv8_rows.cu", "kv8_rows_blocks"), ("k_kv8_select.cu", "kv8_select_scores")]


def in_range(cu, total, max_new):
    return [0 <= cu[b] <= cu[b + 1] <= total and cu[b + 1] - cu[b] <= max_new for b in range(len(cu) - 1)]


def that_count(cu, total, max_new):
    """The requests that are in range and begin behind the end of all before them that are and have rows."""
    out, end = [], 0
    for b, ok in enumerate(in_range(cu, total, max_new)):
        if ok and cu[b] >= end:
            out.append(b)
        if ok and cu[b + 1] > cu[b]:
            end = max(end, cu[b + 1])
    return out


def blocks(cu, requests, group, rows):
    return sum(((cu[b + 1] - cu[b]) * group + rows - 1) // rows for b in requests)


def room(batch, total, group, rows):
    return total * group // rows + min(batch, total)


def rows_of(group):
    return 64 * group if group < 4 else 256


def test_requests_in_range_by_themselves_may_need_more_than_there_is_room_for():
    cu = [0, 100, 0, 100]
    alone = [b for b, ok in enumerate(in_range(cu, 100, 100)) if ok]
    assert alone == [0, 2] and blocks(cu, alone, 8, 256) == 8 > room(3, 100, 8, 256) == 6
    assert that_count(cu, 100, 100) == [0] and blocks(cu, [0], 8, 256) == 4


@pytest.mark.parametrize("seed", range(40))
def test_those_that_count_never_do(seed):
    rng = random.Random(seed)
    for _ in range(200):
        batch, total = rng.randint(1, 60), rng.choice([1, 5, 64, 300, 3000])
        cu = [rng.randint(-2, total + 2) for _ in range(batch + 1)]
        if rng.random() < 0.5:
            cu = sorted(max(0, min(total, x)) for x in cu)
            for _ in range(rng.randint(0, 4)):
                cu[rng.randrange(batch + 1)] = rng.randint(-1, total + 1)
        most = rng.choice([total, max(1, total // 3)])
        some = that_count(cu, total, most)
        taken = [t for b in some for t in range(cu[b], cu[b + 1])]
        assert len(taken) == len(set(taken)) <= total
        for group in (1, 2, 3, 4, 5, 8, 16):
            for rows in (8 * group, 32 * group, rows_of(group)):  # tiles of 8 and of 32 tokens, and blocks
                assert blocks(cu, some, group, rows) <= room(batch, total, group, rows)
        if all(a <= b for a, b in zip(cu, cu[1:])):  # every one in range, then
            assert some == [b for b, ok in enumerate(in_range(cu, total, most)) if ok]
        else:
            assert not all(in_range(cu, total, most))  # somebody is reported


@pytest.mark.parametrize("file,kernel", KERNELS)
def test_the_kernels_lay_out_those_alone(file, kernel):
    source = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())
    body = source[source.index(kernel + "("):]
    body = body[: body.index("__global__") if "__global__" in body else len(body)]
    assert "locate_rows(" in body and not re.search(r"\blocate\(", body)


def last_that_begins(cu, token):
    """A search of cu_new by halves, 32 parts at a time, which counts the places that do not lie behind the token."""
    lo, n = 0, len(cu) - 1
    while n > 1:
        step = (n + 31) // 32
        w = max(0, sum(i * step < n and cu[lo + i * step] <= token for i in range(32)) - 1)
        lo, n = lo + w * step, min(step, n - w * step)
    return lo


def test_a_search_finds_a_tokens_request_only_while_all_are_in_range():
    """Request 2 of these is in range and shares no row, but the search for its token ends at request 1."""
    cu = [0, 9, 4, 6]
    assert that_count(cu, 6, 6) == [2] and last_that_begins(cu, 4) == 1
    for seed in range(200):
        rng = random.Random(seed)
        cu = [0] + sorted(rng.randint(0, 90) for _ in range(rng.randint(1, 70)))
        for token in range(cu[-1]):
            b = last_that_begins(cu, token)
            assert cu[b] <= token < cu[b + 1]


def test_select_searches_only_while_all_are_in_range():
    source = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "k_kv8_select.cu")).read())
    body = source[source.index("kv8_select_pick("):]
    search = re.sub(r"\s+", " ", body[: body.index("RowIn in;")])
    assert search.endswith("if (strange) { lo = owner_of(a, token); its = lo >= 0 && kv8_request(a, lo, false, row0, n_new, past); } "
                           "if (!its) return; const int64_t unit = (int64_t)lo * a.Hkv + h; ")
    assert [m for m in re.findall(r"if \(([^{;]*)\) return;", search)][1:] == ["token >= a.cu[a.B] && !strange", "!its"]
