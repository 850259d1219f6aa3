"""Attention over lists for more tokens than are laid out at a time, without a GPU: what its workspace takes, and that a turn's blocks have room."""
import random

import pytest

from sparse_attention_tiered_gb300 import _binding as B

from test_kv8_refusals import cache
from test_kv8_requests_in_order import room, rows_of

GB4 = 4 << 30


def blocks(cu, t0, t1, group):
    """Of a head: each request's rows between the tokens t0 and t1."""
    R = rows_of(group)
    return sum((max(0, min(z, t1) - max(a, t0)) * group + R - 1) // R for a, z in zip(cu, cu[1:]))


@pytest.mark.parametrize("kv_heads,group", [(1, 1), (1, 3), (2, 4), (8, 5), (8, 8), (4, 16), (4096, 1)])
def test_the_workspace_is_bounded(kv_heads, group):
    for batch in (1, 300, 16384):
        for max_pages in (1, 500, 1 << 24):
            c = cache(batch=batch, kv_heads=kv_heads, q_heads=kv_heads * group, max_pages=max_pages)
            rest = B.spin_kv8_workspace(c)
            for topk in (1, 40, 512):
                lists = batch * kv_heads * topk * 4  # of single tokens
                sizes = [B.spin_kv8_attend_rows_workspace(c, n, topk) - rest for n in (1, 5, 500, 65536, 1 << 20, (1 << 31) - 1)]
                tokens = (rows_of(group) - 1) // group + (2 if rows_of(group) % group else 1)
                block = kv_heads * (64 + 32 * (min(tokens * (topk + 1), max_pages) + 1))  # at least one, of all heads: 4.3 GB for 4096
                assert sizes == sorted(sizes) and 16 + block <= sizes[0] and sizes[-1] <= max(GB4 + 16, 16 + block, lists)


def test_what_fitted_takes_one_turn_as_before():
    """A prompt chunk and a batch of drafts: room for all of their blocks."""
    for batch, tokens, topk, max_pages in ((1, 2048, 32, 500), (1, 8192, 128, 4096), (256, 1280, 128, 4096), (1024, 5120, 128, 4096)):
        c = cache(batch=batch, kv_heads=8, q_heads=64, max_pages=max_pages)
        items = 2 * (min(33 * (topk + 1), max_pages) + 1)
        want = 16 + room(batch, tokens, 8, 256) * 8 * (64 + 16 * items)
        got = B.spin_kv8_attend_rows_workspace(c, tokens, topk) - B.spin_kv8_workspace(c)
        assert want * 0.95 < got <= want


@pytest.mark.parametrize("seed", range(20))
def test_turns_have_room_and_take_every_row_once(seed):
    rng = random.Random(seed)
    for _ in range(100):
        batch, group = rng.randint(1, 40), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        cu = [0]
        for _ in range(batch):
            cu.append(cu[-1] + rng.choice([0, 1, 2, 3, 17, 64, 65, rng.randint(0, 400)]))
        total, R = cu[-1] + rng.randint(0, 5), rows_of(group)
        turn = rng.randint(1, max(1, total))
        taken = []
        for t0 in range(0, total, turn):
            t1 = min(total, t0 + turn)
            assert blocks(cu, t0, t1, group) <= room(batch, t1 - t0, group, R)
            for a, z in zip(cu, cu[1:]):
                n = (max(0, min(z, t1) - max(a, t0)) * group + R - 1) // R
                for k in range(n):  # the kernel's numbers
                    first = max(0, t0 - a) * group + k * R
                    n_new = (min(min(z - a, t1 - a) * group, first + R) + group - 1) // group
                    rows = min(R, n_new * group - first)
                    assert rows > 0
                    taken += [a * group + r for r in range(first, first + rows)]
        assert sorted(taken) == list(range(cu[-1] * group))
