"""What the attention kernels of the 8-bit cache do once a bounded wait has run out, restated: every warp comes to its end."""
import itertools

import pytest

PAIR_BARRIERS = 9  # of the two tiles' warps in a shared block: the sums, four times 32 columns there and back


def softmax_warp(segments, lost, agree):
    """A softmax warp of k_kv8_prefill.cu: yields where it waits at the barrier that it has with the other tile's warp of
    the same rows, and is told what that barrier's vote came to. `lost`: the number of its waits after which one has run
    out and no other succeeds (None: never). A segment is (shared, waits of this warp)."""
    waits = 0

    def ok():
        return lost is None or waits <= lost

    for shared, mine in segments:
        waits += 1  # for the segment's announcement, which is there
        well = ok()
        if agree:
            well = yield ("vote", well)
        if not well:
            return
        waits += mine
        for _ in range(PAIR_BARRIERS if shared else 0):
            yield ("sync", True)


def ends(a, b):
    """Two warps and their barrier: whether both come to their end."""
    say = [next(a, None), next(b, None)]
    while say[0] is not None and say[1] is not None:
        if say[0][0] != say[1][0]:
            return False
        vote = say[0][1] and say[1][1]
        for i, w in enumerate((a, b)):
            try:
                say[i] = w.send(vote)
            except StopIteration:
                say[i] = None
    return say[0] is None and say[1] is None


def all_losses(agree):
    kinds = [(True, (1, 1)), (True, (2, 1)), (True, (1, 0)), (False, (2, 3)), (False, (0, 2))]
    for segments in itertools.product(kinds, repeat=3):
        per_warp = [[(shared, waits[i]) for shared, waits in segments] for i in range(2)]
        most = [sum(1 + n for _, n in s) for s in per_warp]
        for lost in itertools.product([None, *range(most[0] + 1)], [None, *range(most[1] + 1)]):
            yield ends(*(softmax_warp(s, x, agree) for s, x in zip(per_warp, lost)))


def test_the_two_tiles_warps_leave_together():
    """Wherever either of them loses its waits."""
    assert all(all_losses(agree=True))


def test_they_would_not_without_the_vote():
    """The restatement sees what the vote is for."""
    assert not all(all_losses(agree=False))


SETTLE, LANDED = 0.25, 0.01  # seconds: settle_down(), and when any copy has landed


def end_of_cta(issued, ran_out, consumers_settle):
    """When the last warp of a CTA of k_kv8_attend.cu leaves: copies issued at these times, a consumer's wait that runs
    out at another. The producer leaves with its last copy; it settles only if it has seen the abort by then."""
    producer = max(issued) if max(issued) <= ran_out else ran_out + SETTLE
    return max(producer, ran_out + (SETTLE if consumers_settle else 0.0))


@pytest.mark.parametrize("last", [0.0, 1.0, 1.995, 1.9999, 2.0])
def test_no_copy_is_in_flight_when_a_cta_ends(last):
    issued = [t for t in (0.0, 0.5, 1.5) if t < last] + [last]
    assert end_of_cta(issued, 2.0, True) >= last + LANDED


def test_one_would_be_if_the_consumers_did_not_settle():
    assert end_of_cta([0.0, 1.9999], 2.0, False) < 1.9999 + LANDED
