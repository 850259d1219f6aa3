"""The workspaces that a handle makes for its calls, without a GPU: how they grow, and what stays of those that were outgrown."""
import pytest

import sparse_attention_tiered_gb300 as spin


class Bytes:
    made = 0

    def __init__(self, n):
        self.n, self.at = n, 1 << 40 | Bytes.made << 20
        Bytes.made += 1

    def numel(self):
        return self.n

    def data_ptr(self):
        return self.at


class Torch:
    """What a handle asks of torch when a workspace has to be made."""

    uint8 = "uint8"

    def __init__(self):
        self.cuda, self.capturing, self.waits = self, False, 0

    def device(self, kind, index):
        return kind, index

    def empty(self, n, dtype, device):
        assert dtype == "uint8" and device == ("cuda", 3) and not self.capturing
        return Bytes(n)

    def is_current_stream_capturing(self):
        return self.capturing

    def synchronize(self, device):
        self.waits += 1


def handle():
    h = spin.SpinKV8.__new__(spin.SpinKV8)
    h._torch, h.device, h._spaces = Torch(), 3, {}
    return h


@pytest.mark.parametrize("step", [1, 3, 200000, 2359424])
def test_a_batch_that_grows_a_row_at_a_time_makes_few(step):
    h = handle()
    for rows in range(1, 2049):
        asked = 45000000 + rows * step
        at, n = h._space("attend_rows", asked, None)
        held = h._spaces["attend_rows"]
        assert n >= asked and at == held[-1].data_ptr()
        assert sum(t.numel() for t in held) < 4 * asked
    assert len(held) == h._torch.waits <= 1 + (2049 * step // 45000000 + 1).bit_length()


def test_the_first_is_what_was_asked_for_and_smaller_calls_use_it():
    h = handle()
    first = h._space("select", 1000, None)
    assert first[1] == 1000 and h._space("select", 10, None) == first and h._space("select", 1000, None) == first
    assert h._space("pool", 50, None)[1] == 50 and len(h._spaces["select"]) == 1
    assert h._space("select", 5000, None)[1] == 5000 and len(h._spaces["select"]) == 2  # (the first stays)


def test_one_that_has_to_grow_during_a_capture_is_refused():
    h = handle()
    first = h._space("select", 1000, None)
    h._torch.capturing = True
    assert h._space("select", 900, None) == first
    with pytest.raises(ValueError, match="before capturing"):
        h._space("select", 1001, None)
    assert len(h._spaces["select"]) == 1
