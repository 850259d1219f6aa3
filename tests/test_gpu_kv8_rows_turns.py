"""Attention over lists for more tokens than are laid out at a time, on the GPU."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv8_rows_ref as R  # noqa: E402
from kv8_ref import decode_e4m3  # noqa: E402
from test_gpu_kv8 import D, PAGE, ints, spin  # noqa: E402
from test_gpu_kv8_rows import SCALE  # noqa: E402

G, P, K = 16, 16384, 512
BLOCKS = (4 << 30) // (64 + 32 * (16 * (K + 1) + 1))  # of 16 tokens, that are laid out at a time: 16,346


class Large:
    """Requests over a pool of few pages; lists of few pages in rows of 512."""

    def __init__(self, past, new):
        self.past, self.new = past, new
        B, g = len(past), torch.Generator(device="cuda").manual_seed(1)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        self.cu, T = cu, cu[-1]
        rand = lambda *shape: torch.randint(0, 1 << 30, shape, generator=g, device="cuda")  # noqa: E731
        self.pages = (rand(40, 2, PAGE, D) % 127 & 0x37 | 0x20 | rand(40, 2, PAGE, D) % 2 << 7).to(torch.uint8)
        self.scales = torch.exp2((rand(40, 2) % 3 - 6).float())
        full = max(a + n for a, n in zip(past, new)) // PAGE
        self.table = torch.full((B, 1, P), -1, dtype=torch.int32, device="cuda")
        self.table[:, :, :full] = (rand(B, 1, full) % 40).to(torch.int32)
        self.tails = torch.randn((B, 1, 2, PAGE, D), generator=g, device="cuda").to(torch.bfloat16)
        self.q = torch.randn((T, G, D), generator=g, device="cuda").to(torch.bfloat16)
        self.sel = torch.full((T, 1, K), -1, dtype=torch.int32, device="cuda")
        self.sel[:, :, 5:9] = (rand(T, 1, 4) % max(1, full)).to(torch.int32)
        self.h = spin().SpinKV8(B, G, 1, P, 40, pages=self.pages, scales=self.scales, tails=self.tails, table=self.table)
        self.step = spin().SpinKV8Step(ints(past), ints(cu), T + 3, max(new))

    def run(self):
        from sparse_attention_tiered_gb300 import _binding as B

        T = self.cu[-1]
        one = B.spin_kv8_attend_rows_workspace(self.h.c, T + 3, K)
        assert B.spin_kv8_attend_rows_workspace(self.h.c, 1 << 30, K) == one  # it takes turns
        q = torch.cat([self.q, self.q[:3]])
        sel = torch.cat([self.sel, self.sel[:3]])
        out = self.h.attend_rows(self.step, q, torch.full_like(q, 7.0), sel)
        self.h.check()
        assert (out[T:] == 7.0).all()
        again = self.h.attend_rows(self.step, q, q, sel)  # in place
        assert torch.equal(again[:T], out[:T])
        return out[:T]


def test_many_short_requests():
    new = [1 + b % 4 for b in range(16384)]
    c = Large([(b * 37) % 400 for b in range(16384)], new)
    out = c.run().cpu()
    pages, scales = c.pages.cpu(), c.scales.cpu()
    turn = BLOCKS * 256 // (256 + G)  # tokens: each may be its request's only one
    meet = [b for b in range(16384) if any(c.cu[b] - 3 <= x <= c.cu[b + 1] + 3 for x in range(turn, c.cu[-1], turn))]
    assert len(meet) > 4
    for b in [*range(0, 16384, 199), *meet, 16383]:
        r0, r1 = c.cu[b], c.cu[b + 1]
        want, bound = R.attend_rows(c.q[r0:r1].cpu(), pages, scales, c.tails[b:b + 1].cpu(), c.table[b:b + 1, :, :16].cpu(), [c.past[b]], [0, r1 - r0],
                                    SCALE, c.sel[r0:r1, :, 5:9].cpu())
        assert ((out[r0:r1].double() - want).abs() <= bound).all(), b


def test_one_long_request():
    """Two turns meet inside of it."""
    past, new = [333, 100], [300000, 7]
    c = Large(past, new)
    out = c.run()
    pages, scales = c.pages.cpu(), c.scales.cpu()
    values = decode_e4m3(pages) * scales.double()[:, :, None, None]
    n = past[0] + new[0]
    turn = (BLOCKS - len(new)) * 256 // G
    assert turn < 299000
    for t in [0, 1, 17, 63, 100, 5000, 131071, *range(turn - 40, turn + 40), 270000, 299990, 299998, 299999]:
        see = past[0] + t + 1
        # The same as the next token of `see` - 1: the page that it is in becomes the tail, its values are bf16 numbers.
        last = see // PAGE
        tail = c.tails[0:1].cpu()
        if last < n // PAGE:
            tail = values[int(c.table[0, 0, last])].to(torch.bfloat16)[None, None]
        want, bound = R.attend_rows(c.q[t:t + 1].cpu(), pages, scales, tail, c.table[0:1].cpu(), [see - 1], [0, 1], SCALE, c.sel[t:t + 1, :, 5:9].cpu())
        assert ((out[t:t + 1].cpu().double() - want).abs() <= bound).all(), t
