"""Attention over a list of pages for each token on the GPU, against the 64-bit restatement in kv8_rows_ref.py."""
import math
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv8_rows_ref as R  # noqa: E402
from test_gpu_kv8 import D, PAGE, ints, spin, step_of  # noqa: E402

SCALE = 1.0 / math.sqrt(D)


class Case:
    """A cache of random pages, random queries and lists."""

    def __init__(self, heads, group, past, new, k, n_pages=40, seed=0, pad=0, max_new=None, spread=0.0, lists="random", max_pages=None):
        g = torch.Generator().manual_seed(seed)
        rng = random.Random(seed)
        self.H, self.G, self.k, self.past, self.new = heads, group, k, list(past), list(new)
        B = len(past)
        P = max_pages or max(1, max((a + n) // PAGE for a, n in zip(past, new)))
        self.pages = torch.randint(0, 127, (n_pages, 2, PAGE, D), dtype=torch.uint8, generator=g)
        self.pages |= torch.randint(0, 2, self.pages.shape, dtype=torch.uint8, generator=g) << 7
        # most codes are of middling size, as a page's are
        self.pages = torch.where(torch.rand(self.pages.shape, generator=g) < 0.9, (self.pages & 0x87) | 0x28 | (self.pages & 0x10), self.pages)
        self.scales = torch.exp2(torch.randint(-6, -3, (n_pages, 2), generator=g).float() + spread * torch.randn((n_pages, 2), generator=g).round())
        self.table = torch.randint(0, n_pages, (B, heads, P), generator=g).to(torch.int32)
        self.tails = torch.randn((B, heads, 2, PAGE, D), generator=g).to(torch.bfloat16)
        T = sum(new) + pad
        self.q = torch.randn((T, heads * group, D), generator=g).to(torch.bfloat16)
        self.sel = torch.full((T, heads, k), -1, dtype=torch.int32)
        at = 0
        for a, n in zip(past, new):
            for i in range(n):
                seen = (a + i + 1) // PAGE
                for h in range(heads):
                    if lists == "random":
                        pick = sorted(rng.sample(range(seen), min(k, seen)))
                    elif lists == "near":  # what neighbours have in common
                        pick = sorted({(j * 7 + (i // 5 if j % 3 == 0 else 0)) % seen for j in range(k)}) if seen else []
                    elif lists == "apart":  # the first 16 tokens of 32, and the others, have nothing in common; some have nothing
                        lo, hi = (0, seen // 3) if i % 32 < 16 else (seen // 3, seen)
                        pick = sorted(rng.sample(range(lo, hi), min(k if i % 7 else 0, hi - lo)))
                    elif lists == "late":  # the first 16 tokens of 32 list nothing
                        pick = sorted(rng.sample(range(seen), min(k, seen))) if i % 32 >= 16 else []
                    elif lists == "wild":  # any order, twice, outside, in the future
                        pick = [rng.choice([-1, -5, seen, seen + 1, 10 ** 9, rng.randrange(seen) if seen else -1, 0]) for _ in range(k)]
                    else:
                        pick = []
                    self.sel[at, h, : len(pick)] = torch.tensor(pick, dtype=torch.int32)
                at += 1
        self.pad, self.max_new = pad, max_new

    def run(self, q=None, out=None, scale=None, sel=None, stream=0, check=True):
        c = spin().SpinKV8(len(self.past), self.H * self.G, self.H, self.table.shape[2], self.pages.shape[0], pages=self.pages.cuda(),
                           scales=self.scales.cuda(), tails=self.tails.cuda(), table=self.table.cuda())
        s, self.cu = step_of(self.past, self.new, self.pad, self.max_new)
        q = self.q.cuda() if q is None else q
        out = torch.full_like(q, 7.0) if out is None else out
        c.attend_rows(s, q, out, self.sel.cuda() if sel is None else sel, scale=scale, stream=stream)
        torch.cuda.synchronize()
        self.c = c
        if check:
            c.check()
        return out.cpu()

    def same(self, out, scale=SCALE, q=None):
        want, bound = R.attend_rows(self.q if q is None else q, self.pages, self.scales, self.tails, self.table, self.past, self.cu, scale, self.sel)
        n = self.cu[-1]
        got, want, bound = out[:n].double(), want[:n], bound[:n]
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        miss = torch.where(nan, 0.0, (got - want).abs() - bound)
        assert float(miss.max()) <= 0 if n else True, (float(miss.max()), float((got - want).nan_to_num().abs().max()),
                                                       [int(x) for x in torch.nonzero(miss == miss.max())[0]])
        return want


def check(*args, scale=None, **kw):
    c = Case(*args, **kw)
    out = c.run(scale=scale)
    c.same(out, SCALE if scale is None else scale)
    if c.pad:
        assert (out[c.cu[-1]:] == 7.0).all()


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8, 11, 16])
def test_groups(group):
    check(2, group, [700, 64, 1000], [1, 3, 9], 4, seed=group)


@pytest.mark.parametrize("lists", ["random", "near", "wild", "none"])
def test_lists(lists):
    check(2, 4, [0, 640, 63, 1999, 127], [5, 3, 2, 40, 0], 6, lists=lists, seed=3)


@pytest.mark.parametrize("past", [0, 1, 62, 63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("new", [1, 2, 70])
def test_lengths(past, new):
    """Rows that see nothing, one token, whole pages and nothing else; newest tokens in the tail and in a page that the step completed."""
    check(1, 5, [past], [new], 1, lists="none" if past < 70 else "random", seed=past + new)


@pytest.mark.parametrize("k", [1, 2, 15, 33, 512])
def test_lengths_of_lists(k):
    check(1, 8, [3000], [6], k, seed=k)


@pytest.mark.parametrize("batch", [1, 33, 129, 200])
def test_batches_of_single_tokens(batch):
    rng = random.Random(batch)
    check(1, 4, [rng.choice([0, 63, 64, 500, 1300]) for _ in range(batch)], [1] * batch, 5, seed=batch, pad=3)


def test_a_chunk():
    check(2, 8, [1500, 0], [150, 90], 8, lists="near", seed=9, pad=5, max_new=2000)


@pytest.mark.parametrize("lists", ["apart", "late", "near", "random"])
@pytest.mark.parametrize("group,new,k", [(8, 32, 9), (8, 70, 2), (5, 60, 7), (16, 40, 5), (1, 200, 3), (3, 90, 6)])
def test_tiles_with_pages_of_their_own(lists, group, new, k):
    """Blocks of two tiles: pages of both, of one, of the other, and tiles that attend nothing."""
    check(1, group, [1984, 70], [new, 3], k, lists=lists, seed=group + new)


def test_one_long_list():
    """A tile that many CTAs share, beside small ones."""
    check(1, 2, [64 * 500, 100], [2, 1], 500, seed=12)


@pytest.mark.parametrize("pages", [2047, 2049, 5000, 100000])
def test_far_pages(pages):
    check(1, 3, [pages * PAGE - 5, 10], [7, 3], 9, seed=pages)


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0])
def test_scales_of_scores(scale):
    check(1, 4, [900], [4], 6, scale=scale, seed=1)


@pytest.mark.parametrize("spread", [1.0, 6.0])
def test_pages_of_very_different_scales(spread):
    check(2, 4, [2000, 1300], [5, 1], 12, spread=spread, seed=4)


@pytest.mark.parametrize("size", [1e-30, 1e-3, 1e3, 1e6, 1e15])
def test_scores_of_any_size(size):
    """Queries so large that one key takes all; so small that all count the same."""
    c = Case(1, 4, [1200], [5], 8, seed=5)
    c.q = (c.q.float() * size).to(torch.bfloat16)
    c.same(c.run())


def test_queries_of_mixed_size():
    c = Case(1, 8, [1200], [9], 8, seed=6)
    c.q = (c.q.float() * torch.exp2(torch.randint(-40, 12, (9, 8, 1)).float())).to(torch.bfloat16)
    c.q[:, :, ::3] *= 2.0 ** -9
    c.same(c.run())


def test_equal_scores_of_any_size():
    """Keys that are all the same: the mean of the values, however large the score."""
    for size in (1.0, 1e4, 1e9):
        c = Case(1, 2, [701], [3], 5, seed=7)  # (the last row sees whole pages alone)
        c.pages[:, 0] = c.pages[0, 0, 0]
        c.scales[:, 0] = 2.0 ** -4
        c.q = (c.q.float() * size).to(torch.bfloat16)
        c.same(c.run())


def test_what_is_not_finite():
    c = Case(2, 3, [700, 130], [6, 2], 3, seed=8, n_pages=60)
    c.scales[5, 0] = math.nan
    c.scales[9, 1] = math.nan
    c.scales[11] = math.nan
    c.tails[0, 0, 0, 3, 77] = math.inf
    c.tails[1, 1, 1, 2, 5] = math.nan
    c.q[1, 2, 9] = math.nan
    c.q[3, 4, 100] = -math.inf
    want = c.same(c.run())
    assert torch.isnan(want).any() and not torch.isnan(want).all()


def test_rows_that_see_nothing_are_zeros():
    """Whatever their queries hold."""
    c = Case(1, 4, [63, 127], [1, 1], 3, lists="none")
    c.q[0, 1, 5] = math.nan
    out = c.run()
    assert (out[:2] == 0).all()


def test_stale_rows_of_a_tail_and_unlisted_pages_may_hold_anything():
    c = Case(1, 4, [700], [3], 3, seed=2, n_pages=30)
    used = {int(c.table[0, 0, p]) for p in set(c.sel.flatten().tolist()) if p >= 0}
    out = c.run()
    c.tails[0, 0, :, 703 % 64:] = math.nan
    for i in range(30):
        if i not in used:
            c.pages[i], c.scales[i] = 0x7F, math.nan
    assert torch.equal(c.run(), out)


def test_bad_pages_are_left_out():
    c = Case(1, 4, [900, 900], [2, 1], 4, seed=3)
    a, b = int(c.sel[0, 0, 0]), int(c.sel[2, 0, 1])
    c.table[0, 0, a], c.table[1, 0, b] = -1, 10 ** 6
    c.same(c.run(check=False))
    assert int(c.c.error) == 32


def test_requests_that_are_out_of_range_are_left_out():
    c = Case(1, 2, [200, 100, 300], [2, 2, 2], 2, seed=3)
    c.past[1] = -3
    out = c.run(check=False)
    assert (out[2:4] == 7.0).all() and int(c.c.error) == 32
    c.past[1], c.new[1] = 100, 2
    want = c.run()
    assert torch.equal(out[:2], want[:2]) and torch.equal(out[4:], want[4:])


@pytest.mark.parametrize("new", [1, 11])
def test_layouts(new):
    """Queries inside a projection's output, heads before tokens, outputs in place."""
    c = Case(3, 4, [500, 1000], [new, new], 5, seed=new)
    plain = c.run()
    wide = torch.full((2 * new, 20, D), 3.0, dtype=torch.bfloat16, device="cuda")
    inside = wide[:, 4:16]
    inside.copy_(c.q)
    assert torch.equal(c.run(q=inside), plain)
    swapped = c.q.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(c.run(q=swapped, out=torch.empty_like(swapped)), plain)
    assert torch.equal(c.run(q=inside, out=inside), plain)
    assert (wide[:, :4] == 3.0).all() and (wide[:, 16:] == 3.0).all()


def test_results_do_not_change_from_run_to_run():
    c = Case(2, 8, [5000, 300], [40, 7], 30, lists="near", seed=1)
    first = c.run()
    for _ in range(3):
        assert torch.equal(c.run(), first)


@pytest.mark.parametrize("group,new", [(8, 96), (16, 9), (8, 20)])
def test_many_calls_in_a_row(group, new):
    """Blocks of many and of few steps, shared and not, on CTAs that are never in the same state: no wait runs out."""
    c = Case(2, group, [2500, 300, 64], [new, 7, 2], 16, lists="near", seed=new)
    first = c.run()
    st, _ = step_of(c.past, c.new)
    q, sel = c.q.cuda(), c.sel.cuda()
    outs = [torch.zeros_like(q) for _ in range(16)]
    for n in range(400):
        c.c.attend_rows(st, q, outs[n % 16], sel)
    torch.cuda.synchronize()
    c.c.check()
    for out in outs:
        assert torch.equal(out.cpu(), first)


def test_streams_and_graphs():
    c = Case(2, 4, [900, 1700], [3, 1], 6, seed=4)
    first = c.run()
    st, _ = step_of(c.past, c.new)
    q, sel = c.q.cuda(), c.sel.cuda()
    out = torch.zeros_like(q)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        c.c.attend_rows(st, q, out, sel, stream=side.cuda_stream)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), first)
    c.sel = c.sel.flip(0).contiguous()
    sel.copy_(c.sel)
    graph.replay()
    torch.cuda.synchronize()
    c.same(out.cpu())


def test_a_captured_call_keeps_the_workspace_that_it_was_captured_with():
    """Two graphs and eager calls of one handle, before and after its workspace grows; a capture that would make it grow is refused."""
    c = Case(2, 8, [2000, 300], [60, 7], 12, lists="near", seed=3)
    few, many = Case(2, 8, [2000, 300], [2, 0], 12, lists="near", seed=4), c
    want = many.run()
    h = spin().SpinKV8(2, 16, 2, c.table.shape[2], pages=c.c.pages, scales=c.c.scales, tails=c.c.tails, table=c.c.table)
    side, graphs, outs = torch.cuda.Stream(), [], []
    st, _ = step_of(few.past, few.new)
    q, sel = few.q.cuda(), few.sel.cuda()
    small = h.attend_rows(st, q, torch.zeros_like(q), sel).clone()
    large, lq, lsel = step_of(many.past, many.new)[0], many.q.cuda(), many.sel.cuda()
    torch.cuda.synchronize()
    for _ in range(2):
        outs.append(torch.zeros_like(q))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            h.attend_rows(st, q, outs[-1], sel, stream=side.cuda_stream)
    refused = torch.cuda.CUDAGraph()
    with torch.cuda.graph(refused, stream=side):
        with pytest.raises(ValueError, match="before capturing"):
            h.attend_rows(large, lq, torch.empty_like(lq), lsel, stream=side.cuda_stream)
    got = torch.zeros_like(lq)
    for _ in range(3):
        for g in graphs:
            g.replay()
        h.attend_rows(large, lq, got, lsel, stream=torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(got.cpu(), want)
        for o in outs:
            assert torch.equal(o, small)
            o.zero_()


def test_layers_share_what_their_calls_need():
    """A handle given as the workspace: the two have one between them, whichever of them makes it grow."""
    small, large = Case(2, 4, [900], [2], 6, seed=4), Case(2, 4, [900, 1700], [130, 1], 6, seed=5)
    wants = [small.run(), large.run()]
    handles = []
    for c in (large, small):
        handles.append(spin().SpinKV8(len(c.past), c.H * c.G, c.H, c.table.shape[2], pages=c.c.pages, scales=c.c.scales, tails=c.c.tails,
                                      table=c.c.table, workspace=handles[0] if handles else None))
    assert handles[0].workspace is handles[1].workspace
    for _ in range(2):
        for c, h, want in zip((small, large), handles[::-1], wants):
            q = c.q.cuda()
            assert torch.equal(h.attend_rows(step_of(c.past, c.new)[0], q, torch.full_like(q, 7.0), c.sel.cuda()).cpu(), want)
    assert len(handles[0]._spaces["attend_rows"]) == 2


def test_calls_at_the_same_time_with_workspaces_of_their_own():
    s = spin()
    c = Case(2, 8, [5000, 300], [40, 7], 30, lists="near", seed=1)
    want = c.run()
    st, _ = step_of(c.past, c.new)
    q, sel, n = c.q.cuda(), c.sel.cuda(), s.spin_kv8_attend_rows_workspace(c.c.c, sum(c.new), 30)
    streams = [torch.cuda.Stream() for _ in range(3)]
    spaces = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in streams]
    outs = [torch.zeros_like(q) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(30):
        for x, w, o in zip(streams, spaces, outs):
            c.c.attend_rows(st, q, o, sel, workspace=w, stream=x.cuda_stream)
    torch.cuda.synchronize()
    c.c.check()
    for o in outs:
        assert torch.equal(o.cpu(), want)


def test_the_handle_refuses():
    c = Case(2, 2, [100], [1], 3)
    c.run()
    st, _ = step_of([100], [1])
    q = c.q.cuda()
    for bad in (c.sel.cuda()[:, :1], c.sel.cuda()[0], c.sel.cuda().long()):
        with pytest.raises(ValueError, match="sel"):
            c.c.attend_rows(st, q, q, bad.contiguous())
    with pytest.raises(spin().SpinError, match="workspace"):
        c.c.attend_rows(st, q, q, c.sel.cuda(), workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("group,new", [(5, 1), (8, 5), (4, 90)])
def test_the_whole_path(group, new):
    """reserve, append, select and attend_rows, as a step runs them. With lists of all pages the answer is dense attention's; with
    short ones the restatement's over what the call listed."""
    s = spin()
    B, H, P = 3, 2, 24
    g = torch.Generator(device="cuda").manual_seed(new)
    rows = lambda n, h: torch.randn((n, h, D), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    c = s.SpinKV8(B, H * group, H, P, B * H * P, summaries=True, refs=True, rope=s.SpinRope.from_base(1e4))
    past = [0] * B
    for lens in ([1000, 63, 700], [new] * B, [new] * B):
        st, cu = step_of(past, lens)
        T = cu[-1]
        q, k, v = rows(T, H * group), rows(T, H), rows(T, H)
        c.reserve(st)
        c.append(st, q, k, v)
        for k_ in (6, P):
            sel = torch.empty((T, H, k_), dtype=torch.int32, device="cuda")
            c.select(st, q, sel)
            out = c.attend_rows(st, q, torch.empty_like(q), sel)
            c.check()
            if max(lens) > 100:
                continue
            want, bound = R.attend_rows(q.cpu(), c.pages.cpu(), c.scales.cpu(), c.tails.cpu(), c.table.cpu(), past, cu, SCALE, sel.cpu())
            assert ((out.cpu().double() - want).abs() <= bound).all()
        dense = c.attend(st, q, torch.empty_like(q))
        assert (out.float() - dense.float()).abs().max() < 0.02
        past = [a + n for a, n in zip(past, lens)]
