"""The page pool of the 8-bit cache on the GPU, against the restatement in kv8_pool_ref.py: bit for bit."""
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv8_pool_ref as R  # noqa: E402
from test_gpu_kv8 import D, PAGE, ints, spin, step_of  # noqa: E402


class Both:
    """A cache with random contents beside the restatement, in which a row is the number of its copy's origin."""

    def __init__(self, batch, heads, max_pages, n_pages, lengths=None, summaries=True, seed=0, shared=0):
        self.rng = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        self.B, self.H, self.P, self.N = batch, heads, max_pages, n_pages
        self.len = list(lengths) if lengths else [0] * batch
        order = list(range(n_pages))
        self.rng.shuffle(order)
        table, refs = [[[-1] * max_pages for _ in range(heads)] for _ in range(batch)], [0] * n_pages
        for b in range(batch):
            for h in range(heads):
                for p in range(self.len[b] // PAGE):
                    x = table[0][h][p] if b and p < min(shared, self.len[0] // PAGE) else order.pop()
                    table[b][h][p] = x
                    refs[x] += 1
        self.tails = torch.randn((batch, heads, 2, PAGE, D), generator=g).to(torch.bfloat16)
        self.sums = torch.randn((batch, heads, max_pages, D), generator=g)
        self.pages = torch.randint(0, 256, (n_pages, 2, PAGE, D), dtype=torch.uint8, generator=g)
        self.scales = torch.randn((n_pages, 2), generator=g)
        ids = lambda *shape: torch.arange(torch.tensor(shape).prod()).view(shape).tolist()  # noqa: E731
        self.ref = R.Pool(table, refs, ids(batch, heads, 2 * PAGE), ids(batch, heads, max_pages) if summaries else None)
        self.c = spin().SpinKV8(batch, heads, heads, max_pages, n_pages, table=ints(table), refs=ints(refs), tails=self.tails.cuda(),
                                pages=self.pages.cuda(), scales=self.scales.cuda(), summaries=self.sums.cuda() if summaries else False)
        self.free = torch.full((1,), -7, dtype=torch.int32, device="cuda")

    def same(self, error=0):
        assert self.c.table.cpu().tolist() == self.ref.table
        assert self.c.refs.cpu().tolist() == self.ref.refs
        want = self.tails.reshape(-1, D)[torch.tensor(self.ref.tails).flatten()].view(self.tails.shape)
        assert torch.equal(self.c.tails.cpu().view(torch.int16), want.view(torch.int16))
        if self.c.summaries is not None:
            want = self.sums.reshape(-1, D)[torch.tensor(self.ref.summaries).flatten()].view(self.sums.shape)
            assert torch.equal(self.c.summaries.cpu(), want)
        assert self.ref.error == error and int(self.c.error) == error
        if not error:
            self.c.check()

    def reserve(self, new, stream=0):
        s, _ = step_of(self.len, new)
        self.c.reserve(s, free_pages=self.free, stream=stream)
        torch.cuda.synchronize()
        assert int(self.free) == self.ref.reserve(self.len, new)

    def fork(self, src):
        length = ints(self.len)
        self.c.fork(length, ints(src))
        self.ref.fork(self.len, src)
        assert length.tolist() == self.len

    def compact(self):
        self.c.compact(free_pages=self.free)
        free, go = self.ref.compact()
        assert int(self.free) == free
        for a, z in go.items():
            self.pages[z], self.scales[z] = self.pages[a], self.scales[a]
        assert torch.equal(self.c.pages.cpu(), self.pages) and torch.equal(self.c.scales.cpu(), self.scales)


@pytest.mark.parametrize("n_pages", [1, 31, 33, 1023, 1024, 1025, 5000])
def test_reserve_takes_the_lowest_free_pages(n_pages):
    r = Both(3, 2, 40, n_pages, [min(64 * (n_pages // 8), 2000) // 3 * k for k in range(3)])
    r.reserve([0, 1, 200 if n_pages > 30 else 0])
    r.same()
    r.reserve([0, 1, 200 if n_pages > 30 else 0])  # again: entries that have a page keep it
    r.same()
    r.len = [n + 1 for n in r.len]
    r.reserve([63, 64, 0])
    r.same(R.CAPACITY if r.ref.error else 0)


@pytest.mark.parametrize("batch,heads,new", [(1, 1, 64), (1, 8, 8191), (37, 3, 700), (300, 1, 64), (130, 8, 1)])
def test_reserve_batches(batch, heads, new):
    rng = random.Random(batch)
    lengths = [rng.choice([0, 1, 63, 64, 65, 127, 500]) for _ in range(batch)]
    need = sum((n + new) // PAGE for n in lengths) * heads
    r = Both(batch, heads, (500 + new) // PAGE + 1, need + 77, lengths, summaries=False, seed=batch)
    r.reserve([rng.choice([new, new, 0, rng.randint(0, new)]) for _ in range(batch)])
    r.same()


def test_reserve_takes_all_or_nothing():
    r = Both(4, 2, 8, 12, [64, 0, 128, 0])  # 6 of 12 pages
    r.reserve([0, 64, 0, 256])              # 2 + 8 more
    r.same(R.CAPACITY)
    with pytest.raises(spin().SpinError, match="free pages"):
        r.c.check()
    r.c.error.zero_()
    r.ref.error = 0
    r.reserve([64, 64, 64, 0])              # 6: the last ones
    r.same()
    assert int(r.free) == 0


def test_reserve_leaves_out_what_is_out_of_range():
    r = Both(4, 2, 3, 40, [64, 0, 100, 0])
    r.len[1] = -5
    r.reserve([64, 64, 192, 70])
    r.same(R.INDEX | R.CAPACITY)  # request 2 would outgrow its row
    assert (r.c.table[1:3, :, 2] == -1).all()


@pytest.mark.parametrize("summaries", [False, True])
@pytest.mark.parametrize("src", [[0, 0, 0, 0, 0], [1, 2, 3, 4, 0], [1, 0, 2, 2, -1], [-1] * 5, [0, 1, 2, 3, 4], [4, 4, 1, 1, 3],
                                 [2, 2, 2, -1, 3]], ids=str)
@pytest.mark.parametrize("shared", [0, 2])
def test_fork_maps(src, summaries, shared):
    r = Both(5, 3, 11, 200, [300, 129, 64 * 11 + 63, 0, 191], summaries, shared=shared)
    r.reserve([64, 64, 0, 64, 70])  # entries beyond the complete pages: nobody's but their owner's
    r.fork(src)
    r.same()
    r.fork([0, 0, 1, 3, 3])
    r.same()


def test_fork_leaves_out_what_is_out_of_range():
    r = Both(6, 2, 4, 60, [200, 100, 300, 50, 10, 0])
    r.len[4], r.len[2] = -1, 10 ** 9
    r.fork([0, 7, 2, -2, 3, 1])
    r.same(R.INDEX)
    r.fork([4, 2, 2, 3, 4, 0])
    r.same(R.INDEX | R.CAPACITY)


@pytest.mark.parametrize("batch,max_pages", [(700, 5), (2500, 2), (4500, 1), (16384, 1)])
def test_fork_large_batches(batch, max_pages):
    """More rows than a CTA holds at 16 bytes each, and requests that change places in long cycles."""
    rng = random.Random(batch)
    r = Both(batch, 1, max_pages, batch * max_pages, [rng.randint(0, 64 * max_pages + 63) for _ in range(batch)], seed=batch)
    src = list(range(batch))
    rng.shuffle(src)
    for b in rng.sample(range(batch), batch // 10):
        src[b] = rng.choice([-1, rng.randrange(batch)])
    r.fork(src)
    r.same()


@pytest.mark.parametrize("n_pages,keep", [(64, 1.0), (64, 0.0), (1000, 0.5), (1025, 0.1), (3001, 0.9), (5000, 0.02)])
def test_compact(n_pages, keep):
    per = max(1, n_pages // 8)
    r = Both(4, 2, per, n_pages, [int(PAGE * per * keep)] * 4, seed=n_pages, shared=per // 3)
    r.compact()
    r.same()
    r.compact()  # nothing to do
    r.same()


def test_compact_reports_entries_of_free_pages():
    r = Both(2, 1, 4, 16, [128, 128])
    x = r.ref.refs.index(0)
    r.ref.table[0][0][3], r.ref.table[1][0][3] = x, 99
    r.c.table[0, 0, 3], r.c.table[1, 0, 3] = x, 99
    r.c.compact()
    _, go = r.ref.compact()
    for a, z in go.items():
        r.pages[z] = r.pages[a]
    r.same(R.INDEX)


@pytest.mark.parametrize("seed", range(4))
def test_a_run_of_calls(seed):
    rng = random.Random(seed)
    B, P = 9, 12
    r = Both(B, 2, P, 160, seed=seed)
    for _ in range(30):
        what = rng.choice(["step", "step", "fork", "compact"])
        if what == "step":
            new = [rng.randint(0, max(0, min(150, PAGE * P - n))) for n in r.len]
            r.reserve(new)
            if r.ref.error:
                r.same(R.CAPACITY)
                r.ref.error = 0
                r.c.error.zero_()
                continue
            r.len = [a + n for a, n in zip(r.len, new)]
        elif what == "fork":
            r.fork([rng.choice([b, b, -1, rng.randrange(B)]) for b in range(B)])
        else:
            r.compact()
        r.same()


def test_forks_answer_like_their_source():
    """A prompt, forked and compacted in between, then grown apart: attention of the copies is that of requests of their own."""
    s = spin()
    B, H, G, P = 4, 2, 3, 12
    g = torch.Generator(device="cuda").manual_seed(3)
    rows = lambda n, h: torch.randn((n, h, D), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    pooled = s.SpinKV8(B, H * G, H, P, B * H * P, summaries=True, refs=True)
    alone = s.SpinKV8(B, H * G, H, P, B * H * P, summaries=True, table=torch.randperm(B * H * P, device="cuda").to(torch.int32).view(B, H, P))
    n = 333
    k, v, q = rows(n, H), rows(n, H), rows(n, H * G)
    one, _ = step_of([0] * B, [n, 0, 0, 0])
    pooled.reserve(one)
    pooled.append(one, None, k, v)
    each, _ = step_of([0] * B, [n] * B)
    alone.append(each, None, *(x.repeat(B, 1, 1) for x in (k, v)))
    lengths = ints([n, 0, 0, 0])
    pooled.fork(lengths, ints([0, 0, 0, 0]))
    assert lengths.tolist() == [n] * B
    assert int((pooled.refs > 0).sum()) == H * (n // PAGE) and int(pooled.refs.max()) == B
    grow, _ = step_of([n] * B, [200, 3, 64, 130])
    T = grow.total_new
    k, v, q = rows(T, H), rows(T, H), rows(T, H * G)
    pooled.compact()
    pooled.reserve(grow)
    outs = []
    for c in (pooled, alone):
        c.append(grow, None, k, v)
        out = torch.empty_like(q)
        c.attend(grow, q, out)
        c.check()
        outs.append(out)
    assert torch.equal(*outs)
    for b, m in enumerate([200, 3, 64, 130]):
        whole = (n + m) // PAGE
        assert torch.equal(pooled.summaries[b, :, :whole], alone.summaries[b, :, :whole])


def test_captured_calls_replay():
    r = Both(3, 2, 6, 50, [100, 0, 64])
    step, _ = step_of(r.len, [64, 64, 64])
    lengths, src = ints(r.len), ints([0, 0, 2])
    before = [t.clone() for t in (r.c.table, r.c.refs, r.c.tails, r.c.summaries, r.c.pages, r.c.scales, lengths)]
    st = torch.cuda.Stream()
    with pytest.raises(ValueError, match="before capturing"):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            r.c.reserve(step, stream=st.cuda_stream)
    torch.cuda.synchronize()
    r.c._space("pool", r.c._pool_bytes, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        r.c.reserve(step, free_pages=r.free, stream=st.cuda_stream)
        r.c.fork(lengths, src, stream=st.cuda_stream)
        r.c.compact(stream=st.cuda_stream)
    for _ in range(3):
        for t, x in zip((r.c.table, r.c.refs, r.c.tails, r.c.summaries, r.c.pages, r.c.scales, lengths), before):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        ref = R.Pool(before[0].tolist(), before[1].tolist())
        ref.reserve(r.len, [64] * 3)
        n = list(r.len)
        ref.fork(n, [0, 0, 2])
        ref.compact()
        assert r.c.table.tolist() == ref.table and r.c.refs.tolist() == ref.refs and lengths.tolist() == n
    r.c.check()


@pytest.mark.parametrize("batch", [3413, 3414, 4094, 4095, 4096, 4097])
def test_fork_batches_at_the_borders_of_shared_memory(batch):
    """40 and 48 KB of a CTA's list of moves, and the last batch that a CTA holds 16 bytes each of."""
    rng = random.Random(batch)
    r = Both(batch, 1, 1, batch, [rng.randint(0, 127) for _ in range(batch)], seed=batch)
    src = [rng.choice([-1, rng.randrange(batch)]) for _ in range(batch)]
    src[0], src[-1] = batch - 1, 0
    r.fork(src)
    r.same()


@pytest.mark.parametrize("n_pages", [10485760, 10486784, 12050000, 12300000, 12545000, 12582912, 12583936, 1 << 24])
def test_large_pools(n_pages):
    """Pools whose sums take 40, 48 and 64 KB. No page moves, so that there need be none: their counts alone are looked at."""
    from sparse_attention_tiered_gb300 import _binding as B

    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    h = spin().SpinKV8(2, 1, 1, 4, 8, table=ints([[[0, 1, -1, -1], [2, -1, -1, -1]]]).view(2, 1, 4))
    refs[:3] = 1
    c = h.c
    c.n_pages = n_pages
    free, ws = ints([0]), torch.empty(B.spin_kv8_pool_workspace(c), dtype=torch.uint8, device="cuda")
    step, _ = step_of([128, 64], [64, 128])
    B.spin_kv8_compact(c, refs.data_ptr(), free.data_ptr(), ws.data_ptr(), ws.numel())
    assert int(free) == n_pages - 3
    B.spin_kv8_reserve(c, step.c, refs.data_ptr(), free.data_ptr(), ws.data_ptr(), ws.numel())
    assert int(free) == n_pages - 6
    B.spin_kv8_compact(c, refs.data_ptr(), free.data_ptr(), ws.data_ptr(), ws.numel())
    assert int(free) == n_pages - 6
    assert h.table.flatten().tolist() == [0, 1, 3, -1, 2, 4, 5, -1]
    refs[:] = 1  # the last page is the one that is left
    refs[-1] = 0
    h.table[0, 0, 3] = -1
    one, _ = step_of([192, 0], [64, 0])
    B.spin_kv8_reserve(c, one.c, refs.data_ptr(), free.data_ptr(), ws.data_ptr(), ws.numel())
    assert int(free) == 0 and int(h.table[0, 0, 3]) == n_pages - 1 and int(refs.min()) == 1
    B.spin_kv8_status(c)
