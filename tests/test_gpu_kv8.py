"""The 8-bit paged cache on the GPU, against the 64-bit restatement in kv8_ref.py."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv8_ref as R  # noqa: E402

D, PAGE = 128, 64


def spin():
    import sparse_attention_tiered_gb300 as s
    return s


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def step_of(past, new, pad=0, max_new=None):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return spin().SpinKV8Step(ints(past), ints(cu), cu[-1] + pad, max_new or max(1, max(new))), cu


def freqs(rot, base=10000.0):
    return [base ** (-2.0 * j / rot) for j in range(rot // 2)]


class Pair:
    """The library's cache beside the reference's, fed the same rows."""

    def __init__(self, batch, kv_heads, group, max_pages, rot=128, interleaved=False, summaries=False, seed=0, spare=5):
        self.g = torch.Generator().manual_seed(seed)
        self.B, self.H, self.G = batch, kv_heads, group
        self.f = freqs(rot) if rot else []
        n = batch * kv_heads * max_pages + spare
        table = torch.randperm(n, generator=self.g)[: batch * kv_heads * max_pages].view(batch, kv_heads, max_pages)
        self.c = spin().SpinKV8(batch, kv_heads * group, kv_heads, max_pages, n, rope=spin().SpinRope(self.f, interleaved),
                                table=table.to(torch.int32).cuda(), summaries=summaries)
        self.c.pages.fill_(0x55)
        self.ref = R.Cache(batch, kv_heads, self.f, interleaved)
        self.len = [0] * batch

    def rand(self, *shape, scale=1.0):
        return (torch.randn(shape, generator=self.g) * scale).to(torch.bfloat16)

    def append(self, new, pad=0, k=None, v=None, q=None, positions=None, stream=0):
        s, cu = step_of(self.len, new, pad)
        T = s.total_new
        k = self.rand(T, self.H, D) if k is None else k
        v = self.rand(T, self.H, D) if v is None else v
        q = self.rand(T, self.H * self.G, D) if q is None else q
        qd = q.cuda()
        pos = None if positions is None else positions.to(torch.int32).cuda()
        out = torch.full_like(qd, 7.0)
        self.c.append(s, qd, k.cuda(), v.cuda(), out, positions=pos, stream=stream)
        self.ref.append(k, v, cu, positions)
        self.last = (s, cu, q, out, list(self.len))
        self.len = [a + b for a, b in zip(self.len, new)]
        return s, cu, q, out

    def state(self):
        c = self.c
        return c.pages.cpu(), c.scales.cpu(), c.tails.cpu(), c.table.cpu()

    def check_queries(self, positions=None):
        s, cu, q, out, past = self.last
        got = out.cpu().double()
        for b in range(self.B):
            r0, r1 = cu[b], cu[b + 1]
            if r1 == r0:
                continue
            pos = torch.arange(past[b], past[b] + r1 - r0) if positions is None else positions[r0:r1]
            x = q[r0:r1].double()
            want = R.rotate(x, pos, self.f, self.ref.i)
            slack = R.rotate_slack(x, self.f, self.ref.i)
            tol = R.EPS_BF16 * (want.abs() + slack) + slack  # one rounding to bf16
            assert ((got[r0:r1] - want).abs() <= tol).all()
        assert (got[cu[-1]:] == 7.0).all()  # rows behind the last request

    def check_cache(self):
        pages, scales, tails, table = self.state()
        used = set()
        for b in range(self.B):
            n = self.len[b]
            for h in range(self.H):
                slack = R.rotate_slack(self.ref.x[b][:, h:h + 1], self.f, self.ref.i)[:, 0]
                for p in range(n // PAGE):
                    i = int(table[b, h, p])
                    used.add(i)
                    at = slice(p * PAGE, (p + 1) * PAGE)
                    want_v, sv = R.quantise(self.ref.v[b][at, h])
                    assert float(scales[i, 1]) == sv or (math.isnan(sv) and math.isnan(float(scales[i, 1])))
                    assert torch.equal(R.decode_e4m3(pages[i, 1]), want_v)
                    x = self.ref.x[b][at, h]
                    near = (x.abs() + slack[at]) * (1 + R.EPS_BF16)  # a bf16 key is at most this
                    far = (x.abs() - slack[at]) * (1 - R.EPS_BF16)
                    sk = float(scales[i, 0])
                    assert R.scale_for(float(far.max())) <= sk <= R.scale_for(float(near.max()))
                    got = R.decode_e4m3(pages[i, 0]) * sk
                    # bf16, then e4m3: half a step each (2^-8, 2^-4, or half of the smallest step of 2^-9)
                    tol = slack[at] + R.EPS_BF16 * near + torch.maximum(near * 2.0 ** -4, torch.full_like(x, sk * 2.0 ** -10))
                    assert ((got - x).abs() <= tol).all()
                    if self.c.summaries is not None:
                        mean = x.mean(0)
                        mtol = (slack[at] + R.EPS_BF16 * near).mean(0) + 64 * 2.0 ** -24 * x.abs().mean(0)
                        assert ((self.c.summaries[b, h, p].cpu().double() - mean).abs() <= mtol).all()
                at = slice(n - n % PAGE, n)
                t = tails[b, h, :, : n % PAGE].double()
                assert torch.equal(t[1], self.ref.v[b][at, h])
                x = self.ref.x[b][at, h]
                assert ((t[0] - x).abs() <= slack[at] + R.EPS_BF16 * (x.abs() + slack[at])).all()
        for i in range(self.c.n_pages):  # pages that hold nothing yet
            if i not in used:
                assert (pages[i] == 0x55).all()
        self.c.check()

    def check_attend(self, q=None, scale=None, sel=None, step=None, cu=None, past=None):
        if step is None:
            step, cu, _, _, past = self.last
        T = step.total_new
        q = self.rand(T, self.H * self.G, D, scale=2.0) if q is None else q
        out = torch.full((T, self.H * self.G, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.c.attend(step, q.cuda(), out, scale=scale, sel=None if sel is None else sel.cuda())
        want, tol = R.attend(q, *self.state(), past, cu, 1 / math.sqrt(D) if scale is None else scale, sel)
        got = out.cpu().double()
        assert (got[cu[-1]:] == 7.0).all()  # rows behind the last request
        got, want, tol = got[: cu[-1]], want[: cu[-1]], tol[: cu[-1]]
        nan = torch.isnan(want)
        assert torch.equal(nan, torch.isnan(got))
        bad = ((got - want).abs() > tol) & ~nan
        assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol)[~nan].max()))
        self.c.check()
        return got


# ---------------------------------------------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (64, False), (96, True), (32, False), (16, True), (0, False)])
def test_append_rotations(rot, interleaved):
    p = Pair(3, 2, 3, 4, rot, interleaved, summaries=True, seed=rot)
    for new in ([5, 1, 0], [70, 63, 64], [1, 130, 1]):
        p.append(new)
        p.check_queries()
    p.check_cache()


@pytest.mark.parametrize("H,G", [(1, 1), (3, 5), (8, 8), (2, 16), (5, 1)])
def test_append_head_layouts(H, G):
    p = Pair(2, H, G, 3, seed=H * 100 + G)
    for new in ([1, 129], [63, 1], [1, 1]):
        p.append(new)
        p.check_queries()
    p.check_cache()


def test_append_many_requests_one_token():
    """More requests than one probe of the search covers, some without a token, some completing a page."""
    B = 70
    p = Pair(B, 1, 2, 2, seed=1)
    p.append([(b * 7) % 64 for b in range(B)])
    p.check_queries()
    for i in range(3):
        p.append([0 if b % 11 == i else 1 for b in range(B)], pad=i)
        p.check_queries()
    p.append([63 if b % 3 else 0 for b in range(B)])
    p.check_cache()


def test_append_padding_rows_are_left():
    p = Pair(2, 2, 2, 2, seed=2)
    p.append([3, 66], pad=9)
    p.check_queries()
    p.check_cache()


def test_append_in_pieces_changes_no_bit():
    """One prompt at once, and the same prompt in pieces that end everywhere in a page."""
    n = 64 * 5 + 17
    a, b = Pair(1, 2, 1, 6, summaries=True, seed=3), Pair(1, 2, 1, 6, summaries=True, seed=3)
    k, v, q = a.rand(n, 2, D), a.rand(n, 2, D), a.rand(n, 2, D)
    a.append([n], k=k, v=v, q=q)
    whole, at, pieces = a.last[3].clone(), 0, []
    for m in (1, 62, 1, 1, 63, 65, 100, 3, 41):
        b.append([m], k=k[at:at + m], v=v[at:at + m], q=q[at:at + m])
        pieces.append(b.last[3].clone())
        at += m
    assert at == n
    assert torch.equal(torch.cat(pieces), whole)
    rest = n % PAGE
    assert torch.equal(a.c.pages, b.c.pages) and torch.equal(a.c.scales, b.c.scales)
    assert torch.equal(a.c.tails[..., :rest, :], b.c.tails[..., :rest, :])
    assert torch.equal(a.c.summaries, b.c.summaries)
    a.check_cache()


def test_append_codes_are_the_bf16_rows_nearest():
    """63 rows read back from the tail, then the 64th: the codes are exactly the rounding of those rows."""
    p = Pair(1, 3, 1, 1, seed=4)
    p.append([63])
    t = p.c.tails.clone().cpu()
    p.append([1])
    pages, scales, tails, table = p.state()
    for h in range(3):
        i = int(table[0, h, 0])
        last = p.ref.k[0][63:, h]
        rows = torch.cat([t[0, h, 0, :63].double(), last])
        want, s = R.quantise(rows)
        assert float(scales[i, 0]) == s
        assert torch.equal(R.decode_e4m3(pages[i, 0])[:63], want[:63])


def test_append_far_positions():
    """Positions of any size, given row by row: the angle's error does not grow with them."""
    p = Pair(2, 1, 2, 2, seed=5)
    pos = torch.tensor([0, 1, 2 ** 20 + 3, 2 ** 31 - 1, 12345678, 7, 2 ** 30, 99, 3, 2 ** 24 + 1])
    p.append([4, 6], positions=pos)
    p.check_queries(pos)
    p.check_cache()


def test_append_positions_with_rows_behind():
    """positions has a row for every row of k, those behind the last request's among them."""
    p = Pair(2, 1, 2, 2, seed=8)
    pos = torch.tensor([5, 6, 70, 1, 0, 9, 10, 11, 12, 13, 2 ** 30, -1, 8, 8, 8])
    p.append([4, 6], pad=5, positions=pos)
    p.check_queries(pos)
    p.check_cache()


def test_append_strided_and_in_place():
    """q, k and v as slices of one projection, q rotated in place, heads-first keys."""
    p = Pair(2, 2, 3, 3, seed=6)
    T, new = 70, [66, 4]
    rows = p.rand(T, (6 + 2 + 2) * D).cuda()
    q = rows[:, : 6 * D].view(T, 6, D)
    k = rows[:, 6 * D:8 * D].view(T, 2, D)
    v = rows[:, 8 * D:].view(T, 2, D)
    kk, vv, qq = k.cpu(), v.cpu(), q.cpu()
    k_first = k.transpose(0, 1).contiguous().transpose(0, 1)
    s, cu = step_of([0, 0], new)
    assert p.c.append(s, q, k_first, v) is q
    p.ref.append(kk, vv, cu)
    p.last, p.len = (s, cu, qq, q, [0, 0]), new
    p.check_queries()
    p.check_cache()
    assert torch.equal(k.cpu(), kk) and torch.equal(v.cpu(), vv)
    # keys and values alone
    p2 = Pair(2, 2, 3, 3, seed=6)
    p2.c.append(s, None, k, v)
    p2.ref.append(kk, vv, cu)
    p2.len = new
    p2.check_cache()


def test_append_values_at_the_borders():
    """All-zero halves, halves at 448 * 2^n exactly and just above, the smallest and largest bf16 values,
    infinities and NaN (not rotated, so that they reach the page as they are)."""
    p = Pair(1, 1, 1, 9, rot=0, seed=7)
    k, v = torch.zeros(64 * 8, 1, D), torch.zeros(64 * 8, 1, D)
    base = torch.linspace(-1, 1, 64 * D).view(64, 1, D)
    k[64:128], v[64:128] = base * 448, base * 449.5          # bf16(449.5) = 450 > 448
    k[128:192], v[128:192] = base * 2.0 ** -80, base * 2.0 ** -70
    k[192:256], v[192:256] = base * 3e38, base * 2.0 ** 120
    k[256:320] = base
    k[300, 0, 5] = math.inf
    v[256:320] = base
    v[320:384] = base
    v[383, 0, 127] = math.nan
    k[320:384] = base
    k[384, 0, 0], v[447, 0, 127] = 1.0, -2.0 ** -64 * 448
    k[448:512], v[448:512] = base * 1.75, base * 1.7578125
    p.append([512], k=k.to(torch.bfloat16), v=v.to(torch.bfloat16))
    p2 = Pair(1, 1, 1, 9, rot=0, seed=7)
    for at in range(0, 512, 61):
        p2.append([min(61, 512 - at)], k=k[at:at + 61].to(torch.bfloat16), v=v[at:at + 61].to(torch.bfloat16))
    for c in (p, p2):
        pages, scales, tails, table = c.state()
        for page in range(8):
            i = int(table[0, 0, page])
            for half, x in ((0, c.ref.k[0]), (1, c.ref.v[0])):
                want, s = R.quantise(x[page * 64:(page + 1) * 64, 0])
                assert float(scales[i, half]) == s or (math.isnan(s) and math.isnan(float(scales[i, half])))
                assert torch.equal(R.decode_e4m3(pages[i, half]), want)


# ---------------------------------------------------------------------------------------------------------------
# attend
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 1000, 4097])
def test_attend_one_token(n):
    p = Pair(1, 2, 4, n // 64 + 1, seed=n)
    if n > 1:
        p.append([n - 1])
    p.append([1])
    p.check_attend()


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 12, 16])
def test_attend_groups(G):
    p = Pair(3, 2, G, 8, seed=G)
    p.append([200, 64, 399])
    p.append([1, 1, 1])
    p.check_attend()
    p.append([3, 0, 2])
    p.check_attend()


@pytest.mark.parametrize("new", [[2, 3], [5, 0], [8, 8], [16, 1], [33, 7], [64, 64], [100, 1], [257, 130], [600, 5]], ids=str)
@pytest.mark.parametrize("G", [1, 5, 8])
def test_attend_several_tokens(new, G):
    p = Pair(2, 2, G, 20, seed=new[0] * 10 + G)
    p.append([77, 320])
    p.append(new, pad=3)
    p.check_attend()


@pytest.mark.parametrize("n", [1, 2, 64, 65, 128, 129, 300, 1025])
def test_attend_prompt_from_nothing(n):
    p = Pair(2, 1, 8, 20, seed=n)
    p.append([n, max(1, n // 3)])
    p.check_attend()


def test_attend_ragged_batch_with_empty_requests():
    new = [0, 1, 1, 0, 1, 1, 1, 0]
    p = Pair(8, 2, 5, 40, seed=11)
    p.append([0, 0, 2500, 3, 64, 128, 1, 0])
    p.append(new, pad=2)
    p.check_attend()


def test_attend_mixed_batch():
    """A prompt, a chunk and single tokens in one call."""
    p = Pair(4, 2, 5, 40, seed=12)
    p.append([0, 700, 2000, 64])
    p.append([300, 64, 1, 1])
    p.check_attend()


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 0.02])
def test_attend_scales(scale):
    p = Pair(1, 2, 4, 5, seed=13)
    p.append([250])
    p.append([1])
    p.check_attend(scale=scale)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
def test_attend_scales_of_many_rows(scale):
    p = Pair(2, 2, 4, 5, seed=53)
    p.append([200, 30])
    p.append([40, 9])
    p.check_attend(scale=scale)


@pytest.mark.parametrize("new", [1, 3, 30, 90], ids=["one", "few", "shared", "many"])
@pytest.mark.parametrize("steep", [8.0, 40.0, -40.0])
def test_attend_scores_that_rise_and_fall(new, steep):
    """Scores along the cache rise (or fall) by up to 2^60 in weight from page to page, and the values' scales
    jump: what was added up so far is scaled down again and again, and a page may outweigh all before it."""
    p = Pair(1, 2, 5, 12, rot=0, seed=54)
    n = 64 * 10 + 37 + new
    u = p.rand(1, 1, D).sign().float()
    along = torch.linspace(0, 1, n)[:, None, None]
    k = u * along * steep + torch.randn((n, 2, D), generator=p.g)
    size = torch.exp2(torch.randint(-25, 25, (12,), generator=p.g).float()).repeat_interleave(64)[:n, None, None]
    v = torch.randn((n, 2, D), generator=p.g) * size
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    p.append([n - new], k=k[:-new], v=v[:-new])
    p.append([new], k=k[-new:], v=v[-new:])
    p.check_attend(q=(u * torch.ones(new, 10, 1) + 0.3 * torch.randn((new, 10, D), generator=p.g)).to(torch.bfloat16))


@pytest.mark.parametrize("new", [[2, 1], [30, 5], [90, 3]], ids=str)
@pytest.mark.parametrize("x", [math.nan, math.inf, -math.inf])
def test_attend_queries_that_are_not_finite(new, x):
    """NaN for the rows whose query holds one, and for no other."""
    p = Pair(2, 2, 3, 6, seed=55)
    p.append([300, 100])
    p.append(new)
    q = p.rand(sum(new), 6, D)
    q[1, 4, 17] = q[sum(new) - 1, 0, 127] = x
    s, cu, _, _, past = p.last
    out = torch.empty_like(q, device="cuda")
    p.c.attend(s, q.cuda(), out)
    got = out.cpu().double()
    hit = torch.zeros(got.shape[:2], dtype=torch.bool)
    hit[1, 4] = hit[-1, 0] = True
    assert torch.isnan(got[hit]).all()
    want, tol = R.attend(torch.nan_to_num(q, nan=0.0, posinf=0.0, neginf=0.0), *p.state(), past, cu, 1 / math.sqrt(D))
    assert ((got - want).abs() <= tol)[~hit].all()


@pytest.mark.parametrize("batch,most", [(32, 1), (33, 1), (400, 1), (700, 3), (40, 17), (700, 17), (4100, 17)])
def test_attend_many_requests(batch, most):
    """More requests than threads, than warps' lanes, than the many-row launch plans at once; most of them short,
    some without new tokens."""
    p = Pair(batch, 1, 2, 3, rot=0, seed=batch + most)
    past = torch.randint(0, 140, (batch,), generator=p.g).tolist()
    new = [[1, 0, 1, 1, 2][i % 5] if most > 1 else [1, 1, 0][i % 3] for i in range(batch)]
    if most > 1:
        new[batch // 2] = new[batch - 2] = most
    p.append(past)
    p.append(new, pad=1)
    p.check_attend()


@pytest.mark.parametrize("bound", [8, 40, 2000])
def test_attend_within_a_larger_bound(bound):
    """max_new is a bound: what a captured step of drafts or chunks does when it replays with fewer tokens."""
    p = Pair(3, 2, 4, 9, seed=56)
    p.append([300, 64, 0])
    p.append([1, 0, 5], pad=4)
    _, cu, _, _, past = p.last
    s, _ = step_of(past, [1, 0, 5], pad=4, max_new=bound)
    p.check_attend(step=s, cu=cu, past=past)


@pytest.mark.parametrize("new", [[1, 1, 1], [4, 1, 9]])
def test_attend_selected_pages(new):
    p = Pair(3, 2, 4, 32, seed=14)
    p.append([1500, 640 - new[1], 100])
    p.append(new)
    full = [n // 64 for n in p.len]
    sel = torch.full((6, 7), -1, dtype=torch.int32)
    for u in range(6):
        f = full[u // 2]
        some = torch.randperm(f, generator=p.g)[:5].sort().values
        sel[u, : len(some)] = some
        sel[u, 6] = f + (u % 3)  # not complete: no page
    sel[3] = -1                  # request 1's tail is empty: its rows see nothing
    assert p.len[1] % 64 == 0
    got = p.check_attend(sel=sel)
    r = p.last[1][1]
    assert (got[r:r + new[1], 4:8] == 0).all()
    p.check_attend(sel=sel.flip(1).contiguous())  # any order


def test_attend_large_and_small_values():
    """Blocks of very different sizes in one cache: no block's weight or values are lost."""
    p = Pair(1, 1, 2, 12, rot=0, seed=15)
    n = 64 * 9 + 20
    k, v = torch.randn((n, 1, D), generator=p.g), torch.randn((n, 1, D), generator=p.g)
    size_k = torch.exp2(torch.randint(-6, 3, (10,), generator=p.g).float()).repeat_interleave(64)[:n, None, None]
    size_v = torch.exp2(torch.tensor([-40, 30, -20, 0, 3, 60, -60, 10, -3, 5]).float()).repeat_interleave(64)[:n, None, None]
    p.append([n - 1], k=(k * size_k)[:-1].to(torch.bfloat16), v=(v * size_v)[:-1].to(torch.bfloat16))
    p.append([1], k=(k * size_k)[-1:].to(torch.bfloat16), v=(v * size_v)[-1:].to(torch.bfloat16))
    p.check_attend()
    # the same without the block that outweighs all others
    q = p.rand(1, 2, D)
    p.check_attend(q=q, sel=torch.tensor([[0, 2, 3, 6]], dtype=torch.int32))
    p.check_attend(q=q, sel=torch.tensor([[0, 6]], dtype=torch.int32))
    p.check_attend(q=q * 60, sel=torch.tensor([[0, 1, 2, 3, 4]], dtype=torch.int32))


def test_attend_all_zero_keys_and_values():
    p = Pair(1, 1, 3, 4, rot=0, seed=16)
    z = torch.zeros((130, 1, D), dtype=torch.bfloat16)
    p.append([130], k=z, v=z)
    p.check_attend()
    p.append([1], k=z[:1], v=p.rand(1, 1, D))
    p.check_attend()


@pytest.mark.parametrize("where", ["page", "tail"])
@pytest.mark.parametrize("what", ["key", "value"])
@pytest.mark.parametrize("x", [math.nan, math.inf, -math.inf])
def test_attend_values_that_are_not_finite(where, what, x):
    """A query that sees the token (its page, once complete) gets NaN; one that does not is exact."""
    p = Pair(1, 1, 2, 6, rot=0, seed=17)
    n = 64 * 3 + 30
    k, v = p.rand(n, 1, D), p.rand(n, 1, D)
    bad = 64 * 2 + 5 if where == "page" else 64 * 3 + 20
    (k if what == "key" else v)[bad, 0, 3] = x
    p.append([100], k=k[:100], v=v[:100])
    p.append([n - 100], k=k[100:], v=v[100:])
    s, cu, _, _, past = p.last
    q = p.rand(n - 100, 2, D)
    out = torch.empty((n - 100, 2, D), dtype=torch.bfloat16, device="cuda")
    p.c.attend(s, q.cuda(), out)
    first = (128 if where == "page" else bad) - 100  # the first row that sees it
    got = out.cpu()
    assert torch.isnan(got[first:]).all()
    # the rows before, against a cache whose bad token is finite
    pages, scales, tails, table = p.state()
    scales, tails = torch.nan_to_num(scales, nan=1.0), torch.nan_to_num(tails, nan=0.0, posinf=0.0, neginf=0.0)
    want, tol = R.attend(q, pages, scales, tails, table, past, cu, 1 / math.sqrt(D))
    assert ((got.double() - want).abs() <= tol)[:first].all()


def test_attend_strided_rows():
    p = Pair(2, 2, 3, 4, seed=18)
    p.append([100, 20])
    p.append([2, 1])
    s, cu, _, _, past = p.last
    q = p.rand(3, 6, D)
    wide = torch.zeros((3, 9, D), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:8] = q.cuda()
    first = torch.full((6, 5, D), 7.0, dtype=torch.bfloat16, device="cuda")  # heads first, with room
    p.c.attend(s, wide[:, 2:8], first[:, 1:4].transpose(0, 1))
    want, tol = R.attend(q, *p.state(), past, cu, 1 / math.sqrt(D))
    assert ((first[:, 1:4].transpose(0, 1).cpu().double() - want).abs() <= tol).all()
    assert (first[:, 0] == 7).all() and (first[:, 4] == 7).all()


def test_attend_twice_gives_the_same_bits():
    p = Pair(5, 2, 8, 60, seed=19)
    p.append([3000, 17, 900, 64, 2222])
    p.append([1, 1, 1, 1, 1])
    q = p.rand(5, 16, D).cuda()
    outs = [torch.empty_like(q) for _ in range(3)]
    for o in outs:
        p.c.attend(p.last[0], q, o)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ---------------------------------------------------------------------------------------------------------------
# what the device reports
# ---------------------------------------------------------------------------------------------------------------
def code_of(c):
    from sparse_attention_tiered_gb300._binding import SpinError
    with pytest.raises(SpinError) as e:
        c.check()
    return e.value.code


def test_page_ids_outside_the_pool():
    from sparse_attention_tiered_gb300._binding import SPIN_ERR_INVALID
    for bad in (-1, 10 ** 6):
        p = Pair(2, 1, 2, 3, seed=20)
        p.append([60, 130])
        p.c.check()
        p.c.table[0, 0, 0] = bad
        before = p.c.pages.clone()
        p.append([10, 1])
        assert code_of(p.c) == SPIN_ERR_INVALID
        assert torch.equal(p.c.pages, before)
        # attention leaves the page out, and says so
        p.c.error.zero_()
        s, cu, _, _, past = p.last
        q = p.rand(11, 2, D)
        out = torch.empty((11, 2, D), dtype=torch.bfloat16, device="cuda")
        p.c.attend(s, q.cuda(), out)
        assert code_of(p.c) == SPIN_ERR_INVALID
        want, tol = R.attend(q, *p.state(), past, cu, 1 / math.sqrt(D))
        assert ((out.cpu().double() - want).abs() <= tol).all()


def test_lengths_out_of_range():
    from sparse_attention_tiered_gb300._binding import SPIN_ERR_CAPACITY, SPIN_ERR_INVALID
    sp = spin()
    for past, cu, total, most, code in (([0, -1], [0, 1, 2], 2, 1, SPIN_ERR_INVALID), ([0, 3 * 64], [0, 1, 65], 65, 64, SPIN_ERR_CAPACITY),
                                        ([0, 5], [0, 1, 9], 2, 8, SPIN_ERR_INVALID), ([0, 5], [0, 1, 4], 4, 2, SPIN_ERR_INVALID)):
        p = Pair(2, 1, 2, 3, seed=21)
        s = sp.SpinKV8Step(ints(past), ints(cu), total, most)
        q, k, v = (p.rand(total, h, D).cuda() for h in (2, 1, 1))
        out = torch.full_like(q, 7.0)
        pages, tails = p.c.pages.clone(), p.c.tails[1].clone()
        p.c.append(s, q, k, v, out)
        assert code_of(p.c) == code
        assert torch.equal(p.c.pages, pages) and torch.equal(p.c.tails[1], tails)
        assert (out[1:] == 7.0).all() and not (out[0] == 7.0).all()
        assert torch.equal(p.c.tails[0, 0, 1, 0], v[0, 0])
        p.c.error.zero_()
        out.fill_(7.0)
        p.c.attend(s, q, out)
        assert code_of(p.c) == code
        assert (out[1:] == 7.0).all()
        assert ((out[0].double() - v[0].double()).abs() <= 2.0 ** -8 * v[0].double().abs()).all()  # one token: its value


def test_last_row_of_the_table():
    """A request that fills its table row, and the tail behind it."""
    p = Pair(1, 1, 1, 2, seed=22)
    p.append([64 * 2 + 62])
    p.append([1])
    p.check_cache()
    p.check_attend()


# ---------------------------------------------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------------------------------------------
def test_prompt_then_tokens_with_selection():
    """As a serving loop runs them: a prompt, then for each token the append, Select over the summaries the
    append wrote, and the attention over the selected pages and the tail."""
    sp = spin()
    H, G, k = 2, 5, 4
    p = Pair(1, H, G, 12, summaries=True, seed=30)
    p.append([700])
    p.check_attend()
    for i in range(70):
        _, cu, _, q = p.append([1])
        parts = p.len[0] // 64
        summ = p.c.summaries[0, :, :parts].contiguous()
        sel = torch.empty((H, k), dtype=torch.int32, device="cuda")
        sp.spin_select_noalloc(summ.data_ptr(), q.data_ptr(), H, parts, G, k, sel.data_ptr())
        if i % 10 == 0:
            assert (sel >= 0).all() and (sel < parts).all()
            p.check_attend(q=q.cpu(), sel=sel.cpu())
    p.check_cache()


def test_captured_step_replays_with_new_lengths():
    """Append and attention of one token captured once and replayed; the past grows on the device."""
    B, H, G = 3, 2, 4
    p, e = Pair(B, H, G, 6, seed=31), Pair(B, H, G, 6, seed=31)
    start = [62, 0, 200]
    k0, v0, q0 = p.rand(sum(start), H, D), p.rand(sum(start), H, D), p.rand(sum(start), H * G, D)
    for c in (p, e):
        c.append(start, k=k0, v=v0, q=q0)
    s, _ = step_of(start, [1] * B)
    q, k, v = (torch.zeros((B, n, D), dtype=torch.bfloat16, device="cuda") for n in (H * G, H, H))
    qr, out = torch.empty_like(q), torch.empty_like(q)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        p.c.append(s, q, k, v, qr, stream=st.cuda_stream)
        p.c.attend(s, qr, out, stream=st.cuda_stream)
        s.past.add_(1)
    for _ in range(5):
        kk, vv, qq = p.rand(B, H, D), p.rand(B, H, D), p.rand(B, H * G, D)
        q.copy_(qq), k.copy_(kk), v.copy_(vv)
        torch.cuda.synchronize()
        graph.replay()
        e.append([1] * B, k=kk, v=vv, q=qq)
        want = torch.empty_like(out)
        e.c.attend(e.last[0], e.last[3], want)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(qr, e.last[3])
    assert torch.equal(p.c.pages, e.c.pages)
    p.c.check()


@pytest.mark.parametrize("before", ["nothing", "memset", "copy", "kernel", "event", "append", "attend"])
@pytest.mark.parametrize("new", [1, 40])
def test_captured_behind_other_work(before, new):
    """The attention's first launch as the successor of each kind of node, and of none."""
    p = Pair(2, 2, 4, 30, seed=47)
    p.append([23 * 64, 70])  # no page is completed below, so that an append of the same rows changes nothing
    p.append([new, 1])
    s = p.last[0]
    q = p.rand(new + 1, 8, D).cuda()
    k, v = p.rand(new + 1, 2, D).cuda(), p.rand(new + 1, 2, D).cuda()
    q2 = torch.zeros_like(q)
    want, out = torch.empty_like(q), torch.zeros_like(q)
    if before == "append":
        p.c.append(s, None, k, v)
    p.c.attend(s, q, want)
    torch.cuda.synchronize()
    st, other = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        src = q
        if before == "memset":
            out.zero_()
        elif before == "copy":
            q2.copy_(q)
            src = q2
        elif before == "kernel":
            torch.add(q, 0, out=q2)
            src = q2
        elif before == "event":
            other.wait_stream(st)
            with torch.cuda.stream(other):
                q2.copy_(q)
            st.wait_stream(other)
            src = q2
        elif before == "append":
            p.c.append(s, None, k, v, stream=st.cuda_stream)
        elif before == "attend":
            p.c.attend(s, q, q2, stream=st.cuda_stream)
        p.c.attend(s, src, out, stream=st.cuda_stream)
    for _ in range(3):
        out.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    p.c.check()


def test_attend_follows_what_writes_its_inputs():
    """Calls back to back: each reads what the one before it wrote, the append among them."""
    p, e = Pair(2, 2, 4, 30, rot=0, seed=48), Pair(2, 2, 4, 30, rot=0, seed=48)
    q0 = p.rand(2, 8, D)
    k, v = p.rand(60, 2, D), p.rand(60, 2, D)
    for c in (p, e):
        c.append([1000, 70], k=k.repeat(18, 1, 1)[:1070], v=v.repeat(18, 1, 1)[:1070])
    chain, steps = q0.cuda(), []
    past = [1000, 70]
    for i in range(20):
        steps.append(step_of(past, [1, 1])[0])
        past = [n + 1 for n in past]
    kd, vd = k.cuda(), v.cuda()
    kp = [kd[2 * i:2 * i + 2] for i in range(20)]
    vp = [vd[2 * i:2 * i + 2] for i in range(20)]
    torch.cuda.synchronize()
    for i in range(20):
        p.c.append(steps[i], None, kp[i], vp[i])
        p.c.attend(steps[i], chain, chain)
    torch.cuda.synchronize()
    slow = q0.cuda()
    for i in range(20):
        e.c.append(steps[i], None, kp[i], vp[i])
        torch.cuda.synchronize()
        e.c.attend(steps[i], slow, slow)
        torch.cuda.synchronize()
    assert torch.equal(chain, slow) and torch.equal(p.c.pages, e.c.pages)


def test_two_streams_with_workspaces_of_their_own():
    """Two caches' attention at once, on two streams."""
    ps = [Pair(4, 2, 8, 50, seed=40 + i) for i in range(2)]
    for p in ps:
        p.append([3000, 800, 64, 1])
        p.append([1, 1, 1, 1])
    q = [p.rand(4, 16, D).cuda() for p in ps]
    alone = [torch.empty_like(x) for x in q]
    for p, x, o in zip(ps, q, alone):
        p.c.attend(p.last[0], x, o)
    both = [[torch.empty_like(x) for _ in range(20)] for x in q]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for j in range(20):
        for p, x, o, s in zip(ps, q, both, streams):
            p.c.attend(p.last[0], x, o[j], stream=s.cuda_stream)
    torch.cuda.synchronize()
    for want, got in zip(alone, both):
        for o in got:
            assert torch.equal(o, want)
    # one cache on two streams, with a second workspace
    ws = ps[0].c.new_workspace()
    o = [torch.empty_like(q[0]) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        ps[0].c.attend(ps[0].last[0], q[0], o[0], stream=streams[0].cuda_stream)
        ps[0].c.attend(ps[0].last[0], q[0], o[1], workspace=ws, stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(o[0], alone[0]) and torch.equal(o[1], alone[0])


def test_layers_share_a_workspace():
    """Caches whose calls follow one another on a stream need one workspace between them."""
    a = Pair(3, 2, 4, 30, seed=45)
    b = spin().SpinKV8(3, 8, 2, 30, a.c.n_pages, rope=spin().SpinRope(a.f), pages=a.c.pages, scales=a.c.scales, tails=a.c.tails,
                       table=a.c.table, workspace=a.c.workspace)
    assert b.workspace is a.c.workspace
    a.append([1500, 60, 700])
    a.append([3, 1, 2])
    q = a.rand(6, 8, D).cuda()
    outs = [torch.empty_like(q) for _ in range(4)]
    for i, o in enumerate(outs):
        (a.c, b)[i % 2].attend(a.last[0], q, o)
    want, tol = R.attend(q.cpu(), *a.state(), a.last[4], a.last[1], 1 / math.sqrt(D))
    for o in outs:
        assert torch.equal(o, outs[0])
    assert ((outs[0].cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("new", [[1, 1, 1], [3, 0, 2], [40, 1, 7], [200, 90, 3]], ids=str)
def test_attend_in_place(new):
    """out may be q itself: a unit's rows are written once all that reads them has."""
    p = Pair(3, 2, 5, 60, seed=57)
    p.append([3000, 64, 500])
    p.append(new)
    q = p.rand(sum(new), 10, D).cuda()
    out = torch.empty_like(q)
    p.c.attend(p.last[0], q, out)
    assert p.c.attend(p.last[0], q, q) is q
    assert torch.equal(q, out)


def test_a_page_listed_twice_counts_twice():
    p = Pair(1, 1, 2, 6, rot=0, seed=58)
    p.append([64 * 4])
    p.append([1])
    sel = torch.tensor([[2, 0, 2]], dtype=torch.int32)
    s, cu, _, _, past = p.last
    q = p.rand(1, 2, D)
    out = torch.empty((1, 2, D), dtype=torch.bfloat16, device="cuda")
    p.c.attend(s, q.cuda(), out, sel=sel.cuda())
    want, tol = R.attend(q, *p.state(), past, cu, 1 / math.sqrt(D), sel)
    assert ((out.cpu().double() - want).abs() <= tol).all()


def test_shared_prefix_pages():
    """Two requests whose tables share the pages of a prompt."""
    p = Pair(2, 2, 4, 6, seed=50)
    k, v = p.rand(320, 2, D), p.rand(320, 2, D)
    p.append([320, 0], k=k, v=v)
    p.c.table[1, :, :5] = p.c.table[0, :, :5]
    p.len[1] = 320
    s, cu = step_of([320, 320], [2, 3])
    q = p.rand(5, 8, D)
    kk, vv = p.rand(5, 2, D), p.rand(5, 2, D)
    p.c.append(s, None, kk.cuda(), vv.cuda())
    p.check_attend(q=q, step=s, cu=cu, past=[320, 320])


def test_empty_step():
    p = Pair(2, 1, 1, 2, seed=51)
    e = torch.empty((0, 1, D), dtype=torch.bfloat16, device="cuda")
    s, _ = step_of([0, 0], [0, 0])
    p.c.append(s, e, e, e, e)
    p.c.attend(s, e, e)
    p.c.check()


def test_large_pool_offsets():
    """A pool of more than 4 GiB: pages at both of its ends, and a table whose row is long."""
    n = 270000
    table = torch.full((1, 1, 3), -1, dtype=torch.int32)
    table[0, 0] = torch.tensor([n - 1, 0, 262145])
    c = spin().SpinKV8(1, 2, 1, 3, n, table=table.cuda())
    g = torch.Generator().manual_seed(52)
    k, v = (torch.randn((190, 1, D), generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((190, 2, D), generator=g).to(torch.bfloat16)
    s, cu = step_of([0], [190])
    c.append(s, None, k.cuda(), v.cuda())
    out = torch.empty((190, 2, D), dtype=torch.bfloat16, device="cuda")
    c.attend(s, q.cuda(), out)
    ids = table[0, 0, :2].long()
    small = torch.tensor([[[0, 1, -1]]], dtype=torch.int32)
    want, tol = R.attend(q, c.pages[ids.cuda()].cpu(), c.scales[ids.cuda()].cpu(), c.tails.cpu(), small, [0], cu, 1 / math.sqrt(D))
    assert ((out.cpu().double() - want).abs() <= tol).all()
    c.check()
