"""Select over the 8-bit cache on the GPU: the pages of exact scores, whatever the sizes and however close the scores."""
import math
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_kv8 import D, PAGE, ints, spin, step_of  # noqa: E402


def handle(batch, heads, group, summaries):
    return spin().SpinKV8(batch, heads * group, heads, summaries.shape[2], 1, summaries=summaries,
                          table=torch.zeros(summaries.shape[:3], dtype=torch.int32, device="cuda"))


def want(q, summaries, past, new, group, k):
    """int32 [rows][heads][k] by a stable sort of 64-bit scores."""
    H = summaries.shape[1]
    out = torch.full((sum(new), H, k), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, (a, n) in enumerate(zip(past, new)):
        for h in range(H):
            qs = q[at:at + n, h * group:(h + 1) * group].double().sum(1)
            score = (qs[:, None, :] * summaries[b, h].double()[None]).sum(-1) if n * summaries.shape[2] < 20000 else \
                qs @ summaries[b, h].double().T
            score = torch.nan_to_num(score, nan=-math.inf, posinf=math.inf, neginf=-math.inf)
            for i in range(n):
                seen = (a + i + 1) // PAGE
                take = score[i, :seen].sort(descending=True, stable=True).indices[:k].sort().values
                out[at + i, h, : take.numel()] = take.to(torch.int32)
        at += n
    return out


def run(q, summaries, past, new, group, k, pad=0, max_new=None, stream=0):
    c = handle(len(past), summaries.shape[1], group, summaries)
    s, _ = step_of(past, new, pad, max_new)
    sel = torch.full((s.total_new, summaries.shape[1], k), -77, dtype=torch.int32, device="cuda")
    c.select(s, q, sel, stream=stream)
    torch.cuda.synchronize()
    c.check()
    assert (sel[sum(new):] == -77).all()
    return sel[: sum(new)]


def rand(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * scale


def case(batch, heads, group, past, new, k, seed=0, pad=0, max_new=None, pages=None):
    P = pages or max(1, max((a + n) // PAGE for a, n in zip(past, new)))
    q = rand(seed, sum(new) + pad, heads * group, D).to(torch.bfloat16)
    summaries = rand(seed + 1, batch, heads, P, D) * torch.exp(0.7 * rand(seed + 2, heads, 1, D))
    got = run(q, summaries, past, new, group, k, pad, max_new)
    assert torch.equal(got, want(q, summaries, past, new, group, k))


@pytest.mark.parametrize("k", [1, 7, 32, 512])
@pytest.mark.parametrize("group", [1, 5, 16])
def test_ragged_batches(k, group):
    past = [0, 63, 64, 5000, 127, 16384, 2048 * PAGE - 3, 70000]
    case(8, 2, group, past, [1, 1, 1, 5, 0, 33, 2, 70], k, seed=k)


@pytest.mark.parametrize("batch", [1, 31, 32, 33, 129, 300])
def test_batches_of_single_tokens(batch):
    rng = random.Random(batch)
    case(batch, 3, 4, [rng.choice([0, 62, 63, 64, 639, 4000, rng.randint(0, 9000)]) for _ in range(batch)], [1] * batch, 9, seed=batch, pad=2)


@pytest.mark.parametrize("pages", [1, 31, 32, 256, 257, 512, 513, 1024, 1025, 2047, 2048])
def test_numbers_of_pages(pages):
    case(2, 1, 2, [pages * PAGE - 1, pages * PAGE + 30], [1, 3], min(pages, 17), seed=pages)


@pytest.mark.parametrize("pages,new", [(2049, 1), (5000, 3), (33000, 1)])
def test_long_requests(pages, new):
    case(2, 2, 3, [pages * PAGE - new, 500], [new, 1], 65, seed=pages)


@pytest.mark.parametrize("batch,new", [(1, 700), (170, 1)])
def test_many_rows_of_up_to_2048_pages(batch, new):
    """More rows than a CTA each would pay for: a warp a row, 64 scores a lane."""
    case(batch, 6 if batch > 1 else 2, 3, [2048 * PAGE - new - 7 * i for i in range(batch)], [new] * batch, 40, seed=batch, pages=2048)


def test_a_chunk():
    case(2, 2, 8, [3001, 0], [700, 333], 12, seed=5, pad=9)


@pytest.mark.parametrize("new", [1, 8, 9, 40])
def test_rows_of_another_layout(new):
    """Queries inside a projection's output, heads before tokens."""
    past, G, H, k = [1000, 3000], 2, 3, 6
    summaries = rand(1, 2, H, (3000 + new) // PAGE, D)
    wide = rand(2, 2 * new, (G + 2) * H * D).to(torch.bfloat16)
    q = wide[:, : G * H * D].view(2 * new, G * H, D)
    swapped = q.transpose(0, 1).contiguous().transpose(0, 1)
    expect = want(q, summaries, past, [new, new], G, k)
    for x in (q, swapped):
        assert torch.equal(run(x, summaries, past, [new, new], G, k), expect)


@pytest.mark.parametrize("pages", [40, 1500, 3000])
@pytest.mark.parametrize("kind", ["same", "two kinds", "zero", "close", "few kinds"])
def test_ties_go_to_the_lower_page(kind, pages):
    k, new = 11, 3
    base = rand(3, 1, 1, 1, D)
    s = base.expand(1, 1, pages, D).clone()
    if kind == "two kinds":
        s[:, :, ::3] = rand(4, 1, 1, 1, D)
    elif kind == "zero":
        s.zero_()
    elif kind == "close":  # a step of fp32 in one dimension, where the first scores see nothing of it
        s[0, 0, :, 5] = torch.nextafter(s[0, 0, :, 5], torch.where(torch.arange(pages, device="cuda") % 7 == 3, math.inf, s[0, 0, :, 5]))
    elif kind == "few kinds":
        s = rand(4, 1, 1, 5, D)[:, :, torch.arange(pages, device="cuda") * 7919 % 5].contiguous()
    q = rand(6, new, 4, D).to(torch.bfloat16)
    past = [pages * PAGE - new + 1]
    assert torch.equal(run(q, s, past, [new], 4, k), want(q, s, past, [new], 4, k))


@pytest.mark.parametrize("size", [1e-42, 1e-30, 1e-18, 1e10, 1e25, 3e38])
@pytest.mark.parametrize("pages", [100, 2500])
def test_sizes(size, pages):
    s = (rand(1, 1, 2, pages, D).clamp(-1, 1).double() * size).float()
    q = rand(2, 9, 4, D).to(torch.bfloat16)
    past = [pages * PAGE - 9]
    assert torch.equal(run(q, s, past, [9], 2, 13), want(q, s, past, [9], 2, 13))


def test_pages_of_very_different_size():
    s = rand(1, 1, 1, 400, D) * torch.exp2(torch.linspace(-60, 40, 400, device="cuda"))[:, None]
    q = rand(2, 12, 3, D).to(torch.bfloat16)
    assert torch.equal(run(q, s, [400 * PAGE - 12], [12], 3, 37), want(q, s, [400 * PAGE - 12], [12], 3, 37))


def test_groups_that_cancel():
    """Heads whose sum is far smaller than they are."""
    q = rand(2, 20, 16, D, scale=1000.0)
    q[:, 1::2] = -q[:, ::2] + 1e-2 * rand(3, 20, 8, D)
    q = q.to(torch.bfloat16)
    s = rand(1, 1, 1, 700, D)
    assert torch.equal(run(q, s, [700 * PAGE - 20], [20], 16, 50), want(q, s, [700 * PAGE - 20], [20], 16, 50))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("pages", [30, 3000])
def test_numbers_that_are_not_finite(value, pages):
    s = rand(1, 1, 2, pages, D)
    s[0, 0, 3, 17] = s[0, 0, pages - 2, 1] = value
    s[0, 1, :, 5] = value
    q = rand(2, 4, 4, D).to(torch.bfloat16)
    q[2, 1, 9] = value
    past = [pages * PAGE - 4]
    for k in (5, 25):
        assert torch.equal(run(q, s, past, [4], 2, k), want(q, s, past, [4], 2, k))


def test_what_lies_behind_is_not_looked_at():
    """Summaries of pages that are not complete may hold anything."""
    s = rand(1, 2, 1, 50, D)
    past, new = [1000, 2000], [3, 40]
    for b in range(2):
        s[b, :, (past[b] + new[b]) // PAGE:] = math.nan
    q = rand(2, 43, 2, D).to(torch.bfloat16)
    clean = torch.nan_to_num(s)
    assert torch.equal(run(q, s, past, new, 2, 6), want(q, clean, past, new, 2, 6))


def test_splits_do_not_matter():
    """The same tokens one by one, in drafts and as a chunk, alone and among others."""
    s = rand(1, 1, 2, 300, D)
    s[:, :, 100:200] = s[:, :, :100]
    q = rand(2, 60, 6, D).to(torch.bfloat16)
    past = 300 * PAGE - 60
    whole = run(q, s, [past], [60], 3, 20)
    for size in (1, 7, 30):
        parts = [run(q[i:i + size], s, [past + i], [min(size, 60 - i)], 3, 20) for i in range(0, 60, size)]
        assert torch.equal(torch.cat(parts), whole)
    both = run(torch.cat([q, q]), s.expand(2, -1, -1, -1).contiguous(), [past, past], [60, 60], 3, 20)
    assert torch.equal(both, torch.cat([whole, whole]))


def test_more_rows_than_the_workspace_takes_at_once():
    """max_pages that make a gigabyte of a few rows: they go in turns."""
    P, new = 1 << 20, 90
    c = spin().SpinKV8(2, 2, 1, P, 1, summaries=torch.empty((2, 1, P, D), device="cuda"),
                       table=torch.zeros((2, 1, P), dtype=torch.int32, device="cuda"))
    s = rand(1, 2, 1, 120, D)
    c.summaries[:, :, :120] = s
    q = rand(2, 2 * new, 2, D).to(torch.bfloat16)
    past = [120 * PAGE - new, 3000]
    sel = torch.full((2 * new, 1, 9), -77, dtype=torch.int32, device="cuda")
    st, _ = step_of(past, [new, new])
    c.select(st, q, sel)
    c.check()
    assert torch.equal(sel, want(q, s, past, [new, new], 2, 9))


def test_requests_that_are_out_of_range_are_left_out():
    s = rand(1, 3, 1, 10, D)
    c = handle(3, 1, 2, s)
    q = rand(2, 6, 2, D).to(torch.bfloat16)
    sel = torch.full((6, 1, 3), -77, dtype=torch.int32, device="cuda")
    st = spin().SpinKV8Step(ints([500, -1, 10 * PAGE + 62]), ints([0, 2, 4, 6]), 6, 2)
    c.select(st, q, sel)
    assert torch.equal(sel[:2], want(q[:2], s[:1], [500], [2], 2, 3))
    assert (sel[2:] == -77).all()
    assert int(c.error) == 1 | 32
    c.error.zero_()
    st = spin().SpinKV8Step(ints([500, 100, 200]), ints([0, 2, 4, 6]), 6, 1)  # more new tokens than max_new
    c.select(st, q, sel.fill_(-77))
    assert (sel == -77).all() and int(c.error) == 32


def test_streams_and_graphs():
    s = rand(1, 4, 2, 200, D)
    c = handle(4, 2, 2, s)
    past, k = [1000, 5000, 12000, 64], 8
    q = rand(2, 4, 4, D).to(torch.bfloat16)
    st, _ = step_of(past, [1] * 4)
    sel = torch.empty((4, 2, k), dtype=torch.int32, device="cuda")
    c.select(st, q, sel)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.select(st, q, sel, stream=side.cuda_stream)
    for seed in (5, 6):
        q.copy_(rand(seed, 4, 4, D).to(torch.bfloat16))
        st.past.add_(1)
        past = [n + 1 for n in past]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(sel, want(q, s, past, [1] * 4, 2, k))


def test_the_handle_refuses():
    s = rand(1, 1, 2, 5, D)
    c = handle(1, 2, 2, s)
    st, _ = step_of([100], [1])
    q = rand(2, 1, 4, D).to(torch.bfloat16)
    for bad in (torch.zeros((1, 2), dtype=torch.int32, device="cuda"), torch.zeros((1, 1, 4), dtype=torch.int32, device="cuda"),
                torch.zeros((1, 2, 4), dtype=torch.int64, device="cuda"),
                torch.zeros((1, 2, 8), dtype=torch.int32, device="cuda")[:, :, ::2]):
        with pytest.raises(ValueError, match="sel"):
            c.select(st, q, bad)
    sel = torch.zeros((1, 2, 4), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        c.select(st, q, sel, workspace=torch.zeros(8, device="cuda"))
    with pytest.raises(spin().SpinError, match="workspace"):
        c.select(st, q, sel, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))


def test_a_batch_that_grows_a_request_at_a_time():
    """The handle's workspaces stay in proportion to what the largest call needs."""
    from sparse_attention_tiered_gb300 import _binding as B

    P, most = 4000, 48
    s = rand(1, 1, 1, P, D).expand(most, -1, -1, -1).contiguous()
    c, q = handle(most, 1, 2, s), rand(2, most, 2, D).to(torch.bfloat16)
    expect = want(q, s, [P * PAGE - 1] * most, [1] * most, 2, 7)
    for n in range(1, most + 1):
        st, _ = step_of([P * PAGE - 1] * most, [1] * n + [0] * (most - n))
        sel = torch.full((n, 1, 7), -77, dtype=torch.int32, device="cuda")
        c.select(st, q[:n], sel)
        assert torch.equal(sel, expect[:n])
        assert sum(t.numel() for t in c._spaces["select"]) < 4 * B.spin_kv8_select_workspace(c.c, n)
    assert len(c._spaces["select"]) <= 7
    c.check()


@pytest.mark.parametrize("k", [1, 17, 512])
@pytest.mark.parametrize("pages", [8191, 8192, 8193, 12000, 16383, 16384, 16385, 40000])
def test_numbers_of_pages_of_a_wide_row(pages, k):
    """16 or 32 keys a thread, and more than it holds."""
    case(2, 1, 2, [pages * PAGE - 1, pages * PAGE + 30], [1, 3], k, seed=pages)


@pytest.mark.parametrize("k", [11, 512])
@pytest.mark.parametrize("pages", [5000, 12000, 19900])
@pytest.mark.parametrize("kind", ["same", "two kinds", "zero", "close", "few kinds"])
def test_ties_of_a_wide_row(kind, pages, k):
    """More doubtful pages than a lane each: 64-bit keys, a search of their bits, and ties by rank."""
    base = rand(3, 1, 1, 1, D)
    s = base.expand(1, 1, pages, D).clone()
    if kind == "two kinds":
        s[:, :, ::3] = rand(4, 1, 1, 1, D)
    elif kind == "zero":
        s.zero_()
    elif kind == "close":
        s[0, 0, :, 5] = torch.nextafter(s[0, 0, :, 5], torch.where(torch.arange(pages, device="cuda") % 7 == 3, math.inf, s[0, 0, :, 5]))
    elif kind == "few kinds":
        s = rand(4, 1, 1, 5, D)[:, :, torch.arange(pages, device="cuda") * 7919 % 5].contiguous()
    q = rand(6, 1, 4, D).to(torch.bfloat16)
    past = [pages * PAGE - 1]
    assert torch.equal(run(q, s, past, [1], 4, k), want(q, s, past, [1], 4, k))


@pytest.mark.parametrize("spread", [2, 20, 33, 300])
@pytest.mark.parametrize("pages", [600, 1500, 3000, 12000, 19900])
def test_doubtful_pages_around_the_last_place(pages, spread):
    """So many pages that the first scores cannot tell apart, at the k-th place: fewer than a lane each, and more."""
    q = rand(6, 1, 4, D).to(torch.bfloat16)
    s = rand(3, 1, 1, pages, D)
    order = (s[0, 0].double() @ q.double().sum(1)[0]).sort(descending=True).indices
    k = 60
    some = order[k - spread // 2 - 1:][:spread] if spread < 2 * k else order[:spread]
    s[0, 0, some] = s[0, 0, order[k - 1]].clone()
    s[0, 0, some[::2], 7] = torch.nextafter(s[0, 0, some[::2], 7], torch.full_like(s[0, 0, some[::2], 7], math.inf))
    past = [pages * PAGE - 1]
    assert torch.equal(run(q, s, past, [1], 4, k), want(q, s, past, [1], 4, k))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("pages", [5000, 12000, 19900])
def test_numbers_that_are_not_finite_in_a_wide_row(value, pages):
    s = rand(1, 1, 2, pages, D)
    s[0, 0, 3, 17] = s[0, 0, pages - 2, 1] = value
    s[0, 1, :, 5] = value
    q = rand(2, 2, 4, D).to(torch.bfloat16)
    q[1, 1, 9] = value
    past = [pages * PAGE - 2]
    for k in (5, 512):
        assert torch.equal(run(q, s, past, [2], 2, k), want(q, s, past, [2], 2, k))


@pytest.mark.parametrize("size", [1e-42, 1e-18, 1e25, 3e38])
@pytest.mark.parametrize("pages", [12000, 19900])
def test_sizes_of_a_wide_row(size, pages):
    s = (rand(1, 1, 1, pages, D).clamp(-1, 1).double() * size).float()
    q = rand(2, 2, 2, D).to(torch.bfloat16)
    past = [pages * PAGE - 2]
    assert torch.equal(run(q, s, past, [2], 2, 99), want(q, s, past, [2], 2, 99))


@pytest.mark.parametrize("width", [513, 1025, 2049, 8193, 16385, 70000])
def test_tables_wider_than_the_requests(width):
    """Rows of all lengths in a table made for longer ones."""
    past, new = [0, 63, 700, 300 * PAGE - 2, 500 * PAGE, 5000], [1, 1, 70, 4, 1, 0]
    case(6, 2, 3, past, new, 20, seed=width, pages=width, pad=3)
