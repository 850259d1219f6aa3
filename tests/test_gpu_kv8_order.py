"""Steps whose cu_new does not ascend, on the GPU: requests that count are answered, the rows of the others are not written."""
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv8_rows_ref as R  # noqa: E402
from test_gpu_kv8 import D, PAGE, ints, spin  # noqa: E402
from test_gpu_kv8_rows import SCALE, Case  # noqa: E402
from test_gpu_kv8_select import handle, rand, want  # noqa: E402
from test_kv8_requests_in_order import in_range, that_count  # noqa: E402


def orders(seed, batch, total, most):
    """cu_new of a batch that ascends but for some entries."""
    rng = random.Random(seed)
    cu = [0]
    for b in range(batch):
        cu.append(min(total, cu[-1] + rng.randint(0, min(most, 2 * total // batch + 1))))
    for _ in range(max(1, batch // 20)):
        cu[rng.randrange(1, batch + 1)] = rng.choice([0, -1, total + 1, rng.randint(0, total)])
    return cu


STEPS = [([0, 100, 0, 100], 100), ([0, 9, 4, 6], 6), ([0, 5, 3], 5), ([0, 4, 2, 6], 6), ([0, 3, 3, 1, 1, 8], 8), ([4, 0, 4, 8], 8),
         ([0, 70, -1, 70, 90], 90), ([0, 40, 0, 40, 0, 40, 0, 40], 40), ([5, 0], 5)]
STEPS += [(orders(s, 9, 60, 40), 60) for s in range(4)] + [(orders(s, 150, 200, 9), 200) for s in range(2)]


@pytest.mark.parametrize("group", [3, 8])
@pytest.mark.parametrize("cu,total", STEPS, ids=lambda x: str(x)[:30])
def test_attention_over_lists(cu, total, group):
    B, most = len(cu) - 1, max(2, total)
    rng = random.Random(total)
    past = [rng.choice([0, 50, 300, 700]) for _ in range(B)]
    c = Case(2, group, past, [0] * B, 4, pad=total, max_pages=(700 + total) // PAGE + 1, seed=B)
    c.sel = torch.randint(-1, 12, c.sel.shape, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    h = spin().SpinKV8(B, 2 * group, 2, c.table.shape[2], c.pages.shape[0], pages=c.pages.cuda(), scales=c.scales.cuda(),
                       tails=c.tails.cuda(), table=c.table.cuda())
    q = c.q.cuda()
    out = torch.full_like(q, 7.0)
    h.attend_rows(spin().SpinKV8Step(ints(past), ints(cu), total, most), q, out, c.sel.cuda())
    torch.cuda.synchronize()
    out = out.cpu()
    ok, some = in_range(cu, total, most), that_count(cu, total, most)
    left = set(range(total))
    for b in some:
        r0, r1 = cu[b], cu[b + 1]
        if B > 20 and b % 7:  # (the restatement takes its time)
            left -= set(range(r0, r1))
            continue
        one = [r0] * (b + 1) + [r1] * (B - b)
        want, bound = R.attend_rows(c.q, c.pages, c.scales, c.tails, c.table, past, one, SCALE, c.sel)
        assert ((out[r0:r1].double() - want[r0:r1]).abs() <= bound[r0:r1]).all(), b
        left -= set(range(r0, r1))
    assert (out[sorted(left)] == 7.0).all()
    assert int(h.error) == (0 if all(ok) else 32)


@pytest.mark.parametrize("pages,turns", [(30, False), (700, False), (2100, False), (1 << 20, True)])
@pytest.mark.parametrize("cu,total", STEPS, ids=lambda x: str(x)[:30])
def test_select(cu, total, pages, turns):
    B, most, group, heads, k = len(cu) - 1, max(2, total), 2, 1, 5
    if turns and B > 20:
        pytest.skip("the summaries would be large")
    rng = random.Random(total + pages)
    seen = min(pages, 2100) - (total + 63) // PAGE - 1
    past = [rng.choice([0, 100, rng.randint(0, seen * PAGE)]) for _ in range(B)]
    s = rand(1, B, heads, min(pages, 2100), D)
    if turns:
        wide = torch.empty((B, heads, pages, D), device="cuda")
        wide[:, :, : s.shape[2]] = s
        c = handle(B, heads, group, wide)
    else:
        c = handle(B, heads, group, s)
    q = rand(2, total, heads * group, D).to(torch.bfloat16)
    sel = torch.full((total, heads, k), -77, dtype=torch.int32, device="cuda")
    step = spin().SpinKV8Step(ints(past), ints(cu), total, most)
    for _ in range(2):  # what the workspace holds of the last call does not matter
        c.select(step, q, sel)
    left = set(range(total))
    for b in that_count(cu, total, most):
        r0, r1 = cu[b], cu[b + 1]
        assert torch.equal(sel[r0:r1], want(q[r0:r1], s[b:b + 1], [past[b]], [r1 - r0], group, k)), b
        left -= set(range(r0, r1))
    assert (sel[sorted(left)] == -77).all()
    assert int(c.error) == (0 if all(in_range(cu, total, most)) else 32)


def test_select_in_order_after_a_step_that_was_not():
    s, past, q = rand(1, 3, 1, 40, D), [2000, 1000, 2300], rand(2, 6, 2, D).to(torch.bfloat16)
    c = handle(3, 1, 2, s)
    sel = torch.full((6, 1, 4), -77, dtype=torch.int32, device="cuda")
    cu = ints([0, 4, 2, 6])
    step = spin().SpinKV8Step(ints(past), cu, 6, 6)
    c.select(step, q, sel)
    assert (sel[4:] == -77).all() and (sel[:4] >= 0).all()
    cu.copy_(ints([0, 2, 4, 6]))
    c.error.zero_()
    c.select(step, q, sel)
    assert torch.equal(sel, want(q, s, past, [2, 2, 2], 2, 4))
    c.check()


def test_captured_calls_replay_with_steps_in_and_out_of_order():
    """cu_new is read by each replay: one that descends leaves out whom it leaves out, and nothing of it is left for the next."""
    B, H, G, k, total = 4, 2, 3, 4, 120
    past = [500, 900, 64, 1300]
    c = Case(H, G, past, [0] * B, k, pad=total, max_pages=32, seed=3)
    summaries = rand(1, B, H, 32, D)
    h = spin().SpinKV8(B, H * G, H, 32, c.pages.shape[0], pages=c.pages.cuda(), scales=c.scales.cuda(), tails=c.tails.cuda(),
                       table=c.table.cuda(), summaries=summaries)
    q, cu = c.q.cuda(), ints([0, 30, 60, 90, 120])
    sel, out = torch.empty((total, H, k), dtype=torch.int32, device="cuda"), torch.empty_like(q)
    step = spin().SpinKV8Step(ints(past), cu, total, total)
    h.select(step, q, sel)
    h.attend_rows(step, q, out, sel)
    torch.cuda.synchronize()
    first = sel.clone(), out.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        h.select(step, q, sel, stream=side.cuda_stream)
        h.attend_rows(step, q, out, sel, stream=side.cuda_stream)
    for now in ([0, 30, 0, 90, 120], [0, 30, 60, 90, 120], [0, 100, 0, 100, 0], [0, 30, 60, 90, 120]):
        cu.copy_(ints(now))
        sel.fill_(-1)
        out.fill_(7.0)
        h.error.zero_()
        graph.replay()
        torch.cuda.synchronize()
        some = that_count(now, total, total)
        assert int(h.error) == (0 if all(in_range(now, total, total)) else 32)
        if len(some) == B:
            assert torch.equal(sel, first[0]) and torch.equal(out, first[1])
        left = torch.ones(total, dtype=torch.bool)
        for b in some:
            r0, r1 = now[b], now[b + 1]
            left[r0:r1] = False
            assert torch.equal(sel[r0:r1], want(q[r0:r1], summaries[b:b + 1], [past[b]], [r1 - r0], G, k))
            one = [r0] * (b + 1) + [r1] * (B - b)
            exact, bound = R.attend_rows(c.q, c.pages, c.scales, c.tails, c.table, past, one, SCALE, sel.cpu())
            assert ((out[r0:r1].cpu().double() - exact[r0:r1]).abs() <= bound[r0:r1]).all()
        assert (out.cpu()[left] == 7.0).all()


def test_selects_at_the_same_time_with_workspaces_of_their_own():
    """One of them over a step that is out of order."""
    from sparse_attention_tiered_gb300 import _binding as B

    past, k, total = [3000, 5000, 900], 6, 90
    s, q = rand(1, 3, 2, 100, D), rand(2, total, 4, D).to(torch.bfloat16)
    c = handle(3, 2, 2, s)
    n = B.spin_kv8_select_workspace(c.c, total)
    orders = ([0, 30, 60, 90], [0, 30, 10, 90], [0, 1, 89, 90])
    steps = [spin().SpinKV8Step(ints(past), ints(cu), total, total) for cu in orders]
    streams = [torch.cuda.Stream() for _ in orders]
    spaces = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in orders]
    sels = [torch.full((total, 2, k), -77, dtype=torch.int32, device="cuda") for _ in orders]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, x, w, sel in zip(steps, streams, spaces, sels):
            c.select(st, q, sel, workspace=w, stream=x.cuda_stream)
    torch.cuda.synchronize()
    for cu, sel in zip(orders, sels):
        left = torch.ones(total, dtype=torch.bool)
        for b in that_count(cu, total, total):
            r0, r1 = cu[b], cu[b + 1]
            left[r0:r1] = False
            assert torch.equal(sel[r0:r1], want(q[r0:r1], s[b:b + 1], [past[b]], [r1 - r0], 2, k))
        assert (sel.cpu()[left] == -77).all()
