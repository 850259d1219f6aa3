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
         ([0, 70, -1, 70, 90], 90), ([0, 40, 0, 40, 0, 40, 0, 40], 40)]
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
