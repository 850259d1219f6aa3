"""Calls of the 8-bit cache's attention at the borders of what its header allows."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv8_ref as R  # noqa: E402
from test_gpu_kv8 import D, Pair, spin, step_of  # noqa: E402


@pytest.mark.parametrize("new", [1, 3, 30, 128], ids=["one", "few", "shared", "many"])
@pytest.mark.parametrize("x", [math.nan, math.inf, -math.inf])
def test_a_query_that_is_not_finite_and_sees_nothing(new, x):
    """Zeros, as for any row that sees nothing; NaN for the head that sees something."""
    p = Pair(1, 2, 2, 8, seed=new)
    p.append([384 - new])
    p.append([new])
    s = p.last[0]
    q = p.rand(new, 4, D)
    q[0, :, 5] = q[new - 1, :, 127] = x
    sel = torch.tensor([[-1, -1, -1], [0, -1, -1]], dtype=torch.int32, device="cuda")
    out = torch.full((new, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    p.c.attend(s, q.cuda(), out, sel=sel)
    got = out.cpu().double()
    assert (got[:, :2] == 0).all()
    assert torch.isnan(got[0, 2:]).all() and torch.isnan(got[-1, 2:]).all()
    assert torch.isfinite(got[1:-1, 2:]).all()
    p.c.check()


@pytest.mark.parametrize("new", [1, 4, 9, 40, 200], ids=["one", "few", "sixteen", "shared", "many"])
@pytest.mark.parametrize("reach", [3, 30, 52])
def test_scales_that_are_no_powers_of_two(new, reach):
    """A cache that another program wrote: any codes, any normal scales from 2^-reach to 2^reach, for keys and values."""
    p = Pair(2, 2, 2, 8, rot=0, seed=new + reach)
    p.append([470 - new, 130])
    p.append([new, 1])
    g = p.g
    codes = torch.randint(0, 127, p.c.pages.shape, generator=g) | (torch.randint(0, 2, p.c.pages.shape, generator=g) << 7)
    p.c.pages.copy_(codes.to(torch.uint8))
    size = torch.empty((p.c.n_pages, 2)).uniform_(-reach, reach, generator=g)
    size[:, 0] = size[:, 0] / reach * 3 - 12  # keys: codes of up to 448 make scores of some tens
    p.c.scales.copy_(torch.exp2(size))
    p.check_attend(q=p.rand(new + 1, 4, D, scale=0.05))


def test_attend_many_rows_twice_gives_the_same_bits():
    p = Pair(3, 2, 8, 60, seed=3)
    p.append([3000, 17, 900])
    p.append([33, 300, 5])
    q = p.rand(338, 16, D).cuda()
    outs = [torch.empty_like(q) for _ in range(4)]
    for o in outs:
        p.c.attend(p.last[0], q, o)
    for o in outs[1:]:
        assert torch.equal(outs[0], o)


def test_append_of_broadcast_keys_and_values():
    """One row for all heads, or for all tokens: strides of 0."""
    p = Pair(2, 4, 2, 4, seed=5)
    s, cu = step_of([0, 0], [70, 3])
    k = p.rand(73, 1, D).cuda().expand(73, 4, D)
    v = p.rand(1, 4, D).cuda().expand(73, 4, D)
    p.c.append(s, None, k, v)
    p.ref.append(k.cpu(), v.cpu(), cu)
    p.last, p.len = (s, cu, None, None, [0, 0]), [70, 3]
    p.check_cache()
    p.check_attend()


def test_selection_for_a_ragged_batch():
    """Select takes one count of partitions a call: requests of different lengths are selected one by one, from a
    dense copy of the summaries of their complete pages, and attended together."""
    sp = spin()
    H, G, k = 2, 4, 3
    p = Pair(3, H, G, 20, summaries=True, seed=6)
    p.append([1200, 64 * 3, 500])
    _, cu, _, q = p.append([1, 1, 1])
    p.c.summaries[1, :, 3:] = 1e4  # a former request's: behind this one's pages, and not to be picked
    sel = torch.full((3 * H, k), -1, dtype=torch.int32, device="cuda")
    for b in range(3):
        parts = p.len[b] // 64
        summ = p.c.summaries[b, :, :parts].contiguous()
        sp.spin_select_noalloc(summ.data_ptr(), q[b].data_ptr(), H, parts, G, k, sel[b * H].data_ptr())
    got = sel.cpu()
    full = torch.tensor([n // 64 for n in p.len]).repeat_interleave(H)
    assert (got >= 0).all() and (got < full[:, None]).all()  # k pages for every unit
    score = torch.einsum("bhgd,bhpd->bhp", q.cpu().float().view(3, H, G, D), p.c.summaries.cpu())
    for u in range(3 * H):
        best = score[u // H, u % H, : full[u]].topk(k).indices.sort().values
        assert torch.equal(best, got[u].long())
    p.check_attend(q=q.cpu(), sel=got)
