"""The 8-bit cache's attention where scores are so large that float32 holds them in steps of 4 to 2^12."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv8_ref as R  # noqa: E402
from test_gpu_kv8 import D, Pair  # noqa: E402

MANY = [17, 40, 130, 300]  # new tokens, of groups of 2: a shared block, one of two tiles, several


def build(new, keys, values, batch=1, seed=0):
    """A cache of one KV head and two query heads, `new` tokens of it from the last call; keys and values [n][128]."""
    n = keys.shape[0]
    p = Pair(batch, 1, 2, n // 64 + 1, rot=0, seed=seed)
    k, v = (x.to(torch.bfloat16)[:, None] for x in (keys, values))
    if n > new:
        p.append([n - new] * batch, k=k[:-new].repeat(batch, 1, 1), v=v[:-new].repeat(batch, 1, 1))
    p.append([new] * batch, k=k[-new:].repeat(batch, 1, 1), v=v[-new:].repeat(batch, 1, 1))
    return p


def attended(p, q, scale=None):
    """The kernel's result and the 64-bit one, for the last step."""
    s, cu, _, _, past = p.last
    out = torch.full((s.total_new, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    p.c.attend(s, q.to(torch.bfloat16).cuda(), out, scale=scale)
    want, _ = R.attend(q.to(torch.bfloat16), *p.state(), past, cu, 1 / math.sqrt(D) if scale is None else scale)
    p.c.check()
    return out.cpu().double(), want


def values_of(n, seed):
    """Pages whose values' scales differ by up to 2^10."""
    g = torch.Generator().manual_seed(seed)
    size = torch.exp2(torch.randint(-7, 4, (n // 64 + 1,), generator=g).float()).repeat_interleave(64)[:n, None]
    return torch.randn((n, D), generator=g) * size


def check_equal(new, size, sign, n, batch):
    """All queries and keys alike: every row is the mean of the values that it sees. Scores' terms and their partial sums
    are exact, so all scores are the same float32 number, and a weight is a power of two that fp16 holds. What is left
    is fp32 sums over n tokens, and one rounding to bf16."""
    p = build(new, torch.full((n, D), float(size)), values_of(n, n + new), batch, seed=new)
    got, want = attended(p, torch.full((new * batch, 2, D), float(sign * size)))
    off = (n + 64) * 2.0 ** -23 * float(p.ref.v[0].abs().mean(0).max())
    bound = off + R.EPS_BF16 * (want.abs() + off)
    assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / bound).max())


def check_steps(new, size, n, falling=False):
    """Scores of 2^25 to 2^27 that rise (or fall) by some 33 in base 2 from page to page (the last dimension alone makes the
    difference): a row is the mean over the last (or first) page that it sees. float32 rounds these scores by 8 at most."""
    q = torch.full((new, 2, D), float(size))
    q[..., -1] = 8.0
    k = torch.full((n, D), float(size))
    step = torch.arange(n) // 64 + 1
    k[:, -1] = 32.0 * (8 - step if falling else step)
    p = build(new, k, values_of(n, n + new + 1), seed=new + 1)
    got, want = attended(p, q)
    # the next page's weight: 2^-32 and twice the scores' rounding, and the values' sizes differ by up to 2^10
    off = 64 * 2.0 ** (-32 + 16) * float(p.ref.v[0].abs().max())
    bound = off + R.EPS_BF16 * (want.abs() + off)
    assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / bound).max())


def check_jump(new, size, n, at):
    """One key twice as large as the others: rows that see it get its value, the others the mean of theirs."""
    k = torch.full((n, D), float(size))
    k[at] *= 2
    p = build(new, k, values_of(n, n + at), seed=new + 2)
    got, want = attended(p, torch.full((new, 2, D), float(size)))
    off = (n + 64) * 2.0 ** -23 * float(p.ref.v[0].abs().mean(0).max())
    bound = off + R.EPS_BF16 * (want.abs() + off)
    assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / bound).max())


def check_scale(new, n):
    """Ordinary queries and keys, and a softmax scale of 2^24: the largest score takes all. Where the two largest are
    closer to one another than float32 tells apart, either may."""
    g = torch.Generator().manual_seed(new)
    p = build(new, torch.randn((n, D), generator=g), values_of(n, n), seed=new + 3)
    q = torch.randn((new, 2, D), generator=g)
    got, want = attended(p, q, 2.0 ** 24)
    k, v, pos = R.keys_and_values(*p.state(), 0, 0, n)
    s = torch.einsum("igd,jd->igj", q.to(torch.bfloat16).double(), k) * 2.0 ** 24
    s = s.masked_fill(pos[None, None] > (n - new + torch.arange(new))[:, None, None], -math.inf)
    top = s.topk(2, -1).values
    size = torch.einsum("igd,jd->igj", q.to(torch.bfloat16).double().abs(), k.abs()).amax(-1) * 2.0 ** 24
    clear = top[..., 0] - top[..., 1] > 128 * 2.0 ** -22 * size + 40  # 128 additions' roundings; e^-40 is nothing
    assert clear.double().mean() > 0.9
    bound = R.EPS_BF16 * want.abs() + 2.0 ** -20 * float(v.abs().max())
    assert ((got - want).abs() <= bound)[clear].all()
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("new", MANY)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [1536, 2560, 2 ** 14])
def test_many_rows_equal_scores(new, sign, size):
    check_equal(new, size, sign, 64 * 7 + 21 + new, 1)


def test_many_rows_equal_scores_of_many_requests():
    """Units that one CTA does alone, and units that two share."""
    check_equal(20, 2560, 1, 150, 90)


@pytest.mark.parametrize("new", MANY)
@pytest.mark.parametrize("falling", [False, True])
@pytest.mark.parametrize("size", [1536, 2560])
def test_many_rows_scores_in_steps(new, falling, size):
    check_steps(new, size, 64 * 7, falling)


@pytest.mark.parametrize("new", MANY)
@pytest.mark.parametrize("at", [0, 100, 300, 447])
def test_many_rows_one_large_score(new, at):
    check_jump(new, 2560, 64 * 7 + 2, at)


@pytest.mark.parametrize("new", MANY)
def test_many_rows_large_softmax_scale(new):
    check_scale(new, 64 * 9 + 5 + new)


FEW = [1, 2, 4, 5, 8]  # new tokens, of groups of 2: units of up to 8 rows, and of up to 16


@pytest.mark.parametrize("new", FEW)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [1536, 2560, 2 ** 14])
def test_few_rows_equal_scores(new, sign, size):
    check_equal(new, size, sign, 64 * 7 + 21 + new, 1)


@pytest.mark.parametrize("new", [1, 6])
def test_few_rows_equal_scores_of_many_requests(new):
    check_equal(new, 2560, 1, 150, 90)


@pytest.mark.parametrize("new", FEW)
@pytest.mark.parametrize("falling", [False, True])
@pytest.mark.parametrize("size", [1536, 2560])
def test_few_rows_scores_in_steps(new, falling, size):
    check_steps(new, size, 64 * 7, falling)


@pytest.mark.parametrize("new", FEW)
@pytest.mark.parametrize("at", [0, 100, 300, 447])
def test_few_rows_one_large_score(new, at):
    check_jump(new, 2560, 64 * 7 + 2, at)


@pytest.mark.parametrize("new", FEW)
def test_few_rows_large_softmax_scale(new):
    check_scale(new, 64 * 9 + 5 + new)


@pytest.mark.parametrize("new", [1, 5, 40, 300])
@pytest.mark.parametrize("scale", [3.0, 30.0, 100.0, 1000.0])
def test_scores_on_both_sides_of_where_differences_come_first(new, scale):
    """Rows' largest scores from some hundred to some ten thousands, in base 2, in one block, over pages whose values'
    scales differ: what is worked out in one operation and what takes the difference first, side by side."""
    g = torch.Generator().manual_seed(new)
    n = 64 * 20 + 30 + new
    p = build(new, torch.randn((n, D), generator=g), values_of(n, n), seed=new + 4)
    q = torch.randn((new, 2, D), generator=g) * torch.exp2(torch.randint(-3, 2, (new, 2, 1), generator=g).float())
    p.check_attend(q=q.to(torch.bfloat16), scale=scale)
