"""The page pool of the 8-bit cache without a GPU: its refusals, and the restatement that its GPU tests compare with."""
import random

import pytest

import sparse_attention_tiered_gb300 as spin
from sparse_attention_tiered_gb300 import _binding as B

import kv8_pool_ref as R
from test_kv8_refusals import A, BAD_CACHE, BAD_STEP, cache, refused, step


def reserve(c=None, s=None, refs=A, free=None, ws=A, ws_bytes=1 << 40):
    B.spin_kv8_reserve(c or cache(), s or step(), refs, free, ws, ws_bytes)


def fork(c=None, refs=A, length=A, src=2 * A):
    B.spin_kv8_fork(c or cache(), refs, length, src)


def compact(c=None, refs=A, free=None, ws=A, ws_bytes=1 << 40):
    B.spin_kv8_compact(c or cache(), refs, free, ws, ws_bytes)


@pytest.mark.parametrize("call", [reserve, fork, compact])
@pytest.mark.parametrize("bad,word", BAD_CACHE, ids=str)
def test_bad_caches(call, bad, word):
    refused(call, word, c=cache(**bad))
    refused(call, "spin_kv8_", c=cache(**bad))


@pytest.mark.parametrize("bad,word", BAD_STEP, ids=str)
def test_bad_steps(bad, word):
    refused(reserve, word, s=step(**bad))


@pytest.mark.parametrize("call,kw,word", [
    (reserve, dict(refs=None), "refs"), (reserve, dict(refs=A + 2), "aligned"), (reserve, dict(free=A + 1), "aligned"),
    (reserve, dict(ws=None), "workspace"), (reserve, dict(ws=A + 8), "workspace"), (reserve, dict(ws_bytes=8), "workspace"),
    (compact, dict(refs=None), "refs"), (compact, dict(free=A + 1), "aligned"), (compact, dict(ws=A + 8), "workspace"),
    (compact, dict(ws_bytes=8), "workspace"), (compact, dict(ws=None), "workspace"),
    (fork, dict(refs=None), "refs"), (fork, dict(length=None), "len"), (fork, dict(src=None), "src"), (fork, dict(src=A), "two arrays"),
    (fork, dict(src=A + 2), "aligned"), (fork, dict(length=A + 2), "aligned")], ids=str)
def test_bad_arguments(call, kw, word):
    refused(call, word, **kw)


def test_null_structures_and_workspace():
    lib = spin.load()
    assert lib.spin_kv8_reserve(None, None, None, None, None, 0, None) == B.SPIN_ERR_INVALID
    assert lib.spin_kv8_fork(None, None, None, None, None) == B.SPIN_ERR_INVALID
    assert lib.spin_kv8_compact(None, None, None, None, 0, None) == B.SPIN_ERR_INVALID
    assert lib.spin_kv8_pool_workspace(None, None) == B.SPIN_ERR_INVALID
    assert 0 < B.spin_kv8_pool_workspace(cache()) < B.spin_kv8_pool_workspace(cache(n_pages=5000))


def test_without_a_gpu_the_calls_fail_cleanly():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (reserve, fork, compact):
        with pytest.raises(B.SpinError) as e:
            call()
        assert e.value.code == B.SPIN_ERR_CUDA


def counts(pool):
    n = [0] * len(pool.refs)
    for head in pool.table:
        for row in head:
            for x in row:
                if x >= 0:
                    n[x] += 1
    return n


@pytest.mark.parametrize("seed", range(6))
def test_the_restatement_keeps_its_books(seed):
    """Counts are those of the table after every call, and a page has one owner's contents."""
    rng = random.Random(seed)
    B_, H, P, N = 5, 2, 7, 60
    pool = R.Pool([[[-1] * P for _ in range(H)] for _ in range(B_)], [0] * N)
    length, holds = [0] * B_, {}
    for _ in range(60):
        what = rng.choice(["step", "step", "fork", "compact"])
        if what == "step":
            new = [rng.randint(0, max(0, min(90, R.PAGE * P - n))) for n in length]
            free = pool.reserve(length, new)
            assert free == pool.refs.count(0)
            if pool.error:
                pool.error = 0
                continue
            length = [a + n for a, n in zip(length, new)]
        elif what == "fork":
            src = [rng.choice([b, b, -1, rng.randrange(B_)]) for b in range(B_)]
            pool.fork(length, src)
        else:
            before = [r for r in pool.refs if r]
            free, go = pool.compact()
            assert all(pool.refs[: len(pool.refs) - free]) and not any(pool.refs[len(pool.refs) - free:])
            assert sorted(before) == sorted(r for r in pool.refs if r)
        assert counts(pool) == pool.refs
        for b in range(B_):
            for h in range(H):
                assert all(x >= 0 for x in pool.table[b][h][: length[b] // R.PAGE])
    assert not pool.error
