"""Attention over a list of pages for each token, without a GPU: its refusals."""
import math

import pytest

import sparse_attention_tiered_gb300 as spin
from sparse_attention_tiered_gb300 import _binding as B

from test_kv8_refusals import A, BAD_CACHE, BAD_ROWS, BAD_STEP, cache, refused, rows, step


def attend(c=None, s=None, q=None, out=None, scale=0.1, sel=A, topk=4, ws=A, ws_bytes=1 << 40):
    B.spin_kv8_attend_rows(c or cache(), s or step(), q or rows(), out or rows(), scale, sel, topk, ws, ws_bytes)


@pytest.mark.parametrize("bad,word", BAD_CACHE, ids=str)
def test_bad_caches(bad, word):
    refused(attend, word, c=cache(**bad))


@pytest.mark.parametrize("bad,word", BAD_STEP, ids=str)
def test_bad_steps(bad, word):
    refused(attend, word, s=step(**bad))


@pytest.mark.parametrize("bad,word", BAD_ROWS, ids=str)
def test_bad_rows(bad, word):
    refused(attend, word, q=rows(**bad))
    refused(attend, word, out=rows(**bad))


@pytest.mark.parametrize("kw,word", [(dict(scale=math.nan), "scale"), (dict(scale=math.inf), "scale"), (dict(topk=0), "topk"),
                                     (dict(topk=513), "topk"), (dict(sel=None), "sel"), (dict(sel=A + 2), "aligned"),
                                     (dict(ws=None), "workspace"), (dict(ws=A + 8), "workspace"), (dict(ws_bytes=64), "workspace")], ids=str)
def test_bad_arguments(kw, word):
    refused(attend, word, **kw)


def test_outputs_that_overlap_and_other_strides_in_place():
    refused(attend, "overlap", out=rows(token_stride=120))
    refused(attend, "in place", q=rows(ptr=2 * A), out=rows(ptr=2 * A, token_stride=2048))


def test_workspace():
    lib = spin.load()
    assert lib.spin_kv8_attend_rows(None, None, None, None, 0.1, None, 1, None, 0, None) == B.SPIN_ERR_INVALID
    assert lib.spin_kv8_attend_rows_workspace(None, 1, 1, None) == B.SPIN_ERR_INVALID
    for bad in ((-1, 4), (1, 0), (1, 513)):
        with pytest.raises(B.SpinError, match="total_new"):
            B.spin_kv8_attend_rows_workspace(cache(), *bad)
    sizes = [B.spin_kv8_attend_rows_workspace(cache(), n, k) for n, k in ((0, 1), (1, 1), (1, 9), (500, 9), (500, 512))]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_without_a_gpu_it_fails_cleanly():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    with pytest.raises(B.SpinError) as e:
        attend()
    assert e.value.code == B.SPIN_ERR_CUDA
