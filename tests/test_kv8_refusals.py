"""The 8-bit cache's entry points without a GPU: every argument check refuses before anything is
enqueued, with a message that names the entry point. The addresses are never followed."""
import ctypes
import math

import pytest

import sparse_attention_tiered_gb300 as spin
from sparse_attention_tiered_gb300 import _binding as B

FREQ = (ctypes.c_double * 64)(*[10000.0 ** (-j / 64) for j in range(64)])
A = 1 << 20  # an aligned address


def cache(**kw):
    d = dict(batch=2, q_heads=8, kv_heads=2, max_pages=4, n_pages=16, pages=A, scales=A, tails=A, summaries=None,
             table=A, error=A, device=0, rot_dim=128, interleaved=0, reserved=0, inv_freq=ctypes.addressof(FREQ))
    d.update(kw)
    return B.spin_kv8(**d)


def step(**kw):
    d = dict(past=A, cu_new=A, total_new=3, max_new=2)
    d.update(kw)
    return B.spin_kv8_step(**d)


def rows(heads=8, **kw):
    d = dict(ptr=A, token_stride=heads * 128, head_stride=128)
    d.update(kw)
    return B.spin_rows(**d)


def append(c=None, s=None, q=None, q_out=None, k=None, v=None, positions=None):
    B.spin_kv8_append(c or cache(), s or step(), q or rows(), q_out or rows(), k or rows(2), v or rows(2), positions)


def attend(c=None, s=None, q=None, out=None, scale=0.1, sel=None, topk=0, ws=A, ws_bytes=1 << 40):
    B.spin_kv8_attend(c or cache(), s or step(), q or rows(), out or rows(), scale, sel, topk, ws, ws_bytes)


def refused(call, word, **kw):
    with pytest.raises(B.SpinError) as e:
        call(**kw)
    assert e.value.code == B.SPIN_ERR_INVALID, e.value
    assert word in str(e.value), e.value


BAD_CACHE = [(dict(batch=0), "batch"), (dict(batch=16385), "batch"), (dict(q_heads=7), "q_heads"), (dict(kv_heads=0), "kv_heads"),
             (dict(q_heads=34), "group"), (dict(max_pages=0), "max_pages"), (dict(n_pages=0), "n_pages"),
             (dict(n_pages=(1 << 24) + 1), "n_pages"), (dict(pages=None), "pages"), (dict(scales=None), "scales"),
             (dict(tails=None), "tails"), (dict(table=None), "table"), (dict(error=None), "error"), (dict(pages=A + 64), "aligned"),
             (dict(tails=A + 8), "aligned"), (dict(scales=A + 4), "aligned"), (dict(table=A + 2), "aligned"),
             (dict(summaries=A + 8), "aligned"), (dict(device=-1), "device"), (dict(reserved=1), "reserved")]
BAD_STEP = [(dict(past=None), "past"), (dict(cu_new=None), "cu_new"), (dict(past=A + 2), "aligned"), (dict(total_new=-1), "total_new"),
            (dict(max_new=0), "max_new"), (dict(max_new=(1 << 20) + 1), "max_new")]
BAD_ROWS = [(dict(ptr=None), "NULL"), (dict(ptr=A + 8), "aligned"), (dict(token_stride=1028), "multiples"), (dict(head_stride=132), "multiples")]


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("bad,word", BAD_CACHE, ids=str)
def test_bad_caches(call, bad, word):
    refused(call, word, c=cache(**bad))
    refused(call, "spin_kv8_", c=cache(**bad))


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("bad,word", BAD_STEP, ids=str)
def test_bad_steps(call, bad, word):
    refused(call, word, s=step(**bad))


@pytest.mark.parametrize("bad,word", BAD_ROWS, ids=str)
def test_bad_rows(bad, word):
    for name, heads in (("q", 8), ("q_out", 8), ("k", 2), ("v", 2)):
        refused(append, word, **{name: rows(heads, **bad)})
    for name in ("q", "out"):
        refused(attend, word, **{name: rows(**bad)})


@pytest.mark.parametrize("strides", [dict(token_stride=1016), dict(token_stride=0), dict(head_stride=120), dict(head_stride=0),
                                     dict(token_stride=120, head_stride=1024), dict(token_stride=128, head_stride=376)], ids=str)
def test_overlapping_outputs(strides):
    refused(append, "overlap", q_out=rows(ptr=2 * A, **strides))
    refused(attend, "overlap", out=rows(**strides))


@pytest.mark.parametrize("strides", [dict(token_stride=2048), dict(token_stride=128, head_stride=1024)], ids=str)
def test_other_strides_in_place(strides):
    refused(attend, "in place", q=rows(ptr=2 * A), out=rows(ptr=2 * A, **strides))


@pytest.mark.parametrize("bad,word", [(dict(rot_dim=8), "rot_dim"), (dict(rot_dim=144), "rot_dim"), (dict(rot_dim=-16), "rot_dim"),
                                      (dict(inv_freq=None), "inv_freq"), (dict(interleaved=2), "interleaved")], ids=str)
def test_bad_rotations(bad, word):
    refused(append, word, c=cache(**bad))


def test_frequencies_that_are_not_finite():
    for f in (math.nan, math.inf):
        bad = (ctypes.c_double * 64)(*([1.0] * 63 + [f]))
        refused(append, "inv_freq[63]", c=cache(inv_freq=ctypes.addressof(bad)))


def test_queries_and_their_output_come_together():
    with pytest.raises(B.SpinError, match="both"):
        B.spin_kv8_append(cache(), step(), rows(), None, rows(2), rows(2))
    with pytest.raises(B.SpinError, match="both"):
        B.spin_kv8_append(cache(), step(), None, rows(), rows(2), rows(2))
    refused(append, "in place", q_out=rows(token_stride=2048))
    refused(append, "positions", positions=A + 2)


@pytest.mark.parametrize("kw,word", [(dict(scale=math.nan), "scale"), (dict(scale=math.inf), "scale"), (dict(sel=A), "topk"),
                                     (dict(topk=3), "sel"), (dict(sel=A, topk=-1), "topk"), (dict(sel=A + 1, topk=2), "aligned"),
                                     (dict(ws=None), "workspace"), (dict(ws=A + 8), "workspace"), (dict(ws_bytes=8), "workspace")], ids=str)
def test_bad_attention_arguments(kw, word):
    refused(attend, word, **kw)


def test_null_structures_and_workspace():
    lib = spin.load()
    assert lib.spin_kv8_append(None, None, None, None, None, None, None, None) == B.SPIN_ERR_INVALID
    assert lib.spin_kv8_attend(None, None, None, None, 0.1, None, 0, None, 0, None) == B.SPIN_ERR_INVALID
    assert lib.spin_kv8_workspace(None, None) == B.SPIN_ERR_INVALID
    assert lib.spin_kv8_status(None, None) == B.SPIN_ERR_INVALID
    assert B.spin_kv8_workspace(cache()) > 0
    big, small = (B.spin_kv8_workspace(cache(q_heads=h, kv_heads=2)) for h in (32, 2))
    assert big >= small


def test_handle_refuses_what_the_library_cannot_see():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="CUDA tensor"):
        spin.SpinKV8Step(torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 2, 1)
    with pytest.raises(ValueError, match="pages"):
        spin.SpinKV8(1, 1, 1, 1, pages=torch.zeros((1, 2, 64, 128), dtype=torch.uint8), device=0)
    with pytest.raises(ValueError, match="CUDA tensors"):
        spin.SpinKV8(1, 1, 1, 1, pages=torch.zeros((1, 2, 64, 128), dtype=torch.uint8))


def test_without_a_gpu_the_calls_fail_cleanly():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (append, attend):
        with pytest.raises(B.SpinError) as e:
            call()
        assert e.value.code == B.SPIN_ERR_CUDA
