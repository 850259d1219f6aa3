"""Select over the 8-bit cache without a GPU: its refusals, and the bound on the first scores' error that it relies on."""
import pytest

import sparse_attention_tiered_gb300 as spin
from sparse_attention_tiered_gb300 import _binding as B

from test_kv8_refusals import A, BAD_CACHE, BAD_ROWS, BAD_STEP, cache, refused, rows, step


def select(c=None, s=None, q=None, topk=4, sel=A, ws=A, ws_bytes=1 << 40):
    B.spin_kv8_select(c or cache(summaries=A), s or step(), q or rows(), topk, sel, ws, ws_bytes)


@pytest.mark.parametrize("bad,word", BAD_CACHE, ids=str)
def test_bad_caches(bad, word):
    refused(select, word, c=cache(**dict(dict(summaries=A), **bad)))


@pytest.mark.parametrize("bad,word", BAD_STEP, ids=str)
def test_bad_steps(bad, word):
    refused(select, word, s=step(**bad))


@pytest.mark.parametrize("bad,word", BAD_ROWS, ids=str)
def test_bad_rows(bad, word):
    refused(select, word, q=rows(**bad))


@pytest.mark.parametrize("kw,word", [(dict(c=cache()), "summaries"), (dict(topk=0), "topk"), (dict(topk=513), "topk"), (dict(sel=None), "sel"),
                                     (dict(sel=A + 2), "aligned"), (dict(ws=None), "workspace"), (dict(ws=A + 8), "workspace"),
                                     (dict(ws_bytes=64), "workspace")], ids=lambda x: "" if isinstance(x, dict) else x)
def test_bad_arguments(kw, word):
    refused(select, word, **kw)


def test_workspace():
    lib = spin.load()
    assert lib.spin_kv8_select(None, None, None, 1, None, None, 0, None) == B.SPIN_ERR_INVALID
    assert lib.spin_kv8_select_workspace(None, 1, None) == B.SPIN_ERR_INVALID
    with pytest.raises(B.SpinError, match="total_new"):
        B.spin_kv8_select_workspace(cache(), -1)
    sizes = [B.spin_kv8_select_workspace(cache(max_pages=512), n) for n in (0, 1, 2, 1000, 100000, 10000000)]
    assert sizes == sorted(sizes) and 0 < sizes[0] and sizes[1] < sizes[2]
    assert sizes[3] < sizes[4] == sizes[5] < 1.2e9  # more rows than that are taken in turns


def test_without_a_gpu_it_fails_cleanly():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    with pytest.raises(B.SpinError) as e:
        select()
    assert e.value.code == B.SPIN_ERR_CUDA


@pytest.mark.parametrize("seed", range(8))
def test_error_of_split_products(seed):
    """x = h + l + r: three products of bf16 numbers, added in fp32, are off by less than 2^-15 of the norms' product; the
    group's sum in fp32 by less than 2^-20 of the sum of absolute values."""
    torch = pytest.importorskip("torch")
    g = torch.Generator().manual_seed(seed)
    heads = torch.randn((200, 16, 128), generator=g) * torch.exp2(torch.randint(-12, 12, (200, 16, 1), generator=g).float())
    heads = heads.to(torch.bfloat16)
    heads[:, 1::2] = torch.where(torch.rand((200, 8, 128), generator=g) < 0.5, -heads[:, 0::2], heads[:, 1::2])
    q = torch.zeros((200, 128))
    for i in range(16):
        q += heads[:, i].float()
    s = torch.randn((200, 128), generator=g) * torch.exp(2 * torch.randn((200, 128), generator=g))

    def split(x):
        h = x.to(torch.bfloat16).float()
        return h, (x - h).to(torch.bfloat16).float()

    (qh, ql), (sh, sl) = split(q), split(s)
    got = (qh * sh).cumsum(1)[:, -1] + ((qh * sl).cumsum(1)[:, -1] + (ql * sh).cumsum(1)[:, -1])
    want = (heads.double().sum(1) * s.double()).sum(1)
    a = heads.float().abs().sum(1)
    bound = 2.0 ** -15 * (q.norm(dim=1) + a.norm(dim=1) / 32) * s.norm(dim=1)
    assert ((got.double() - want).abs() < bound).all()
