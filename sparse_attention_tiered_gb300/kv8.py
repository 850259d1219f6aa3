"""A Python handle around one layer's 8-bit paged cache (spin_kv8 in include/spin.h).

Marshalling only: PyTorch supplies device memory and streams, every operation is one call
into libspin.so. Streams are passed as ints (``torch.cuda.current_stream().cuda_stream``);
0 is the legacy default stream. Calls on one handle, and handles that share tensors, must be
ordered on one stream or by events. A handle is used from one host thread at a time.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional, Sequence

from . import _binding as B


_SCALE = 1.0 / math.sqrt(B.HEAD_DIM)
_ROWS2, _ROWS4 = struct.Struct("Pqq" * 2), struct.Struct("Pqq" * 4)  # spin_rows, so many of them
_ROW_BYTES = ctypes.sizeof(B.spin_rows)


def _tensor(name, t, dtype, shape=None, device=None):
    """Checks what the C side cannot see: type, shape, device and layout."""
    if t.dtype is not dtype or not t.is_cuda:
        raise ValueError(f"{name}: need a CUDA tensor of {dtype}, got {t.dtype} on {t.device}")
    if device is not None and t.device.index != device:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: need shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


class SpinRope:
    """Position rotation: pair j of a head turns by position * inv_freq[j] radians.

    The first 2 * len(inv_freq) dimensions are rotated (a multiple of 16, at most 128; none for
    an empty list). Dimension j pairs with j + len(inv_freq), or 2j with 2j + 1 where
    interleaved."""

    def __init__(self, inv_freq: Sequence[float], interleaved: bool = False):
        self.inv_freq = [float(f) for f in inv_freq]
        self.interleaved = bool(interleaved)
        self.dim = 2 * len(self.inv_freq)
        self._c = (ctypes.c_double * max(1, len(self.inv_freq)))(*self.inv_freq)

    @classmethod
    def from_base(cls, base: float, dim: int = 128, interleaved: bool = False) -> "SpinRope":
        return cls([base ** (-2.0 * j / dim) for j in range(dim // 2)], interleaved)


class SpinKV8Step:
    """The new tokens of one step, the same for every layer: past int32 [batch] (tokens in the
    cache before it), cu_new int32 [batch + 1] (request b's rows), and their host bounds. A
    captured graph replays with whatever the two tensors hold by then, within the bounds."""

    def __init__(self, past, cu_new, total_new: int, max_new: int):
        import torch
        _tensor("past", past, torch.int32)
        if past.dim() != 1:
            raise ValueError("past: need shape [batch]")
        _tensor("cu_new", cu_new, torch.int32, (past.numel() + 1,), past.device.index)
        self.past, self.cu_new = past, cu_new
        self.batch, self.device = past.numel(), past.device.index
        self.c = B.spin_kv8_step(past.data_ptr(), cu_new.data_ptr(), int(total_new), int(max_new))
        self._at = ctypes.addressof(self.c)

    @property
    def total_new(self) -> int:
        return self.c.total_new

    @property
    def max_new(self) -> int:
        return self.c.max_new


class SpinKV8:
    """One layer's cache: the page pool, scales, tails and table, and the calls on them.

    Tensors that are not given are allocated: a pool of n_pages pages, zeroed scales and tails,
    and (summaries=True) the fp32 mean keys that Select scores, a dense copy of the complete pages' rows at a
    time. The table (int32
    [batch][kv_heads][max_pages]) says which pool page holds page p of a head; the caller fills
    it, before the call that completes or reads the page, or leaves it to the pool's calls (reserve, fork,
    compact). Those keep refs (int32 [n_pages]: the table entries that name each page; refs=True: zeros, for a new cache).

    workspace: another handle's, or new_workspace()'s, for attend (some 43 MB); or the other handle itself, for all calls'. The
    layers of a model, whose calls follow one another on a stream, need one between them. Calls that may run at the same time,
    of one handle or of two that share, need one each: every call but fork takes one of its own."""

    def __init__(self, batch: int, q_heads: int, kv_heads: int, max_pages: int, n_pages: Optional[int] = None, *,
                 rope: Optional[SpinRope] = None, pages=None, scales=None, tails=None, table=None, summaries=False,
                 refs=False, workspace=None, device: Optional[int] = None):
        import torch
        self._torch = torch
        given = [t for t in (table, pages, scales, tails) if t is not None]
        if device is None:
            device = given[0].device.index if given else torch.cuda.current_device()
        if device is None:
            raise ValueError(f"need CUDA tensors, got one on {given[0].device}")
        self.batch, self.q_heads, self.kv_heads, self.max_pages = int(batch), int(q_heads), int(kv_heads), int(max_pages)
        self.device = int(device)
        if n_pages is None:
            n_pages = pages.shape[0] if pages is not None else self.batch * self.kv_heads * self.max_pages
        self.n_pages = int(n_pages)
        dev, D, P = torch.device("cuda", self.device), B.HEAD_DIM, B.PART_TOKENS
        unit = (self.batch, self.kv_heads)

        def own(name, t, dtype, shape, make):
            return make(shape, dtype=dtype, device=dev) if t is None else _tensor(name, t, dtype, shape, self.device)

        self.pages = own("pages", pages, torch.uint8, (self.n_pages, 2, P, D), torch.empty)
        self.scales = own("scales", scales, torch.float32, (self.n_pages, 2), torch.zeros)
        self.tails = own("tails", tails, torch.bfloat16, unit + (2, P, D), torch.zeros)
        self.table = own("table", table, torch.int32, unit + (self.max_pages,), lambda s, **kw: torch.full(s, -1, **kw))
        self.summaries = None
        if summaries is not False:
            self.summaries = own("summaries", None if summaries is True else summaries, torch.float32,
                                 unit + (self.max_pages, D), torch.zeros)
        self.refs = None
        if refs is not False:
            self.refs = own("refs", None if refs is True else refs, torch.int32, (self.n_pages,), torch.zeros)
        self.error = torch.zeros(1, dtype=torch.int32, device=dev)
        self.rope = rope or SpinRope([])
        self.c = B.spin_kv8(self.batch, self.q_heads, self.kv_heads, self.max_pages, self.n_pages, self.pages.data_ptr(),
                            self.scales.data_ptr(), self.tails.data_ptr(),
                            None if self.summaries is None else self.summaries.data_ptr(), self.table.data_ptr(),
                            self.error.data_ptr(), self.device, self.rope.dim, int(self.rope.interleaved), 0,
                            ctypes.addressof(self.rope._c))
        lib = B.load()
        self._append, self._attend = lib.spin_kv8_append, lib.spin_kv8_attend
        self._select, self._attend_rows = lib.spin_kv8_select, lib.spin_kv8_attend_rows
        self._reserve, self._fork, self._compact = lib.spin_kv8_reserve, lib.spin_kv8_fork, lib.spin_kv8_compact
        self._pool_bytes = B.spin_kv8_pool_workspace(self.c)
        self._sizes = {}
        self._spaces = {}  # workspaces of the other calls, by kind: the last of each list is in use
        if isinstance(workspace, SpinKV8):
            self._spaces, workspace = workspace._spaces, workspace.workspace
        self._c_at = ctypes.addressof(self.c)
        self.workspace = self.new_workspace() if workspace is None else _tensor("workspace", workspace, torch.uint8, None, self.device)
        self._bf16 = torch.bfloat16
        self._rows = (ctypes.c_char * (4 * _ROW_BYTES))()
        at = ctypes.addressof(self._rows)
        self._rows_at = tuple(at + i * _ROW_BYTES for i in range(4))

    def new_workspace(self):
        """Workspace for one stream of attend calls; the handle has one of its own."""
        n = B.spin_kv8_workspace(self.c)
        return self._torch.empty(n, dtype=self._torch.uint8, device=self._torch.device("cuda", self.device))

    def _row(self, name, t, rows, heads):
        """The three words of a spin_rows."""
        if t.dtype is not self._bf16 or t.get_device() != self.device:
            raise ValueError(f"{name}: need a bfloat16 tensor on cuda:{self.device}, got {t.dtype} on {t.device}")
        if t.shape != (rows, heads, 128):
            raise ValueError(f"{name}: need shape {(rows, heads, 128)}, got {tuple(t.shape)}")
        ts, hs, es = t.stride()
        if es != 1:
            raise ValueError(f"{name}: the head dimension must be contiguous")
        if heads <= 1:  # a stride that nothing steps over
            hs = 128
        if rows <= 1:
            ts = hs * heads
        return t.data_ptr(), ts, hs

    def _step(self, step):
        if step.batch != self.batch or step.device != self.device:
            raise ValueError(f"the step is for {step.batch} requests on cuda:{step.device}, the cache for {self.batch} "
                             f"on cuda:{self.device}")
        return step._at, step.c.total_new

    def append(self, step: SpinKV8Step, q, k, v, q_out=None, positions=None, stream: int = 0):
        """Rotates q [total_new][q_heads][128] into q_out (q itself when q_out is None; q None:
        keys and values alone), rotates k and appends k and v [total_new][kv_heads][128], all
        bf16. positions: int32 [total_new] instead of past + i. Returns q_out."""
        sp, n = self._step(step)
        hq, hk = self.q_heads, self.kv_heads
        at_q, at_out, at_k, at_v = self._rows_at
        if q is not None:
            q_out = q if q_out is None else q_out
            _ROWS4.pack_into(self._rows, 0, *self._row("q", q, n, hq), *self._row("q_out", q_out, n, hq),
                             *self._row("k", k, n, hk), *self._row("v", v, n, hk))
        elif q_out is not None:
            raise ValueError("q_out needs q")
        else:
            at_q = at_out = None
            _ROWS2.pack_into(self._rows, 2 * _ROW_BYTES, *self._row("k", k, n, hk), *self._row("v", v, n, hk))
        pos = None
        if positions is not None:
            pos = _tensor("positions", positions, self._torch.int32, (n,), self.device).data_ptr()
        rc = self._append(self._c_at, sp, at_q, at_out, at_k, at_v, pos, stream)
        if rc:
            B._check(rc)
        return q_out

    def attend(self, step: SpinKV8Step, q, out, scale: Optional[float] = None, sel=None, workspace=None,
               stream: int = 0):
        """out [total_new][q_heads][128] = attention of the rotated q over the cache as it is after
        the step's append, each row up to its own token. out may be q itself. scale: 1/sqrt(128) by default.
        sel: int32 [batch * kv_heads][topk], the pages to attend (with the tail) instead of all; -1 is
        none. workspace: instead of the handle's own."""
        sp, n = self._step(step)
        _ROWS2.pack_into(self._rows, 0, *self._row("q", q, n, self.q_heads), *self._row("out", out, n, self.q_heads))
        sel_ptr, topk = None, 0
        if sel is not None:
            if sel.dim() != 2:
                raise ValueError("sel: need shape [batch * kv_heads][topk]")
            topk = sel.shape[1]
            sel_ptr = _tensor("sel", sel, self._torch.int32, (self.batch * self.kv_heads, topk), self.device).data_ptr()
        ws = self.workspace if workspace is None else _tensor("workspace", workspace, self._torch.uint8, None, self.device)
        rc = self._attend(self._c_at, sp, self._rows_at[0], self._rows_at[1], _SCALE if scale is None else scale, sel_ptr, topk,
                          ws.data_ptr(), ws.numel(), stream)
        if rc:
            B._check(rc)
        return out

    def _space(self, kind, nbytes, given):
        """(address, bytes) of the given workspace, or of one of the handle's own that is large enough. Those that were
        outgrown stay, for the graphs that were captured with them; each is at least twice the one before, so that a batch that
        grows a row at a time makes few, and all of them hold less than four times the most that was asked for."""
        if given is not None:
            _tensor("workspace", given, self._torch.uint8, None, self.device)
            return given.data_ptr(), given.numel()
        held = self._spaces.setdefault(kind, [])
        if not held or held[-1].numel() < nbytes:
            torch, dev = self._torch, self._torch.device("cuda", self.device)
            if torch.cuda.is_current_stream_capturing():
                raise ValueError(f"the handle's workspace of {kind} has to grow: call it once at this size before capturing, "
                                 "or give one")
            held.append(torch.empty(max(nbytes, 2 * held[-1].numel() if held else 0), dtype=torch.uint8, device=dev))
            torch.cuda.synchronize(dev)  # nothing on another stream uses that memory any more
        return held[-1].data_ptr(), held[-1].numel()

    def _lists(self, sel, rows):
        """topk of a list of pages for each row and KV head."""
        if sel.dim() != 3:
            raise ValueError("sel: need shape [total_new][kv_heads][topk]")
        _tensor("sel", sel, self._torch.int32, (rows, self.kv_heads, sel.shape[2]), self.device)
        return sel.shape[2]

    def select(self, step: SpinKV8Step, q, sel, workspace=None, stream: int = 0):
        """sel int32 [total_new][kv_heads][topk] = the topk pages of those that each row of the rotated q [total_new][q_heads][128]
        sees whole, by the products of its group's queries with the summaries; ascending, -1 behind the last. After the step's
        append. Returns sel."""
        sp, n = self._step(step)
        topk = self._lists(sel, n)
        _ROWS2.pack_into(self._rows, 0, *self._row("q", q, n, self.q_heads), 0, 0, 0)
        at, size = self._space("select", self._bytes(B.spin_kv8_select_workspace, n) if workspace is None else 0, workspace)
        rc = self._select(self._c_at, sp, self._rows_at[0], topk, sel.data_ptr(), at, size, stream)
        if rc:
            B._check(rc)
        return sel

    def attend_rows(self, step: SpinKV8Step, q, out, sel, scale: Optional[float] = None, workspace=None, stream: int = 0):
        """out [total_new][q_heads][128] = attention of the rotated q over the pages that each row lists for each KV head
        (sel int32 [total_new][kv_heads][topk], as select writes it) and its newest tokens up to itself. After the step's append.
        out may be q itself. scale: 1/sqrt(128) by default."""
        sp, n = self._step(step)
        topk = self._lists(sel, n)
        _ROWS2.pack_into(self._rows, 0, *self._row("q", q, n, self.q_heads), *self._row("out", out, n, self.q_heads))
        at, size = self._space("attend_rows", self._bytes(B.spin_kv8_attend_rows_workspace, n, topk) if workspace is None else 0, workspace)
        rc = self._attend_rows(self._c_at, sp, self._rows_at[0], self._rows_at[1], _SCALE if scale is None else scale,
                               sel.data_ptr(), topk, at, size, stream)
        if rc:
            B._check(rc)
        return out

    def _bytes(self, of, *sizes):
        key = (of, *sizes)
        if key not in self._sizes:
            self._sizes[key] = of(self.c, *sizes)
        return self._sizes[key]

    def _counts(self, free_pages):
        if self.refs is None:
            raise ValueError("the pool's calls need a handle with refs")
        return None if free_pages is None else _tensor("free_pages", free_pages, self._torch.int32, (1,), self.device).data_ptr()

    def reserve(self, step: SpinKV8Step, free_pages=None, workspace=None, stream: int = 0):
        """Before the step's append: takes free pages of the pool for the pages that the step completes. Entries that name a page
        already keep it. With too few free pages nothing is taken (check() raises). free_pages: int32 [1], gets the number of
        those that are left."""
        sp, _ = self._step(step)
        count = self._counts(free_pages)
        at, n = self._space("pool", self._pool_bytes, workspace)
        rc = self._reserve(self._c_at, sp, self.refs.data_ptr(), count, at, n, stream)
        if rc:
            B._check(rc)

    def fork(self, lengths, src, stream: int = 0):
        """Between steps: request b becomes what request src[b] was, all at once; -1: empty, and its pages are free unless others
        share them. src, lengths (tokens in the cache; updated): int32 [batch]."""
        self._counts(None)
        at = [_tensor(n, t, self._torch.int32, (self.batch,), self.device).data_ptr() for n, t in (("lengths", lengths), ("src", src))]
        rc = self._fork(self._c_at, self.refs.data_ptr(), *at, stream)
        if rc:
            B._check(rc)

    def compact(self, free_pages=None, workspace=None, stream: int = 0):
        """Moves the pages in use to the front of the pool, and the table's entries with them. free_pages: int32 [1], gets the
        number of the others."""
        count = self._counts(free_pages)
        at, n = self._space("pool", self._pool_bytes, workspace)
        rc = self._compact(self._c_at, self.refs.data_ptr(), count, at, n, stream)
        if rc:
            B._check(rc)

    def check(self, stream: int = 0):
        """Waits for the stream; raises where a call on this cache met what only the device can see."""
        B.spin_kv8_status(self.c, stream)
