"""The 8-bit paged K/V cache over torch tensors (the spec_kv8_* calls of include/spec.h).

Argument checks and marshalling only: buffers are torch tensors, every computation is a call into libspec.so on the
current stream, and no call synchronises or copies to the host.

    cache = KV8Cache(n_layers, n_kv_heads, n_pages, page=64)
    pages = cache.page_state(n_seqs, max_blocks)                  # lengths, tables, ring, state: all pages free
    plan = cache.plan(pages.lengths, add, pages.tables, pages.ring, pages.state, max_rows)
    cache.append(layer, k, v, plan.slots)                         # each layer
    out, lse = cache.attention(layer, q, pages.tables, pages.lengths, offsets, max_prefix=..., k_new=k, v_new=v,
                               parents=parents)                   # before the rows are appended, or without k_new
"""

from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional

import torch

from . import spec as S

HEAD_DIM = 128
_DTYPE = {torch.float32: S.SPEC_DTYPE_F32, torch.bfloat16: S.SPEC_DTYPE_BF16, torch.float16: S.SPEC_DTYPE_F16}
# the argument structures, field by field as include/spec.h declares them
_PLAN = struct.Struct("@11P4i")
_APPEND = struct.Struct("@4P4q3i4x")
_ATTN = struct.Struct("@11PN7q8if4x")
_I32 = torch.int32


class PageState(NamedTuple):
    lengths: torch.Tensor  # int32 [n_seqs]
    tables: torch.Tensor   # int32 [n_seqs][max_blocks]
    ring: torch.Tensor     # int32 [n_pages]
    state: torch.Tensor    # int32 [2]: head and count of the free pages in the ring


class PagePlan(NamedTuple):
    offsets: torch.Tensor  # int32 [batch + 1]: the first new row of every entry
    slots: torch.Tensor    # int32 [max_rows]: slots of the new rows, then -1
    lengths: torch.Tensor  # int32 [n_seqs]: lengths after the step
    state: torch.Tensor    # int32 [2]: the ring's state after the step
    status: torch.Tensor   # int32 [1]: 0, or SPEC_KV8_* bits: nothing was done


def _ints(t: torch.Tensor, name: str, device, shape) -> int:
    """The address of a contiguous int32 tensor of this shape (None: any extent)."""
    if t.dtype is not _I32 or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor on %s" % (name, device))
    if t.dim() != len(shape) or any(w is not None and w != g for w, g in zip(shape, t.shape)):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, device, heads: int):
    """Checks [rows][heads][128] with contiguous heads' values; (address, row stride, head stride)."""
    if t.device != device or t.dim() != 3 or t.shape[1] != heads or t.shape[2] != HEAD_DIM:
        raise ValueError("%s must be [rows][%d][%d] on %s, got %s on %s" % (name, heads, HEAD_DIM, device,
                                                                            tuple(t.shape), t.device))
    r, h, c = t.stride()
    if c != 1:
        raise ValueError("%s must have contiguous values (last stride 1, got %d)" % (name, c))
    return t.data_ptr(), r, h


class KV8Cache:
    """One 8-bit paged cache: codes uint8 [n_layers][K, V][n_pages][n_kv_heads][page][128] (e4m3 bits) and exps uint8
    [n_layers][K, V][n_pages][n_kv_heads] (the page's scale is 2^(byte - 127)), allocated here unless given."""

    def __init__(self, n_layers: int, n_kv_heads: int, n_pages: int, page: int = 64,
                 codes: Optional[torch.Tensor] = None, exps: Optional[torch.Tensor] = None, device=None):
        self.h = None
        self.cfg = S.spec_kv8_config(n_layers=n_layers, n_kv_heads=n_kv_heads, head_dim=HEAD_DIM, page=page,
                                     n_pages=n_pages)
        nc = S.spec_kv8_code_bytes(ctypes.byref(self.cfg))
        ne = S.spec_kv8_exp_bytes(ctypes.byref(self.cfg))
        if nc == 0:
            raise S.SpecError(S.SPEC_ERR_ARG, "cache configuration rejected")
        if (codes is None) != (exps is None):
            raise ValueError("codes and exps go together")
        if codes is None:
            device = torch.device("cuda" if device is None else device)
            codes = torch.empty((n_layers, 2, n_pages, n_kv_heads, page, HEAD_DIM), dtype=torch.uint8, device=device)
            exps = torch.empty((n_layers, 2, n_pages, n_kv_heads), dtype=torch.uint8, device=device)
        for t, shape, n in ((codes, (n_layers, 2, n_pages, n_kv_heads, page, HEAD_DIM), nc),
                            (exps, (n_layers, 2, n_pages, n_kv_heads), ne)):
            if t.dtype is not torch.uint8 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != shape:
                raise ValueError("expected a contiguous uint8 CUDA tensor of shape %s" % (shape,))
        if codes.device != exps.device:
            raise ValueError("codes and exps are on different devices")
        self.codes, self.exps = codes, exps
        self.device = codes.device
        self.n_layers, self.n_kv_heads, self.n_pages, self.page = n_layers, n_kv_heads, n_pages, page
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            rc = S.spec_kv8_open(ctypes.byref(self.cfg), codes.data_ptr(), nc, exps.data_ptr(), ne, ctypes.byref(h))
        if rc != S.SPEC_OK:
            raise S.SpecError(rc, "spec_kv8_open failed")
        self.h = h
        lib = S.lib()
        self._c_plan, self._c_append, self._c_attn = lib.spec_kv8_plan, lib.spec_kv8_append, lib.spec_kv8_attention

    def close(self):
        if getattr(self, "h", None):
            S.spec_kv8_close(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------------ helpers
    def _call(self, fn, *args):
        """fn(handle, *args, stream) on the cache's device and torch's current stream there."""
        if torch.cuda.current_device() == self.device.index:
            rc = fn(self.h, *args, torch.cuda.current_stream().cuda_stream)
        else:
            with torch.cuda.device(self.device):
                rc = fn(self.h, *args, torch.cuda.current_stream().cuda_stream)
        if rc != S.SPEC_OK:
            raise S.SpecError(rc, S.spec_kv8_last_error(self.h).decode())

    # ------------------------------------------------------------------ pages
    def page_state(self, n_seqs: int, max_blocks: int) -> PageState:
        """Empty sequences, every page free."""
        dev = self.device
        return PageState(torch.zeros(n_seqs, dtype=_I32, device=dev),
                         torch.full((n_seqs, max_blocks), -1, dtype=_I32, device=dev),
                         torch.arange(self.n_pages, dtype=_I32, device=dev),
                         torch.tensor([0, self.n_pages], dtype=_I32, device=dev))

    def plan_buffers(self, batch: int, n_seqs: int, max_rows: int) -> PagePlan:
        """Output buffers for plan(..., out=): a program that keeps them allocates nothing per step."""
        def new(n):
            return torch.empty(n, dtype=_I32, device=self.device)
        return PagePlan(new(batch + 1), new(max_rows), new(n_seqs), new(2), new(1))

    def plan(self, lengths: torch.Tensor, add: torch.Tensor, tables: torch.Tensor, ring: torch.Tensor,
             state: torch.Tensor, max_rows: int, seq_ids: Optional[torch.Tensor] = None,
             out: Optional[PagePlan] = None) -> PagePlan:
        """Pages, slots and lengths of a step (spec_kv8_plan).  Entry b, sequence seq_ids[b] (or b), goes from
        lengths to max(0, lengths + add[b]) tokens.  tables and ring are updated in place (only entries beyond the old
        lengths and free places change); the new lengths and state are in the result, whose buffers (`out`) may be
        lengths and state themselves."""
        dev, batch, (n_seqs, max_blocks) = self.device, add.shape[0], tables.shape
        if out is None:
            out = self.plan_buffers(batch, n_seqs, max_rows)
        args = _PLAN.pack(
            _ints(lengths, "lengths", dev, (n_seqs,)), _ints(add, "add", dev, (batch,)),
            0 if seq_ids is None else _ints(seq_ids, "seq_ids", dev, (batch,)),
            _ints(tables, "tables", dev, (n_seqs, max_blocks)), _ints(ring, "ring", dev, (self.n_pages,)),
            _ints(state, "state", dev, (2,)), _ints(out.offsets, "offsets", dev, (batch + 1,)),
            _ints(out.slots, "slots", dev, (max_rows,)), _ints(out.lengths, "lengths", dev, (n_seqs,)),
            _ints(out.state, "state", dev, (2,)), _ints(out.status, "status", dev, (1,)),
            batch, n_seqs, max_blocks, max_rows)
        self._call(self._c_plan, args)
        return out

    # ------------------------------------------------------------------ rows
    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
               src_rows: Optional[torch.Tensor] = None) -> None:
        """Store rows of k and v ([rows][n_kv_heads][128], fp32, bf16 or fp16, any row and head stride) at `slots`;
        row i is source row src_rows[i] (or i).  Negative slots store nothing (spec_kv8_append)."""
        dev = self.device
        if k.dtype is not v.dtype or k.dtype not in _DTYPE:
            raise ValueError("k and v must both be fp32, bf16 or fp16")
        if k.shape[0] != v.shape[0]:
            raise ValueError("k and v have %d and %d rows" % (k.shape[0], v.shape[0]))
        kp, kr, kh = _rows(k, "k", dev, self.n_kv_heads)
        vp, vr, vh = _rows(v, "v", dev, self.n_kv_heads)
        rows = slots.shape[0]
        args = _APPEND.pack(kp, vp, _ints(slots, "slots", dev, (rows,)),
                            0 if src_rows is None else _ints(src_rows, "src_rows", dev, (rows,)),
                            kr, kh, vr, vh, _DTYPE[k.dtype], rows, k.shape[0])
        self._call(self._c_append, layer, args)

    def attention_workspace(self, batch: int, n_q_heads: int, max_nodes: int, max_prefix: int) -> torch.Tensor:
        """A workspace for attention() within these bounds.  A program keeps one per stream; calls (or graphs) that
        may run at the same time need one each."""
        n = S.spec_kv8_attention_workspace(self.h, batch, n_q_heads, max_nodes, max_prefix)
        if n == 0:
            raise S.SpecError(S.SPEC_ERR_ARG, "attention bounds rejected")
        return torch.zeros(n, dtype=torch.uint8, device=self.device)

    def attention(self, layer: int, q: torch.Tensor, tables: torch.Tensor, lengths: torch.Tensor,
                  offsets: torch.Tensor, max_prefix: int, max_nodes: int = 128,
                  k_new: Optional[torch.Tensor] = None, v_new: Optional[torch.Tensor] = None,
                  parents: Optional[torch.Tensor] = None, seq_ids: Optional[torch.Tensor] = None, scale: float = 0.0,
                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None):
        """Attention of q's rows ([rows][n_q_heads][128], bf16 or fp16) over the cached prefixes and, with k_new and
        v_new ([rows][n_kv_heads][128]), the step's own rows (spec_kv8_attention).  Entry b holds rows offsets[b] ..
        offsets[b + 1] - 1, at most max_nodes, of a sequence of at most max_prefix cached tokens.  Returns (out, lse);
        rows outside every entry are left as they were."""
        dev = self.device
        rows, hq = q.shape[0], q.shape[1]
        batch, (n_seqs, max_blocks) = offsets.shape[0] - 1, tables.shape
        dt = q.dtype
        if dt is not torch.bfloat16 and dt is not torch.float16:
            raise ValueError("q must be bf16 or fp16")
        qp, qr, qh = _rows(q, "q", dev, hq)
        if (k_new is None) != (v_new is None):
            raise ValueError("k_new and v_new go together")
        kp = kr = kh = vp = vr = vh = 0
        if k_new is not None:
            if k_new.dtype is not dt or v_new.dtype is not dt:
                raise ValueError("k_new and v_new must have q's dtype")
            if k_new.shape[0] != rows or v_new.shape[0] != rows:
                raise ValueError("k_new and v_new must have q's %d rows" % rows)
            kp, kr, kh = _rows(k_new, "k_new", dev, self.n_kv_heads)
            vp, vr, vh = _rows(v_new, "v_new", dev, self.n_kv_heads)
        if out is None:
            out = torch.empty((rows, hq, HEAD_DIM), dtype=dt, device=dev)
        elif out.dtype is not dt or out.shape != q.shape or (rows and out.stride()[1:] != (HEAD_DIM, 1)):
            raise ValueError("out must have q's dtype and shape, its heads contiguous")
        if lse is None:
            lse = torch.empty((rows, hq), dtype=torch.float32, device=dev)
        elif lse.dtype is not torch.float32 or tuple(lse.shape) != (rows, hq) or not lse.is_contiguous() or \
                lse.device != dev:
            raise ValueError("lse must be contiguous fp32 [%d][%d] on %s" % (rows, hq, dev))
        op, orow, _ = _rows(out, "out", dev, hq)
        if workspace is None:
            workspace = self.attention_workspace(batch, hq, max_nodes, max_prefix)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous on %s" % dev)
        args = _ATTN.pack(
            qp, kp, vp, 0 if parents is None else _ints(parents, "parents", dev, (rows,)),
            _ints(offsets, "offsets", dev, (batch + 1,)), _ints(tables, "tables", dev, (n_seqs, max_blocks)),
            _ints(lengths, "lengths", dev, (n_seqs,)),
            0 if seq_ids is None else _ints(seq_ids, "seq_ids", dev, (batch,)),
            op, lse.data_ptr(), workspace.data_ptr(), workspace.nbytes, qr, qh, kr, kh, vr, vh, orow,
            _DTYPE[dt], batch, n_seqs, max_blocks, hq, rows, max_nodes, max_prefix, scale)
        self._call(self._c_attn, layer, args)
        return out, lse
