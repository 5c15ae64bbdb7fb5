"""The 8-bit paged K/V cache over torch tensors (the spec_kv8_* calls of include/spec.h).

Argument checks and marshalling only: buffers are torch tensors, every computation is a call into libspec.so on the
current stream, and no call synchronises or copies to the host.

    cache = KV8Cache(n_layers, n_kv_heads, n_pages, page=64)
    pages = cache.page_state(n_seqs, max_blocks)                  # lengths, tables, ring, state: all pages free
    plan = cache.plan(pages.lengths, add, pages.tables, pages.ring, pages.state, max_rows)
    cache.append(layer, k, v, plan.slots)                         # each layer
    ws = cache.attention_workspace(batch, n_q_heads, max_nodes, max_prefix)       # once, for the largest bounds
    out, lse = cache.attention(layer, q, pages.tables, pages.lengths, offsets, max_prefix=..., k_new=k, v_new=v,
                               parents=parents, workspace=ws)     # before the rows are appended, or without k_new
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import spec as S

try:
    from . import _kv8
except ImportError as e:  # not built
    raise ImportError("the torch binding is not built; run `python -m speculative_decoding_06_b200.build`") from e

HEAD_DIM = 128
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
        # what every call passes first: the handle, the device and the kv heads
        self._id = (h.value, self.device.index, n_kv_heads)

    def close(self):
        if getattr(self, "h", None):
            S.spec_kv8_close(self.h)
            self.h = None
            self._id = (0,) + self._id[1:]

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _fail(self, rc):
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
        if out is None:
            out = self.plan_buffers(add.shape[0], tables.shape[0], max_rows)
        rc = _kv8.plan(*self._id, self.n_pages, lengths, add, tables, ring, state, max_rows, seq_ids, *out)
        if rc:
            self._fail(rc)
        return out

    # ------------------------------------------------------------------ rows
    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
               src_rows: Optional[torch.Tensor] = None) -> None:
        """Store rows of k and v ([rows][n_kv_heads][128], fp32, bf16 or fp16, any row and head stride) at `slots`;
        row i is source row src_rows[i] (or i).  Negative slots store nothing (spec_kv8_append)."""
        rc = _kv8.append(*self._id, layer, k, v, slots, src_rows)
        if rc:
            self._fail(rc)

    def attention_workspace(self, batch: int, n_q_heads: int, max_nodes: int, max_prefix: int) -> torch.Tensor:
        """A workspace for attention() within these bounds: for fewer sequences or nodes and shorter prefixes too.  A
        program keeps one per stream, made for its largest bounds; calls (or graphs) that may run at the same time need
        one each."""
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
        offsets[b + 1] - 1, at most max_nodes, of a sequence of at most max_prefix cached tokens.  Returns (out, lse).
        Rows outside every entry, and those of an entry that is out of range (its sequence id, length or row count),
        are left as they were in `out` and `lse`; where these are new, the former are 0 and -inf, the latter NaN.
        Without `workspace` each call makes one and clears its first 64 KB.  max_prefix decides how decoding is split: a
        bound near the longest sequence is faster than the tables' capacity."""
        rc, out, lse = _kv8.attention(*self._id, layer, q, tables, lengths, offsets, max_prefix, max_nodes, k_new,
                                      v_new, parents, seq_ids, scale, out, lse, workspace)
        if rc:
            self._fail(rc)
        return out, lse
