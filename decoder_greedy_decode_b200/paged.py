"""A paged KV cache: pages of a shared pool, the sequences that hold them, the
append of rotated rows and the attention that reads them.

Marshalling only: torch provides device memory and streams, every operation
runs in libdec.so's kernels (dec_pages_*, dec_paged_append,
dec_paged_attention).
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import capi, tensors
from .rotary import Rope


class PagedKV:
    """A pool of pages and the map of its sequences, over the caller's tensors.

    k, v     [n_layers, n_pages, n_kv_heads, page_rows, head_dim], bf16, or
             uint8 E4M3 codes with k_scale, v_scale fp32 [n_layers, n_pages,
             n_kv_heads, page_rows].  Layers and pages may be strided (the
             rows of one page of one head are contiguous, its heads follow one
             another); k and v have the same strides.
    table    int32 [n_seqs, width], -1 behind a sequence's last page
    rows     int32 [n_seqs], rows that each sequence holds
    refs     int32 [n_pages], how many table entries name a page

    `create` makes all of them for an empty cache.  Errors found on the device
    (a page that is not assigned, too few free pages) are collected in
    `status`; `check` reads and clears it.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, rows: torch.Tensor,
                 refs: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        if k.dim() != 5 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must be alike, [layers, pages, kv_heads, page_rows, head_dim]")
        self.n_layers, self.n_pages, self.n_kv_heads, self.page_rows, self.head_dim = k.shape
        D, page = self.head_dim, self.page_rows * self.head_dim
        if k.stride(4) != 1 or k.stride(3) != D or (self.n_kv_heads > 1 and k.stride(2) != page):
            raise ValueError("the rows of a page must be contiguous")
        if k.dtype == torch.bfloat16:
            code = capi.DEC_KV_BF16
            if k_scale is not None or v_scale is not None:
                raise ValueError("a bf16 pool has no scales")
        elif k.dtype == torch.uint8:
            code = capi.DEC_KV_FP8_E4M3
            if k_scale is None or v_scale is None:
                raise ValueError("an E4M3 pool needs k_scale and v_scale")
        else:
            raise ValueError(f"k must be bfloat16 or uint8 (E4M3 codes), got {k.dtype}")
        # (torch leaves the stride of a dimension of length 1 open)
        ls = k.stride(0) if self.n_layers > 1 else max(k.stride(0), self.n_kv_heads * page)
        ps = k.stride(1) if self.n_pages > 1 else max(k.stride(1), self.n_kv_heads * page)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is None:
                continue
            if t.dtype != torch.float32 or t.shape != k.shape[:4] or t.stride(3) != 1 or \
                    (self.n_kv_heads > 1 and t.stride(2) != self.page_rows) or \
                    (self.n_layers > 1 and t.stride(0) * D != ls) or \
                    (self.n_pages > 1 and t.stride(1) * D != ps):
                raise ValueError(f"{name} must be fp32 with the layout of k's rows")
        self.device = k.device
        tensors.same_device(self.device, v=v, k_scale=k_scale, v_scale=v_scale)
        if table.dim() != 2:
            raise ValueError("table must be [n_seqs, width]")
        self.n_seqs, self.width = table.shape
        tensors.check_tensor(table, "table", torch.int32, None, self.device)
        tensors.check_tensor(rows, "rows", torch.int32, (self.n_seqs,), self.device)
        tensors.check_tensor(refs, "refs", torch.int32, (self.n_pages,), self.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.table, self.rows, self.refs = table, rows, refs
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.pool = capi.dec_pages(
            k.data_ptr(), v.data_ptr(), None if k_scale is None else k_scale.data_ptr(),
            None if v_scale is None else v_scale.data_ptr(), self.n_layers, self.n_pages,
            self.page_rows, self.n_kv_heads, D, code, ls, ps)
        self.map = capi.dec_page_map(table.data_ptr(), rows.data_ptr(), refs.data_ptr(),
                                     self.n_seqs, self.width)
        self._ws_bytes = capi.dec_pages_workspace_bytes(self.pool, self.map)
        if self._ws_bytes == 0:
            raise ValueError("unsupported pool or map (page_rows a power of two in 8..1024, "
                             "head_dim 64 or 128, at most 4096 sequences, 16-byte aligned)")
        self._refs = (ctypes.byref(self.pool), ctypes.byref(self.map))
        self._status = self.status.data_ptr()
        self._attend_bytes = {}

    @classmethod
    def create(cls, n_layers: int, n_pages: int, page_rows: int, n_kv_heads: int, head_dim: int,
               n_seqs: int, max_rows: int, dtype: str = "bf16", device="cuda") -> "PagedKV":
        """An empty cache: a pool of n_pages pages and room for n_seqs sequences
        of up to max_rows rows."""
        shape = (n_layers, n_pages, n_kv_heads, page_rows, head_dim)
        scales = {}
        if dtype == "bf16":
            kv = [torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(2)]
        elif dtype == "fp8":
            kv = [torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2)]
            scales = {n: torch.zeros(shape[:4], dtype=torch.float32, device=device)
                      for n in ("k_scale", "v_scale")}
        else:
            raise ValueError(dtype)
        width = -(-max_rows // page_rows)
        table = torch.full((n_seqs, width), -1, dtype=torch.int32, device=device)
        rows = torch.zeros(n_seqs, dtype=torch.int32, device=device)
        refs = torch.zeros(n_pages, dtype=torch.int32, device=device)
        return cls(kv[0], kv[1], table, rows, refs, **scales)

    # (scratch comes from torch's allocator call by call: calls on several
    # streams and several captured graphs never share it)

    def resize(self, new_rows: torch.Tensor, stream=None) -> None:
        """Every sequence s holds new_rows[s] rows (int32; negative: as it is)."""
        dev = self.device
        if tensors.elsewhere(dev, stream):
            with tensors.guard(dev, stream):
                return self.resize(new_rows)
        tensors.check_tensor(new_rows, "new_rows", torch.int32, (self.n_seqs,), dev)
        ws = torch.empty(self._ws_bytes, dtype=torch.uint8, device=dev)
        rc = capi.lib().dec_pages_resize(*self._refs, new_rows.data_ptr(), ws.data_ptr(),
                                         self._ws_bytes, self._status, tensors.current_stream_of(dev))
        if rc:
            raise capi.DecError(rc, "dec_pages_resize")

    def fork(self, parents: torch.Tensor, stream=None) -> None:
        """Sequence s becomes a copy of sequence parents[s] (int32; negative:
        empty), all at once, by sharing pages."""
        dev = self.device
        if tensors.elsewhere(dev, stream):
            with tensors.guard(dev, stream):
                return self.fork(parents)
        tensors.check_tensor(parents, "parents", torch.int32, (self.n_seqs,), dev)
        rc = capi.lib().dec_pages_fork(*self._refs, parents.data_ptr(), self._status,
                                       tensors.current_stream_of(dev))
        if rc:
            raise capi.DecError(rc, "dec_pages_fork")

    def compact(self, stream=None) -> torch.Tensor:
        """Live pages move to the lowest numbers; returns their count (int32 [1])."""
        dev = self.device
        if tensors.elsewhere(dev, stream):
            with tensors.guard(dev, stream):
                return self.compact()
        live = torch.empty(1, dtype=torch.int32, device=dev)
        ws = torch.empty(self._ws_bytes, dtype=torch.uint8, device=dev)
        rc = capi.lib().dec_pages_compact(*self._refs, live.data_ptr(), ws.data_ptr(),
                                          self._ws_bytes, self._status,
                                          tensors.current_stream_of(dev))
        if rc:
            raise capi.DecError(rc, "dec_pages_compact")
        return live

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
               seqs: Optional[torch.Tensor] = None, rope: Optional[Rope] = None,
               q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
               q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None,
               eps: float = 1e-6, stream=None) -> Optional[torch.Tensor]:
        """Store the rows k, v [tokens, n_kv_heads, head_dim] of new tokens at
        `positions` of sequences `seqs` (int32; None: token i is sequence i),
        k normalised by k_norm and rotated by `rope`, and q [tokens,
        n_q_heads, head_dim] likewise into q_out (bf16; a new one, zero
        where tokens are skipped, if None), which is returned.  Tokens at negative positions are skipped."""
        dev = self.device
        if tensors.elsewhere(dev, stream):
            with tensors.guard(dev, stream):
                return self.append(layer, k, v, positions, seqs, rope, q, q_out, q_norm, k_norm, eps)
        D, H = self.head_dim, self.n_kv_heads
        shape = tensors.check_heads(k, "k", dev)
        T = shape[0]
        if shape != (T, H, D) or tensors.check_heads(v, "v", dev) != shape or v.dtype != k.dtype:
            raise ValueError(f"k and v must be alike, [tokens, {H}, {D}]")
        tensors.check_tensor(positions, "positions", torch.int32, (T,), dev)
        io = capi.dec_append(T, tensors.dtype_code(k, "k"))
        if q is not None:
            shape = tensors.check_heads(q, "q", dev)
            if shape[0] != T or shape[2] != D or q.dtype != k.dtype:
                raise ValueError(f"q must be [{T}, heads, {D}] of {k.dtype}")
            if q_out is None:
                q_out = q.new_empty(shape, dtype=torch.bfloat16)
                io.zero_skipped = 1
            else:
                tensors.check_tensor(q_out, "q_out", torch.bfloat16, shape, dev)
            io.n_q_heads, io.q, io.q_stride = shape[1], q.data_ptr(), q.stride(0)
            io.q_out = q_out.data_ptr()
        elif q_out is not None:
            raise ValueError("q_out without q")
        io.k, io.k_stride, io.v, io.v_stride = k.data_ptr(), k.stride(0), v.data_ptr(), v.stride(0)
        io.positions, io.eps = positions.data_ptr(), eps
        if seqs is not None:
            tensors.check_tensor(seqs, "seqs", torch.int32, (T,), dev)
            io.seqs = seqs.data_ptr()
        if q_norm is not None:
            tensors.check_tensor(q_norm, "q_norm", torch.bfloat16, (D,), dev)
            io.q_norm = q_norm.data_ptr()
        if k_norm is not None:
            tensors.check_tensor(k_norm, "k_norm", torch.bfloat16, (D,), dev)
            io.k_norm = k_norm.data_ptr()
        if rope is not None:
            if rope.device != dev:
                raise ValueError(f"rope must be on {dev}, got {rope.device}")
            io.rope = rope.pointer
        rc = capi.lib().dec_paged_append(*self._refs, layer, ctypes.byref(io), self._status,
                                         tensors.current_stream_of(dev))
        if rc:
            raise capi.DecError(rc, "dec_paged_append")
        return q_out

    def attend(self, layer: int, q: torch.Tensor, rows: Optional[torch.Tensor] = None,
               window: int = 0, out: Optional[torch.Tensor] = None, return_lse: bool = False,
               stream=None):
        """Attention of one new token per sequence: q bf16 [batch, n_q_heads,
        head_dim] over the first rows[b] rows (int32; None: self.rows) of
        sequences 0 .. batch-1, the last `window` of them if that is not 0
        (several new tokens of one sequence have no call of their own yet).
        Returns out fp32 [batch, n_q_heads, head_dim], with return_lse also
        the log of the softmax sums [batch, n_q_heads]."""
        dev = self.device
        if tensors.elsewhere(dev, stream):
            with tensors.guard(dev, stream):
                return self.attend(layer, q, rows, window, out, return_lse)
        B, Hq, D = shape = tensors.check_heads(q, "q", dev)
        if q.dtype != torch.bfloat16 or D != self.head_dim:
            raise ValueError(f"q must be bfloat16 [batch, heads, {self.head_dim}]")
        if rows is not None:
            tensors.check_tensor(rows, "rows", torch.int32, (B,), dev)
        if out is None:
            out = q.new_empty(shape, dtype=torch.float32)
        else:
            tensors.check_tensor(out, "out", torch.float32, shape, dev)
        nb = self._attend_bytes.get((B, Hq))
        if nb is None:
            nb = capi.dec_paged_attention_workspace_bytes(self.pool, B, Hq)
            self._attend_bytes[(B, Hq)] = nb
        lse = q.new_empty((B, Hq), dtype=torch.float32) if return_lse else None
        ws = torch.empty(nb or 256, dtype=torch.uint8, device=dev)
        rc = capi.lib().dec_paged_attention(
            *self._refs, layer, B, Hq, q.data_ptr(), q.stride(0),
            None if rows is None else rows.data_ptr(), window, out.data_ptr(),
            None if lse is None else lse.data_ptr(), ws.data_ptr(), nb, self._status,
            tensors.current_stream_of(dev))
        if rc:
            raise capi.DecError(rc, "dec_paged_attention")
        return (out, lse) if return_lse else out

    def check(self) -> int:
        """The device errors since the last check (DEC_DEV_* bits; waits for
        the work on the current stream).  An error that a call on another
        stream finds meanwhile is in this check's bits or in the next one's."""
        dev = self.device
        if tensors.elsewhere(dev, None):
            with tensors.guard(dev, None):
                return self.check()
        taken = torch.empty(1, dtype=torch.int32, device=dev)
        rc = capi.lib().dec_status_take(self._status, taken.data_ptr(),
                                        tensors.current_stream_of(dev))
        if rc:
            raise capi.DecError(rc, "dec_status_take")
        return int(taken.item())
