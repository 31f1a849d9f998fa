"""A paged latent cache whose pages are torch CUDA tensors, driving the cca_paged_* calls of the
C ABI: append with the rotation on the way, attention over the pages, dense read-back.  Holds
memory and marshals arguments only."""
from __future__ import annotations

import contextlib

import torch

from . import (CCA_BF16, CCA_F16, CCA_F32, cca_paged_append, cca_paged_attention,
               cca_paged_attention_workspace_size, cca_paged_cache_t, cca_paged_check,
               cca_paged_gather, cca_rows_t)

_DTYPES = {torch.float32: CCA_F32, torch.bfloat16: CCA_BF16, torch.float16: CCA_F16}


class PagedCache:
    """Keys and values of ``n_kv_heads`` heads, ``head_dim`` wide, in pages of ``page_size``
    tokens, 16 bits (float16 or bfloat16) or 4 (codes with a float16 scale and zero per vector).

    ``page_table`` [batch, max_pages] and ``lengths`` [batch] (int32, on the device) are the
    caller's to fill: lengths count the tokens of the call they are passed to, its new ones
    included.  With ``n_pages`` None every sequence owns ``max_pages`` pages and the table says
    so; otherwise the table starts at zero.

    New tokens come as [tokens, heads, d] with ``cu_seqlens`` (int32 [batch + 1] on the device),
    or, without it, the same number for every sequence, as [tokens, heads, d] or
    [batch, tokens per sequence, heads, d] of any strides (channels contiguous).  ``stream`` is a
    torch stream (default: the device's current one); results are allocated on it."""

    def __init__(self, batch: int, max_pages: int, page_size: int, n_kv_heads: int, head_dim: int,
                 bits: int = 4, dtype: torch.dtype = torch.float16, n_pages: int | None = None,
                 device="cuda"):
        pages = batch * max_pages if n_pages is None else n_pages
        shape = (pages, n_kv_heads, page_size)
        row = (head_dim // 2, torch.uint8) if bits == 4 else (head_dim, dtype)
        k, v = (torch.zeros(*shape, row[0], dtype=row[1], device=device) for _ in range(2))
        scales = torch.zeros(*shape, 4, dtype=torch.float16, device=device) if bits == 4 else None
        table = torch.zeros(batch, max_pages, dtype=torch.int32, device=device)
        if n_pages is None:
            table.copy_(torch.arange(pages, dtype=torch.int32).view(batch, max_pages))
        lengths = torch.zeros(batch, dtype=torch.int32, device=device)
        self._take(k, v, table, lengths, scales)

    @classmethod
    def from_pages(cls, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor,
                   lengths: torch.Tensor, scales: torch.Tensor | None = None,
                   status: torch.Tensor | None = None) -> "PagedCache":
        """A cache over existing tensors: k, v [n_pages, n_kv_heads, page_size, head_dim] of
        float16 or bfloat16, or [.., head_dim / 2] uint8 with ``scales`` [.., page_size, 4]
        float16; ``status`` an int32 of one element (None: kernel-side errors go unrecorded)."""
        self = cls.__new__(cls)
        self._take(k, v, page_table, lengths, scales, status, own_status=False)
        return self

    def _take(self, k, v, table, lengths, scales, status=None, own_status=True):
        self.device = k.device
        self.bits = 16 if scales is None else 4
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v are [n_pages, n_kv_heads, page_size, row] of one type")
        if (k.dtype != torch.uint8) if self.bits == 4 else (k.dtype not in (torch.float16, torch.bfloat16)):
            raise ValueError(f"pages of {self.bits} bits cannot be {k.dtype}")
        n_pages, n_kv, page_size, row = k.shape
        if scales is not None and (scales.shape != (n_pages, n_kv, page_size, 4)
                                   or scales.dtype != torch.float16):
            raise ValueError("scales are [n_pages, n_kv_heads, page_size, 4] float16")
        if (table.dim() != 2 or lengths.shape != table.shape[:1] or table.dtype != torch.int32
                or lengths.dtype != torch.int32):
            raise ValueError("page_table is int32 [batch, max_pages], lengths int32 [batch]")
        if own_status:
            status = torch.zeros(1, dtype=torch.int32, device=self.device)
        if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
            raise ValueError("status is an int32 tensor of one element")
        for t in (k, v, table, lengths, scales, status):
            if t is not None and (t.device != self.device or not t.is_contiguous()):
                raise ValueError("the cache's tensors are contiguous and on one device")
        self.k, self.v, self.scales = k, v, scales
        self.page_table, self.lengths, self.status = table, lengths, status
        self.batch, self.max_pages = table.shape
        self.n_kv_heads, self.page_size = n_kv, page_size
        self.head_dim = row * 2 if self.bits == 4 else row
        self.struct = cca_paged_cache_t(
            k.data_ptr(), v.data_ptr(), None if scales is None else scales.data_ptr(),
            table.data_ptr(), lengths.data_ptr(), None if status is None else status.data_ptr(),
            self.batch, self.max_pages, n_pages, page_size, n_kv, self.head_dim, self.bits,
            CCA_F16 if self.bits == 4 else _DTYPES[k.dtype])
        self.conv_state = self.vshift_state = None     # a layer's (CCALayer.new_paged_cache)

    # ------------------------------------------------------------------ marshalling
    def _on(self, stream):
        """The device and, where given, the stream that the call's allocations belong to."""
        if stream is not None:
            return torch.cuda.stream(stream)
        if torch.cuda.current_device() == self.device.index:
            return contextlib.nullcontext()
        return torch.cuda.device(self.device)

    def _tokens(self, t: torch.Tensor, cu) -> int:
        if t.dim() == 4:
            if cu is not None or t.shape[0] != self.batch:
                raise ValueError("[batch, tokens, heads, d] rows are for uniform batches")
            return t.shape[0] * t.shape[1]
        if t.dim() != 3:
            raise ValueError("rows are [tokens, heads, d] or [batch, tokens, heads, d]")
        return t.shape[0]

    def _rows(self, t: torch.Tensor, like=None, heads: int | None = None) -> cca_rows_t:
        if t.device != self.device or t.dtype not in _DTYPES:
            raise ValueError(f"rows must be floating and on {self.device}")
        if t.shape[-1] != self.head_dim or (t.shape[-1] > 1 and t.stride(-1) != 1):
            raise ValueError(f"rows end in {self.head_dim} contiguous channels")
        if heads is not None and t.shape[-2] != heads:
            raise ValueError(f"{t.shape[-2]} heads, {heads} expected")
        if like is not None and t.shape[:-2] != like.shape[:-2]:
            raise ValueError(f"rows of {tuple(t.shape[:-2])} tokens beside {tuple(like.shape[:-2])}")
        if t.dim() == 4:
            return cca_rows_t(t.data_ptr(), _DTYPES[t.dtype], t.stride(0), t.stride(1), t.stride(2))
        per = t.shape[0] // self.batch
        return cca_rows_t(t.data_ptr(), _DTYPES[t.dtype], per * t.stride(0), t.stride(0), t.stride(1))

    def _cu(self, cu):
        if cu is not None and (cu.dtype != torch.int32 or cu.device != self.device
                               or cu.numel() != self.batch + 1 or not cu.is_contiguous()):
            raise ValueError("cu_seqlens is a contiguous int32 tensor of batch + 1 on the cache's device")
        return cu

    # ------------------------------------------------------------------ the operators
    def append(self, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor | None = None,
               cu_seqlens: torch.Tensor | None = None, rope_base: float = 0.0,
               q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
        """Stores the new tokens' keys and values in their pages; with rope_base > 1 keys and
        queries are rotated to their positions on the way.  Returns the rotated queries."""
        cu = self._cu(cu_seqlens)
        n = self._tokens(k, cu)
        kr, vr = self._rows(k, None, self.n_kv_heads), self._rows(v, k, self.n_kv_heads)
        with self._on(stream):
            qr = qo = None
            if q is not None:
                qr = self._rows(q, k)
                if q_out is None:
                    q_out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
                qo = self._rows(q_out, k, q.shape[-2])
            cca_paged_append(self.struct, qr, kr, vr, qo, q.shape[-2] if q is not None else 0, cu, n,
                             rope_base, stream)
        return q_out if q is not None else None

    def attend(self, q: torch.Tensor, cu_seqlens: torch.Tensor | None = None,
               scale: float | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Causal attention of the new tokens' queries over their sequences' pages (which hold
        the new tokens already); scale None: 1 / sqrt(head_dim)."""
        cu = self._cu(cu_seqlens)
        n, heads = self._tokens(q, cu), q.shape[-2]
        if scale is not None and scale == 0.0:
            raise ValueError("a scale of 0 is not taken (None means 1 / sqrt(head_dim))")
        qr = self._rows(q)
        with self._on(stream):
            if out is None:
                out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
            orow = self._rows(out, q, heads)
            # scratch of its own for every call: captured graphs and streams never share one
            ws = torch.empty(cca_paged_attention_workspace_size(self.struct, heads, n),
                             dtype=torch.uint8, device=self.device)
            cca_paged_attention(self.struct, qr, orow, heads, cu, n, scale or 0.0, ws, stream)
        return out

    def gather(self, tokens: int | None = None, cu_seqlens: torch.Tensor | None = None,
               k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
               dtype: torch.dtype | None = None, stream=None):
        """The cached rows, dense: (k, v) of [tokens, n_kv_heads, d] with room for sequence b at
        cu_seqlens[b], or the given outputs (uniform rows of any strides; packed with
        cu_seqlens).  Rows behind a sequence's end are left as they are."""
        cu = self._cu(cu_seqlens)
        with self._on(stream):
            if k_out is None:
                dt = dtype or (torch.float16 if self.bits == 4 else self.k.dtype)
                shape = (tokens, self.n_kv_heads, self.head_dim)
                k_out, v_out = (torch.empty(shape, dtype=dt, device=self.device) for _ in range(2))
            n = self._tokens(k_out, cu)
            cca_paged_gather(self.struct, self._rows(k_out, None, self.n_kv_heads),
                             self._rows(v_out, k_out, self.n_kv_heads), cu, n, stream)
        return k_out, v_out

    def check(self, stream=None):
        """Waits for the stream and raises CCAError if a kernel recorded an error since."""
        with self._on(stream):
            cca_paged_check(self.struct, stream)
