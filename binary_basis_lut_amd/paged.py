"""A layer's attention over a paged cache: rotation and append, attention, as a class on tensors.

`PagedAttention` owns a cache and what goes with it; `rope_frequencies` gives the angles per position that
its rotation takes.
"""
from __future__ import annotations

import math

WORKSPACE = 72 << 20  # bytes: fluxbin_paged_attention asks for no more


def rope_frequencies(rotary_dim: int, theta: float = 10000.0, linear: float = 1.0, by_parts=None):
    """fp64 [rotary_dim / 2] on the CPU: theta^(-2j / rotary_dim), scaled for contexts longer than the model's own.

    linear: every frequency divided by it.  by_parts = (factor, low, high, length): frequencies of which a
    text of `length` positions holds fewer than `low` turns are divided by factor, those of more than `high`
    turns kept, those between mixed in proportion.
    """
    import torch

    f = theta ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim) / linear
    if by_parts is not None:
        factor, low, high, length = by_parts
        if not (factor > 0 and high > low and length > 0):
            raise ValueError(f"by_parts: {by_parts}")
        turns = length * f / (2 * math.pi)
        kept = ((turns - low) / (high - low)).clamp(0, 1)
        f = f * kept + f / factor * (1 - kept)
    return f


class PagedAttention:
    """Attention of `heads` query heads over a paged cache of `kv_heads` heads, for up to max_tokens new rows
    of up to max_seqs sequences at a time.

    The caller fills `page_table` (int32 [max_seqs][max_pages], -1: no page) and `kv_lens` (int32 [max_seqs],
    the lengths with the new tokens), on the device, before the work of attend() runs; the cache is
    `k_cache`, `v_cache` [pages][kv_heads][page_size][dim].  attend() enqueues fluxbin_rope_append and
    fluxbin_paged_attention on the current stream and returns a view of a buffer that the next call
    overwrites; it allocates nothing, so it can be captured in a graph, which then serves every step of a
    decode.  Calls of one object share its buffers: the caller orders calls on different streams.
    """

    def __init__(self, heads: int, kv_heads: int, dim: int, pages: int, page_size: int, max_seqs: int, max_pages: int,
                 max_tokens: int, dtype=None, device="cuda", freq=None, rotary_dim: int | None = None, pairs: int = 0,
                 rope_scale: float = 1.0, q_norm=None, k_norm=None, eps: float = 1e-5, window: int = 0):
        import torch
        from . import fluxbin as F

        dtype = torch.float16 if dtype is None else dtype
        if dtype not in (torch.float16, torch.bfloat16):
            raise ValueError(f"dtype: {dtype}, not fp16 or bf16")
        if not 0 <= window < 1 << 31:  # attention alone takes it, behind an append that would have run
            raise ValueError(f"window: {window}, not in [0, 2^31)")
        self.F, self.heads, self.kv_heads, self.dim, self.window, self.eps = F, heads, kv_heads, dim, window, eps
        self.dtype, self.scale, self.pairs, self.rope_scale = dtype, 1 / math.sqrt(dim), pairs, rope_scale
        self.rotary_dim = dim if rotary_dim is None else rotary_dim
        dev = torch.device(device)
        self.device = dev = torch.device(dev.type, torch.cuda.current_device()) if dev.index is None else dev
        self._check_current()
        if freq is None:
            freq = rope_frequencies(self.rotary_dim)
        self.freq = freq.to(dev, torch.float64).contiguous()
        if tuple(self.freq.shape) != (self.rotary_dim // 2,):
            raise ValueError(f"freq: {tuple(self.freq.shape)}, not ({self.rotary_dim // 2},)")
        for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
            if w is not None:
                self._check(name, w, dtype, (dim,))
        self.q_norm, self.k_norm = (None if w is None else w.contiguous() for w in (q_norm, k_norm))
        new = lambda *shape, dtype=dtype: torch.zeros(shape, dtype=dtype, device=dev)
        self.k_cache, self.v_cache = new(pages, kv_heads, page_size, dim), new(pages, kv_heads, page_size, dim)
        self.page_table = torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=dev)
        self.kv_lens = new(max_seqs, dtype=torch.int32)
        self.q, self.out = new(max_tokens, heads * dim), new(max_tokens, heads * dim)
        self.workspace = torch.empty(WORKSPACE, dtype=torch.uint8, device=dev)
        b = self.batch = F.PagedBatch()
        b.abi_version, b.dtype = F.ABI_VERSION, F.DT_F16 if dtype == torch.float16 else F.DT_BF16
        b.heads, b.kv_heads, b.dim, b.page_size = heads, kv_heads, dim, page_size
        b.kv_lens, b.page_table = self.kv_lens.data_ptr(), self.page_table.data_ptr()
        b.table_ld = b.table_pages = max_pages
        b.k_cache, b.v_cache, b.cache_pages = self.k_cache.data_ptr(), self.v_cache.data_ptr(), pages
        b.page_stride, b.head_stride, b.token_stride = kv_heads * page_size * dim, page_size * dim, dim
        F.fluxbin_paged_attention_workspace_size(b)  # refuses what the kernels do not take
        torch.cuda.current_stream().synchronize()  # the cache and the frequencies are there for a call on any stream

    def _check(self, name, t, dtype, shape) -> None:
        if t.dtype != dtype or t.device != self.device or tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, not {dtype} {tuple(shape)} on {self.device}")

    def _check_current(self) -> None:
        import torch

        if torch.cuda.current_device() != self.device.index:  # where the launches go
            raise ValueError(f"the cache is on {self.device}, the current device is cuda:{torch.cuda.current_device()}")

    def attend(self, qkv, seq_starts=None, seqs: int | None = None, max_kv_len: int = 0, positions=None):
        """qkv: [rows][(heads + 2 kv_heads) * dim] in dtype, queries, keys, values, any row stride.

        seq_starts: int32 [seqs + 1] on the device, or None: a row to a sequence.  Rows of the result behind
        the last sequence are left as they were.  positions: int32 [rows], or None: the places in the cache.
        max_kv_len: what no length passes, 0: whatever the page table holds, which divides the work of short
        sequences as if they were as long.
        """
        import torch

        rows, h, kv, d = qkv.shape[0], self.heads, self.kv_heads, self.dim
        if rows > self.q.shape[0]:
            raise ValueError(f"qkv {tuple(qkv.shape)}: at most {self.q.shape[0]} rows")
        self._check("qkv", qkv, self.dtype, (rows, (h + 2 * kv) * d))
        if qkv.stride(1) != 1:
            raise ValueError(f"qkv: the elements of a row lie {qkv.stride(1)} apart, not side by side")
        if seq_starts is None:
            seqs = rows if seqs is None else seqs
            if seqs != rows:
                raise ValueError(f"{rows} rows of {seqs} sequences without seq_starts")
        else:
            seqs = seq_starts.shape[0] - 1 if seqs is None else seqs
            self._check("seq_starts", seq_starts, torch.int32, (seqs + 1,))
            if not seq_starts.is_contiguous():
                raise ValueError("seq_starts: not contiguous")
        if seqs > self.kv_lens.shape[0]:
            raise ValueError(f"{seqs} sequences: at most {self.kv_lens.shape[0]}")
        if positions is not None:
            self._check("positions", positions, torch.int32, (rows,))
            if not positions.is_contiguous():
                raise ValueError("positions: not contiguous")
        self._check_current()
        F, b = self.F, self.batch
        b.tokens, b.seqs, b.max_kv_len = rows, seqs, max_kv_len
        b.seq_starts = None if seq_starts is None else seq_starts.data_ptr()
        ld = qkv.stride(0) if rows > 1 else qkv.shape[1]  # a single row's stride can be any number
        F.fluxbin_rope_append(b, qkv, ld, qkv[:, h * d:], ld, qkv[:, (h + kv) * d:], ld, self.q_norm, self.k_norm, self.eps,
                              self.freq if self.rotary_dim else None, self.rotary_dim, self.pairs, self.rope_scale, positions,
                              self.q, h * d)
        F.fluxbin_paged_attention(b, self.q, h * d, self.scale, self.window, self.out, h * d, None, self.workspace,
                                  self.workspace.numel())
        return self.out[:rows]
