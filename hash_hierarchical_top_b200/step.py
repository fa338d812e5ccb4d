"""Buffer ownership for one decode layer: the caller-side plumbing around the C ABI.

``LayerCache`` holds the per-layer retrieval metadata (page summaries, codes,
block means) next to the caller's K/V cache; ``DecodeStep`` owns the workspaces
and outputs of one decode step and runs append-encode -> select -> sparse
attention through the C ABI on one stream. ``KV8Cache`` is a layer's 8-bit K/V
cache; ``DenseStep`` attends to every key of a cache (bf16 or 8-bit), and
``BlockStep`` selects blocks by their mean keys and attends to those, for one
token or a chunk of queries per sequence. PyTorch only allocates memory here
(and takes 1 from the lengths where block means are kept); every step of the path
runs in the library's kernels.
"""
from __future__ import annotations

import math

import torch

from . import hhr


class _NewestRow:
    """The newest row of every sequence, as the `start` and `n_new` of an append."""

    def __init__(self, d: hhr.Dims, device):
        self.start, self.one = (torch.ones(d.batch, dtype=torch.int32, device=device)
                                for _ in range(2))

    def position(self, seq_len, stream):
        """seq_len - 1, on `stream` (a torch stream, a raw handle, or None for the current one)."""
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream))
        with torch.cuda.stream(stream):
            return torch.sub(seq_len.reshape(-1)[:len(self.start)], 1, out=self.start)


class LayerCache:
    """Retrieval metadata of one layer, laid out as include/hhr.h documents."""

    def __init__(self, d: hhr.Dims, device, hashing=True, block_means=False):
        n, G, P = d.n_phys_pages, d.n_kv_heads, d.page_size
        # Zero-filled, so that slots past a sequence's end have deterministic contents.
        sdt = torch.float16 if d.summary_fp16 else torch.float32
        self.page_minmax = (torch.zeros(n, G, 2, d.head_dim, dtype=sdt, device=device)
                            if hashing else None)
        self.codes = (torch.zeros(n, G, P, d.code_bits // 32, dtype=torch.int32, device=device)
                      if hashing else None)
        self.block_mean = (torch.zeros(n, G, d.head_dim, dtype=torch.float32, device=device)
                           if block_means else None)


class DecodeStep:
    """Workspaces and outputs of one decode step (hash mode) or one selection (indexer)."""

    def __init__(self, d: hhr.Dims, mode: int, m_pages: int, keep_div: int, top_k: int, device,
                 attention: bool = True, sink_pages: int = 0, local_pages: int = 0):
        self.d, self.mode, self.m_pages, self.keep_div, self.top_k = d, mode, m_pages, keep_div, top_k
        self.opts = hhr.make_opts(sink_pages, local_pages)  # forced pages (hash mode variant)
        rows = hhr.sel_rows(d) if mode == hhr.HHR_MODE_HASH else d.n_q_heads
        ws = hhr.hhr_select_workspace_bytes(d, mode, m_pages, keep_div, top_k)
        if ws == 0:
            raise ValueError("unsupported selection parameters")
        self.sel_ws = torch.empty(ws, dtype=torch.uint8, device=device)
        self.idx = torch.empty(d.batch, rows, top_k, dtype=torch.int32, device=device)
        self.count = torch.empty(d.batch, rows, dtype=torch.int32, device=device)
        self.m_max = hhr.hhr_kept_max(d, m_pages, keep_div)
        self.attention = attention and mode == hhr.HHR_MODE_HASH
        self.fused_ws = self.newest = None  # made by the first fused_step that needs them
        if self.attention:
            aws = hhr.hhr_attn_workspace_bytes(d, top_k)
            self.attn_ws = torch.empty(aws, dtype=torch.uint8, device=device)
            self.out = torch.empty(d.batch, d.n_q_heads, d.head_dim, dtype=torch.float32,
                                   device=device)

    def encode(self, k_cache, page_table, start, n_new, max_new, R, W, cache: LayerCache,
               stream=None):
        hhr.hhr_encode_keys(self.d, k_cache, page_table, start, n_new, max_new, R, W,
                            cache.page_minmax, cache.codes, cache.block_mean, stream)

    def select(self, q, seq_len, page_table, cache: LayerCache, R=None, W=None, k_cache=None,
               q_pos=None, trace=None, stream=None):
        hhr.hhr_select(self.d, self.mode, q, seq_len, q_pos, page_table, R, W, cache.page_minmax,
                       cache.codes, cache.block_mean, k_cache, self.m_pages, self.keep_div,
                       self.top_k, self.idx, self.count, self.sel_ws, trace, stream, self.opts)

    def attend(self, q, k_cache, v_cache, page_table, seq_len, scale=None, stream=None):
        if scale is None:
            scale = 1.0 / math.sqrt(self.d.head_dim)
        hhr.hhr_sparse_attn(self.d, q, k_cache, v_cache, page_table, seq_len, self.idx,
                            self.count, self.top_k, scale, self.out, self.attn_ws, stream)

    def fused_step(self, q, k_cache, v_cache, page_table, seq_len, R, W, cache: LayerCache,
                   k_new=None, v_new=None, scale=None, stream=None):
        """One decode step through hhr_decode_step (the fused single-call path), which encodes the
        newest row; the block means of a cache that has them are brought up to date behind it."""
        if self.fused_ws is None:
            n = hhr.hhr_decode_step_workspace_bytes(self.d, self.m_pages, self.keep_div,
                                                    self.top_k)
            self.fused_ws = torch.empty(n, dtype=torch.uint8, device=self.idx.device)
        if scale is None:
            scale = 1.0 / math.sqrt(self.d.head_dim)
        hhr.hhr_decode_step(self.d, q, k_new, v_new, k_cache, v_cache, page_table, seq_len, R, W,
                            cache.page_minmax, cache.codes, self.m_pages, self.keep_div,
                            self.top_k, scale, self.idx, self.count, self.out, self.fused_ws,
                            stream, self.opts)
        if cache.block_mean is not None:
            if self.newest is None:
                self.newest = _NewestRow(self.d, self.idx.device)
            hhr.hhr_encode_keys(self.d, k_cache, page_table, self.newest.position(seq_len, stream),
                                self.newest.one, 1, None, None, None, None, cache.block_mean, stream)
        return self.out

    def step(self, q, k_cache, v_cache, page_table, seq_len, R, W, cache: LayerCache,
             append_start, append_n, stream=None):
        """One HHR decode step: encode the appended key(s), select, attend."""
        self.encode(k_cache, page_table, append_start, append_n, 1, R, W, cache, stream)
        self.select(q, seq_len, page_table, cache, R=R, W=W, stream=stream)
        self.attend(q, k_cache, v_cache, page_table, seq_len, stream=stream)
        return self.out


class KV8Cache:
    """A layer's 8-bit K/V cache (e4m3 with one exponent byte per row), and optionally the mean
    key of every page, laid out as include/hhr.h documents."""

    def __init__(self, d: hhr.Dims, device, block_means=False):
        shape = (d.n_phys_pages, d.n_kv_heads, d.page_size)
        self.d = d
        self.k, self.v = (torch.zeros(*shape, d.head_dim, dtype=torch.uint8, device=device)
                          .view(torch.float8_e4m3fn) for _ in range(2))
        self.k_exp, self.v_exp = (torch.zeros(shape, dtype=torch.uint8, device=device)
                                  for _ in range(2))
        self.block_mean = (torch.zeros(d.n_phys_pages, d.n_kv_heads, d.head_dim,
                                       dtype=torch.float32, device=device)
                           if block_means else None)

    def append(self, k_new, v_new, start, n_new, page_table, stream=None):
        """Quantise new rows [B][max_new][G][d] into positions [start, start + n_new)."""
        hhr.hhr_append_kv8(self.d, k_new, v_new, start, n_new, page_table, self.k, self.v,
                           self.k_exp, self.v_exp, self.block_mean, stream)

    def read(self, start, n, page_table, k_out, v_out, stream=None):
        """Read positions [start, start + n) back as bf16 [B][max_n][G][d]."""
        hhr.hhr_read_kv8(self.d, self.k, self.v, self.k_exp, self.v_exp, page_table, start, n,
                         k_out, v_out, stream)


def _cache_args(cache):
    """(k, v, k_exp, v_exp) of a KV8Cache, or of a (k_cache, v_cache) pair in bf16."""
    if isinstance(cache, KV8Cache):
        return cache.k, cache.v, cache.k_exp, cache.v_exp
    k, v = cache
    return k, v, None, None


class DenseStep:
    """Workspace and outputs of dense decode attention: one new token per sequence over every key
    of its cache."""

    def __init__(self, d: hhr.Dims, device, out_dtype=torch.float32):
        self.d = d
        n = hhr.hhr_paged_attn_workspace_bytes(d)
        if n == 0:
            raise ValueError("unsupported dims")
        self.ws = torch.empty(n, dtype=torch.uint8, device=device)
        self.out = torch.empty(d.batch, d.n_q_heads, d.head_dim, dtype=out_dtype, device=device)
        self.lse = torch.empty(d.batch, d.n_q_heads, dtype=torch.float32, device=device)
        self.newest = _NewestRow(d, device)

    def attend(self, q, cache, page_table, seq_len, k_new=None, v_new=None, scale=None,
               stream=None):
        """cache: a KV8Cache, or (k_cache, v_cache) in bf16. k_new, v_new [B][G][d]: the rows of
        position seq_len - 1, written by the same call. A KV8Cache with block means has them brought
        up to date by an append of these rows behind it. Of a bf16 cache only the rows are written:
        its page summaries, codes and block means (LayerCache) are the encoder's."""
        if scale is None:
            scale = 1.0 / math.sqrt(self.d.head_dim)
        k, v, k_exp, v_exp = _cache_args(cache)
        hhr.hhr_paged_attn(self.d, q, k_new, v_new, k, v, k_exp, v_exp, page_table, seq_len, scale,
                           self.out, self.ws, self.lse, stream)
        if k_new is not None and isinstance(cache, KV8Cache) and cache.block_mean is not None:
            k_new, v_new = (x.reshape(-1, 1, self.d.n_kv_heads, self.d.head_dim)[:self.d.batch]
                            for x in (k_new, v_new))
            cache.append(k_new, v_new, self.newest.position(seq_len, stream), self.newest.one,
                         page_table, stream)
        return self.out


class BlockStep:
    """Workspaces, block lists and outputs of block-sparse attention for n_queries tokens per
    sequence."""

    def __init__(self, d: hhr.Dims, n_queries: int, m_pages: int, device, sink_pages: int = 0,
                 local_pages: int = 0, out_dtype=torch.float32):
        self.d, self.m_pages = d, m_pages
        self.opts = hhr.make_opts(sink_pages, local_pages)
        m_max = hhr.hhr_kept_max(d, m_pages, 0)
        sel = hhr.hhr_block_select_workspace_bytes(d, n_queries)
        att = hhr.hhr_block_attn_workspace_bytes(d, n_queries, m_max)
        if m_max < 1 or sel == 0 or att == 0:
            raise ValueError("unsupported block selection parameters")
        u8 = dict(dtype=torch.uint8, device=device)
        self.sel_ws, self.attn_ws = torch.empty(sel, **u8), torch.empty(att, **u8)
        B, T, rows = d.batch, n_queries, hhr.sel_rows(d)
        self.blocks = torch.empty(B, T, rows, m_max, dtype=torch.int32, device=device)
        self.count = torch.empty(B, T, rows, dtype=torch.int32, device=device)
        self.out = torch.empty(B, T, d.n_q_heads, d.head_dim, dtype=out_dtype, device=device)
        self.lse = torch.empty(B, T, d.n_q_heads, dtype=torch.float32, device=device)

    def select(self, q, seq_len, page_table, block_mean, q_pos=None, stream=None):
        hhr.hhr_block_select(self.d, q, seq_len, q_pos, page_table, block_mean, self.m_pages,
                             self.blocks, self.count, self.sel_ws, stream, self.opts)

    def attend(self, q, cache, page_table, seq_len, q_pos=None, scale=None, stream=None):
        if scale is None:
            scale = 1.0 / math.sqrt(self.d.head_dim)
        k, v, k_exp, v_exp = _cache_args(cache)
        hhr.hhr_block_attn(self.d, q, k, v, k_exp, v_exp, page_table, seq_len, q_pos, self.blocks,
                           self.count, scale, self.out, self.attn_ws, self.lse, stream)
        return self.out

    def step(self, q, cache, page_table, seq_len, block_mean=None, q_pos=None, stream=None):
        """Select by block_mean (a KV8Cache's own when None), then attend."""
        mean = cache.block_mean if block_mean is None else block_mean
        self.select(q, seq_len, page_table, mean, q_pos, stream)
        return self.attend(q, cache, page_table, seq_len, q_pos, stream=stream)
