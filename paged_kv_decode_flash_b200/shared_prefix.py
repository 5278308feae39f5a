"""Decode attention for a batch whose sequences share a long prefix.

Argument marshalling for paged_attn_decode_shared (include/pagedattn.h): the
prefix's keys are read and scored once for the query rows of all sequences,
then joined with each sequence's own keys.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as _b


class SharedPrefixDecode(_b.PagedDecode):
    """A PagedDecode configuration with room for a shared prefix of up to
    ``prefix_blocks`` blocks.  The inherited calls (plain decode, partial,
    cache_write, ...) work on the same workspace."""

    def __init__(self, *, num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                 block_size: int, max_blocks_per_seq: int, num_blocks: int, n_query: int,
                 prefix_blocks: int, device=None, workspace=None):
        d = _b.Dims(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                    max_blocks_per_seq, num_blocks, None, 0)
        need = int(_b.lib().paged_attn_shared_workspace_size(ctypes.byref(d), n_query,
                                                             int(prefix_blocks)))
        if need == 0:
            raise _b.PagedAttnError(_b.PA_ERR_INVALID_ARG, "shared_workspace_size (bad shapes)")
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device="cuda" if device is None else device)
        elif workspace.numel() * workspace.element_size() < need:
            raise _b.PagedAttnError(_b.PA_ERR_WORKSPACE, "workspace too small")
        with torch.cuda.device(workspace.device):
            super().__init__(num_seqs=num_seqs, num_q_heads=num_q_heads, num_kv_heads=num_kv_heads,
                             head_dim=head_dim, block_size=block_size,
                             max_blocks_per_seq=max_blocks_per_seq, num_blocks=num_blocks,
                             n_query=n_query, workspace=workspace)
        self.workspace_bytes = need
        self.prefix_blocks = int(prefix_blocks)
        self._caches = {kv: _b.cache_shape(kv, num_blocks, num_kv_heads, block_size, head_dim)
                        for kv in (_b.KV_FP16, _b.KV_Q8_0, _b.KV_INT8_ROW)}

    @classmethod
    def for_case(cls, case, prefix_blocks, device=None):
        return cls(num_seqs=case.num_seqs, num_q_heads=case.num_q_heads,
                   num_kv_heads=case.num_kv_heads, head_dim=case.head_dim,
                   block_size=case.block_size, max_blocks_per_seq=case.max_blocks_per_seq,
                   num_blocks=case.num_blocks, n_query=case.n_query, prefix_blocks=prefix_blocks,
                   device=device)

    def check_shared(self, prefix_table, prefix_len):
        """The addresses of the prefix's tensors, checked."""
        dev = self.workspace.device
        return (_b._given(prefix_table, "prefix_table", torch.int32, (self.prefix_blocks,), dev),
                _b._given(prefix_len, "prefix_len", torch.int32, (1,), dev))

    def __call__(self, q, k_cache, v_cache, block_table, context_lens, prefix_table=None,
                 prefix_len=None, *, causal: int, window: int, scale: float, kv_dtype: int,
                 out=None, stream=None):
        """paged_attn_decode_shared: the first prefix_len[0] keys of every
        sequence are those of prefix_table (int32 [prefix_blocks]); without
        both a plain decode."""
        if prefix_table is None and prefix_len is None:
            return super().__call__(q, k_cache, v_cache, block_table, context_lens, causal=causal,
                                    window=window, scale=scale, kv_dtype=kv_dtype, out=out,
                                    stream=stream)
        d, dev = self.dims, self.workspace.device
        qshape = (d.num_seqs, self.n_query, d.num_q_heads, d.head_dim)
        kind = self._caches.get(kv_dtype)
        if kind is None:
            _b.cache_shape(kv_dtype, 1, 1, 16, 128)  # raises
        dtype, shape = kind
        args = (_b._given(q, "q", torch.float16, qshape, dev),
                _b._given(k_cache, "k_cache", dtype, shape, dev),
                _b._given(v_cache, "v_cache", dtype, shape, dev),
                _b._given(block_table, "block_table", torch.int32,
                          (d.num_seqs, d.max_blocks_per_seq), dev),
                _b._given(context_lens, "context_lens", torch.int32, (d.num_seqs,), dev),
                *self.check_shared(prefix_table, prefix_len))
        if out is None:
            out = _b._like(q, stream)
        op = _b._given(out, "out", torch.float16, qshape, dev)
        _b._check(_b._on(dev.index, stream, lambda st: _b.lib().paged_attn_decode_shared(
            d, *args, self.prefix_blocks, self.n_query, int(causal), int(window), float(scale),
            int(kv_dtype), op, st)), "paged_attn_decode_shared")
        return out
