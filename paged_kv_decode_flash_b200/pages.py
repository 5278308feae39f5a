"""The pages of a paged KV cache: fork, resize (grow, truncate, free), compact
and copy.

Argument marshalling for the page operations of include/pagedattn.h: every
step runs on the device and nothing is copied to the host.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import binding as _b


@dataclasses.dataclass
class Moves:
    """A compaction: pages src[i] -> dst[i] for i < count[0] (-1 behind), and
    where every page went (-1: free)."""
    src: torch.Tensor
    dst: torch.Tensor
    count: torch.Tensor
    remap: torch.Tensor


class PagePool:
    """The books of one pool of KV blocks and the operations on them.

    ``block_table`` int32 [num_seqs][max_blocks_per_seq], ``context_lens``
    int32 [num_seqs], ``ref_counts`` int32 [num_blocks]: given, or made empty
    here.  Pass the first two to the decode and cache-write calls.  Requests
    are int32 device tensors.  What the device refused shows in get_error().
    """

    def __init__(self, *, num_seqs: int, num_kv_heads: int, head_dim: int, block_size: int,
                 max_blocks_per_seq: int, num_blocks: int, block_table=None, context_lens=None,
                 ref_counts=None, device=None, workspace=None):
        self.dims = _b.Dims(num_seqs, num_kv_heads, num_kv_heads, head_dim, block_size,
                            max_blocks_per_seq, num_blocks, None, 0)
        need = int(_b.lib().paged_attn_pages_workspace_size(ctypes.byref(self.dims)))
        if need == 0:
            raise _b.PagedAttnError(_b.PA_ERR_INVALID_ARG, "pages_workspace_size (bad shapes)")
        given = [t for t in (workspace, block_table, context_lens, ref_counts) if t is not None]
        device = torch.device(device if device is not None else
                              given[0].device if given else "cuda")
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device = device
        self._caches = {kv: _b.cache_shape(kv, num_blocks, num_kv_heads, block_size, head_dim)
                        for kv in (_b.KV_FP16, _b.KV_Q8_0, _b.KV_INT8_ROW)}
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        elif workspace.numel() * workspace.element_size() < need:
            raise _b.PagedAttnError(_b.PA_ERR_WORKSPACE, "workspace too small")
        elif workspace.device != device:
            raise ValueError(f"workspace is on {workspace.device}, expected {device}")
        books = {"block_table": ((num_seqs, max_blocks_per_seq), block_table, -1),
                 "context_lens": ((num_seqs,), context_lens, 0),
                 "ref_counts": ((num_blocks,), ref_counts, 0)}
        for name, (shape, t, fill) in books.items():
            if t is None:
                t = torch.full(shape, fill, dtype=torch.int32, device=device)
            self._given(t, name, shape)
            setattr(self, name, t)
        self.workspace_bytes = need
        self.workspace = workspace
        self.dims.workspace = _b._dptr(workspace)
        self.dims.workspace_bytes = workspace.numel() * workspace.element_size()
        with torch.cuda.device(device):
            _b._check(_b.lib().paged_attn_pages_workspace_init(ctypes.byref(self.dims),
                                                               _b._stream_ptr(None)),
                      "pages_workspace_init")

    def _given(self, t, name, shape):
        return _b._given(t, name, torch.int32, shape, self.device)

    def _books(self):
        return (self.block_table.data_ptr(), self.context_lens.data_ptr(),
                self.ref_counts.data_ptr())

    def _new(self, sizes, stream):
        """int32 tensors of these sizes, in one allocation."""
        t, = _b._outputs(stream, lambda: torch.empty(sum(sizes), dtype=torch.int32,
                                                     device=self.device))
        return t.split(sizes)

    def fork(self, parents, children, *, stream=None) -> None:
        """paged_attn_fork: the empty rows ``children`` become copies of the
        rows ``parents`` and hold the same pages."""
        n = children.numel()
        pp = self._given(parents, "parents", (n,))
        cp = self._given(children, "children", (n,))
        _b._check(_b._on(self.device.index, stream, lambda st: _b.lib().paged_attn_fork(
            self.dims, *self._books(), pp, cp, n, st)), "paged_attn_fork")

    def resize(self, rows, new_lens=None, *, copy_src=None, copy_dst=None, stream=None):
        """paged_attn_resize: ``rows`` get the lengths ``new_lens`` (None: 0).
        Returns (src, dst) int32 [n]: the pages to copy (-1: none) on every
        layer before the new tokens are written."""
        n = rows.numel()
        rp = self._given(rows, "rows", (n,))
        lp = None if new_lens is None else self._given(new_lens, "new_lens", (n,))
        if copy_src is None or copy_dst is None:
            src, dst = _b._like(rows, stream), _b._like(rows, stream)
            sp, dp = src.data_ptr(), dst.data_ptr()
        if copy_src is not None:
            src, sp = copy_src, self._given(copy_src, "copy_src", (n,))
        if copy_dst is not None:
            dst, dp = copy_dst, self._given(copy_dst, "copy_dst", (n,))
        _b._check(_b._on(self.device.index, stream, lambda st: _b.lib().paged_attn_resize(
            self.dims, *self._books(), rp, lp, n, sp, dp, st)), "paged_attn_resize")
        return src, dst

    def free(self, rows, *, stream=None) -> None:
        """The rows end: length 0, their pages given up (of damaged entries
        those that name a held page)."""
        self.resize(rows, stream=stream)

    def compact(self, *, stream=None) -> Moves:
        """paged_attn_compact: the live pages become the first ones of the
        pool.  Returns the moves, to be copied on every layer."""
        room = max(1, self.dims.num_blocks // 2)
        m = Moves(*self._new((room, room, 1, self.dims.num_blocks), stream))
        _b._check(_b._on(self.device.index, stream, lambda st: _b.lib().paged_attn_compact(
            self.dims, *self._books(), m.src.data_ptr(), m.dst.data_ptr(), m.count.data_ptr(),
            m.remap.data_ptr(), st)), "paged_attn_compact")
        return m

    def copy(self, k_cache, v_cache, src, dst, *, kv_dtype: int, count=None, stream=None) -> None:
        """paged_attn_copy_blocks on one layer's caches: page dst[i] becomes a
        copy of page src[i] (negative src: skipped)."""
        kind = self._caches.get(kv_dtype)
        if kind is None:
            _b.cache_shape(kv_dtype, 1, 1, 16, 128)  # raises
        dtype, shape = kind
        kp = _b._given(k_cache, "k_cache", dtype, shape, self.device)
        vp = _b._given(v_cache, "v_cache", dtype, shape, self.device)
        n = src.numel()
        sp, dp = self._given(src, "src", (n,)), self._given(dst, "dst", (n,))
        cp = None if count is None else self._given(count, "count", (1,))
        _b._check(_b._on(self.device.index, stream, lambda st: _b.lib().paged_attn_copy_blocks(
            self.dims, sp, dp, n, cp, int(kv_dtype), kp, vp, st)), "paged_attn_copy_blocks")

    def get_error(self, stream=None) -> int:
        """Synchronises and returns (and clears) what the device refused."""
        return _b._on(self.device.index, stream,
                      lambda st: _b.lib().paged_attn_get_error(self.dims, st))
