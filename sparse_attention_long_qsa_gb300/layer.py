"""Device-resident state of one QSA layer and its step.

QSALayer owns the caller-side buffers of include/qsa.h (caches, block tables,
the pooled block-key cache, workspaces, outputs) as torch CUDA tensors and
runs a step as the C-ABI calls on one stream:

    step:       pool_update(dirty) -> index_topk(tokens) -> sparse_attn(tokens)
    full_step:  kv_append(new cells, re-pooling the blocks they dirty) ->
                index_attn(tokens)  (index top-k and sparse attention in one call)

and around the steps: norm_rope (the step's q, k_new and q_idx from the
projections), fork (a sequence sharing another's blocks) and release (freeing
what no sequence holds, optionally moving the rest together).

Layers of the same model that attend densely or over a window run paged_attn in
place of the index calls, after kv_append; evict cuts sequences back to the blocks
that gathered most attention, and release then frees the others' cells.

It holds no arithmetic of its own.
"""
from __future__ import annotations

import contextlib
from typing import Optional

import numpy as np
import torch

from . import qsa


def _dev(x, dtype=None, device="cuda"):
    t = torch.from_numpy(np.ascontiguousarray(x))
    if dtype is not None:
        t = t.to(dtype)
    return t.to(device)


def _on(stream):
    """Tensors made within belong to `stream` (a torch stream, its handle, or
    None for the current one): filled before what is launched there, and on
    memory that no other stream still uses."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


class QSALayer:
    def __init__(self, cfg: dict, idx_k, k_cache, v_cache, n_cells: int, blk_cells, slot_block_idx,
                 seq_blk_off, seq_blk_slots, norm_w, max_blocks: int, max_tokens: int,
                 device: str = "cuda"):
        self.cfgd = dict(cfg)
        self.cfg = qsa.config_from_dict(cfg)
        self.device = device
        self.n_cells = int(n_cells)
        self.max_blocks = max(int(max_blocks), 1)
        self.max_tokens = int(max_tokens)
        self.idx_k = _dev(idx_k, device=device)
        kv_dtype = torch.float16 if cfg["kv_type"] == "f16" else torch.uint8
        self.k_cache = _dev(k_cache, device=device).view(kv_dtype)
        self.v_cache = _dev(v_cache, device=device).view(kv_dtype)
        self.blk_cells = _dev(blk_cells, device=device)
        self.slot_block_idx = _dev(slot_block_idx, device=device)
        self.seq_blk_off = _dev(seq_blk_off, device=device)
        self.seq_blk_slots = _dev(seq_blk_slots, device=device)
        self.norm_w = _dev(norm_w, device=device)
        self.n_slots = int(self.blk_cells.shape[0])
        self.max_list = max(int(np.diff(np.asarray(seq_blk_off)).max(initial=1)), 1)   # entries of a sequence's list
        self.pooled = torch.zeros((self.n_slots, cfg["idx_dim"]), dtype=torch.float32, device=device)
        self.pitch = qsa.cells_per_token(self.cfg)
        T = self.max_tokens
        self.cells = torch.full((T, self.pitch), -1, dtype=torch.int32, device=device)
        self.count = torch.zeros(T, dtype=torch.int32, device=device)
        self.out = torch.zeros((T, cfg["n_q_heads"], cfg["head_dim"]), dtype=torch.float32, device=device)
        # zero-filled once; the library leaves its control words zero after every call
        self.ws_index = torch.zeros(qsa.index_topk_workspace_size(self.cfg, T, self.max_blocks),
                                    dtype=torch.uint8, device=device)
        self.ws_attn = torch.empty(qsa.sparse_attn_workspace_size(self.cfg, T),
                                   dtype=torch.uint8, device=device)
        self._dirty = None
        self._heads = self._sweep = self._ws_sweep = self._evicted = None
        self._ws_paged = {}
        self.block_weight = None

    @classmethod
    def from_workload(cls, wl, step: int = 0, max_tokens: Optional[int] = None, device="cuda"):
        """Upload a qsa_workload.Workload with the block table as it stands
        before steps[step] (that step's cells not yet appended)."""
        T = max_tokens or max(len(s.tok_pos) for s in wl.steps)
        return cls(wl.cfg, wl.idx_k, wl.k_cache, wl.v_cache, wl.n_cells, wl.blk_cells_state(step),
                   wl.slot_block_idx, wl.seq_blk_off, wl.seq_blk_slots, wl.norm_w,
                   wl.max_blocks(), T, device=device)

    # ---- the three calls
    def pool_update(self, dirty, stream=None):
        d = dirty if isinstance(dirty, torch.Tensor) else _dev(np.asarray(dirty, dtype=np.int32), device=self.device)
        qsa.pool_update(self.cfg, self.idx_k, self.blk_cells, self.slot_block_idx, d, self.norm_w,
                        self.pooled, stream)

    def index_topk(self, tok_seq, tok_pos, q_idx, w_idx, recomputed=None, stream=None):
        T = int(tok_pos.numel())
        qsa.index_topk(self.cfg, q_idx, w_idx, tok_seq, tok_pos, self.pooled, self.blk_cells,
                       self.seq_blk_off, self.seq_blk_slots, self.max_blocks, self.n_cells,
                       self.cells[:T], self.count[:T], self.ws_index, self.max_tokens,
                       recomputed, stream)

    def index_attn(self, tok_seq, tok_pos, q_idx, w_idx, q, recomputed=None, stream=None, in_cluster=False,
                   out=None, union=False):
        """index_topk then sparse_attn in one call (qsa_index_attn); out:
        where the attention output goes (default the layer's buffer; may be a
        pinned host tensor); union: token pairs attend over the union of
        their lists."""
        T = int(tok_pos.numel())
        qsa.index_attn(self.cfg, q_idx, w_idx, tok_seq, tok_pos, self.pooled, self.blk_cells,
                       self.seq_blk_off, self.seq_blk_slots, self.max_blocks, q, self.k_cache, self.v_cache,
                       self.n_cells, self.cells[:T], self.count[:T], self.out[:T] if out is None else out,
                       self.ws_index, self.max_tokens, recomputed, stream, in_cluster=in_cluster, union=union)

    def sparse_attn(self, q, n_tokens: int, stream=None, union=False):
        T = int(n_tokens)
        qsa.sparse_attn(self.cfg, q, self.k_cache, self.v_cache, self.n_cells, self.cells[:T],
                        self.count[:T], self.out[:T], self.ws_attn, stream, union=union)

    def step(self, tok_seq, tok_pos, q, q_idx, w_idx, dirty, stream=None):
        """One QSA step for T tokens; returns the out[:T] view (fp32)."""
        d = dirty if isinstance(dirty, torch.Tensor) else _dev(np.asarray(dirty, dtype=np.int32), device=self.device)
        self.pool_update(d, stream)
        self.index_topk(tok_seq, tok_pos, q_idx, w_idx, recomputed=d, stream=stream)
        self.sparse_attn(q, int(tok_pos.numel()), stream)
        return self.out[:int(tok_pos.numel())]

    def kv_append(self, tok_seq, tok_pos, cells, k_new, v_new, idx_new, stream=None, pool=False):
        """Write the step's new cells and build the dirty list on the device
        (with pool=True also re-pool the dirtied blocks in the same launch);
        returns the dirty-list view (padded to a power of two >= max(4, T))."""
        T = int(tok_pos.numel())
        nd = 4
        while nd < T:
            nd *= 2
        if self._dirty is None or self._dirty.numel() < nd:
            self._dirty = torch.full((max(nd, 4),), -1, dtype=torch.int32, device=self.device)
        d = self._dirty[:nd]
        extra = dict(slot_block_idx=self.slot_block_idx, norm_w=self.norm_w, pooled=self.pooled) if pool else {}
        qsa.kv_append(self.cfg, tok_seq, tok_pos, cells, k_new, v_new, idx_new, self.k_cache, self.v_cache,
                      self.idx_k, self.blk_cells, self.seq_blk_off, self.seq_blk_slots, d, stream=stream, **extra)
        return d

    def full_step(self, tok_seq, tok_pos, q, q_idx, w_idx, cells, k_new, v_new, idx_new, stream=None,
                  in_cluster=False, out=None, union=False, **_):
        """The whole layer step from the new tokens on: append of their cells
        (K/V, indexer keys, table, device dirty list) with the pool update of
        the blocks they dirty in the same launch, then index top-k and sparse
        attention in one qsa_index_attn call (in_cluster: the selection inside
        the attention clusters; union: token pairs over the union of their
        lists).  The step's inputs and `out` may be pinned
        host tensors.  Returns the output (fp32 [T][n_q_heads][head_dim])."""
        # the append re-pooled only the query tokens' own blocks: score work on
        # the other blocks may start before it finishes
        self.kv_append(tok_seq, tok_pos, cells, k_new, v_new, idx_new, stream, pool=True)
        self.index_attn(tok_seq, tok_pos, q_idx, w_idx, q, recomputed="query_blocks", stream=stream,
                        in_cluster=in_cluster, out=out, union=union)
        return self.out[:int(tok_pos.numel())] if out is None else out

    def norm_rope(self, rope, pos, q_in, k_in, q_norm_w, k_norm_w, q_idx_in, idx_pos, q_idx_norm_w, stream=None):
        """Head norms and rotation of T tokens' projections into the layer's
        buffers (more than max_tokens: into new ones, the layer's stay where
        they are); returns (q, k_new, q_idx) as full_step takes them."""
        T, c = int(q_in.shape[0]), self.cfgd
        heads = self._heads
        if heads is None or T > self.max_tokens:
            def new(h, d, t):
                return torch.empty((max(T, self.max_tokens), h, d), dtype=t, device=self.device)
            with _on(stream):
                heads = (new(c["n_q_heads"], c["head_dim"], torch.float16),
                         new(c["n_kv_heads"], c["head_dim"], torch.float16),
                         new(c["n_idx_heads"], c["idx_dim"], torch.float32))
            if T <= self.max_tokens:
                self._heads = heads
        q, k, qi = (x[:T] for x in heads)
        qsa.qk_norm_rope(self.cfg, rope, pos, q_in, k_in, q_norm_w, k_norm_w, q, k, q_idx_in, idx_pos,
                         q_idx_norm_w, qi, stream)
        return q, k, qi

    def paged_attn(self, tok_seq, tok_pos, q, window=0, n_sink=0, weigh=False, out=None, stream=None):
        """Attention of T tokens over all cells of their sequences up to
        themselves, or over the last `window` of them and the first n_sink
        (qsa_paged_attn); weigh: the probabilities are added to
        self.block_weight, one fp32 value per entry of seq_blk_slots (zeros at
        first).  Returns `out`, by default the layer's buffer (of more than
        max_tokens tokens: a new tensor, and a workspace for the call)."""
        T = int(tok_pos.numel())
        max_len = self.max_list * self.cfgd["compress_ratio"]
        ws = self._ws_paged.get(weigh)
        with _on(stream):
            if weigh and self.block_weight is None:
                self.block_weight = torch.zeros(self.seq_blk_slots.numel(), dtype=torch.float32, device=self.device)
            if ws is None or T > self.max_tokens:
                ws = torch.empty(qsa.paged_attn_workspace_size(self.cfg, max(T, self.max_tokens), max_len, weigh),
                                 dtype=torch.uint8, device=self.device)
                if T <= self.max_tokens:
                    self._ws_paged[weigh] = ws
            if out is None:
                out = self.out[:T] if T <= self.max_tokens else \
                    torch.empty((T, *self.out.shape[1:]), dtype=torch.float32, device=self.device)
        qsa.paged_attn(self.cfg, q, tok_seq, tok_pos, self.k_cache, self.v_cache, self.n_cells, self.blk_cells,
                       self.seq_blk_off, self.seq_blk_slots, max_len, out, ws, window=window, n_sink=n_sink,
                       block_weight=self.block_weight if weigh else None, stream=stream)
        return out

    def evict(self, seq_len, keep, n_sink=0, n_recent=1, stream=None):
        """Cut sequences of more than `keep` blocks back to the first n_sink,
        the last n_recent and the others of largest block_weight
        (qsa_cache_evict; seq_len: int32 CUDA tensor, positions each one
        holds): the block lists and weights close up in place.  Returns (new
        lengths, blocks evicted), the layer's own tensors, which the next call
        writes again; release(new lengths) then frees the cells, and the
        sequences' next tokens go to positions from the new lengths on."""
        n = int(seq_len.numel())
        with _on(stream):
            if self.block_weight is None:
                self.block_weight = torch.zeros(self.seq_blk_slots.numel(), dtype=torch.float32, device=self.device)
            if self._evicted is None:
                self._evicted = torch.empty((2, n), dtype=torch.int32, device=self.device)
        new_len, gone = self._evicted
        qsa.cache_evict(self.cfg, keep, n_sink, n_recent, seq_len, self.seq_blk_off, self.seq_blk_slots,
                        self.block_weight, self.max_list, new_len, self.seq_blk_slots, self.block_weight, gone, stream)
        return new_len, gone

    def kv_read(self, cells, stream=None):
        """K and V rows of the listed cells as fp16 [n][n_kv_heads][head_dim]."""
        shape = (int(cells.numel()), self.cfgd["n_kv_heads"], self.cfgd["head_dim"])
        with _on(stream):
            k, v = (torch.zeros(shape, dtype=torch.float16, device=self.device) for _ in range(2))
        qsa.kv_read(self.cfg, cells, self.k_cache, self.v_cache, self.n_cells, k, v, stream)
        return k, v

    def fork(self, src_seq, dst_seq, n_pos, tail_slot, tail_cells, stream=None):
        """Sequence dst_seq[f] becomes the first n_pos[f] positions of
        src_seq[f] (int32 CUDA tensors; tail_cells [n_fork][r]; at most the
        layer's max_blocks whole blocks, as for the steps): the block lists and
        tables, the shared blocks' weights (of the others of dst's list: 0), and
        this layer's rows of the private tail cells.
        Returns the (source, destination) cell pairs, for other layers."""
        n, r = int(src_seq.numel()), self.cfgd["compress_ratio"]
        with _on(stream):
            pairs = torch.empty((2, n, r), dtype=torch.int32, device=self.device)
        qsa.seq_fork(self.cfg, src_seq, dst_seq, n_pos, tail_slot, tail_cells, self.seq_blk_off, self.seq_blk_slots,
                     self.blk_cells, self.slot_block_idx, self.max_blocks, pairs[0], pairs[1], self.n_cells, stream,
                     self.block_weight)
        qsa.cells_copy(self.cfg, pairs[0], pairs[1], self.k_cache, self.v_cache, self.idx_k, self.n_cells,
                       stream=stream)
        return pairs[0], pairs[1]

    def release(self, seq_len, compact=False, stream=None):
        """Free what the sequences no longer hold (seq_len: int32 CUDA tensor,
        positions each one keeps), their blocks' weights with it; compact: also
        move the held cells to the front, this layer's rows with them.  Returns a dict of the sweep's
        outputs (counts, cell_map, free_cells, free_slots, move_src, move_dst):
        the layer's own tensors, which the next call writes again."""
        n, dev = self.n_cells, self.device
        if self._sweep is None:
            def i32(m):
                return torch.full((m,), -1, dtype=torch.int32, device=dev)
            with _on(stream):
                self._sweep = dict(counts=i32(4), cell_map=i32(n), free_cells=i32(n), free_slots=i32(self.n_slots),
                                   move_src=i32(n // 2), move_dst=i32(n // 2))
                self._ws_sweep = torch.empty(qsa.cache_sweep_workspace_size(self.cfg, n, self.n_slots),
                                             dtype=torch.uint8, device=dev)
        s = self._sweep
        qsa.cache_sweep(self.cfg, seq_len, self.seq_blk_off, self.seq_blk_slots, self.blk_cells, self.blk_cells, n,
                        s["counts"], self._ws_sweep, compact, s["cell_map"], s["free_cells"], s["free_slots"],
                        s["move_src"], s["move_dst"], stream)
        if self.block_weight is not None:
            qsa.weight_trim(self.cfg, seq_len, self.seq_blk_off, self.block_weight, stream)
        if compact:
            qsa.cells_copy(self.cfg, s["move_src"], s["move_dst"], self.k_cache, self.v_cache, self.idx_k, n,
                           s["counts"][3:], stream)
        return s

    def set_cells(self, slots, rows):
        """Write block-table rows (the append of new cells), device side."""
        s = _dev(np.asarray(slots, dtype=np.int64), device=self.device)
        self.blk_cells[s] = _dev(np.asarray(rows, dtype=np.int32), device=self.device)

    def warm(self, dirty_all):
        """Pool every listed slot (cold start / rebuild from the key cache)."""
        self.pool_update(dirty_all)


def step_inputs(st, device="cuda", new_cells=False):
    """Device tensors of a qsa_workload.Step (with new_cells: also the
    step's own cells and their rows, the inputs of full_step)."""
    d = dict(tok_seq=_dev(st.tok_seq, device=device), tok_pos=_dev(st.tok_pos, device=device),
             q=_dev(st.q, device=device), q_idx=_dev(st.q_idx, device=device),
             w_idx=_dev(st.w_idx, device=device), dirty=_dev(st.dirty, device=device))
    if new_cells:
        d.update(cells=_dev(st.cells, device=device), k_new=_dev(st.k_new, device=device),
                 v_new=_dev(st.v_new, device=device), idx_new=_dev(st.idx_new, device=device))
    return d


class PackedInputs:
    """A step's input tensors laid out back to back (256-byte aligned) in one
    pinned host buffer and one device buffer, so that moving a step's inputs
    to the device is a single copy.  `views` are the device tensors to pass to
    the layer's calls; `pack` fills a pinned host buffer from host arrays and
    `host_views` gives the tensors of such a buffer, which the calls can also
    take directly (read in place over the host link)."""

    def __init__(self, fields: dict, device="cuda", pin=True):
        self.fields = {}
        off = 0
        for k, (shape, dtype) in fields.items():
            n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
            self.fields[k] = (off, tuple(shape), dtype, n)
            off += -(-n // 256) * 256
        self.nbytes = off
        self.pin = pin
        self.dev = torch.empty(max(off, 256), dtype=torch.uint8, device=device)
        self.views = {k: self.dev[o:o + n].view(dtype).view(shape) for k, (o, shape, dtype, n) in self.fields.items()}

    def pack(self, arrays: dict):
        """A (pinned) host buffer holding `arrays` (numpy, same shapes and
        dtypes as the fields) in this layout."""
        host = torch.zeros(max(self.nbytes, 256), dtype=torch.uint8)
        if self.pin:
            host = host.pin_memory()
        hv = host.numpy()
        for k, (o, shape, dtype, n) in self.fields.items():
            a = np.ascontiguousarray(arrays[k])
            if a.nbytes != n or tuple(a.shape) != shape:
                raise ValueError(f"{k}: expected {shape} ({n} bytes), got {a.shape} ({a.nbytes} bytes)")
            hv[o:o + n] = a.view(np.uint8).reshape(-1)
        return host

    def host_views(self, host):
        """Tensors of the fields of a pinned host buffer made by `pack`."""
        return {k: host[o:o + n].view(dtype).view(shape) for k, (o, shape, dtype, n) in self.fields.items()}

    def upload(self, host, stream=None):
        """One host-to-device copy of a packed step (asynchronous on `stream`,
        default the current stream)."""
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            self.dev[:host.numel()].copy_(host, non_blocking=True)


def append_rows(wl, step: int):
    """Block-table rows changed by steps[step]: (slots, rows) of the state
    after the step's cells are appended (only the blocks the step touches)."""
    r = wl.r
    lens = wl.seq_len_after(step + 1)
    slots, rows = [], []
    for s, ps in enumerate(wl.steps[step].new_pos):
        if len(ps) == 0:
            continue
        off = int(wl.seq_blk_off[s])
        for j in sorted({int(p) // r for p in ps}):
            row = np.full(r, -1, dtype=np.int32)
            hi = min(lens[s], (j + 1) * r)
            row[:hi - j * r] = wl.seq_cells[s][j * r:hi]
            slots.append(int(wl.seq_blk_slots[off + j]))
            rows.append(row)
    return np.array(slots, dtype=np.int64), np.array(rows, dtype=np.int32).reshape(-1, r)
