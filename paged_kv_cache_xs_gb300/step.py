"""One continuous-batching decode step over a paged KV cache.

``PagedDecodeStep`` owns nothing but the split-K workspace; the KV pools,
block tables and lengths belong to the caller.  A step is

1. slot resolution + KV append (the pages' reshape_and_cache_batched_bf16,
   "xserv compare phase10...cf1e9e4", attention.rs);
2. paged decode attention over split-K partitions;
3. the split-K combine (only when a sequence can span several partitions).

``run`` enqueues all three as one launch (``xs_paged_decode_step``);
``run_unfused`` enqueues them as the separate calls ``xs_kv_append_paged``,
``xs_paged_decode_attn`` and ``xs_paged_decode_reduce`` (``append``,
``attend`` and ``reduce`` below).

``run_from_host`` is the same step fed from pinned host buffers: it copies
the step's inputs to the device, runs the step and copies the output back.
"""
from __future__ import annotations

import torch

from . import ops


class PagedDecodeStep:
    """sinks ([Hq] tensor of q's dtype, or None) and window (0 = all tokens)
    select the gpt-oss variant: per-head sink logits and a sliding window.
    ``fused`` picks the partition heuristic for ``run`` (True) or for
    ``run_unfused`` (False); both forms work with either."""

    def __init__(self, B: int, Hq: int, Hkv: int, D: int, max_blocks_per_seq: int, dtype,
                 device, total_context_tokens: int = 0, max_context_len: int | None = None,
                 partition_tokens: int | None = None, sinks=None, window: int = 0,
                 fused: bool = True):
        self.B, self.Hq, self.Hkv, self.D = B, Hq, Hkv, D
        self.sinks, self.window = sinks, int(window)
        self.dtype = dtype
        self.device = torch.device(device)
        self.max_blocks_per_seq = max_blocks_per_seq
        self.ws = ops.DecodeWorkspace(B, Hq, Hkv, D, max_blocks_per_seq, self.device,
                                      total_context_tokens=total_context_tokens,
                                      max_context_len=max_context_len,
                                      partition_tokens=partition_tokens, fused=fused)
        self.err_flag = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._dev_inputs = None

    @property
    def partition_tokens(self) -> int:
        return self.ws.partition_tokens

    @property
    def max_partitions(self) -> int:
        return self.ws.max_partitions

    def cluster_size(self, fused: bool = True) -> int:
        """Cluster size the one-launch step runs with on the current device
        (0: the persistent grid, whose split is partition_tokens)."""
        if not fused:
            return 0
        return ops.xs_paged_decode_step_cluster_size(self.B, self.Hq, self.Hkv, self.D,
                                                     self.max_blocks_per_seq, self.window,
                                                     self.dtype)

    def launches_per_step(self, fused: bool = True) -> int:
        if fused:
            return 1
        return 3 if self.ws.max_partitions > 1 else 2

    def append(self, k_new, v_new, k_cache, v_cache, block_tables, context_lens):
        ops.xs_kv_append_paged(k_new, v_new, k_cache, v_cache, block_tables, context_lens,
                               err_flag=self.err_flag)

    def attend(self, out, q, k_cache, v_cache, block_tables, context_lens, scale):
        ws = self.ws
        if self.sinks is None and self.window == 0:
            ops.xs_paged_decode_attn(out, ws.part_o, ws.part_m, ws.part_l, q, k_cache, v_cache,
                                     block_tables, context_lens, scale, ws.partition_tokens,
                                     ws.max_partitions, err_flag=self.err_flag,
                                     work_counters=ws.work)
        else:
            ops.xs_paged_decode_attn_sinks(out, ws.part_o, ws.part_m, ws.part_l, q, k_cache,
                                           v_cache, block_tables, context_lens, scale,
                                           ws.partition_tokens, ws.max_partitions,
                                           sinks=self.sinks, window=self.window,
                                           err_flag=self.err_flag, work_counters=ws.work)

    def reduce(self, out, context_lens):
        ws = self.ws
        if ws.max_partitions <= 1:
            return
        if self.sinks is None and self.window == 0:
            ops.xs_paged_decode_reduce(out, ws.part_o, ws.part_m, ws.part_l, context_lens,
                                       ws.partition_tokens, ws.max_partitions)
        else:
            ops.xs_paged_decode_reduce_sinks(out, ws.part_o, ws.part_m, ws.part_l, context_lens,
                                             ws.partition_tokens, ws.max_partitions,
                                             sinks=self.sinks, window=self.window)

    def run(self, out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, scale,
            early_reads: bool = False, persistent: bool = False):
        """Append this step's K/V, attend and combine in one launch; all
        tensors on the device.  ``early_reads``: the launch reads lengths,
        tables and its first pages before the previous kernel on the stream
        completes (that kernel must write none of them: e.g. another layer's
        step, or a projection).  ``persistent``: the persistent grid even
        where the launch would run as clusters."""
        ws = self.ws
        ops.xs_paged_decode_step(out, q, k_new, v_new, k_cache, v_cache, block_tables,
                                 context_lens, scale, ws.partition_tokens, ws.max_partitions,
                                 ws.part_o, ws.part_m, ws.part_l, ws.work, sinks=self.sinks,
                                 window=self.window, err_flag=self.err_flag,
                                 early_reads=early_reads, persistent=persistent)
        return out

    def run_unfused(self, out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens,
                    scale):
        """The same step as three launches: append, attention, combine."""
        self.append(k_new, v_new, k_cache, v_cache, block_tables, context_lens)
        self.attend(out, q, k_cache, v_cache, block_tables, context_lens, scale)
        self.reduce(out, context_lens)
        return out

    def run_from_host(self, out_host, q, k_new, v_new, block_tables, context_lens, k_cache,
                      v_cache, scale):
        """Step fed from (pinned) host tensors q, k_new, v_new, block_tables and
        context_lens; the pools stay on the device.  Writes out_host and waits
        for it."""
        if self._dev_inputs is None or self._dev_inputs[0].shape != q.shape \
                or self._dev_inputs[3].shape != block_tables.shape:
            self._dev_inputs = tuple(torch.empty(t.shape, dtype=t.dtype, device=self.device)
                                     for t in (q, k_new, v_new, block_tables, context_lens))
            self._dev_out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
        dq, dk, dv, dbt, dcl = self._dev_inputs
        for d, h in zip(self._dev_inputs, (q, k_new, v_new, block_tables, context_lens)):
            d.copy_(h, non_blocking=True)
        self.run(self._dev_out, dq, dk, dv, k_cache, v_cache, dbt, dcl, scale)
        out_host.copy_(self._dev_out, non_blocking=True)
        torch.cuda.current_stream().synchronize()
        return out_host

    def error_flags(self) -> int:
        return int(self.err_flag.item())


class CapturedStep:
    """A decode step (any sequence of library calls, e.g. every layer's
    append + attention + reduce) captured once into a CUDA graph and
    replayed.

    Every kernel of the path reads its per-step data (lengths, block tables,
    q, the new K/V rows) from device memory and takes only fixed sizes from
    the host, so a replay sees whatever the caller has written into the same
    buffers since the last one.  The split-K work counters reset themselves
    at the end of every launch, so replays need no host action."""

    def __init__(self, fn, warmup: int = 1):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(warmup):  # fills the library's per-kernel caches
                fn()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            fn()

    def replay(self):
        self.graph.replay()


class Kv4DecodeStep:
    """The decode step on a 4-bit cache, from one layer's q, k and v as they
    leave their projection: norm of each head and rotation, append into the
    4-bit pages, attention (``xs_qk_norm_rope_append_paged``, then
    ``xs_kv4_decode``).

    Owns the attention's workspace and the rotated q.  A sequence whose new
    token lies behind cos_sin is not appended and its output is NaN (with
    XS_FLAG_BAD_LEN).  q_weight, k_weight
    ([D], bf16, or None: no norm) and cos_sin (``ops.rope_table``, or None: no
    rotation) are arguments of ``run``, since they differ from layer to layer;
    sinks and window as in PagedDecodeStep."""

    def __init__(self, B: int, Hq: int, Hkv: int, D: int, device, eps: float = 1e-6,
                 interleaved: bool = False, sinks=None, window: int = 0):
        self.B, self.Hq, self.Hkv, self.D = B, Hq, Hkv, D
        self.eps, self.interleaved = float(eps), bool(interleaved)
        self.sinks, self.window = sinks, int(window)
        self.device = torch.device(device)
        self.ws = ops.Kv4Workspace(B, Hq, Hkv, D, self.device)
        self.q = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=self.device)
        self.err_flag = torch.zeros(1, dtype=torch.int32, device=self.device)

    def run(self, out, q, k_new, v_new, q_weight, k_weight, cos_sin, k_cache, v_cache,
            block_tables, context_lens, scale):
        """q [B, Hq, D], k_new and v_new [B, Hkv, D] may be slices of one
        projection's output; sequence b's new token is at position
        context_lens[b] - 1."""
        ops.xs_qk_norm_rope_append_paged(self.q, q, k_new, v_new, q_weight, k_weight, self.eps,
                                         cos_sin, k_cache, v_cache, block_tables, context_lens,
                                         interleaved=self.interleaved, err_flag=self.err_flag)
        ops.xs_kv4_decode(out, self.q, k_cache, v_cache, block_tables, context_lens, scale,
                          self.ws, sinks=self.sinks, window=self.window, err_flag=self.err_flag)

    def error_flags(self) -> int:
        """Device error bits raised so far (synchronises)."""
        return int(self.err_flag.item())


class BoundedDecodeStep:
    """Decode steps on caches that are kept to a budget of tokens: each layer's
    new rows are normed, rotated and appended, attention counts what weight each
    cached token got (``run``, once a layer), and sequences that have grown
    beyond ``limit`` tokens are cut to ``budget`` of them, the ``first`` first,
    the ``recent`` last and the heaviest between (``bound``, once a step).

    A sequence's length is then less than its position: positions (int32 [B],
    the new tokens' places in their texts) are the caller's.  Owns the scores
    [layers, B, Hkv, max_blocks * 16], the attention's workspace and the rotated
    q.  ``start(slots)`` forgets the scores of slots whose sequences are new (or
    were prefilled: a prompt's tokens begin to be counted with the next step).

    A step's first ``run`` (by layers: one that is not above the last) counts
    no more scored tokens than the sequence has behind its new one, so a sequence
    may be shortened between steps (``ops.xs_block_truncate``: a rejected draft):
    the tokens that replace the lost ones start from zero.  If more than one token is
    appended to it before the next ``run``, its slot needs ``start``.

    A sequence is not cut while it shares a page that it would write (``bound``
    raises XS_FLAG_SHARED each time): it grows until the others are released."""

    def __init__(self, B: int, Hq: int, Hkv: int, D: int, max_blocks_per_seq: int, layers: int,
                 dtype: torch.dtype, device, budget: int, limit: int | None = None,
                 first: int = 4, recent: int | None = None, eps: float = 1e-6,
                 interleaved: bool = False):
        self.B, self.layers, self.budget = B, layers, int(budget)
        self.limit = self.budget if limit is None else int(limit)
        self.first = min(int(first), self.budget)
        self.recent = (self.budget - self.first) // 2 if recent is None else int(recent)
        if self.budget <= 0 or self.recent < 0 or self.first < 0 or self.limit < self.budget or \
                self.first + self.recent > self.budget:
            raise ValueError("0 <= first, recent; first + recent <= budget <= limit; budget > 0")
        if self.limit >= max_blocks_per_seq * ops.BLOCK_SIZE:
            raise ValueError("no sequence grows beyond the limit: the table holds "
                             f"{max_blocks_per_seq * ops.BLOCK_SIZE} tokens")
        self.eps, self.interleaved = float(eps), bool(interleaved)
        self.device = torch.device(device)
        i32 = dict(dtype=torch.int32, device=self.device)
        self.ws = ops.BoundedWorkspace(B, Hq, Hkv, D, self.device, max_blocks_per_seq)
        self.scores = torch.zeros(layers, B, Hkv, max_blocks_per_seq * ops.BLOCK_SIZE,
                                  dtype=torch.float32, device=self.device)
        self.scored = torch.zeros(B, **i32)
        self.behind = torch.zeros(B, **i32)     # tokens behind the new one
        self.layer = None                       # of the last run of this step
        self.kept = torch.empty(layers, B, Hkv, self.budget, **i32)
        self.new_lens = torch.empty(B, **i32)
        self.slots = torch.arange(B, **i32)
        self.q = torch.zeros(B, Hq, D, dtype=dtype, device=self.device)
        self.slot_mapping = torch.empty(B, dtype=torch.int64, device=self.device)
        self.err_flag = torch.zeros(1, **i32)

    def start(self, slots):
        """Forget the scores of slots (int64 tensor or list)."""
        self.scored[slots] = 0

    def run(self, layer, out, q, k_new, v_new, q_weight, k_weight, cos_sin, positions, k_cache,
            v_cache, block_tables, context_lens, scale):
        """One layer: q [B, Hq, D], k_new and v_new [B, Hkv, D] may be slices of
        one projection's output; sequence b's new token becomes row
        context_lens[b] - 1 of its cache.  q_weight, k_weight (or None: no norm)
        and cos_sin (``ops.rope_table``, or None: no rotation) as in
        ``ops.xs_qk_norm_rope_append``."""
        if self.layer is None or layer <= self.layer:
            torch.sub(context_lens, 1, out=self.behind)
            torch.minimum(self.scored, self.behind, out=self.scored)
        self.layer = layer
        ops.xs_slot_mapping(block_tables, context_lens, ops.BLOCK_SIZE, k_cache.shape[0],
                            self.slot_mapping, err_flag=self.err_flag)
        ops.xs_qk_norm_rope_append(self.q, q, k_new, v_new, q_weight, k_weight, self.eps, cos_sin,
                                   positions, k_cache, v_cache, self.slot_mapping,
                                   interleaved=self.interleaved, err_flag=self.err_flag)
        ops.xs_paged_decode_weights(out, self.scores[layer], self.q, k_cache, v_cache, block_tables,
                                    context_lens, scale, self.ws, scored_lens=self.scored,
                                    err_flag=self.err_flag)

    def bound(self, k_pools, v_pools, block_tables, context_lens, free_stack, free_top, extra_refs):
        """After the last layer: cut the sequences beyond the limit in all
        layers' pools [layers, num_blocks, Hkv, 16, D] and give back their
        pages."""
        ops.xs_kv_evict(self.slots, k_pools, v_pools, self.scores, block_tables, context_lens,
                        self.kept, self.new_lens, self.first, self.recent, self.limit,
                        extra_refs=extra_refs, err_flag=self.err_flag)
        if self.first == self.budget and self.budget % ops.BLOCK_SIZE:
            # The first tokens alone are kept, so the eviction wrote nothing, but the next
            # token is written to their last page.
            page = block_tables[:, self.budget // ops.BLOCK_SIZE].clamp(0, extra_refs.numel() - 1)
            shared = (extra_refs[page.long()] > 0) & (self.new_lens >= 0)
            self.new_lens.masked_fill_(shared, -1)
            self.kept.masked_fill_(shared.view(1, -1, 1, 1), -1)
            self.err_flag.bitwise_or_(shared.any().to(torch.int32) * ops.FLAG_SHARED)
        ops.xs_block_truncate(self.slots, self.new_lens, block_tables, context_lens, free_stack,
                              free_top, extra_refs, err_flag=self.err_flag)
        self.scored.copy_(context_lens)
        self.layer = None

    def error_flags(self) -> int:
        """Device error bits raised so far (synchronises)."""
        return int(self.err_flag.item())
