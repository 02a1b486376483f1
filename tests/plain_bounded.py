"""Plain 64-bit forms of the bounded caches' operators, for the tests: written
from the definitions in include/xs_paged.h, sequence by sequence."""
from __future__ import annotations

import math

import numpy as np
import torch

BS = 16
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative to the value


def seen_by(n, first, window):
    """Positions that the query of the n-th token sees, ascending."""
    low = max(0, n - window) if window else 0
    return [t for t in range(n) if t < first or t >= low]


def rows(cache, table, at):
    """[len(at), Hkv, D] of positions `at`, in fp64 (table: a list of block ids)."""
    at = torch.as_tensor(at, dtype=torch.long)
    ids = torch.as_tensor(table, dtype=torch.long)[at // BS]
    return cache[ids, :, at % BS].double()


def attend(q, k, v, scale, sinks=None):
    """q [Hq, D] on rows k, v [n, Hkv, D]: the output, the weights [Hq, n], and for
    each value the size of what it is made of: (sum of p |v|, relative error of
    half a weight)."""
    G = q.shape[0] // k.shape[1]
    k, v, q = k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1), q.double()
    x = (q[None] * k).sum(-1).t() * scale
    size = (q[None] * k).abs().sum(-1).t() * abs(scale)
    top = x.amax(-1, keepdim=True)
    if sinks is not None:
        top = torch.maximum(top, sinks.double()[:, None])
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    if sinks is not None:
        total = total + torch.exp(sinks.double()[:, None] - top)
    p = p / total
    # fp32: the sum of a dot product (two units of 2^-24 a term, in any order: a
    # matrix instruction may cut), the scale and the reference; and for the sums
    # over n tokens as much again for each.
    slack = (size.amax(-1) * (2 * q.shape[1] + 4) + 2 * x.abs().amax(-1) + 16 + 2 * x.shape[-1]) * 2.0 ** -24
    return torch.einsum("hn,nhd->hd", p, v), p, torch.einsum("hn,nhd->hd", p, v.abs()), slack


def out_bound(ref, mag, slack, dtype, weight_bits):
    """One rounding to dtype.  A weight is off by the error of its logit and of
    its row's sum (twice the slack), by exp2 (2^-20) and by the rounding it enters
    the product with (2^-weight_bits)."""
    return HALF[dtype] * ref.abs() * (1 + 2.0 ** -7) + (2 * slack[:, None] + 2.0 ** -20 + 2.0 ** -weight_bits) * mag + 1e-30


def decode(q, k_cache, v_cache, tables, lens, scale, first=0, window=0, sinks=None):
    """Outputs [B, Hq, D], their bounds, and per sequence the weights [Hq, n] of
    its seen positions with theirs."""
    B, Hq, D = q.shape
    out, bound = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D, dtype=torch.float64)
    weights = []
    reach = tables.shape[1] * BS
    for b in range(B):
        n = min(int(lens[b]), reach)
        if n <= 0:
            weights.append(None)
            continue
        at = seen_by(n, first, window)
        o, p, mag, slack = attend(q[b], rows(k_cache, tables[b].tolist(), at), rows(v_cache, tables[b].tolist(), at),
                                  scale, sinks)
        out[b] = o
        bound[b] = out_bound(o, mag, slack, q.dtype, 15 if q.dtype == torch.bfloat16 else 20)
        weights.append((at, p, p * (2 * slack[:, None] + 2.0 ** -20)))
    return out, bound, weights


def prefill(q, k_cache, v_cache, ids, start, scale, first, window):
    T, Hq, D = q.shape
    out, bound = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    for i in range(T):
        at = seen_by(start + i + 1, first, window)
        o, _, mag, slack = attend(q[i], rows(k_cache, ids, at), rows(v_cache, ids, at), scale)
        out[i] = o
        bound[i] = out_bound(o, mag, slack, q.dtype, 8)     # weights of 8 bits
    return out, bound


def keep(scores, n, first, recent, budget):
    """The positions kept of one row of scores (a list of floats)."""
    middle = list(range(first, n - recent))
    value = [-math.inf if math.isnan(scores[t]) else scores[t] + 0.0 for t in middle]
    order = sorted(range(len(middle)), key=lambda i: (-value[i], i))[:budget - first - recent]
    return list(range(first)) + sorted(middle[i] for i in order) + list(range(n - recent, n))


class Evicted:
    """xs_kv_evict on numpy arrays: pools [L, nb, Hkv, 16, D] as bits."""

    def __init__(self, ids, k, v, scores, tables, lens, first, recent, budget, limit, extra=None):
        self.k, self.v, self.scores = k.copy(), v.copy(), scores.copy()
        L, B, H, S = scores.shape
        self.kept = np.full((L, len(ids), H, budget), -1, dtype=np.int32)
        self.new_lens = np.full(len(ids), -1, dtype=np.int32)
        self.flags = 0
        nb = k.shape[1]
        for i, b in enumerate(ids):
            if b < 0 or b >= B or b in ids[:i]:
                self.flags |= 4
                continue
            n = min(int(lens[b]), S)
            if int(lens[b]) > S:
                self.flags |= 2
            if n <= limit:
                continue
            row = tables[b]
            pages = range(first // BS, -(-n // BS))
            if any(row[c] < 0 or row[c] >= nb for c in pages):
                self.flags |= 1
            shared = extra is not None and budget > first and any(0 <= row[c] < nb and extra[row[c]] > 0
                                               for c in pages if c <= (budget - 1) // BS)
            if shared:
                self.flags |= 128
            if shared or any(row[c] < 0 or row[c] >= nb for c in pages):
                continue
            self.new_lens[i] = budget
            for l in range(L):
                for h in range(H):
                    at = keep(scores[l, b, h].tolist(), n, first, recent, budget)
                    self.kept[l, i, h] = at
                    self.scores[l, b, h, :budget] = scores[l, b, h, at]
                    for j, t in enumerate(at):
                        if j >= first:
                            for new, old in ((self.k, k), (self.v, v)):
                                new[l, row[j // BS], h, j % BS] = old[l, row[t // BS], h, t % BS]


def truncate(pool, ids, new_lens):
    """xs_block_truncate on a plain_ops.Pool."""
    gone = []
    for i, (b, to) in enumerate(zip(ids, new_lens)):
        if b < 0 or b >= len(pool.lens) or b in ids[:i]:
            pool.flags |= 4
            continue
        n = pool.lens[b]
        if to < 0 or to >= n:
            continue
        for c in range(-(-to // BS), min(-(-n // BS), len(pool.tables[b]))):
            blk, pool.tables[b][c] = pool.tables[b][c], -1
            if 0 <= blk < len(pool.extra):
                pool.extra[blk] -= 1
                if pool.extra[blk] < 0:
                    gone.append(blk)
            else:
                pool.flags |= 1
        pool.lens[b] = to
    for blk in sorted(gone, reverse=True):
        pool.extra[blk] = 0
        if pool.top < len(pool.stack):
            pool.stack[pool.top] = blk
            pool.top += 1
        else:
            pool.flags |= 32
