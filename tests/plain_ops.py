"""Plain 64-bit forms of the cache operators, for the tests: written from the
definitions in include/xs_paged.h, value by value where that is affordable."""
from __future__ import annotations

import math

import numpy as np
import torch

BS = 16
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative to the value


# ---------------------------------------------------------------- norm and rotation

def norm_rope(x, w, eps, table, pos, rot, interleaved):
    """(y [T, H, D] in fp64, magnitude of what each value was summed from)."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + eps) * w.double()
    out, mag = y.clone(), y.abs()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c = table[pos.long(), i].double()[:, None]
        s = table[pos.long(), rot // 2 + i].double()[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        mag[..., a] = mag[..., b] = y[..., a].abs() + y[..., b].abs()
    return out, mag


def norm_rope_bound(ref, mag, dtype):
    """One rounding to dtype, and fp32 arithmetic: 16 terms and 3 exchanges of
    the sum of squares count half in the root (9.5 units of 2^-24), rsqrt 4,
    the products with it, the weight, 1 / D and eps 4, the rotation 3 on both
    parts: under 24 units of what the value was summed from."""
    return HALF[dtype] * ref.abs() * (1 + 2.0 ** -8) + 24 * 2.0 ** -24 * mag + 2.0 ** -126


# ---------------------------------------------------------------- the 4-bit page

def quantise(x):
    """Codes (0..15) and bf16 scales of rows x [..., D], in fp64."""
    g = x.double().reshape(*x.shape[:-1], -1, 32)
    big = g.abs().amax(-1)
    positive = (g == big[..., None]).any(-1)
    s = (torch.where(positive, big, -big) * -0.125).to(torch.bfloat16)
    sd = s.double()[..., None]
    n = torch.where(sd == 0, torch.zeros_like(g), torch.round(g / torch.where(sd == 0, 1, sd)))
    return (n.clamp(-8, 7) + 8).to(torch.int64).reshape(x.shape), s


def values(codes, s):
    return ((codes.reshape(*s.shape, 32) - 8).double() * s.double()[..., None]).reshape(codes.shape)


def places(D):
    """(nibble of a K page, of a V page, scale of a K page, of a V page) for
    every (row, dim), [16, D]."""
    k, v, sk, sv = (np.zeros((BS, D), dtype=np.int64) for _ in range(4))
    ng = D // 32
    for o in range(BS):
        for d in range(D):
            c, r = divmod(d, 32)
            k[o, d] = (o * (D // 8) + (r // 8) * ng + c) * 8 + r % 8
            v[o, d] = ((o // 2) * (D // 4) + (r // 4) * ng + c) * 8 + 4 * (o % 2) + r % 4
            sk[o, d] = o * ng + c
            sv[o, d] = ((o // 2) * ng + c) * 2 + o % 2
    return tuple(torch.from_numpy(x) for x in (k, v, sk, sv))


def write_rows(pool, is_v, blk, off, x):
    """Quantise rows x [Hkv, D] into row `off` of block `blk` of a CPU pool."""
    D = x.shape[-1]
    p = places(D)
    nib, sc = (p[1], p[3]) if is_v else (p[0], p[2])
    codes, s = quantise(x)
    page = pool[blk]
    for d in range(D):
        at, shift = int(nib[off, d]) // 2, 4 * (int(nib[off, d]) % 2)
        page[:, at] = (page[:, at] & (0xF0 if shift == 0 else 0x0F)) | (codes[:, d] << shift).to(torch.uint8)
    sb = s.contiguous().view(torch.uint8).reshape(x.shape[0], -1, 2)
    for c in range(D // 32):
        at = 8 * D + 2 * int(sc[off, 32 * c])
        page[:, at:at + 2] = sb[:, c]


def page_values(pool, D, is_v):
    """uint8 [..., 9 D] -> fp64 [..., 16, D]."""
    p = places(D)
    nib, sc = ((p[1], p[3]) if is_v else (p[0], p[2]))
    nib, sc = nib.to(pool.device), sc.to(pool.device)
    n = (pool[..., :8 * D][..., nib // 2].to(torch.int64) >> (4 * (nib % 2))) & 15
    s = pool[..., 8 * D:].contiguous().view(torch.bfloat16)[..., sc]
    return (n - 8).double() * s.double()


def pack_pages(x, is_v):
    """Rows x [nb, Hkv, 16, D] as pages, uint8 [nb, Hkv, 9 D] (vectorised, on
    x's device); write_rows says the same row by row."""
    nb, H, _, D = x.shape
    p = places(D)
    nib, sc = ((p[1], p[3]) if is_v else (p[0], p[2]))
    codes, s = quantise(x)
    nibbles = torch.zeros(nb, H, 16 * D, dtype=torch.int64, device=x.device)
    nibbles[..., nib.flatten().to(x.device)] = codes.flatten(-2)
    out = torch.empty(nb, H, 9 * D, dtype=torch.uint8, device=x.device)
    out[..., :8 * D] = (nibbles[..., 0::2] | nibbles[..., 1::2] << 4).to(torch.uint8)
    scales = torch.zeros(nb, H, 16 * D // 32, dtype=torch.bfloat16, device=x.device)
    scales[..., sc[:, ::32].flatten().to(x.device)] = s.flatten(-2)
    out[..., 8 * D:] = scales.view(torch.uint8)
    return out


# ---------------------------------------------------------------- attention

def attend(q, k_of, v_of, lens, scale, sinks=None, window=0):
    """(out [B, Hq, D] fp64, bound on a kernel's error).  k_of(b), v_of(b):
    [n, Hkv, D] values of sequence b's n tokens.

    The bound: each weight is rounded to bf16, and once more with a scale
    (2^-8 each); a logit is an fp32 sum of exact products s (128 + n) q and
    -136 s q, 34 additions to a group of 32, each off by at most 2^-22 of the
    magnitudes that meet in it (matrix instructions may cut where fp32 would
    round), which changes a weight by that amount; the exponential and the
    product with the scale add 2^-21 of the logit's size; the output is
    rounded once (2^-8)."""
    B, Hq, D = q.shape
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        k, v = k_of(b).transpose(0, 1), v_of(b).transpose(0, 1)      # [Hkv, n, D]
        a = max(0, n - window) if window else 0
        k, v = k[:, a:], v[:, a:]
        Hkv = k.shape[0]
        qd = q[b].double().view(Hkv, Hq // Hkv, D)
        x = qd @ k.transpose(1, 2) * scale
        m = x.amax(-1, keepdim=True)
        z = None
        if sinks is not None:
            z = sinks.double().view(Hkv, Hq // Hkv, 1)
            m = torch.maximum(m, z)
        p = torch.exp(x - m)
        total = p.sum(-1, keepdim=True) + (torch.exp(z - m) if z is not None else 0)
        w = p / total
        out[b] = (w @ v).view(Hq, D)
        # |s| of a group is at least an eighth of its largest value; with it,
        # (128 + 15 + 136) |s| bounds what meets in the sums.
        s = k.abs().reshape(*k.shape[:-1], -1, 32).amax(-1) / 7
        sq = qd.abs().reshape(Hkv, Hq // Hkv, -1, 32).sum(-1)
        size = abs(scale) * 279 * (sq @ s.transpose(1, 2))
        off = 34 * 2.0 ** -22 * size + 2.0 ** -21 * (x - m).abs()
        off = off + (w * off).sum(-1, keepdim=True)
        mag = w @ v.abs()
        bound[b] = ((w * off) @ v.abs() + (2.0 ** -7 + 2.0 ** -15) * mag).view(Hq, D) \
            + 2.0 ** -8 * out[b].abs() + 2.0 ** -24 * mag.view(Hq, D) + 1e-37
    return out, bound


def check(got, ref, bound, what=""):
    d = (got.double() - ref).abs()
    bad = ~(d <= bound)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst {float((d - bound).max()):.3e} over "
        f"its bound, first at {bad.nonzero()[0].tolist()}: {got[tuple(bad.nonzero()[0])]} for "
        f"{ref[tuple(bad.nonzero()[0])]}")


# ---------------------------------------------------------------- pages

class Pool:
    """The page pool as a reader of the definitions would keep it, on lists."""

    def __init__(self, tables, lens, stack, top, extra, bs=BS):
        self.tables = [list(r) for r in tables]
        self.lens, self.extra = list(lens), list(extra)
        self.stack, self.top, self.bs = list(stack), top, bs
        self.flags = 0

    def pages(self, n):
        return -(-n // self.bs) if n > 0 else 0

    def fork(self, parents, children):
        copies, before = [], list(self.lens)
        taken = set()
        for p, c in zip(parents, children):
            pair = (-1, -1)
            B, width = len(self.lens), len(self.tables[0])
            if not (0 <= p < B and 0 <= c < B) or before[p] < 0 or before[c] >= 0 or c in taken:
                self.flags |= 4
            else:
                taken.add(c)
                n = before[p]
                need = n % self.bs != 0
                if self.pages(n) > width:
                    self.flags |= 2
                elif need and self.top == 0:
                    self.flags |= 32
                    self.lens[c] = -1
                else:
                    full = n // self.bs
                    row = [-1] * width
                    for i in range(full):
                        row[i] = self.tables[p][i]
                        self.extra[row[i]] += 1
                    if need:
                        self.top -= 1
                        row[full] = self.stack[self.top]
                        pair = (self.tables[p][full], row[full])
                    self.tables[c], self.lens[c] = row, n
            copies.append(pair)
        return copies

    def release(self, ids, capacity):
        freed = []
        for b in ids:
            if not 0 <= b < len(self.lens):
                self.flags |= 4
                continue
            for i in range(min(self.pages(self.lens[b]), len(self.tables[b]))):
                blk = self.tables[b][i]
                if self.extra[blk] > 0:
                    self.extra[blk] -= 1
                else:
                    freed.append(blk)
            if self.lens[b] >= 0:
                self.tables[b] = [-1] * len(self.tables[b])
                self.lens[b] = -1
        for blk in sorted(freed, reverse=True):
            if self.top == capacity:
                self.flags |= 32
                break
            self.stack[self.top] = blk
            self.top += 1

    def compact(self):
        nb = len(self.extra)
        live = sorted({r[i] for r, n in zip(self.tables, self.lens) for i in range(self.pages(n))})
        L = len(live)
        holes = [b for b in range(L) if b not in set(live)]
        moves = list(zip([b for b in live if b >= L], holes))
        remap = [-1] * nb
        for b in live:
            remap[b] = b
        for s, d in moves:
            remap[s] = d
        extra = [0] * nb
        for b in live:
            extra[remap[b]] = self.extra[b]
        self.extra = extra
        for r, n in zip(self.tables, self.lens):
            for i in range(self.pages(n)):
                r[i] = remap[r[i]]
        for i in range(nb - L):
            self.stack[i] = nb - 1 - i
        self.top = nb - L
        return remap, moves


def uniform_scale(D):
    return 1.0 / math.sqrt(D)
