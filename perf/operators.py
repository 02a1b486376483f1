"""Cases and plain forms of the cache-side operators around the paged decode step.

Five operators, each as a user of the package calls it:

* ``rope``     per-head RMSNorm of q and k, the rotary position rotation and the
               append of the new K/V rows into their pages, in one pass;
* ``store``    a prompt chunk stored in a 4-bit cache, and the sequence's pages
               read back as bf16 pages (what the chunk's attention reads);
* ``attn``     one decode token per sequence attending over a 4-bit cache, and
  ``step``     the whole step: norm, rotation, 4-bit append, attention;
* ``fork``     sequences forked from shared prefixes (tail pages copied), later
               released;
* ``compact``  the live pages of a fragmented pool moved to its front.

The plain forms are elementary torch operations in 32 bits, rounded once.  The
framework's calls are made where ``own`` is true.

The 4-bit page.  A page (block, KV head) holds 16 rows of D values in 9 D bytes.
A row is cut into NG = D / 32 groups of 32 dims.  With e the group's element of
largest magnitude (the positive one of a tie), the group's scale is
s = bf16(-e / 8), a value x is stored as the code n = clamp(rne(x / s), -8, 7) + 8
(8 where s is 0), and stands for s (n - 8).  The first 8 D bytes are the codes,
the last D the scales:

* K page: row o has its D / 8 32-bit words at 4-byte steps; word t NG + c
  (t < 4, c < NG) holds dims 32 c + 8 t + i in bits 4 i .. 4 i + 3.  Scales: [o][c].
* V page: rows 2 i and 2 i + 1 share their words; word g NG + c of pair i
  (g < 8) holds dims 32 c + 4 g + j of row 2 i in bits 4 j .. and of row 2 i + 1
  in bits 16 + 4 j ...  Scales: [i][c][row parity].
"""
import math

import numpy as np
import torch

own = False

BS = 16          # tokens of a page
EPS = 1e-6
THETA = 1e6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # A GPT-2 shaped decode batch in fp32: one new token for each of 61 sequences (one slot empty),
        # half of each head rotated, neighbouring dims paired.  Latency.
        dict(name="rope_decode_f32", kind="rope", form="decode", T=61, Hq=12, Hkv=12, D=64, dtype="f32",
             rot=32, interleaved=True, ctx=1024, empty=1, norm=True),
        # The continuous-batching mix's decode batch: 64 sequences, 32q/8kv x 128.  Latency.
        dict(name="rope_decode_64", kind="rope", form="decode", T=64, Hq=32, Hkv=8, D=128, dtype="bf16",
             rot=128, interleaved=False, ctx=8192, empty=0, norm=True),
        # An 8K-token prompt, one layer: bandwidth.
        dict(name="rope_prefill_8k", kind="rope", form="prefill", T=8192, Hq=32, Hkv=8, D=128, dtype="bf16",
             rot=128, interleaved=False, ctx=8192, empty=0, norm=True),
        # A short odd chunk behind a short prefix, GPT-2 heads, kept in 4 bits.
        dict(name="store_odd_77", kind="store", T=77, start=423, Hkv=12, D=64),
        # The last 4K chunk of a 32K-token prompt: stored, and the 32K tokens read back for its attention.
        dict(name="store_4k_of_32k", kind="store", T=4096, start=28672, Hkv=8, D=128),
        # One stream at 4K tokens of history: latency of the split and its merge.
        dict(name="attn_single_4k", kind="attn", B=1, Hq=32, Hkv=8, D=128, lo=4097, hi=4097, window=0, sinks=False, empty=0),
        # 64q/8kv x 64 with sinks and a sliding window, ragged, two empty slots.
        dict(name="attn_sinks_window", kind="attn", B=23, Hq=64, Hkv=8, D=64, lo=1, hi=8192, window=4096, sinks=True, empty=2),
        # Long contexts in a batch: bandwidth.
        dict(name="attn_long_32", kind="attn", B=32, Hq=32, Hkv=8, D=128, lo=4097, hi=32769, window=0, sinks=False, empty=0),
        # The whole decode step on a 4-bit cache for the continuous-batching mix.
        dict(name="step_mix_64", kind="step", B=64, Hq=32, Hkv=8, D=128, lo=17, hi=8193, window=0, sinks=False, empty=0,
             rot=128, interleaved=False),
        # Eight prompts sampled eight ways each: forked, tails copied in all 36 layers, released.
        dict(name="fork_8x8", kind="fork", parents=8, children=8, lo=512, hi=1024, layers=36, Hkv=8, D=128),
        # Two prompts forked twice in a GPT-2 sized cache: latency.
        dict(name="fork_2x2", kind="fork", parents=2, children=2, lo=33, hi=500, layers=12, Hkv=12, D=64),
        # A pool of 8K pages, 60 % live and scattered, closed up.
        dict(name="compact_8k", kind="compact", B=64, blocks=8192, live=0.6, layers=4, Hkv=8, D=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "rope", "store", "attn", "attn", "step", "fork", "compact"])
    Hkv = rng.choice([1, 2, 4, 8, 8, 12])
    G = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128])
    if kind == "rope":
        form = rng.choice(["decode", "prefill"])
        T = _log(rng, 1, 300) if form == "decode" else _log(rng, 1, 6000)
        ctx = _log(rng, 16, 8192) if form == "decode" else T + _log(rng, 1, 20000)
        rot = rng.choice([D, D, D // 2, 16, 48])
        return dict(kind=kind, form=form, T=T, Hq=min(32, Hkv * G) // Hkv * Hkv, Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    rot=rot, interleaved=rng.random() < 0.3, ctx=ctx, empty=rng.choice([0, 0, 1]) if form == "decode" and T > 1 else 0,
                    norm=rng.random() < 0.8)
    if kind == "store":
        T = _log(rng, 1, 4096)
        return dict(kind=kind, T=T, start=_log(rng, 1, 28000) - 1, Hkv=min(Hkv, 8), D=D)
    if kind in ("attn", "step"):
        B = _log(rng, 1, 48)
        hi = _log(rng, 2, max(64, min(32769, 500000 // B)))
        c = dict(kind=kind, B=B, Hq=min(8, Hkv) * G, Hkv=min(8, Hkv), D=D, lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi,
                 window=rng.choice([0, 0, 0, _log(rng, 1, 5000)]), sinks=rng.random() < 0.3, empty=rng.choice([0, 0, 1]) if B > 1 else 0)
        if kind == "step":
            c.update(rot=rng.choice([D, D, D // 2]), interleaved=rng.random() < 0.3)
        return c
    if kind == "fork":
        hi = _log(rng, 8, 1024)
        return dict(kind=kind, parents=_log(rng, 1, 8), children=_log(rng, 1, 8), lo=max(1, hi // 2), hi=hi,
                    layers=_log(rng, 1, 24), Hkv=min(8, Hkv), D=D)
    blocks = _log(rng, 40, 6000)
    return dict(kind=kind, B=_log(rng, 1, 64), blocks=blocks, live=rng.choice([0.1, 0.3, 0.5, 0.7, 0.9]),
                layers=_log(rng, 1, 4), Hkv=min(8, Hkv), D=D)


# ---------------------------------------------------------------- inputs

def _dev():
    return torch.device("cuda")


def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32).to(dtype)


def _rope_table(rows, rot):
    """[rows, rot] fp32: cos then sin of position * THETA^(-2 i / rot); the angles in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=_dev())
    a = torch.arange(rows, dtype=torch.float64, device=_dev())[:, None] * THETA ** (-2.0 * i / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


def _tables(lens, cpu, width=None, spare=1):
    """Block tables for `lens` out of a shuffled pool with `spare` unused blocks at its end."""
    pages = [(n + BS - 1) // BS for n in lens]
    nb = sum(pages) + spare
    perm = torch.randperm(nb - spare, generator=cpu).to(torch.int32)
    bt = torch.full((len(lens), width or max(pages + [1])), -1, dtype=torch.int32)
    at = 0
    for b, p in enumerate(pages):
        bt[b, :p] = perm[at:at + p]
        at += p
    return bt.to(_dev()), nb


def _spread(n, lo, hi, empty=0):
    """The lengths of a case with `n` slots: spread over [lo, hi], evenly in their logarithm where that range is wide; the
    last `empty` slots hold no sequence.  The seed decides which sequence has which (_shuffled)."""
    m = n - empty
    at = [i / (m - 1) if m > 1 else 1.0 for i in range(m)]
    if lo * 9 > hi:
        v = [round(lo + (hi - lo) * a) for a in at]
    else:
        v = [round(lo * (hi / lo) ** a) for a in at]
    return v + [0] * empty


def _shuffled(v, cpu):
    m = sum(x > 0 for x in v)
    return [v[i] for i in torch.randperm(m, generator=cpu).tolist()] + v[m:]


def _kv4_pools(gen, nb, Hkv, D, k_std=1.0, v_std=1.0):
    """Packed pools [nb, Hkv, 9 D] of normal rows, quantised in pieces."""
    k = torch.empty(nb, Hkv, 9 * D, dtype=torch.uint8, device=_dev())
    v = torch.empty_like(k)
    step = max(1, (1 << 26) // (Hkv * BS * D))
    for a in range(0, nb, step):
        m = min(step, nb - a)
        for pool, pack, std in ((k, _pack_k, k_std), (v, _pack_v, v_std)):
            codes, s = _quantise(_normal(gen, m, Hkv, BS, D) * std)
            pool[a:a + m] = pack(codes, s)
    return k, v


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=_dev()).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    kind = c["kind"]
    s = {"case": c}
    if kind in ("rope", "step"):
        D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
        T = c["B"] if kind == "step" else c["T"]
        dt = torch.float32 if c.get("dtype") == "f32" else torch.bfloat16
        qkv = _normal(gen, T, (Hq + 2 * Hkv) * D, dtype=dt)       # one projection's output
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        s["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        s["qw"] = (1 + 0.1 * _normal(gen, D, dtype=torch.float32)).to(dt) if c.get("norm", True) else None
        s["kw"] = (1 + 0.1 * _normal(gen, D, dtype=torch.float32)).to(dt) if c.get("norm", True) else None
        s["table"] = _rope_table(c["hi"] if kind == "step" else c["ctx"], c["rot"])
        s["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device=_dev())
    if kind == "rope":
        if c["form"] == "decode":
            lens = _shuffled(_spread(T, 1, c["ctx"], c["empty"]), cpu)
            s["tables"], nb = _tables(lens, cpu)
            s["lens"] = torch.tensor(lens, dtype=torch.int32, device=_dev())
        else:
            first = c["ctx"] - T
            ids, nb = _tables([T + first % BS], cpu)
            pos = torch.arange(first, first + T, device=_dev())
            s["positions"] = pos.to(torch.int32)
            at = pos - first // BS * BS
            s["slots"] = ids[0].long()[at // BS] * BS + at % BS
        s["k_cache"] = torch.zeros(nb, Hkv, BS, D, dtype=dt, device=_dev())
        s["v_cache"] = torch.zeros(nb, Hkv, BS, D, dtype=dt, device=_dev())
    elif kind == "store":
        T, first, Hkv, D = c["T"], c["start"], c["Hkv"], c["D"]
        kv = _normal(gen, T, 2 * Hkv * D)
        s["k"], s["v"] = kv[:, :Hkv * D].view(T, Hkv, D), kv[:, Hkv * D:].view(T, Hkv, D)
        ids, nb = _tables([first + T], cpu)
        s["ids"] = ids[0].contiguous()
        pos = torch.arange(first, first + T, device=_dev())
        s["slots"] = s["ids"].long()[pos // BS] * BS + pos % BS
        s["k_cache"], s["v_cache"] = _kv4_pools(gen, nb, Hkv, D)
        n = s["ids"].numel()
        s["k_pages"] = torch.empty(n, Hkv, BS, D, dtype=torch.bfloat16, device=_dev())
        s["v_pages"] = torch.empty_like(s["k_pages"])
    elif kind in ("attn", "step"):
        B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
        lens = _shuffled(_spread(B, c["lo"], c["hi"], c["empty"]), cpu)
        s["tables"], nb = _tables(lens, cpu)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=_dev())
        s["k_cache"], s["v_cache"] = _kv4_pools(gen, nb, Hkv, D)
        if kind == "attn":
            s["q"] = _normal(gen, B, Hq, D)
        s["sinks"] = _normal(gen, Hq) if c["sinks"] else None
        s["out"] = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=_dev())
        if own:
            from paged_kv_cache_xs_gb300 import ops
            s["ws"] = ops.Kv4Workspace(B, Hq, Hkv, D, _dev())
    elif kind == "fork":
        P, C, Hkv, D, L = c["parents"], c["children"], c["Hkv"], c["D"], c["layers"]
        plens = _shuffled(_spread(P, c["lo"], c["hi"]), cpu)
        bt, nb = _tables(plens, cpu, width=(c["hi"] + BS - 1) // BS + 1, spare=0)
        free = P * C + 5
        nb += free                                                  # the free blocks: a shuffled share of the pool
        perm = torch.randperm(nb, generator=cpu).to(torch.int32).to(_dev())
        bt = torch.where(bt >= 0, perm[bt.clamp(min=0).long()], bt)
        freed = perm[nb - free:].sort(descending=True).values       # lowest id on top
        s["tables"] = torch.cat([bt, torch.full((P * C, bt.shape[1]), -1, dtype=torch.int32, device=_dev())])
        s["lens"] = torch.tensor(plens + [-1] * (P * C), dtype=torch.int32, device=_dev())
        s["from"] = torch.arange(P, dtype=torch.int32, device=_dev()).repeat_interleave(C)
        s["to"] = torch.arange(P, P + P * C, dtype=torch.int32, device=_dev())
        s["stack"] = torch.full((nb,), -1, dtype=torch.int32, device=_dev())
        s["stack"][:free] = freed
        s["top"] = torch.tensor([free], dtype=torch.int32, device=_dev())
        s["extra"] = torch.zeros(nb, dtype=torch.int32, device=_dev())
        s["copies"] = torch.empty(P * C, 2, dtype=torch.int64, device=_dev())
        s["k_pools"] = _normal(gen, L, nb, Hkv, BS, D)
        s["v_pools"] = _normal(gen, L, nb, Hkv, BS, D)
    else:
        B, nb, Hkv, D, L = c["B"], c["blocks"], c["Hkv"], c["D"], c["layers"]
        B = min(B, int(nb * c["live"]))
        live = max(B, int(nb * c["live"]))
        cuts = [live * i * (i + 1) // (B * (B + 1)) for i in range(1, B)]
        share = _shuffled([b - a for a, b in zip([0] + cuts, cuts + [live])], cpu)  # own pages of each sequence, short and long
        perm = torch.randperm(nb, generator=cpu).to(torch.int32)
        rows, at = [], 0
        for i, p in enumerate(share):
            prefix = rows[i - 1][:len(rows[i - 1]) // 2] if i % 3 == 2 else []  # each third shares half a neighbour's pages
            rows.append(prefix + perm[at:at + p].tolist())
            at += p
        bt = torch.full((B + 1, 2 * max(share) + 1), -1, dtype=torch.int32)
        for i, r in enumerate(rows):
            bt[i, :len(r)] = torch.tensor(r, dtype=torch.int32)
        lens = [max(0, len(r) * BS - int(torch.randint(0, BS, (1,), generator=cpu))) for r in rows] + [-1]
        s["tables"] = bt.to(_dev())
        s["tables_out"] = torch.full_like(s["tables"], -1)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=_dev())
        used = torch.cat([torch.tensor(r) for r in rows])
        s["extra"] = (torch.bincount(used, minlength=nb) - 1).clamp(min=0).to(torch.int32).to(_dev())
        s["extra_out"] = torch.zeros_like(s["extra"])
        s["stack_out"] = torch.full((nb,), -1, dtype=torch.int32, device=_dev())
        s["top_out"] = torch.zeros(1, dtype=torch.int32, device=_dev())
        s["remap"] = torch.empty(nb, dtype=torch.int32, device=_dev())
        s["moves"] = torch.empty(nb // 2, 2, dtype=torch.int64, device=_dev())
        s["n_moves"] = torch.zeros(1, dtype=torch.int32, device=_dev())
        s["k_pools"] = _normal(gen, L, nb, Hkv, BS, D)
        s["v_pools"] = _normal(gen, L, nb, Hkv, BS, D)
    return s


# ---------------------------------------------------------------- plain forms: norm and rotation

def _norm_rotate(x, w, table, positions, rot, interleaved):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    cs = table[positions.long()][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _decode_slots(tables, lens):
    """Position, block and offset of each slot's new token; which slots hold a sequence."""
    live = lens > 0
    pos = (lens - 1).clamp(min=0)
    blk = tables.gather(1, (pos // BS).long()[:, None])[:, 0].long()
    return live, pos, blk, (pos % BS).long()


# ---------------------------------------------------------------- plain forms: the 4-bit page

def _quantise(x):
    """Codes (uint8, 0..15) and scales (bf16) of rows x [..., D]."""
    g = x.float().unflatten(-1, (-1, 32))
    hi, lo = g.amax(-1), g.amin(-1)
    s = (torch.where(hi >= -lo, hi, lo) * -0.125).bfloat16()
    f = s.float()[..., None]
    n = torch.where(f == 0, torch.zeros_like(g), torch.round(g / f)).clamp(-8, 7) + 8
    return n.to(torch.uint8).flatten(-2), s


def _k_words(codes):
    """[..., D] codes -> [..., D / 2] bytes of a K row."""
    w = codes.unflatten(-1, (-1, 4, 8)).transpose(-3, -2)          # [.., t, c, i]
    return (w[..., 0::2] | w[..., 1::2] << 4).flatten(-3)


def _v_words(codes):
    """[..., D] codes -> [..., 8, NG, 2] bytes of one row's half words."""
    w = codes.unflatten(-1, (-1, 8, 4)).transpose(-3, -2)          # [.., g, c, j]
    return w[..., 0::2] | w[..., 1::2] << 4


def _bytes(s):
    return s.contiguous().view(torch.uint8)


def _pack_k(codes, s):
    return torch.cat([_k_words(codes).flatten(-2), _bytes(s).flatten(-2)], -1)


def _pack_v(codes, s):
    n = codes.shape[:-2]
    w = _v_words(codes).unflatten(-4, (8, 2)).movedim(-4, -2)      # [.., pair, g, c, parity, 2]
    z = s.unflatten(-2, (8, 2)).transpose(-1, -2)                  # [.., pair, c, parity]
    return torch.cat([w.reshape(*n, -1), _bytes(z).reshape(*n, -1)], -1)


def _nibbles(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _unpack_k(p, D):
    """[..., 9 D] page bytes -> values [..., 16, D] fp32."""
    n = _nibbles(p[..., :8 * D].unflatten(-1, (BS, 4, D // 32, 4))).transpose(-3, -2)   # [.., o, c, t, i]
    s = p[..., 8 * D:].contiguous().view(torch.bfloat16).unflatten(-1, (BS, D // 32))
    return ((n.flatten(-2).float() - 8) * s.float()[..., None]).flatten(-2)


def _unpack_v(p, D):
    n = _nibbles(p[..., :8 * D].unflatten(-1, (8, 8, D // 32, 2, 2)))                   # [.., pair, g, c, parity, j]
    n = n.movedim(-2, -4).transpose(-3, -2)                                             # [.., pair, parity, c, g, j]
    s = p[..., 8 * D:].contiguous().view(torch.bfloat16).unflatten(-1, (8, D // 32, 2)).transpose(-1, -2)
    return ((n.flatten(-2).float() - 8) * s.float()[..., None]).flatten(-2).flatten(-3, -2)


def _store(k, v, k_cache, v_cache, blk, off, keep=None):
    """Rows k, v [T, Hkv, D] into row `off` of block `blk`; rows outside `keep` are left as they were."""
    D = k.shape[-1]
    NG = D // 32
    kc, ks = _quantise(k)
    vc, vs = _quantise(v)
    kw = k_cache[..., :8 * D].unflatten(-1, (BS, D // 2))
    kz = k_cache[..., 8 * D:].unflatten(-1, (BS, 2 * NG))
    vw = v_cache[..., :8 * D].unflatten(-1, (8, 8, NG, 2, 2))
    vz = v_cache[..., 8 * D:].unflatten(-1, (8, NG, 2, 2))
    for dst, src, ix in ((kw, _k_words(kc), (blk, slice(None), off)), (kz, _bytes(ks), (blk, slice(None), off)),
                         (vw, _v_words(vc), (blk, slice(None), off // 2, slice(None), slice(None), off % 2)),
                         (vz, _bytes(vs[..., None]), (blk, slice(None), off // 2, slice(None), off % 2))):
        if keep is not None:
            src = torch.where(keep.view(-1, *[1] * (src.dim() - 1)), src, dst[ix])
        dst[ix] = src


def _attend(q, k_cache, v_cache, tables, lens, sinks, window, scale):
    B, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    ids = tables.clamp(min=0).long()
    n = ids.shape[1] * BS
    k = _unpack_k(k_cache[ids], D).transpose(1, 2).reshape(B, Hkv, n, D)
    x = (q.float().view(B, Hkv, Hq // Hkv, D) @ k.transpose(-1, -2)) * scale
    del k
    t = torch.arange(n, device=q.device)
    seen = t < lens[:, None]
    if window:
        seen &= t >= lens[:, None] - window
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    z = sinks.float().view(1, Hkv, Hq // Hkv, 1) if sinks is not None else None
    if z is not None:
        m = torch.maximum(m, z)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    if z is not None:
        total = total + torch.exp(z - m)
    v = _unpack_v(v_cache[ids], D).transpose(1, 2).reshape(B, Hkv, n, D)
    o = (p @ v) / total.clamp(min=1e-38)
    return torch.where(lens[:, None, None] > 0, o.reshape(B, Hq, D), torch.zeros_like(o).reshape(B, Hq, D)).to(q.dtype)


# ---------------------------------------------------------------- plain forms: pages

def _fork(s):
    par, to, tables, lens = s["from"].long(), s["to"].long(), s["tables"], s["lens"]
    n = lens[par]
    full = (n // BS)[:, None]
    tail = n % BS != 0
    rows = tables[par]
    col = torch.arange(rows.shape[1], device=rows.device)
    shared = col < full
    blk = s["stack"][(s["top"] - torch.cumsum(tail, 0)).clamp(min=0)]
    src = rows.gather(1, full.long())[:, 0]
    minus = torch.full_like(rows, -1)
    tables[to] = torch.where(shared, rows, torch.where((col == full) & tail[:, None], blk[:, None], minus))
    lens[to] = n
    s["extra"].index_add_(0, rows.clamp(min=0).flatten().long(), shared.flatten().to(torch.int32))
    s["top"] -= tail.sum().to(torch.int32)
    none = torch.full_like(src, -1)
    s["copies"].copy_(torch.stack([torch.where(tail, src, none), torch.where(tail, blk, none)], -1))


def _copy(pairs, pools, idle):
    """Pairs (src, dst) of blocks in every layer; a pair of -1 copies block `idle`, which nothing else writes, onto itself."""
    src = torch.where(pairs[:, 0] < 0, idle, pairs[:, 0])
    dst = torch.where(pairs[:, 0] < 0, idle, pairs[:, 1])
    for p in pools:
        p[:, dst] = p[:, src]


def _release(s):
    ids, tables, lens, extra = s["to"].long(), s["tables"], s["lens"], s["extra"]
    n = lens[ids]
    rows = tables[ids]
    col = torch.arange(rows.shape[1], device=rows.device)
    used = col < (n[:, None] + BS - 1) // BS
    drop = torch.zeros_like(extra).index_add_(0, rows.clamp(min=0).flatten().long(), used.flatten().to(torch.int32))
    gone = drop > extra
    back = gone.nonzero()[:, 0].flip(0)
    s["stack"][s["top"] + torch.arange(back.numel(), device=back.device)] = back.to(torch.int32)
    s["top"] += back.numel()
    extra.copy_((extra - drop).clamp(min=0))
    tables[ids] = -1
    lens[ids] = -1


def _compact(s):
    tables, lens, nb = s["tables"], s["lens"], s["extra"].numel()
    col = torch.arange(tables.shape[1], device=tables.device)
    used = col < (lens[:, None] + BS - 1) // BS
    hits = torch.zeros(nb, dtype=torch.int32, device=tables.device)
    hits.index_add_(0, tables.clamp(min=0).flatten().long(), used.flatten().to(torch.int32))
    live = hits > 0
    ids = torch.arange(nb, device=tables.device)
    count = live.sum()
    front = ids < count
    src, dst = (live & ~front).nonzero()[:, 0], (~live & front).nonzero()[:, 0]
    s["remap"].copy_(torch.where(live, ids, -torch.ones_like(ids)))
    s["remap"][src] = dst.to(torch.int32)
    s["tables_out"].copy_(torch.where(used, s["remap"][tables.clamp(min=0).long()], tables))
    s["extra_out"].copy_(torch.where(front & live, s["extra"], torch.zeros_like(s["extra"])))
    s["extra_out"][dst] = s["extra"][src]
    s["moves"].fill_(-1)
    s["moves"][:src.numel()] = torch.stack([src, dst], -1)
    s["n_moves"].fill_(src.numel())
    s["stack_out"].copy_(torch.where(ids < nb - count, nb - 1 - ids, s["stack_out"].long()))
    s["top_out"].copy_(nb - count)
    for p in (s["k_pools"], s["v_pools"]):
        p[:, dst] = p[:, src]


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    kind = c["kind"]
    if own:
        from paged_kv_cache_xs_gb300 import ops
        if kind == "rope":
            if c["form"] == "decode":
                ops.xs_qk_norm_rope_append_paged(s["q_out"], s["q"], s["k"], s["v"], s["qw"], s["kw"], EPS, s["table"],
                                                 s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                                 interleaved=c["interleaved"])
            else:
                ops.xs_qk_norm_rope_append(s["q_out"], s["q"], s["k"], s["v"], s["qw"], s["kw"], EPS, s["table"],
                                           s["positions"], s["k_cache"], s["v_cache"], s["slots"],
                                           interleaved=c["interleaved"])
            return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if kind == "store":
            ops.xs_kv4_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])
            ops.xs_kv4_unpack(s["k_pages"], s["v_pages"], s["k_cache"], s["v_cache"], s["ids"])
            return {"k": s["k_pages"], "v": s["v_pages"]}
        if kind in ("attn", "step"):
            q = s["q"]
            if kind == "step":
                ops.xs_qk_norm_rope_append_paged(s["q_out"], s["q"], s["k"], s["v"], s["qw"], s["kw"], EPS, s["table"],
                                                 s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                                 interleaved=c["interleaved"])
                q = s["q_out"]
            ops.xs_kv4_decode(s["out"], q, s["k_cache"], s["v_cache"], s["tables"], s["lens"], 1 / math.sqrt(c["D"]),
                              s["ws"], sinks=s["sinks"], window=c["window"])
            return {"out": s["out"], "q": q} if kind == "step" else {"out": s["out"]}
        if kind == "fork":
            ops.xs_block_fork(s["from"], s["to"], s["tables"], s["lens"], s["stack"], s["top"], s["extra"], s["copies"])
            ops.xs_block_copy(s["k_pools"], s["v_pools"], s["copies"])
            ops.xs_block_release(s["to"], s["tables"], s["lens"], s["stack"], s["top"], s["extra"])
        else:
            ops.xs_block_compact(s["tables"], s["tables_out"], s["lens"], s["extra"], s["extra_out"], s["stack_out"],
                                 s["top_out"], s["remap"], s["moves"], s["n_moves"])
            ops.xs_block_copy(s["k_pools"], s["v_pools"], s["moves"], count=s["n_moves"])
    elif kind in ("rope", "step"):
        if kind == "step" or c["form"] == "decode":
            keep, pos, blk, off = _decode_slots(s["tables"], s["lens"])
        else:
            keep, pos, blk, off = None, s["positions"], s["slots"] // BS, s["slots"] % BS
        q = _norm_rotate(s["q"], s["qw"], s["table"], pos, c["rot"], c["interleaved"])
        k, v = _norm_rotate(s["k"], s["kw"], s["table"], pos, c["rot"], c["interleaved"]), s["v"]
        if keep is not None:
            q = torch.where(keep[:, None, None], q, s["q_out"])
            spare = s["k_cache"].shape[0] - 1                       # slots without a sequence write the unused block back
            blk, off = torch.where(keep, blk, spare), torch.where(keep, off, 0)
        s["q_out"].copy_(q)
        if kind == "step":
            _store(k, v, s["k_cache"], s["v_cache"], blk, off, keep)
            s["out"].copy_(_attend(s["q_out"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["sinks"], c["window"],
                                   1 / math.sqrt(c["D"])))
            return {"out": s["out"], "q": s["q_out"]}
        for pool, x in ((s["k_cache"], k), (s["v_cache"], v)):
            if keep is not None:
                x = torch.where(keep[:, None, None], x, pool[blk, :, off])
            pool[blk, :, off] = x
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    elif kind == "store":
        _store(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"] // BS, s["slots"] % BS)
        ids = s["ids"].long()
        s["k_pages"].copy_(_unpack_k(s["k_cache"][ids], c["D"]))
        s["v_pages"].copy_(_unpack_v(s["v_cache"][ids], c["D"]))
        return {"k": s["k_pages"], "v": s["v_pages"]}
    elif kind == "attn":
        s["out"].copy_(_attend(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["sinks"], c["window"],
                               1 / math.sqrt(c["D"])))
        return {"out": s["out"]}
    elif kind == "fork":
        _fork(s)
        _copy(s["copies"], (s["k_pools"], s["v_pools"]), s["tables"][0, 0].long())
        _release(s)
    else:
        _compact(s)
    if kind == "fork":
        return {n: s[n] for n in ("copies", "tables", "lens", "stack", "top", "extra", "k_pools", "v_pools")}
    return {n: s[n] for n in ("tables_out", "extra_out", "stack_out", "top_out", "remap", "moves", "n_moves", "k_pools", "v_pools")}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    kind = c["kind"]
    D = c["D"]
    if kind == "rope":
        e = 4 if c["dtype"] == "f32" else 2
        row = (c["Hq"] + 2 * c["Hkv"]) * D
        T = c["T"] - c["empty"]
        table = 4 * c["rot"] * (T if c["form"] == "decode" else min(T, c["ctx"]))
        return {"bytes": 2 * e * T * row + table + 2 * e * D + 12 * T, "flops": 8.0 * T * row}
    if kind == "store":
        pages = -(-(c["start"] + c["T"]) // BS)
        new = c["T"] * c["Hkv"] * D * 2
        return {"bytes": new * (2 + 0.5625) + 8 * c["T"] + pages * (2 * c["Hkv"] * (9 * D + 2 * BS * D) + 4),
                "flops": 4.0 * new + 2.0 * pages * BS * c["Hkv"] * D}
    if kind in ("attn", "step"):
        n = c["B"] - c["empty"]
        tokens = sum(min(v, c["window"] or v) for v in _spread(c["B"], c["lo"], c["hi"], c["empty"]))
        b = tokens * (c["Hkv"] * 2 * (D / 2 + D / 16) + 4 / BS) + 2 * 2 * n * c["Hq"] * D
        f = 4.0 * tokens * c["Hq"] * D
        if kind == "step":
            b += n * ((c["Hq"] + 2 * c["Hkv"]) * D * 2 + 4 * c["rot"] + c["Hkv"] * 2 * D * 0.5625)
            f += 8.0 * n * (c["Hq"] + 2 * c["Hkv"]) * D
        return {"bytes": b, "flops": f}
    page = c["Hkv"] * BS * D * 2
    if kind == "fork":
        v = _spread(c["parents"], c["lo"], c["hi"])
        tails = c["children"] * sum(x % BS != 0 for x in v)
        entries = c["children"] * sum(-(-x // BS) for x in v)           # read and written, counted up, counted down
        return {"bytes": tails * c["layers"] * 2 * 2 * page + entries * 4 * 4, "flops": 0.0}
    live = c["live"] * c["blocks"]
    moved = live * (1 - live / c["blocks"])
    return {"bytes": moved * c["layers"] * 2 * 2 * page + 4.0 * (5 * c["blocks"] + 2 * 1.2 * live), "flops": 0.0}


# ---------------------------------------------------------------- the operators in 64 bits

def _exact_rope(x, w, pos, rot, interleaved):
    """Rotation as a product with exp(i angle), in complex128."""
    y = x.double()
    if w is not None:
        y = y / (y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + EPS).sqrt() * w.double()
    i = torch.arange(rot // 2, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos.double()[:, None, None] * torch.pow(THETA, -2 * i / rot))
    head = y[..., :rot]
    pairs = head.unflatten(-1, (rot // 2, 2)) if interleaved else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, y[..., rot:]], -1)


def _code_places(D):
    """For every (row, dim): the nibble of a K page and of a V page that holds it."""
    o, d = np.meshgrid(np.arange(BS), np.arange(D), indexing="ij")
    NG, c = D // 32, d // 32
    k = (o * (D // 8) + (d % 32) // 8 * NG + c) * 8 + d % 8
    v = ((o // 2 * 8 + (d % 32) // 4) * NG + c) * 8 + o % 2 * 4 + d % 4
    sk = o * NG + c
    sv = (o // 2 * NG + c) * 2 + o % 2
    return [torch.from_numpy(x).to(_dev()) for x in (k, v, sk, sv)]


def _exact_values(page, place, scale_at, D):
    """Page bytes [.., 9 D] -> [.., 16, D] in 64 bits, nibble by nibble."""
    byte = page[..., :8 * D][..., place // 2].to(torch.int32)
    n = (byte >> (place % 2 * 4)) & 15
    s = page[..., 8 * D:].contiguous().view(torch.bfloat16)[..., scale_at]
    return (n - 8).double() * s.double()


def _exact_quantised(x):
    """What a 4-bit row stands for, in 64 bits."""
    g = x.double().view(*x.shape[:-1], -1, 32)
    big = g.abs().amax(-1, keepdim=True)
    e = torch.where((g == big).any(-1, keepdim=True), big, -big)
    s = (-e / 8).bfloat16().double()
    n = torch.where(s == 0, torch.zeros_like(g), (g / s).round()).clamp(-8, 7)
    return (n * s).view(x.shape)


def _exact_attention(s, c, k_of, v_of, q):
    B, Hq, D = q.shape
    G = Hq // c["Hkv"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=q.device)
    for b, n in enumerate(s["lens"].tolist()):
        if n <= 0:
            continue
        a = max(0, n - c["window"]) if c["window"] else 0
        pages = s["tables"][b, a // BS:(n + BS - 1) // BS].long()
        k, v = (f(b, pages).transpose(0, 1).flatten(1, 2)[:, a % BS:a % BS + n - a] for f in (k_of, v_of))   # [Hkv, n, D]
        x = torch.einsum("hgd,hnd->hgn", q[b].double().view(-1, G, D), k) / math.sqrt(D)
        if s["sinks"] is not None:
            x = torch.cat([x, s["sinks"].double().view(-1, G, 1)], -1)
        p = torch.softmax(x, -1)[..., :n - a]
        out[b] = torch.einsum("hgn,hnd->hgd", p, v).reshape(Hq, D)
    return out


def _forked_tails(s):
    """(from, to) of the blocks a fork copies, sequence by sequence; the whole numbers of a case have no value here."""
    tables, lens, stack = s["tables"].tolist(), s["lens"].tolist(), s["stack"][:int(s["top"])].tolist()
    for p in s["from"].tolist():
        if lens[p] % BS:
            yield tables[p][lens[p] // BS], stack.pop()


def _closed_up(s):
    """(from, to) of the blocks that a compaction moves: the live ones behind the front into its holes, in order."""
    live = {b for row, n in zip(s["tables"].tolist(), s["lens"].tolist()) for b in row[:-(-max(n, 0) // BS)]}
    holes = (b for b in range(len(live)) if b not in live)
    for b in sorted(live):
        if b >= len(live):
            yield b, next(holes)


def _exact_pools(s, pairs):
    pools = {n: s[n].double() for n in ("k_pools", "v_pools")}
    for a, b in pairs(s):
        for p in pools.values():
            p[:, b] = p[:, a]
    return pools


def exact(case, seed):
    c = dict(case)
    if c["kind"] == "fork":
        return _exact_pools(prepare(c, seed), _forked_tails)
    if c["kind"] == "compact":
        return _exact_pools(prepare(c, seed), _closed_up)
    if c["kind"] == "attn" and (c["lo"] + c["hi"]) * c["B"] * c["Hkv"] * c["D"] > 4e9:
        return None
    s = prepare(c, seed)
    D = c["D"]
    if c["kind"] == "rope":
        if c["form"] == "decode":
            live = (s["lens"] > 0).nonzero()[:, 0]
            pos = s["lens"][live].long() - 1
            slot = s["tables"][live, pos // BS].long() * BS + pos % BS
        else:
            live, pos, slot = torch.arange(c["T"], device=_dev()), s["positions"].long(), s["slots"]
        q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=_dev())
        q[live] = _exact_rope(s["q"][live], s["qw"], pos, c["rot"], c["interleaved"])
        pools = []
        for pool, x in ((s["k_cache"], _exact_rope(s["k"][live], s["kw"], pos, c["rot"], c["interleaved"])), (s["v_cache"], s["v"][live].double())):
            rows = torch.zeros(pool.shape, dtype=torch.float64, device=_dev()).transpose(1, 2).flatten(0, 1)
            rows[slot] = x
            pools.append(rows.unflatten(0, (-1, BS)).transpose(1, 2))
        return {"q": q, "k_cache": pools[0], "v_cache": pools[1]}
    pk, pv, sk, sv = _code_places(D)
    if c["kind"] == "store":
        ids = s["ids"].long()
        k, v = (_exact_values(s[n][ids], p, z, D).transpose(1, 2).flatten(0, 1) for n, p, z in (("k_cache", pk, sk), ("v_cache", pv, sv)))
        k[c["start"]:c["start"] + c["T"]] = _exact_quantised(s["k"])
        v[c["start"]:c["start"] + c["T"]] = _exact_quantised(s["v"])
        return {n: x.unflatten(0, (-1, BS)).transpose(1, 2) for n, x in (("k", k), ("v", v))}
    q = s["q"]
    new = None
    if c["kind"] == "step":
        live = (s["lens"] > 0).nonzero()[:, 0]
        pos = s["lens"][live].long() - 1
        q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=_dev())
        q[live] = _exact_rope(s["q"][live], s["qw"], pos, c["rot"], c["interleaved"])
        k = torch.zeros(s["k"].shape, dtype=torch.float64, device=_dev())
        k[live] = _exact_rope(s["k"][live], s["kw"], pos, c["rot"], c["interleaved"])
        # the cache is fed the bf16 row
        new = (_exact_quantised(k.bfloat16()), _exact_quantised(s["v"]))

    def read(pool, place, at, row):
        def f(b, pages):
            x = _exact_values(pool[pages], place, at, D)
            if row is not None:
                x[-1, :, (int(s["lens"][b]) - 1) % BS] = row[b]
            return x
        return f

    out = _exact_attention(s, c, read(s["k_cache"], pk, sk, None if new is None else new[0]),
                           read(s["v_cache"], pv, sv, None if new is None else new[1]), q)
    return {"out": out, "q": q} if c["kind"] == "step" else {"out": out}
