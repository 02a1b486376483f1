"""Cases and plain forms of the operators that bound a paged cache.

Five operators, each as a user of the package calls it:

* ``decode``    one token per sequence attends to the sequence's first tokens and
                to a sliding window of its last ones;
* ``prompt``    the same mask for a chunk of a prompt;
* ``weights``   one token per sequence attends to all of its cache, and the
                attention weight that each cached token got is added to its score;
* ``evict``     sequences beyond a limit are cut to a budget of tokens: the first
                ones, the last ones and those of largest score, moved together in
                the pages of every layer;
* ``truncate``  sequences give back the pages behind a new length.

The plain forms are elementary torch operations in 32 bits, rounded once.  The
framework's calls are made where ``own`` is true.

A score belongs to (sequence, KV head, token): fp32 [B, Hkv, S], or one such array
for each layer.  A KV head's score of a token is the sum of the softmax weights
that its query heads gave it.
"""
import math

import numpy as np
import torch

own = False

BS = 16          # tokens of a page


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One stream far into a long text: 32K tokens behind it, 4 first tokens and a 4K window seen, the pages
        # between given back.  Latency.
        dict(name="decode_single_32k", kind="decode", B=1, Hq=32, Hkv=8, D=128, dtype="bf16", lo=32769, hi=32769, first=4,
             window=4096, sinks=False, empty=0, freed=True),
        # The continuous-batching mix under a 1K window, all pages kept (another layer attends to everything).
        dict(name="decode_mix_64", kind="decode", B=64, Hq=32, Hkv=8, D=128, dtype="bf16", lo=17, hi=8193, first=4, window=1024,
             sinks=False, empty=1, freed=False),
        # A large batch of long sequences: bandwidth.
        dict(name="decode_long_128", kind="decode", B=128, Hq=32, Hkv=8, D=128, dtype="bf16", lo=4097, hi=32769, first=16,
             window=4096, sinks=False, empty=0, freed=True),
        # A short odd chunk behind a prefix, GPT-2 heads, a small window.
        dict(name="prompt_odd_333", kind="prompt", T=333, start=1201, Hq=12, Hkv=12, D=64, first=4, window=255),
        # The last 4K chunk of a 32K-token prompt under a 4K window: arithmetic.
        dict(name="prompt_4k_of_32k", kind="prompt", T=4096, start=28672, Hq=32, Hkv=8, D=128, first=4, window=4096),
        # One stream at 4K tokens: latency of the split, its merge and the scores.
        dict(name="weights_single_4k", kind="weights", B=1, Hq=32, Hkv=8, D=128, dtype="bf16", lo=4097, hi=4097, fresh=0,
             sinks=False, empty=0),
        # A GPT-2 shaped batch in fp32, one slot empty, some sequences scored for the first time.  Latency.
        dict(name="weights_f32_61", kind="weights", B=61, Hq=12, Hkv=12, D=64, dtype="f32", lo=1, hi=1024, fresh=5, sinks=False,
             empty=1),
        # A large batch whose sequences were bounded to between 2K and 4K tokens: bandwidth.
        dict(name="weights_bounded_128", kind="weights", B=128, Hq=32, Hkv=8, D=128, dtype="bf16", lo=2049, hi=4097, fresh=0,
             sinks=False, empty=0),
        # A 32K-token prompt cut to 2K tokens in 4 layers.
        dict(name="evict_single_32k", kind="evict", B=1, Hkv=8, D=128, dtype="bf16", layers=4, lo=32769, hi=32769, first=4,
             recent=512, budget=2048, limit=2304),
        # 64 sequences that grew past 2K tokens, three in four beyond the limit, 4 layers: bandwidth.
        dict(name="evict_64", kind="evict", B=64, Hkv=8, D=128, dtype="bf16", layers=4, lo=2049, hi=2401, first=4, recent=256,
             budget=2048, limit=2137),
        # Three short sequences roll back a few tokens: latency.
        dict(name="truncate_3", kind="truncate", B=3, lo=33, hi=500, cut=40, spare=100),
        # After an eviction: 64 sequences give back up to 4K tokens of pages, some of them shared, in a pool of 40K blocks.
        dict(name="truncate_64", kind="truncate", B=64, lo=2049, hi=16384, cut=4096, spare=2000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "prompt", "weights", "weights", "evict", "truncate"])
    Hkv = rng.choice([1, 2, 4, 8, 8, 12])
    G = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128])
    if kind == "decode":
        B = _log(rng, 1, 120)
        hi = _log(rng, 2, max(64, min(40000, 2000000 // B)))
        Hkv = min(Hkv, 8)
        return dict(kind=kind, B=B, Hq=Hkv * min(G, 4 if B > 64 else 8), Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]) if B < 60 else "bf16",
                    lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi, first=rng.choice([0, 1, 4, _log(rng, 1, 300)]), window=_log(rng, 1, 4096),
                    sinks=rng.random() < 0.25, empty=rng.choice([0, 0, 1]) if B > 1 else 0, freed=rng.random() < 0.5)
    if kind == "prompt":
        T = _log(rng, 1, 3800)
        Hkv = min(Hkv, 8)
        return dict(kind=kind, T=T, start=_log(rng, 1, 28673) - 1, Hq=Hkv * min(G, 4), Hkv=Hkv, D=D, first=rng.choice([0, 1, 4, _log(rng, 1, 300)]),
                    window=_log(rng, 1, 4096))
    if kind == "weights":
        B = _log(rng, 1, 128)
        hi = _log(rng, 2, max(64, min(9000, 500000 // B)))
        Hkv = min(Hkv, 8)
        return dict(kind=kind, B=B, Hq=Hkv * min(G, 4 if B > 64 else 8), Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]) if B < 60 else "bf16",
                    lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi, fresh=rng.choice([0, 0, min(B, 3)]), sinks=rng.random() < 0.25,
                    empty=rng.choice([0, 0, 1]) if B > 1 else 0)
    if kind == "evict":
        B = _log(rng, 1, 64)
        budget = _log(rng, 1, min(4000, 130000 // B))
        limit = budget + _log(rng, 1, budget + 100) - 1
        hi = max(2, limit + _log(rng, 1, min(20000, 140000 // B)) - 1)
        recent = rng.randint(0, budget)
        return dict(kind=kind, B=B, Hkv=min(Hkv, 8), D=D, dtype=rng.choice(["bf16", "bf16", "f32"]), layers=rng.choice([1, 1, 2]),
                    lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi, first=rng.choice([0, min(4, budget - recent), rng.randint(0, budget - recent)]),
                    recent=recent, budget=budget, limit=limit)
    hi = _log(rng, 4, 16384)
    return dict(kind=kind, B=_log(rng, 1, 64), lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi, cut=_log(rng, 1, 4096), spare=_log(rng, 1, 2000))


# ---------------------------------------------------------------- inputs

def _dev():
    return torch.device("cuda")


def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32).to(dtype)


def _pool(gen, *shape, dtype):
    """A pool of normal rows, filled in pieces."""
    p = torch.empty(shape, dtype=dtype, device=_dev())
    flat = p.view(-1)
    step = 1 << 28
    for a in range(0, flat.numel(), step):
        m = min(step, flat.numel() - a)
        flat[a:a + m] = _normal(gen, m, dtype=dtype)
    return p


def _tables(pages, cpu, spare=1):
    """Block tables for sequences of `pages` pages, out of a shuffled pool with `spare` unused blocks at its end.
    Only pages [a, n) and [0, f) of a triple (f, a, n) have a block."""
    width = max([1] + [n for _, _, n in pages])
    owned = [min(f, n) + max(0, n - max(a, f)) for f, a, n in pages]
    nb = sum(owned) + spare
    perm = torch.randperm(nb - spare, generator=cpu).to(torch.int32)
    bt = torch.full((len(pages), width), -1, dtype=torch.int32)
    at = 0
    for b, (f, a, n) in enumerate(pages):
        f = min(f, n)
        bt[b, :f] = perm[at:at + f]
        at += f
        a = max(a, f)
        bt[b, a:n] = perm[at:at + max(0, n - a)]
        at += max(0, n - a)
    return bt.to(_dev()), nb


def _spread(n, lo, hi, empty=0):
    """The lengths of a case with `n` slots: spread over [lo, hi], evenly in their logarithm where that range is wide; the
    last `empty` slots hold no token.  The seed decides which sequence has which (_shuffled)."""
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


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=_dev())


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=_dev()).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    kind = c["kind"]
    s = {"case": c}
    dt = torch.float32 if c.get("dtype") == "f32" else torch.bfloat16
    if kind in ("decode", "weights"):
        B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
        lens = _shuffled(_spread(B, c["lo"], c["hi"], c["empty"]), cpu)
        pages = [(-(-n // BS), 0, -(-n // BS)) for n in lens]
        if c.get("freed"):                       # pages that the mask hides for good went back to the pool
            pages = [(-(-c["first"] // BS), max(0, n - c["window"]) // BS, -(-n // BS)) for n in lens]
        s["tables"], nb = _tables(pages, cpu)
        s["lens"] = _int(lens)
        s["k_cache"], s["v_cache"] = (_pool(gen, nb, Hkv, BS, D, dtype=dt) for _ in range(2))
        qkv = _normal(gen, B, (Hq + 2 * Hkv) * D, dtype=dt)             # one projection's output
        s["q"] = qkv[:, :Hq * D].view(B, Hq, D)
        s["sinks"] = _normal(gen, Hq, dtype=dt) if c["sinks"] else None
        s["out"] = torch.empty(B, Hq, D, dtype=dt, device=_dev())
        if kind == "weights":
            n = s["tables"].shape[1] * BS
            # sums over a few earlier steps: most tokens got little, some much
            s["scores"] = torch.exp(2 * _normal(gen, B, Hkv, n, dtype=torch.float32)) * (Hq / Hkv / n)
            fresh = torch.randperm(B, generator=cpu)[:c["fresh"]].tolist()
            s["scored"] = None
            if c["fresh"]:
                s["scored"] = _int([0 if b in fresh else max(0, x - 1) for b, x in enumerate(lens)])
        if own:
            from paged_kv_cache_xs_gb300 import ops
            s["ws"] = ops.BoundedWorkspace(B, Hq, Hkv, D, _dev(),
                                          max_blocks_per_seq=s["tables"].shape[1] if kind == "weights" else 0)
    elif kind == "prompt":
        T, start, Hq, Hkv, D = c["T"], c["start"], c["Hq"], c["Hkv"], c["D"]
        n = -(-(start + T) // BS)
        ids, nb = _tables([(n, 0, n)], cpu)
        s["ids"] = ids[0].contiguous()
        s["k_cache"], s["v_cache"] = (_pool(gen, nb, Hkv, BS, D, dtype=dt) for _ in range(2))
        s["q"] = _normal(gen, T, Hq, D)
        s["out"] = torch.empty(T, Hq, D, dtype=dt, device=_dev())
    elif kind == "evict":
        B, Hkv, D, L = c["B"], c["Hkv"], c["D"], c["layers"]
        lens = _shuffled(_spread(B, c["lo"], c["hi"]), cpu)
        s["tables"], nb = _tables([(-(-n // BS), 0, -(-n // BS)) for n in lens], cpu)
        s["lens"] = _int(lens)
        s["k_pools"], s["v_pools"] = (_pool(gen, L, nb, Hkv, BS, D, dtype=dt) for _ in range(2))
        s["ids"] = torch.randperm(B, generator=cpu).to(torch.int32).to(_dev())
        s["extra"] = torch.zeros(nb, dtype=torch.int32, device=_dev())
        x = torch.exp(2 * _normal(gen, L, B, Hkv, s["tables"].shape[1] * BS, dtype=torch.float32))
        s["scores"] = torch.where(x < 0.02, torch.zeros_like(x), x)     # weights that were 0 in every step
        s["kept"] = torch.empty(L, B, Hkv, c["budget"], dtype=torch.int32, device=_dev())
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device=_dev())
    else:
        B = c["B"]
        lens = _shuffled(_spread(B, c["lo"], c["hi"]), cpu)
        pages = [-(-n // BS) for n in lens]
        bt, nb = _tables([(p, 0, p) for p in pages], cpu, spare=c["spare"])
        bt = bt.cpu()
        for b in range(2, B, 3):                 # each third sequence was forked from its neighbour's full pages
            m = min(lens[b], lens[b - 1]) // BS // 2
            bt[b, :m] = bt[b - 1, :m]
        used = torch.cat([bt[b, :p] for b, p in enumerate(pages)]).long()
        count = torch.bincount(used, minlength=nb)
        free = (count == 0).nonzero()[:, 0]
        free = free[torch.randperm(free.numel(), generator=cpu)].to(torch.int32)
        stack = torch.full((nb,), -1, dtype=torch.int32)
        stack[:free.numel()] = free
        cut = [int(x) for x in (torch.rand(B, generator=cpu) * c["cut"]).round()]
        s["ids"] = torch.randperm(B, generator=cpu).to(torch.int32)
        s["new_lens"] = _int([max(0, lens[b] - cut[b]) if cut[b] else -1 for b in s["ids"].tolist()])
        s["ids"] = s["ids"].to(_dev())
        # What the calls change; run() starts from these again.
        s["start"] = [bt.to(_dev()), _int(lens), stack.to(_dev()), _int([free.numel()]), (count - 1).clamp(min=0).to(torch.int32).to(_dev())]
        s["state"] = [x.clone() for x in s["start"]]
    return s


# ---------------------------------------------------------------- plain forms

def _softmax(x, sinks):
    """Weights of logits x [B, Hkv, G, n] (masked ones -infinity), a sink one more logit without a value."""
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    if sinks is None:
        p = torch.exp(x - m)
        return p / p.sum(-1, keepdim=True).clamp(min=1e-38)
    z = sinks.float().view(1, x.shape[1], x.shape[2], 1)
    m = torch.maximum(m, z)
    p = torch.exp(x - m)
    return p / (p.sum(-1, keepdim=True) + torch.exp(z - m))


def _rows(cache, tables, at):
    """Rows [B, Hkv, n, D] of tokens at [B, n] (those without a page: of block 0)."""
    blk = tables.gather(1, (at // BS).clamp(max=tables.shape[1] - 1)).clamp(min=0).long()
    return cache[blk, :, at % BS].transpose(1, 2).float()


def _attend(q, k, v, seen, sinks, scale):
    """Outputs [B, Hq, D] and weights [B, Hkv, G, n] of q [B, Hq, D] on rows [B, Hkv, n, D] of which `seen` [B, n] count."""
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    x = (q.float().view(B, Hkv, Hq // Hkv, D) @ k.transpose(-1, -2)) * scale
    p = _softmax(x.masked_fill(~seen[:, None, None], -math.inf), sinks)
    return (p @ v).reshape(B, Hq, D), p


def _decode(s):
    c, lens = s["case"], s["lens"].long()
    # First tokens, then the window's, each as far as the longest sequence has them.
    f = torch.arange(c["first"], device=lens.device).expand(lens.numel(), -1)
    low = torch.clamp(lens - c["window"], min=0)[:, None]
    w = low + torch.arange(min(c["window"], s["tables"].shape[1] * BS), device=lens.device)
    at = torch.cat([f, w], 1)
    seen = (at < lens[:, None]) & torch.cat([f < low, torch.ones_like(w, dtype=torch.bool)], 1)
    o, _ = _attend(s["q"], _rows(s["k_cache"], s["tables"], at), _rows(s["v_cache"], s["tables"], at), seen, s["sinks"], 1 / math.sqrt(c["D"]))
    s["out"].copy_(torch.where(lens[:, None, None] > 0, o, torch.zeros_like(o)))


def _weights(s):
    c, lens = s["case"], s["lens"].long()
    n = s["scores"].shape[-1]
    at = torch.arange(n, device=lens.device).expand(lens.numel(), -1)
    seen = at < lens[:, None]
    o, p = _attend(s["q"], _rows(s["k_cache"], s["tables"], at), _rows(s["v_cache"], s["tables"], at), seen, s["sinks"], 1 / math.sqrt(c["D"]))
    s["out"].copy_(torch.where(lens[:, None, None] > 0, o, torch.zeros_like(o)))
    scored = (lens - 1 if s["scored"] is None else s["scored"].long())[:, None]
    got = p.sum(2)
    new = torch.where((at < scored)[:, None], s["scores"] + got, got)
    s["scores"].copy_(torch.where(seen[:, None], new, s["scores"]))


def _prompt(s):
    c = s["case"]
    T, start, D, Hkv = c["T"], c["start"], c["D"], c["Hkv"]
    G = c["Hq"] // Hkv
    low = max(0, start - c["window"] + 1)
    at = torch.cat([torch.arange(min(c["first"], low), device=_dev()), torch.arange(low, start + T, device=_dev())])
    blk = s["ids"][at // BS].long()
    k, v = (pool[blk, :, at % BS].transpose(0, 1).float() for pool in (s["k_cache"], s["v_cache"]))     # [Hkv, n, D]
    pos = torch.arange(start, start + T, device=_dev())[:, None]
    seen = (at <= pos) & ((at > pos - c["window"]) | (at < c["first"]))
    q = s["q"].float().view(T, Hkv, G, D).permute(1, 2, 0, 3)
    x = (q @ k[:, None].transpose(-1, -2)) * (1 / math.sqrt(D))
    p = _softmax(x.masked_fill_(~seen, -math.inf), None)
    s["out"].copy_((p @ v[:, None]).permute(2, 0, 1, 3).reshape(T, c["Hq"], D))


def _evict(s):
    c = s["case"]
    lens = s["lens"][s["ids"].long()].long()
    cut = lens > c["limit"]
    s["kept"].fill_(-1)
    s["new_lens"].copy_(torch.where(cut, c["budget"], -1))
    i = cut.nonzero()[:, 0]
    ids, n = s["ids"][i].long(), lens[i][:, None, None]
    x = s["scores"][:, ids]                                                             # [L, m, Hkv, S]
    at = torch.arange(x.shape[-1], device=x.device)
    key = torch.where((at < c["first"]) | (at >= n - c["recent"]), math.inf, x)
    key = torch.where(at < n, key, -math.inf)
    kept = key.sort(dim=-1, descending=True, stable=True).indices[..., :c["budget"]].sort(-1).values
    s["kept"][:, i] = kept.to(torch.int32)
    s["scores"][:, ids, :, :c["budget"]] = x.gather(-1, kept)
    row = s["tables"][ids].clamp(min=0).long()
    to = torch.arange(c["budget"], device=x.device)
    layer = torch.arange(x.shape[0], device=x.device)[:, None, None, None]
    head = torch.arange(x.shape[2], device=x.device)[None, None, :, None]
    from_blk = row[None, :, None].expand(*x.shape[:3], -1).gather(-1, kept // BS)
    to_blk = row[:, to // BS][None, :, None]
    for pool in (s["k_pools"], s["v_pools"]):
        pool[layer, to_blk, head, to % BS] = pool[layer, from_blk, head, kept % BS]


def _truncate(s):
    tables, lens, stack, top, extra = s["state"]
    ids, n = s["ids"].long(), s["new_lens"]
    old = lens[ids]
    cut = (n >= 0) & (n < old)
    rows = tables[ids]
    col = torch.arange(rows.shape[1], device=rows.device)
    gone = cut[:, None] & (col >= (n[:, None] + BS - 1) // BS) & (col < (old[:, None] + BS - 1) // BS)
    drop = torch.zeros_like(extra).index_add_(0, rows.clamp(min=0).flatten().long(), gone.flatten().to(torch.int32))
    back = (drop > extra).nonzero()[:, 0].flip(0)
    stack[top + torch.arange(back.numel(), device=back.device)] = back.to(torch.int32)
    top += back.numel()
    extra.copy_((extra - drop).clamp(min=0))
    tables[ids] = torch.where(gone, -1, rows)
    lens[ids] = torch.where(cut, n, old)


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "truncate":
        torch._foreach_copy_(s["state"], s["start"])
    if own:
        from paged_kv_cache_xs_gb300 import ops
        if kind == "decode":
            ops.xs_paged_decode_first(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], 1 / math.sqrt(c["D"]), s["ws"],
                                      first=c["first"], window=c["window"], sinks=s["sinks"])
        elif kind == "prompt":
            ops.xs_paged_prefill_first(s["out"], s["q"], s["k_cache"], s["v_cache"], s["ids"], c["start"], 1 / math.sqrt(c["D"]),
                                       first=c["first"], window=c["window"])
        elif kind == "weights":
            ops.xs_paged_decode_weights(s["out"], s["scores"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                        1 / math.sqrt(c["D"]), s["ws"], scored_lens=s["scored"], sinks=s["sinks"])
        elif kind == "evict":
            ops.xs_kv_evict(s["ids"], s["k_pools"], s["v_pools"], s["scores"], s["tables"], s["lens"], s["kept"], s["new_lens"],
                            first=c["first"], recent=c["recent"], limit=c["limit"], extra_refs=s["extra"])
        else:
            tables, lens, stack, top, extra = s["state"]
            ops.xs_block_truncate(s["ids"], s["new_lens"], tables, lens, stack, top, extra)
    else:
        {"decode": _decode, "prompt": _prompt, "weights": _weights, "evict": _evict, "truncate": _truncate}[kind](s)
    if kind in ("decode", "prompt"):
        return {"out": s["out"]}
    if kind == "weights":
        return {"out": s["out"], "scores": s["scores"]}
    if kind == "evict":
        return {n: s[n] for n in ("kept", "new_lens", "scores", "k_pools", "v_pools")}
    return dict(zip(("tables", "lens", "stack", "top", "extra"), s["state"]))


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    kind = c["kind"]
    e = 4 if c.get("dtype") == "f32" else 2
    if kind in ("decode", "weights"):
        Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
        lens = _spread(c["B"], c["lo"], c["hi"], c["empty"])
        tokens = sum(min(n, c["first"] + c["window"]) if kind == "decode" else n for n in lens)
        b = tokens * (2 * e * Hkv * D + 4 / BS) + 2 * e * (c["B"] - c["empty"]) * Hq * D
        if kind == "weights":
            b += 2 * 4 * Hkv * tokens
        return {"bytes": b, "flops": 4.0 * tokens * Hq * D}
    if kind == "prompt":
        T, start, W, F = c["T"], c["start"], c["window"], c["first"]
        n = np.arange(start + 1, start + T + 1)
        seen = np.minimum(n, W) + np.minimum(F, np.maximum(0, n - W))
        keys = start + T - max(0, start - W + 1) + min(F, max(0, start - W + 1))
        return {"bytes": 2.0 * (2 * T * c["Hq"] + 2 * keys * c["Hkv"]) * c["D"], "flops": 4.0 * float(seen.sum()) * c["Hq"] * c["D"]}
    if kind == "evict":
        lens = [n for n in _spread(c["B"], c["lo"], c["hi"]) if n > c["limit"]]
        # Each candidate's score read; each kept row behind the first tokens read and written, with its score and place.
        scores = sum(n - c["first"] - c["recent"] for n in lens)
        moved = len(lens) * (c["budget"] - c["first"])
        heads = c["layers"] * c["Hkv"]
        return {"bytes": heads * (4.0 * scores + moved * (2 * 2 * e * c["D"] + 2 * 4) + 4.0 * len(lens) * c["budget"]), "flops": 0.0}
    lens = _spread(c["B"], c["lo"], c["hi"])
    pages = sum(min(n, c["cut"] / 2) / BS for n in lens)
    return {"bytes": pages * 4 * 5 + 16.0 * c["B"], "flops": 0.0}


# ---------------------------------------------------------------- the operators in 64 bits

def _exact_rows(q, k, v, sinks, scale):
    """One sequence: q [Hq, D] on rows [n, Hkv, D], by one einsum for each product; outputs and weights [Hq, n]."""
    G = q.shape[0] // k.shape[1]
    kk, vv = (x.double().repeat_interleave(G, 1) for x in (k, v))
    x = torch.einsum("hd,nhd->hn", q.double(), kk) * scale
    if sinks is not None:
        x = torch.cat([x, sinks.double()[:, None]], 1)
    p = torch.softmax(x, -1)[:, :k.shape[0]]
    return torch.einsum("hn,nhd->hd", p, vv), p


def _exact_prompt(s):
    c = s["case"]
    T, start, W, F, G = c["T"], c["start"], c["window"], c["first"], c["Hq"] // c["Hkv"]
    out = torch.empty(T, c["Hq"], c["D"], dtype=torch.float64, device=_dev())
    every = torch.arange(start + T, device=_dev())
    for a in range(0, T, 256):                       # 256 queries on the tokens that any of them sees
        m = min(256, T - a)
        pos = start + a + torch.arange(m, device=_dev())
        use = every[(every < F) | (every > start + a - W)]
        use = use[use < start + a + m]
        k, v = (pool[s["ids"][use // BS].long(), :, use % BS].double().repeat_interleave(G, 1) for pool in (s["k_cache"], s["v_cache"]))
        x = torch.einsum("thd,nhd->htn", s["q"][a:a + m].double(), k) / math.sqrt(c["D"])
        hidden = (use > pos[:, None]) | ((use >= F) & (use <= pos[:, None] - W))
        out[a:a + m] = torch.einsum("htn,nhd->thd", torch.softmax(x.masked_fill(hidden, -math.inf), -1), v)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    kind = c["kind"]
    if kind == "prompt":
        return {"out": _exact_prompt(s)}
    if kind == "truncate":
        return None
    if kind == "evict":
        kept, scores = np.full(tuple(s["kept"].shape), -1, dtype=np.int32), s["scores"].cpu().numpy()
        lens, ids, after = s["lens"].tolist(), s["ids"].tolist(), scores.astype(np.float64)
        for i, b in enumerate(ids):
            if lens[b] <= c["limit"]:
                continue
            middle = np.arange(c["first"], lens[b] - c["recent"])
            for at in np.ndindex(kept.shape[0], kept.shape[2]):
                x = scores[at[0], b, at[1]]
                best = middle[np.lexsort((middle, -x[middle]))][:c["budget"] - c["first"] - c["recent"]]
                keep = np.concatenate([np.arange(c["first"]), np.sort(best), np.arange(lens[b] - c["recent"], lens[b])])
                kept[at[0], i, at[1]] = keep
                after[at[0], b, at[1], :c["budget"]] = x[keep]
        new = np.array([c["budget"] if lens[b] > c["limit"] else -1 for b in ids], dtype=np.int32)
        return {"kept": kept, "new_lens": new, "scores": after, "k_pools": None, "v_pools": None}
    out = torch.zeros(c["B"], c["Hq"], c["D"], dtype=torch.float64, device=_dev())
    scores = s["scores"].double() if kind == "weights" else None
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        at = torch.arange(n, device=_dev())
        if kind == "decode":
            at = at[(at < c["first"]) | (at >= n - c["window"])]
        blk = s["tables"][b][at // BS].long()
        out[b], p = _exact_rows(s["q"][b], s["k_cache"][blk, :, at % BS], s["v_cache"][blk, :, at % BS], s["sinks"], 1 / math.sqrt(c["D"]))
        if kind == "weights":
            got = p.view(c["Hkv"], -1, n).sum(1)
            old = n - 1 if s["scored"] is None else int(s["scored"][b])
            scores[b, :, :old] += got[:, :old]
            scores[b, :, old:n] = got[:, old:]
    return {"out": out, "scores": scores} if kind == "weights" else {"out": out}
