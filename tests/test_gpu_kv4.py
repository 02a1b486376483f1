"""The 4-bit cache: stores bit for bit, reading back, decode attention."""
import math

import pytest
import torch

from paged_kv_cache_xs_gb300 import ops
from paged_kv_cache_xs_gb300.step import Kv4DecodeStep
from tests import plain_ops as plain
from tests.gpu_helpers import device

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def gen(seed):
    return torch.Generator(device=device()).manual_seed(seed)


def flag():
    return torch.zeros(1, dtype=torch.int32, device=device())


# ---------------------------------------------------------------- store and read back

def awkward_rows(n, D, seed):
    """Rows whose groups hold ties of magnitude, zeros, tiny, huge, one-sided
    values, exact ties of the rounding, infinities and NaN."""
    x = torch.randn(n, D, generator=torch.Generator().manual_seed(seed))
    x[0 % n, :32] = 0
    x[1 % n, :32] = torch.linspace(-1, 1, 32)              # +1 and -1: a tie of magnitude
    x[2 % n, 32:] = x[2 % n, 32:].abs()                    # one-sided
    x[3 % n, :32] *= 1e-38
    x[4 % n, 32:64] *= 1e30
    x[5 % n, :32] = torch.arange(32) * 0.5 - 8             # ties: x / s is a half integer
    x[6 % n, :32] = torch.arange(32) * 1.5 - 24            # the same under a scale of 3
    x[7 % n, 32:64] = -3.0
    x[8 % n, :32] = 1e-40                                  # subnormal
    return x.to(BF)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hkv,T", [(1, 1), (3, 16), (8, 41)])
def test_append_bytes(Hkv, T, D):
    dev = device()
    nb = 6
    cpu = torch.Generator().manual_seed(T)
    k = awkward_rows(T * Hkv, D, 1).view(T, Hkv, D)
    v = awkward_rows(T * Hkv, D, 2).view(T, Hkv, D)
    slots = torch.randperm(nb * 16, generator=cpu)[:T]
    if T > 5:
        slots[3] = -1
    start = torch.randint(0, 256, (2, nb, Hkv, 9 * D), generator=cpu, dtype=torch.uint8)
    kc, vc = start[0].to(dev), start[1].to(dev)
    err = flag()
    both = torch.cat([k, v], 1).to(dev)                    # strided rows
    ops.xs_kv4_append(both[:, :Hkv], both[:, Hkv:], kc, vc, slots.to(dev), err_flag=err)
    want = start.clone()
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            plain.write_rows(want[0], False, s // 16, s % 16, k[t])
            plain.write_rows(want[1], True, s // 16, s % 16, v[t])
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])
    assert int(err) == 0


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_group_with_infinity_or_nan_reads_as_nan(bad):
    dev = device()
    k = torch.ones(1, 2, 64, dtype=BF, device=dev)
    k[0, 1, 40] = bad
    kc, vc = ops.kv4_pools(1, 2, 64, dev)
    ops.xs_kv4_append(k, k, kc, vc, torch.tensor([5], device=dev))
    ko, vo = (torch.empty(1, 2, 16, 64, dtype=BF, device=dev) for _ in range(2))
    ops.xs_kv4_unpack(ko, vo, kc, vc, torch.zeros(1, dtype=torch.int32, device=dev))
    for o in (ko, vo):
        assert bool(o[0, 1, 5, 32:].isnan().all())
        assert bool((o[0, 0, 5] == 1).all()) and bool((o[0, 1, 5, :32] == 1).all())
        o[0, :, 5] = 0
        assert bool((o == 0).all())


def test_all_bf16_quotients_round_as_in_64_bits():
    # Every 8-bit significand under every 8-bit scale: a group is an extreme
    # and 31 values; codes against 64 bits, bit for bit.
    dev = device()
    ext = torch.arange(128, 256, dtype=torch.float32)
    vals = torch.cat([torch.arange(128, 256) * 2.0 ** e for e in (0, -1, -2, -3, -4, -5)])
    vals = torch.cat([vals, -vals])
    vals = torch.nn.functional.pad(vals, (0, -vals.numel() % 31)).view(-1, 31)
    x = torch.cat([(ext[:, None, None] * 1.0).expand(-1, vals.shape[0], 1),
                   vals[None].expand(128, -1, -1)], -1)
    x = torch.where(x.abs() > ext[:, None, None], torch.zeros(()), x).reshape(-1, 1, 32)
    x = torch.cat([x, -x], -1).to(BF)                      # [N, 1, 64]
    n = x.shape[0]
    kc, vc = ops.kv4_pools(-(-n // 16), 1, 64, dev)
    ops.xs_kv4_append(x.to(dev), x.to(dev), kc, vc, torch.arange(n, device=dev))
    codes, s = plain.quantise(x[:, 0])
    want = plain.values(codes, s)
    for pool, is_v in ((kc, False), (vc, True)):
        got = plain.page_values(pool, 64, is_v)[:, 0].reshape(-1, 64)[:n]
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("n,Hkv,D", [(1, 1, 64), (5, 3, 128), (300, 8, 128), (70, 12, 64)])
def test_unpack(n, Hkv, D, dtype):
    dev = device()
    nb = n + 3
    x = torch.randn(2, nb, Hkv, 16, D, generator=gen(n), device=dev)
    kc, vc = plain.pack_pages(x[0], False), plain.pack_pages(x[1], True)
    ids = torch.randperm(nb, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32)
    if n > 4:
        ids[1], ids[3] = -1, nb
    ids = ids.to(dev)
    ko, vo = (torch.full((n, Hkv, 16, D), 9.0, dtype=dtype, device=dev) for _ in range(2))
    err = flag()
    ops.xs_kv4_unpack(ko, vo, kc, vc, ids, err_flag=err)
    ok = (ids >= 0) & (ids < nb)
    for out, pool, is_v in ((ko, kc, False), (vo, vc, True)):
        want = plain.page_values(pool[ids[ok].long()], D, is_v).to(dtype)  # 12 bits: exact in fp32
        assert torch.equal(out[ok], want)
        assert bool((out[~ok] == 9.0).all())
    assert int(err) == (ops.FLAG_BAD_BLOCK if n > 4 else 0)


# ---------------------------------------------------------------- attention

def setup(lens, Hq, Hkv, D, seed, k_std=1.0, spare=2, width=None):
    """Pools whose rows outside the sequences hold 0xff bytes (NaN scales)."""
    dev = device()
    lens = list(lens)
    pages = [max(0, -(-n // 16)) for n in lens]
    nb = sum(pages) + spare
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    width = width or max(pages + [1])
    bt = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, p in enumerate(pages):
        bt[b, :p] = perm[at:at + p]
        at += p
    x = torch.randn(2, nb, Hkv, 16, D, generator=gen(seed), device=dev).to(BF)
    x[0] *= k_std
    kc, vc = plain.pack_pages(x[0], False), plain.pack_pages(x[1], True)
    # garbage in rows at and behind each length, and in unused blocks
    p = [t.to(dev) for t in plain.places(D)]
    gk, gv = torch.full_like(kc, 255), torch.full_like(vc, 255)
    gk[perm[:at].long().to(dev)] = kc[perm[:at].long().to(dev)]
    gv[perm[:at].long().to(dev)] = vc[perm[:at].long().to(dev)]
    for b, n in enumerate(lens):
        if n > 0 and n % 16:
            blk = int(bt[b, n // 16])
            for pool, nib, sc in ((gk, p[0], p[2]), (gv, p[1], p[3])):
                for o in range(n % 16, 16):
                    at_s = 8 * D + 2 * sc[o, ::32]
                    pool[blk][:, at_s] = 255
                    pool[blk][:, at_s + 1] = 255
    q = torch.randn(len(lens), Hq, D, generator=gen(seed + 1), device=dev).to(BF)
    return q, gk, gv, bt.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)


def reader(pool, bt, lens, D, is_v):
    def f(b):
        n = int(lens[b])
        x = plain.page_values(pool[bt[b, :-(-n // 16)].long()], D, is_v)    # [p, H, 16, D]
        return x.transpose(1, 2).flatten(0, 1)[:n]
    return f


def check_decode(q, kc, vc, bt, lens, scale, ws=None, sinks=None, window=0, what=""):
    B, Hq, D = q.shape
    ws = ws or ops.Kv4Workspace(B, Hq, kc.shape[1], D, q.device)
    out = torch.full((B, Hq, D), 5.0, dtype=BF, device=q.device)
    err = flag()
    ops.xs_kv4_decode(out, q, kc, vc, bt, lens, scale, ws, sinks=sinks, window=window, err_flag=err)
    ref, bound = plain.attend(q, reader(kc, bt, lens, D, False), reader(vc, bt, lens, D, True),
                              lens.tolist(), scale, sinks, window)
    plain.check(out, ref, bound, what)
    assert int(err) == 0
    return out


LENS = [1, 15, 16, 17, 0, 31, 33, 128, -1, 129, 257, 500]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,Hkv", [(1, 3), (2, 2), (4, 1), (8, 2)])
def test_decode_lengths(G, Hkv, D):
    check_decode(*setup(LENS, G * Hkv, Hkv, D, seed=G), 1 / math.sqrt(D))


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 10 ** 6])
@pytest.mark.parametrize("sinks", [False, True])
def test_decode_window_and_sinks(window, sinks):
    a = setup(LENS, 8, 2, 64, seed=window % 97)
    z = torch.randn(8, generator=gen(3), device=device()).to(BF) * 3 if sinks else None
    check_decode(*a, 0.125, sinks=z, window=window)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 32, 8), (64, 12, 12)])
@pytest.mark.parametrize("lens", [[4097], [3000, 17, 0, 9001], [700 + 37 * i for i in range(40)],
                                  [20000]])
def test_decode_split(lens, D, Hq, Hkv):
    # Lengths that are cut between blocks, alone and in a ragged batch.
    check_decode(*setup(lens, Hq, Hkv, D, seed=len(lens)), 1 / math.sqrt(D))


@pytest.mark.parametrize("B,Hkv,G,D", [(300, 1, 2, 64), (150, 2, 4, 128), (1, 1, 1, 64), (2, 1, 8, 128)])
def test_decode_many_or_few_sequences(B, Hkv, G, D):
    # More sequences than a CTA has threads, empty ones among them, first and
    # last; and the fewest.
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 90, (B,), generator=g).tolist()
    if B > 10:
        lens[0] = lens[-1] = lens[128] = lens[129] = 0
        lens[7], lens[B - 2] = 1200, 700
    else:
        lens[0] = 3333
    check_decode(*setup(lens, G * Hkv, Hkv, D, seed=B), 1 / math.sqrt(D))
    check_decode(*setup(lens, G * Hkv, Hkv, D, seed=B), 1 / math.sqrt(D), window=33,
                 sinks=torch.randn(G * Hkv, generator=gen(2), device=device()).to(BF))


@pytest.mark.parametrize("Hkv,G,D", [(8, 4, 128), (8, 8, 64), (1, 1, 64), (5, 2, 128)])
@pytest.mark.parametrize("lens", [[240], [257], [4096], [4097], [8100, 3], [12000], [16, 0, 4500, 300],
                                  [5000, 0, 9, 700]])
def test_decode_few_sequences(lens, Hkv, G, D):
    # One CTA, one cluster, or all CTAs to a segment, and empty sequences
    # among them; with tables that hold no more, and with wider ones.
    a = setup(lens, G * Hkv, Hkv, D, seed=sum(lens))
    check_decode(*a, 1 / math.sqrt(D))
    z = torch.randn(G * Hkv, generator=gen(4), device=device()).to(BF) * 3
    check_decode(*setup(lens, G * Hkv, Hkv, D, seed=sum(lens), width=900), 1 / math.sqrt(D), sinks=z,
                 window=max(lens) - 5)


@pytest.mark.parametrize("B,Hkv,G,D", [(5, 8, 4, 128), (17, 8, 8, 128), (18, 8, 8, 64), (70, 2, 1, 64), (100, 1, 2, 128)])
def test_decode_batches_of_short_tables(B, Hkv, G, D):
    # From empty to 128 pages, a CTA or a cluster for each; and a table one wider.
    lens = [(0, 1, 16, 255, 256, 257, 600, 2048, 1999, 3)[i % 10] for i in range(B)]
    z = torch.randn(G * Hkv, generator=gen(4), device=device()).to(BF) * 3
    for width in (128, 129):
        a = setup(lens, G * Hkv, Hkv, D, seed=B, width=width)
        one = check_decode(*a, 1 / math.sqrt(D))
        two = check_decode(*a, 1 / math.sqrt(D), sinks=z, window=300)
        assert not torch.equal(one, two)
    q, kc, vc, bt, n = setup(lens, G * Hkv, Hkv, D, seed=B, width=128)
    n[B - 1] = 128 * 16 + 1                 # past the table: told, and clamped
    bt[B - 1] = bt[7 % B][:1]
    out, err = torch.empty_like(q), flag()
    ops.xs_kv4_decode(out, q, kc, vc, bt, n, 0.1, ops.Kv4Workspace(B, G * Hkv, Hkv, D, device()), err_flag=err)
    assert int(err) == ops.FLAG_BAD_LEN


@pytest.mark.parametrize("n", [5, 40, 300, 5000])
def test_every_token_counts_once(n):
    # q = 0: all weights are 1 / n; V is zero but for one token, so the result
    # is v / n to 3 roundings.  A token dropped or taken twice shows whatever n is.
    dev = device()
    places = sorted({0, 1, 15, 16, n // 2, n // 3, n - 1, max(0, n - 16), max(0, n - 17)} & set(range(n)))
    pages = -(-n // 16)
    B = len(places)
    v = torch.zeros(B * pages, 1, 16, 128, device=dev)
    for b, t in enumerate(places):
        v[b * pages + t // 16, 0, t % 16] = torch.arange(1, 129, device=dev) % 8 + 1.0
    k = torch.randn(B * pages, 1, 16, 128, generator=gen(n), device=dev).to(BF)
    kc, vc = plain.pack_pages(k, False), plain.pack_pages(v, True)
    bt = torch.arange(B * pages, dtype=torch.int32, device=dev).view(B, pages)
    lens = torch.full((B,), n, dtype=torch.int32, device=dev)
    q = torch.zeros(B, 4, 128, dtype=BF, device=dev)
    out = check_decode(q, kc, vc, bt, lens, 0.1)
    assert bool((out != 0).all())


def test_sharp_and_rising_logits():
    # Large logits, and logits that rise along the sequence so that the
    # running maximum moves on page after page; and a descending order.
    dev = device()
    n = 2000
    for sign in (1.0, -1.0):
        k = torch.zeros(125, 2, 16, 128, device=dev)
        ramp = sign * torch.arange(n, device=dev).view(125, 1, 16, 1) / n * 8
        k += ramp.expand(-1, 2, -1, 128) / 128 * 16
        kc = plain.pack_pages(k.to(BF), False)
        vc = plain.pack_pages(torch.randn(125, 2, 16, 128, generator=gen(1), device=dev).to(BF), True)
        bt = torch.arange(125, dtype=torch.int32, device=dev)[None]
        lens = torch.tensor([n - 3], dtype=torch.int32, device=dev)
        q = torch.full((1, 8, 128), 1.0, dtype=BF, device=dev)
        check_decode(q, kc, vc, bt, lens, 8.0 / 16, what=str(sign))
    check_decode(*setup([900, 33, 5000], 8, 2, 128, seed=9, k_std=6.0), 1.0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e", [-120, -100, -60, 60, 100, 112, 120, 125])
def test_queries_of_any_magnitude(e, D):
    # q times 2^e under keys times 2^-e (exact, but for keys that become
    # subnormal, whose values are what the pages then hold): ordinary logits.
    # And under keys of zero: all weights alike, whatever q is.
    a = setup([300, 77], 8, 2, D, seed=abs(e))
    q, kc, vc, bt, lens = a
    q = (q.float() * 2.0 ** e).to(BF)
    x = torch.randn(kc.shape[0], 2, 16, D, generator=gen(e + 200), device=device())
    kc = plain.pack_pages((x * 2.0 ** -e).to(BF), False)
    check_decode(q, kc, vc, bt, lens, 0.1)
    out = check_decode(q, torch.zeros_like(kc), vc, bt, lens, 0.1)
    assert bool(out.isfinite().all())


def test_captured_beside_other_streams():
    """One captured graph with two branches: a bf16 append by itself on a side
    stream, norm + rotation + 4-bit append and attention on the other; a copy
    before and a torch operation behind; then the same once more in a row.
    Replays follow the inputs and equal the calls made one by one."""
    dev = device()
    Hq, Hkv, D, B = 8, 2, 128, 5
    nb = 40
    bt = torch.randperm(nb, generator=torch.Generator().manual_seed(3))[:B * 6].to(torch.int32).view(B, 6).to(dev)
    tab = ops.rope_table(96, D, 1e4, dev)
    src = torch.randn(B, Hq + 2 * Hkv, D, generator=gen(1), device=dev).to(BF)

    def buffers():
        x = torch.zeros_like(src)
        lens = torch.zeros(B, dtype=torch.int32, device=dev)
        bf = torch.zeros(2, nb, Hkv, 16, D, dtype=BF, device=dev)
        return x, lens, bf, ops.kv4_pools(nb, Hkv, D, dev), torch.zeros(2, B, Hq, D, dtype=BF, device=dev)

    def work(x, lens, bf, kv4, out, step, side):
        for _ in range(2):
            x.copy_(src)
            lens.add_(1)
            q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                ops.xs_kv_append_paged(k.contiguous(), v.contiguous(), bf[0], bf[1], bt, lens)
            step.run(out[0], q, k, v, None, None, tab, kv4[0], kv4[1], bt, lens, 0.09)
            main.wait_stream(side)
            ops.xs_kv4_decode(out[1], out[0], kv4[0], kv4[1], bt, lens, 0.09, step.ws)
            x.add_(1.0)

    a, b = buffers(), buffers()
    step = Kv4DecodeStep(B, Hq, Hkv, D, dev)
    side = torch.cuda.Stream()
    work(*a, step, side)                    # builds what a first call builds
    torch.cuda.synchronize()
    for x in (a[0], a[1], a[2], *a[3], a[4]):
        x.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(*a, step, side)
    other = Kv4DecodeStep(B, Hq, Hkv, D, dev)
    for i in range(30):
        src.copy_(torch.randn(src.shape, generator=gen(i), device=dev))
        graph.replay()
        work(*b, other, torch.cuda.current_stream())
        for x, y in zip((a[0], a[1], a[2], *a[3], a[4]), (b[0], b[1], b[2], *b[3], b[4])):
            assert torch.equal(x, y), i
    assert step.error_flags() == 0 and int(a[1][0]) == 60


def test_nan_in_a_sequence_stays_in_its_head():
    q, kc, vc, bt, lens = setup([40, 40], 4, 2, 64, seed=5)
    ws = ops.Kv4Workspace(2, 4, 2, 64, device())
    q[0, 1] = float("nan")
    out = torch.empty_like(q)
    ops.xs_kv4_decode(out, q, kc, vc, bt, lens, 0.125, ws)
    assert bool(out[0, 1].isnan().all())
    out[0, 1] = 0
    assert bool(out.isfinite().all())
    q[0, 1] = 0
    check_decode(q, kc, vc, bt, lens, 0.125, ws=ws, what="the workspace is clean afterwards")


@pytest.mark.parametrize("lens,Hkv,D", [([900, 40], 2, 64), ([9000, 40], 2, 128), ([300] * 50, 2, 128),
                                        ([600, 1200] * 40, 4, 64)])
def test_infinities_stay_where_they_are(lens, Hkv, D):
    # A NaN in one head's query, an infinity in one sequence's K and a NaN in a
    # group of its V, in every form of the call: other heads, sequences and (for
    # V) groups are as without them.
    q, kc, vc, bt, n = setup(lens, 4 * Hkv, Hkv, D, seed=11)
    good = check_decode(q, kc, vc, bt, n, 0.1)
    ws = ops.Kv4Workspace(len(lens), 4 * Hkv, Hkv, D, device())
    q[0, 1] = float("nan")
    one = int(bt[1, 1])                         # block of tokens 16 .. 31 of sequence 1
    row = torch.zeros(1, Hkv, D, dtype=BF, device=device())
    row[0, 0, 3] = float("inf")
    value = torch.zeros(1, Hkv, D, dtype=BF, device=device())
    value[0, 1, 40] = float("nan")
    ops.xs_kv4_append(row, value, kc, vc, torch.tensor([16 * one + 5], device=device()))
    out = torch.empty_like(q)
    ops.xs_kv4_decode(out, q, kc, vc, bt, n, 0.1, ws)
    bad = out.isnan()
    want = torch.zeros_like(bad)
    want[0, 1] = True
    want[1, :4] = True                          # KV head 0 of sequence 1
    want[1, 4:8, 32:64] = True                  # the group of dim 40 of its KV head 1
    assert torch.equal(bad, want)
    same = torch.ones(len(lens), 4 * Hkv, dtype=torch.bool, device=device())
    same[0, 1] = False
    same[1] = False
    assert torch.equal(out[same], good[same])


def test_calls_from_several_threads():
    # Each thread with its stream and workspace, in each of the call's forms.
    import threading

    dev = device()
    cases = [setup([290], 8, 2, 128, seed=1), setup([6000, 20], 64, 8, 128, seed=2),
             setup([310 - i for i in range(9)], 64, 8, 64, seed=3),
             setup([100 + i for i in range(40)], 64, 8, 128, seed=4)]
    want = [check_decode(*c, 0.1) for c in cases]
    torch.cuda.synchronize()
    got = [None] * 8

    def work(i):
        q, kc, vc, bt, n = cases[i % 4]
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            ws = ops.Kv4Workspace(q.shape[0], q.shape[1], kc.shape[1], q.shape[2], dev)
            out = torch.empty_like(q)
            for _ in range(100):
                ops.xs_kv4_decode(out, q, kc, vc, bt, n, 0.1, ws)
            s.synchronize()
        got[i] = out

    threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    for i in range(8):
        assert torch.equal(got[i], want[i % 4]), i


def test_same_result_every_time_and_across_batches():
    # Bit-identical on repetition, on a reused workspace after other batches,
    # on a side stream and from a graph whose lengths change between replays.
    dev = device()
    a = setup([1, 700, 4000, 0, 33], 32, 8, 128, seed=21)
    b = setup([9000, 5], 32, 8, 128, seed=22)
    ws = ops.Kv4Workspace(5, 32, 8, 128, dev)
    first = check_decode(*a, 0.09, ws=ws)
    check_decode(*b, 0.09, ws=ws)
    out = torch.empty_like(first)
    for _ in range(20):
        out.fill_(1.0)
        ops.xs_kv4_decode(out, *a, 0.09, ws)
        assert torch.equal(out, first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out.fill_(1.0)
        ops.xs_kv4_decode(out, *a, 0.09, ws)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, first)
    q, kc, vc, bt, lens = a
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.xs_kv4_decode(out, q, kc, vc, bt, lens, 0.09, ws)
    for change in ([1, 700, 4000, 0, 33], [1, 16, 3999, 0, 0], [0] * 5, [1, 1, 1, 0, 1]):
        lens.copy_(torch.tensor(change, dtype=torch.int32))
        graph.replay()
        ref, bound = plain.attend(q, reader(kc, bt, lens, 128, False), reader(vc, bt, lens, 128, True),
                                  change, 0.09)
        plain.check(out, ref, bound + 0 * ref, str(change))


def test_decode_device_errors():
    q, kc, vc, bt, lens = setup([40, 40, 64], 4, 2, 64, seed=6)
    good = check_decode(q, kc, vc, bt, lens, 0.125)
    bt[0, 1] = kc.shape[0]
    bt[2, 0] = -3
    ws = ops.Kv4Workspace(3, 4, 2, 64, device())
    out, err = torch.empty_like(q), flag()
    ops.xs_kv4_decode(out, q, kc, vc, bt, lens, 0.125, ws, err_flag=err)
    assert int(err) == ops.FLAG_BAD_BLOCK and torch.equal(out[1], good[1])
    bt[0, 1], bt[2, 0] = 0, 0
    lens[2] = 65
    err.zero_()
    ops.xs_kv4_decode(out, q, kc, vc, bt, lens, 0.125, ws, err_flag=err)
    assert int(err) == ops.FLAG_BAD_LEN and torch.equal(out[1], good[1])
    lens[2] = 2 ** 31 - 1
    err.zero_()
    ops.xs_kv4_decode(out, q, kc, vc, bt, lens, 0.125, ws, err_flag=err)
    assert int(err) == ops.FLAG_BAD_LEN and torch.equal(out[1], good[1])


def test_far_blocks():
    # Pages beyond 2^32 bytes of the pools, stored, read back and attended to.
    dev = device()
    Hkv, D = 8, 128
    nb = 2 ** 32 // (Hkv * 9 * D) + 600
    kc = torch.empty(nb, Hkv, 9 * D, dtype=torch.uint8, device=dev)
    vc = torch.empty(nb, Hkv, 9 * D, dtype=torch.uint8, device=dev)
    ids = torch.tensor([nb - 1, 0, nb - 500], dtype=torch.int32, device=dev)
    for pool in (kc, vc):
        pool[ids.long()] = 255
    k = torch.randn(45, Hkv, D, generator=gen(1), device=dev).to(BF)
    v = torch.randn(45, Hkv, D, generator=gen(2), device=dev).to(BF)
    pos = torch.arange(45, device=dev)
    ops.xs_kv4_append(k, v, kc, vc, ids.long()[pos // 16] * 16 + pos % 16)
    ko, vo = (torch.empty(3, Hkv, 16, D, dtype=BF, device=dev) for _ in range(2))
    ops.xs_kv4_unpack(ko, vo, kc, vc, ids)
    for o, x in ((ko, k), (vo, v)):
        want = plain.values(*plain.quantise(x)).to(BF)
        assert torch.equal(o.transpose(1, 2).flatten(0, 1)[:45], want)
    q = torch.randn(1, 32, D, generator=gen(3), device=dev).to(BF)
    check_decode(q, kc, vc, ids[None].contiguous(), torch.tensor([45], dtype=torch.int32, device=dev), 0.09)


# ---------------------------------------------------------------- together

def test_prompt_then_decode_steps():
    """A prompt stored in two chunks, its attention through the read-back
    pages, then decode steps of a small batch through Kv4DecodeStep."""
    dev = device()
    Hq, Hkv, D, n0 = 8, 2, 128, 150
    B, nb = 3, 60
    kc, vc = ops.kv4_pools(nb, Hkv, D, dev)
    bt = torch.randperm(nb, generator=torch.Generator().manual_seed(1)).to(torch.int32)[:45].view(3, 15).to(dev)
    tab = ops.rope_table(240, D, 1e6, dev)
    w = (1 + 0.1 * torch.randn(2, D, generator=gen(5), device=dev)).to(BF)
    scale = 1 / math.sqrt(D)
    k_rows = {b: [] for b in range(B)}          # what each sequence's cache should stand for
    v_rows = {b: [] for b in range(B)}

    def remember(b, k, v):
        k_rows[b] += list(plain.values(*plain.quantise(k)))
        v_rows[b] += list(plain.values(*plain.quantise(v)))

    err = flag()
    for lo, hi in ((0, 100), (100, n0)):        # the prompt of sequence 0
        T = hi - lo
        x = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen(hi), device=dev).to(BF)
        q, k, v = (y.view(T, -1, D) for y in x.split([Hq * D, Hkv * D, Hkv * D], 1))
        pos = torch.arange(lo, hi, device=dev)
        slots = bt[0].long()[pos // 16] * 16 + pos % 16
        qo = torch.empty(T, Hq, D, dtype=BF, device=dev)
        ops.xs_qk_norm_rope_append(qo, q, k, v, w[0], w[1], 1e-6, tab, pos.to(torch.int32), kc, vc, slots,
                                   err_flag=err)
        ko = torch.empty(T, Hkv, D, dtype=BF, device=dev)
        ops.xs_qk_norm_rope(torch.empty_like(qo), ko, q, k, w[0], w[1], 1e-6, tab, pos.to(torch.int32))
        remember(0, ko, v)
        pages = -(-hi // 16)
        kp, vp = (torch.empty(pages, Hkv, 16, D, dtype=BF, device=dev) for _ in range(2))
        ops.xs_kv4_unpack(kp, vp, kc, vc, bt[0, :pages].contiguous(), err_flag=err)
        out = torch.empty_like(qo)
        ops.xs_paged_prefill_tc(out, qo, kp, vp, torch.arange(pages, dtype=torch.int32, device=dev), lo, scale,
                                err_flag=err)
        kv = [torch.stack(r[0]).to(BF).double().transpose(0, 1) for r in (k_rows, v_rows)]
        x = qo.double().transpose(0, 1).view(Hkv, Hq // Hkv, T, D) @ kv[0].transpose(1, 2)[:, None] * scale
        x = x.masked_fill(torch.arange(hi, device=dev) > pos[:, None], -math.inf)
        p = torch.softmax(x, -1)
        ref = (p @ kv[1][:, None]).view(Hq, T, D).transpose(0, 1)
        mag = (p @ kv[1].abs()[:, None]).view(Hq, T, D).transpose(0, 1)
        plain.check(out, ref, 2.0 ** -7 * mag + 2.0 ** -8 * ref.abs(), "prompt")  # weights and output in bf16

    step = Kv4DecodeStep(B, Hq, Hkv, D, dev)
    lens = torch.tensor([n0, 0, 0], dtype=torch.int32, device=dev)
    for i in range(20):
        lens += torch.tensor([1, 1, int(i >= 7)], dtype=torch.int32, device=dev)
        x = torch.randn(B, (Hq + 2 * Hkv) * D, generator=gen(900 + i), device=dev).to(BF)
        q, k, v = (y.view(B, -1, D) for y in x.split([Hq * D, Hkv * D, Hkv * D], 1))
        out = torch.empty(B, Hq, D, dtype=BF, device=dev)
        step.run(out, q, k, v, w[0], w[1], tab, kc, vc, bt, lens, scale)
        ko, qo = torch.empty(B, Hkv, D, dtype=BF, device=dev), torch.zeros(B, Hq, D, dtype=BF, device=dev)
        ops.xs_qk_norm_rope(qo, ko, q, k, w[0], w[1], 1e-6, tab, lens - 1)
        for b in range(B):
            if int(lens[b]) > 0:
                remember(b, ko[b:b + 1], v[b:b + 1])
        ref, bound = plain.attend(qo, lambda b: torch.stack(k_rows[b]), lambda b: torch.stack(v_rows[b]),
                                  lens.tolist(), scale)
        plain.check(out, ref, bound, f"step {i}")
    assert step.error_flags() == 0 and int(err) == 0
