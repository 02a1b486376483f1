"""What the norm + rotation, 4-bit cache and shared-page calls refuse on the
host: before any CUDA call, so these run without a GPU."""
import pytest
import torch

from paged_kv_cache_xs_gb300 import build as xsbuild
from paged_kv_cache_xs_gb300 import ops

A = 1 << 20          # a non-null, aligned address that nothing touches
OK, NULL, SHAPE, DTYPE, ALIGN, UNSUP, WORKSPACE = 0, -1, -2, -3, -4, -5, -6


@pytest.fixture(scope="module")
def lib():
    xsbuild.build()
    return ops.load()


def caller(lib, name, order, **defaults):
    def call(**kw):
        assert set(kw) <= set(order)
        args = {**defaults, **kw}
        return getattr(lib, name)(*[args[n] for n in order])
    return call


ROPE = dict(q_out=A, k_out=A, q=A, q_stride=1024, k=A, k_stride=256, qw=A, kw=A, eps=1e-6, cs=A,
            max_pos=64, rot=128, positions=A, T=0, Hq=8, Hkv=2, D=128, flags=0, dtype=1, err=None,
            stream=None)


def test_norm_rope(lib):
    order = list(ROPE)
    f = caller(lib, "xs_qk_norm_rope", order, **ROPE)
    assert f() == OK                                     # T = 0: nothing is launched
    assert f(qw=None, kw=None) == OK and f(cs=None, positions=None, rot=0) == OK
    for n in ("q_out", "k_out", "q", "k", "cs", "positions"):
        assert f(**{n: None}) == NULL, n
    for kw in (dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(rot=-16), dict(rot=144),
               dict(max_pos=-1), dict(q_stride=1016), dict(k_stride=248), dict(q_stride=-1024)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(D=96, rot=96), dict(rot=8), dict(flags=2), dict(flags=4)):
        assert f(**kw) == UNSUP, kw
    assert f(dtype=2) == DTYPE
    for kw in (dict(q=A + 8), dict(k=A + 2), dict(q_out=A + 8), dict(k_out=A + 8), dict(qw=A + 2),
               dict(kw=A + 2), dict(cs=A + 4), dict(q_stride=1028), dict(k_stride=260)):
        assert f(**kw) == ALIGN, kw


APPEND = dict(q_out=A, q=A, q_stride=1024, k=A, k_stride=256, v=A, v_stride=256, qw=A, kw=A, eps=1e-6,
              cs=A, max_pos=64, rot=128, positions=A, kc=A, vc=A, slots=A, T=0, Hq=8, Hkv=2, D=128,
              bs=16, nb=4, flags=0, dtype=1, err=None, stream=None)


def test_norm_rope_append(lib):
    f = caller(lib, "xs_qk_norm_rope_append", list(APPEND), **APPEND)
    assert f() == OK and f(flags=1) == OK and f(flags=2) == OK and f(flags=3) == OK
    for n in ("q_out", "q", "k", "v", "kc", "vc", "slots", "cs", "positions"):
        assert f(**{n: None}) == NULL, n
    assert f(bs=32) == UNSUP and f(flags=4) == UNSUP and f(flags=2, dtype=0) == UNSUP
    assert f(nb=-1) == SHAPE and f(bs=0) == SHAPE and f(v_stride=128) == SHAPE
    assert f(kc=A + 8) == ALIGN and f(v=A + 8) == ALIGN and f(v_stride=257) == ALIGN


def test_norm_rope_append_paged(lib):
    order = ["q_out", "q", "q_stride", "k", "k_stride", "v", "v_stride", "qw", "kw", "eps", "cs", "max_pos",
             "rot", "kc", "vc", "bt", "maxb", "lens", "B", "Hq", "Hkv", "D", "bs", "nb", "flags", "dtype",
             "err", "stream"]
    f = caller(lib, "xs_qk_norm_rope_append_paged", order, **{**APPEND, "bt": A, "maxb": 4, "lens": A, "B": 0})
    assert f() == OK
    assert f(bt=None) == NULL and f(lens=None) == NULL and f(cs=None) == NULL
    assert f(maxb=-1) == SHAPE and f(B=-1) == SHAPE


def test_kv4(lib):
    assert lib.xs_kv4_page_bytes(128) == 1152 and lib.xs_kv4_page_bytes(64) == 576
    assert lib.xs_kv4_page_bytes(96) == UNSUP
    order = ["k", "ks", "v", "vs", "kc", "vc", "slots", "T", "Hkv", "D", "bs", "nb", "dtype", "err", "stream"]
    d = dict(k=A, ks=256, v=A, vs=256, kc=A, vc=A, slots=A, T=0, Hkv=2, D=128, bs=16, nb=4, dtype=1, err=None,
             stream=None)
    f = caller(lib, "xs_kv4_append", order, **d)
    assert f() == OK
    for n in ("k", "v", "kc", "vc", "slots"):
        assert f(**{n: None}) == NULL, n
    assert f(dtype=0) == UNSUP and f(dtype=7) == DTYPE and f(D=32) == UNSUP and f(ks=128) == SHAPE
    order = order[:6] + ["bt", "maxb", "lens", "B"] + order[8:]
    f = caller(lib, "xs_kv4_append_paged", order, **{**d, "bt": A, "maxb": 3, "lens": A, "B": 0})
    assert f() == OK and f(bt=None) == NULL and f(B=-2) == SHAPE and f(bs=8) == UNSUP
    order = ["ko", "vo", "kc", "vc", "ids", "n", "Hkv", "D", "bs", "nb", "dtype", "err", "stream"]
    f = caller(lib, "xs_kv4_unpack", order, **{**d, "ko": A, "vo": A, "ids": A, "n": 0})
    assert f() == OK and f(dtype=0) == OK
    for n in ("ko", "vo", "kc", "vc", "ids"):
        assert f(**{n: None}) == NULL, n
    assert f(n=-1) == SHAPE and f(D=256) == UNSUP and f(ko=A + 4) == ALIGN and f(dtype=3) == DTYPE


def test_kv4_decode(lib):
    order = ["out", "q", "kc", "vc", "bt", "maxb", "lens", "sinks", "window", "B", "Hq", "Hkv", "D", "bs", "nb",
             "scale", "ws", "wsb", "dtype", "err", "stream"]
    d = dict(out=A, q=A, kc=A, vc=A, bt=A, maxb=4, lens=A, sinks=None, window=0, B=0, Hq=8, Hkv=2, D=128, bs=16,
             nb=4, scale=0.1, ws=A, wsb=1 << 40, dtype=1, err=None, stream=None)
    f = caller(lib, "xs_kv4_decode", order, **d)
    assert f() == OK
    for n in ("out", "q", "kc", "vc", "bt", "lens"):
        assert f(**{n: None}) == NULL, n
    for kw in (dict(B=-1), dict(Hq=7), dict(Hkv=0), dict(window=-1), dict(maxb=-1), dict(nb=-1), dict(B=1, nb=0)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(dtype=0), dict(D=32), dict(Hq=6), dict(Hq=32), dict(bs=32)):
        assert f(**kw) == UNSUP, kw
    assert f(dtype=9) == DTYPE and f(ws=A + 4) == ALIGN and f(q=A + 2) == ALIGN
    assert f(B=1, ws=None) == WORKSPACE and f(B=1, wsb=16) == WORKSPACE
    assert ops.load().xs_kv4_decode_workspace_bytes(0, 8, 2, 128) == 0


def test_shared_pages(lib):
    order = ["parents", "children", "n", "bt", "maxb", "lens", "B", "bs", "stack", "top", "extra", "nb", "copies",
             "err", "stream"]
    d = dict(parents=A, children=A, n=0, bt=A, maxb=4, lens=A, B=2, bs=16, stack=A, top=A, extra=A, nb=9, copies=A,
             err=None, stream=None)
    f = caller(lib, "xs_block_fork", order, **d)
    assert f() == OK
    for n in ("parents", "children", "bt", "lens", "stack", "top", "extra", "copies"):
        assert f(**{n: None}) == NULL, n
    for kw in (dict(n=-1), dict(B=-1), dict(maxb=-1), dict(bs=0), dict(nb=-1), dict(nb=1 << 31)):
        assert f(**kw) == SHAPE, kw
    order = ["ids", "n", "bt", "maxb", "lens", "B", "bs", "stack", "top", "cap", "extra", "nb", "err", "stream"]
    f = caller(lib, "xs_block_release", order, **{**d, "ids": A, "cap": 9})
    assert f() == OK and f(ids=None) == NULL and f(extra=None) == NULL and f(cap=-1) == SHAPE and f(n=-1) == SHAPE
    order = ["bt", "bto", "maxb", "lens", "B", "bs", "extra", "eo", "stack", "top", "nb", "remap", "moves", "nm",
             "err", "stream"]
    f = caller(lib, "xs_block_compact", order, **{**d, "bto": A, "eo": A, "remap": A, "moves": A, "nm": A})
    for n in ("bt", "bto", "lens", "extra", "eo", "stack", "top", "remap", "moves", "nm"):
        assert f(**{n: None}) == NULL, n
    assert f(nb=-1) == SHAPE and f(B=-1) == SHAPE and f(bs=0) == SHAPE
    order = ["k", "v", "layers", "stride", "pairs", "n", "count", "bytes", "nb", "err", "stream"]
    f = caller(lib, "xs_block_copy", order, k=A, v=A, layers=2, stride=9 * 64, pairs=A, n=0, count=None, bytes=64,
               nb=9, err=None, stream=None)
    assert f() == OK and f(n=1, layers=0) == OK
    for n in ("k", "v", "pairs"):
        assert f(**{n: None}) == NULL, n
    for kw in (dict(n=-1), dict(layers=-1), dict(bytes=0), dict(nb=-1), dict(stride=512), dict(nb=1 << 62)):
        assert f(**kw) == SHAPE, kw
    assert f(bytes=24, nb=1) == UNSUP and f(stride=9 * 64 + 8) == UNSUP and f(k=A + 8) == ALIGN


# ---------------------------------------------------------------- the binding's own checks

def meta(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses(lib):
    q, k, w = meta(4, 8, 128), meta(4, 2, 128), meta(128)
    cs, pos = meta(64, 128, dtype=torch.float32), meta(4, dtype=torch.int32)
    good = dict(q_out=q, k_out=k, q=q, k=k, q_weight=w, k_weight=w, eps=1e-6, cos_sin=cs, positions=pos)
    with pytest.raises(ValueError, match="CUDA"):
        ops.xs_qk_norm_rope(**good)                     # nothing runs on the CPU
    for bad in (dict(q_out=meta(4, 8, 64)), dict(k=meta(3, 2, 128)), dict(k=meta(4, 2, 128, dtype=torch.float32)),
                dict(q_weight=meta(64)), dict(positions=meta(4, dtype=torch.int64)), dict(k_out=q),
                dict(cos_sin=meta(64, 128)), dict(k_weight=meta(128, dtype=torch.float32))):
        with pytest.raises(ValueError):
            ops.xs_qk_norm_rope(**{**good, **bad})
    # Slices of a projection are taken (and refused only for being on the CPU);
    # rows whose heads are apart are not.
    with pytest.raises(ValueError, match="CUDA"):
        ops.xs_qk_norm_rope(**{**good, "q": meta(4, 10, 128)[:, :8]})
    for odd in (meta(4, 128, 8).transpose(1, 2), meta(4, 8, 256)[..., :128], meta(4, 16, 128)[:, ::2]):
        with pytest.raises(ValueError, match="contiguous"):
            ops.xs_qk_norm_rope(**{**good, "q": odd})
    with pytest.raises(ValueError, match="tensor"):
        ops.xs_qk_norm_rope(**{**good, "k": None})
    slots = meta(4, dtype=torch.int64)
    app = dict(q_out=q, q=q, k=k, v=k, q_weight=w, k_weight=w, eps=1e-6, cos_sin=cs, positions=pos,
               slot_mapping=slots)
    for kc in (meta(9, 2, 16, 64), meta(9, 3, 16, 128), meta(9, 2, 16, 128, dtype=torch.float32),
               meta(9, 2, 1024, dtype=torch.uint8), meta(9, 2, 16, 144, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="pool"):
            ops.xs_qk_norm_rope_append(**app, k_cache=kc, v_cache=kc)
    for kc in (meta(9, 2, 16, 128), meta(9, 2, 1152, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="CUDA"):
            ops.xs_qk_norm_rope_append(**app, k_cache=kc, v_cache=kc)
    kc = meta(9, 2, 1152, dtype=torch.uint8)
    bt, lens = meta(4, 3, dtype=torch.int32), meta(4, dtype=torch.int32)
    ws = ops.Kv4Workspace(4, 8, 2, 128, "cpu")
    with pytest.raises(ValueError, match="workspace"):
        ops.xs_kv4_decode(meta(5, 8, 128), meta(5, 8, 128), kc, kc, meta(5, 3, dtype=torch.int32),
                          meta(5, dtype=torch.int32), 0.1, ws)
    with pytest.raises(ValueError):
        ops.xs_kv4_decode(q, q, kc, kc, bt[:3], lens, 0.1, ws)
    with pytest.raises(ValueError, match="CUDA"):
        ops.xs_kv4_decode(q, q, kc, kc, bt, lens, 0.1, ws)
    with pytest.raises(ValueError):
        ops.xs_kv4_append(k, k, meta(9, 2, 16, 128), meta(9, 2, 16, 128), meta(4, dtype=torch.int64))
    i = meta(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.xs_block_fork(i, i[:3], bt, lens, i, i[:1], i, meta(4, 2, dtype=torch.int64))
    with pytest.raises(ValueError):
        ops.xs_block_release(i.long(), bt, lens, i, i[:1], i)
    with pytest.raises(ValueError):
        ops.xs_block_copy(kc, kc, meta(4, 2, dtype=torch.int32))


def test_rope_table():
    t = ops.rope_table(100000, 8, 1e4, "cpu")
    assert t.shape == (100000, 8) and t.dtype == torch.float32
    a = 99999 * 1e4 ** (-2 / 8)
    assert t[99999, 1] == torch.tensor(a, dtype=torch.float64).cos().float()
    assert t[99999, 5] == torch.tensor(a, dtype=torch.float64).sin().float()
    assert bool((t[0] == torch.tensor([1.0] * 4 + [0.0] * 4)).all())


def test_bench_finds_the_counters_of_its_kernel():
    # The committed counters belong to the decode kernel's source as it is.
    import bench

    for workload in ("qwen3_8b_long_batch", "qwen3_8b_cb_mix", "qwen3_8b_single_stream", "gpt2_bf16_12layer"):
        assert bench.kernel_traffic(workload) is not None, workload
