"""What the bounded caches' calls refuse on the host, before any CUDA call."""
import pytest
import torch

from paged_kv_cache_xs_gb300 import build as xsbuild
from paged_kv_cache_xs_gb300 import ops
from paged_kv_cache_xs_gb300.step import BoundedDecodeStep
from tests import plain_bounded as plain
from tests.test_operator_refusals import ALIGN, DTYPE, NULL, OK, SHAPE, UNSUP, WORKSPACE, A, caller, meta

I32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    xsbuild.build()
    return ops.load()


DECODE = dict(out=A, q=A, qs=1024, kc=A, vc=A, bt=A, maxb=4, lens=A, sinks=None, first=4, window=8, B=0, Hq=8, Hkv=2,
              D=128, bs=16, nb=4, scale=0.1, ws=A, wsb=1 << 40, dtype=1, err=None, stream=None)


def refusals_of_decode(f):
    assert f() == OK and f(dtype=0) == OK               # B = 0: nothing is launched
    for n in ("out", "q", "kc", "vc", "bt", "lens"):
        assert f(**{n: None}) == NULL, n
    for kw in (dict(B=-1), dict(Hq=7), dict(Hkv=0), dict(maxb=-1), dict(nb=-1), dict(B=1, nb=0), dict(qs=1016), dict(D=0)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(D=32, qs=256), dict(Hq=6), dict(Hq=32, qs=4096), dict(bs=32), dict(qs=1028), dict(nb=1 << 31),
               dict(maxb=(1 << 26) + 1), dict(B=1 << 30)):
        assert f(**kw) == UNSUP, kw
    assert f(dtype=9) == DTYPE
    for n in ("out", "q", "kc", "vc", "ws"):
        assert f(**{n: A + 8}) == ALIGN, n
    assert f(B=1, ws=None) == WORKSPACE and f(B=1, wsb=16) == WORKSPACE


def test_decode_first(lib):
    f = caller(lib, "xs_paged_decode_first", list(DECODE), **DECODE)
    refusals_of_decode(f)
    assert f(first=-1) == SHAPE and f(window=-1) == SHAPE
    assert lib.xs_paged_decode_first_workspace_bytes(0, 8, 2, 128) == 0


def test_decode_weights(lib):
    order = ["out", "scores", "scored"] + [n for n in DECODE if n not in ("out", "first", "window")]
    f = caller(lib, "xs_paged_decode_weights", order, **{**DECODE, "scores": A, "scored": None})
    refusals_of_decode(f)
    assert f(scores=None) == NULL
    need = lib.xs_paged_decode_weights_workspace_bytes(2, 8, 2, 128, 4)
    assert need > lib.xs_paged_decode_first_workspace_bytes(2, 8, 2, 128)
    assert f(B=2, wsb=need - 1) == WORKSPACE
    assert lib.xs_paged_decode_weights_workspace_bytes(2, 8, 2, 128, -1) == 0


def test_prefill_first(lib):
    d = dict(out=A, q=A, kc=A, vc=A, ids=A, n=4, T=0, start=0, first=4, window=8, Hq=8, Hkv=2, D=128, bs=16, nb=4, scale=0.1,
             dtype=1, err=None, stream=None)
    f = caller(lib, "xs_paged_prefill_first", list(d), **d)
    assert f() == OK
    for n in ("out", "q", "kc", "vc", "ids"):
        assert f(**{n: None}) == NULL, n
    for kw in (dict(T=-1), dict(start=-1), dict(first=-1), dict(window=-1), dict(Hq=7), dict(T=65), dict(start=64, T=1)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(dtype=0), dict(D=32), dict(Hq=6), dict(bs=8), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan"))):
        assert f(**kw) == UNSUP, kw
    assert f(dtype=5) == DTYPE and f(q=A + 8) == ALIGN
    assert f(n=1 << 27, start=(1 << 31) - 512) == UNSUP and f(n=1 << 27, start=(1 << 31) - 513) == OK


def test_evict(lib):
    d = dict(ids=A, n=0, k=A, v=A, layers=2, stride=4 * 2 * 16 * 256, scores=A, bt=A, maxb=4, lens=A, B=3, extra=None, first=4,
             recent=8, budget=16, limit=20, Hkv=2, D=128, bs=16, nb=4, dtype=1, kept=A, new=A, err=None, stream=None)
    f = caller(lib, "xs_kv_evict", list(d), **d)
    assert f() == OK                                    # n = 0: nothing is launched
    for n in ("ids", "k", "v", "scores", "bt", "lens", "kept", "new"):
        assert f(**{n: None}) == NULL, n
    for kw in (dict(n=-1), dict(layers=0), dict(layers=-1), dict(B=-1), dict(Hkv=0), dict(first=-1), dict(recent=-1), dict(budget=0),
               dict(limit=15), dict(first=9), dict(nb=-1), dict(nb=5), dict(maxb=-1), dict(first=1 << 30, recent=(1 << 31) - 1)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(D=32), dict(bs=8), dict(stride=4 * 2 * 16 * 256 + 8), dict(n=1 << 30), dict(maxb=(1 << 26) + 1)):
        assert f(**kw) == UNSUP, kw
    assert f(dtype=2) == DTYPE and f(k=A + 8) == ALIGN


def test_truncate(lib):
    d = dict(ids=A, new=A, n=0, bt=A, maxb=4, lens=A, B=2, bs=16, stack=A, top=A, cap=9, extra=A, nb=9, err=None, stream=None)
    f = caller(lib, "xs_block_truncate", list(d), **d)
    assert f() == OK
    for n in ("ids", "new", "bt", "lens", "stack", "top", "extra"):
        assert f(**{n: None}) == NULL, n
    for kw in (dict(n=-1), dict(B=-1), dict(maxb=-1), dict(bs=0), dict(cap=-1), dict(nb=-1), dict(nb=1 << 31)):
        assert f(**kw) == SHAPE, kw


def test_binding_refuses(lib):
    q, kc, kv4 = meta(4, 8, 128), meta(9, 2, 16, 128), meta(9, 2, 1152, dtype=torch.uint8)
    bt, lens = meta(4, 3, dtype=I32), meta(4, dtype=I32)
    ws, scores = ops.BoundedWorkspace(4, 8, 2, 128, "cpu", 3), meta(4, 2, 48, dtype=torch.float32)
    first = dict(out=q, q=q, k_cache=kc, v_cache=kc, block_tables=bt, context_lens=lens, scale=0.1, workspace=ws)
    weights = {**first, "scores": scores}
    for f, good in ((ops.xs_paged_decode_first, first), (ops.xs_paged_decode_weights, weights)):
        with pytest.raises(ValueError, match="CUDA"):
            f(**good)                                   # nothing runs on the CPU
        with pytest.raises(ValueError, match="CUDA"):
            f(**{**good, "q": meta(4, 12, 128)[:, :8]})
        for bad in (dict(k_cache=kv4, v_cache=kv4), dict(v_cache=meta(9, 2, 16, 64)), dict(block_tables=bt[:3]),
                    dict(context_lens=lens.long()), dict(out=q.float()), dict(sinks=meta(7)), dict(q=meta(4, 16, 128)[:, ::2]),
                    dict(workspace=ops.BoundedWorkspace(4, 8, 4, 128, "cpu"))):
            with pytest.raises(ValueError):
                f(**{**good, **bad})
    for bad in (dict(scores=scores[..., :32]), dict(scores=scores.double()), dict(scored_lens=lens.long())):
        with pytest.raises(ValueError):
            ops.xs_paged_decode_weights(**{**weights, **bad})
    ids = meta(5, dtype=I32)
    good = dict(out=q, q=q, k_cache=kc, v_cache=kc, block_ids=ids, start_pos=3, scale=0.1, first=1, window=3)
    with pytest.raises(ValueError, match="CUDA"):
        ops.xs_paged_prefill_first(**good)
    for bad in (dict(block_ids=ids.long()), dict(out=meta(4, 8, 64)), dict(k_cache=kv4, v_cache=kv4), dict(window=1 << 40)):
        with pytest.raises(ValueError):
            ops.xs_paged_prefill_first(**{**good, **bad})
    pools = meta(2, 9, 2, 16, 128)
    good = dict(seq_ids=meta(3, dtype=I32), k_pools=pools, v_pools=pools, scores=meta(2, 4, 2, 48, dtype=torch.float32),
                block_tables=bt, context_lens=lens, kept=meta(2, 3, 2, 16, dtype=I32), new_lens=meta(3, dtype=I32), first=1,
                recent=2, limit=20)
    with pytest.raises(ValueError, match="CUDA"):
        ops.xs_kv_evict(**good)
    for bad in (dict(k_pools=pools[0]), dict(v_pools=pools.float()), dict(kept=meta(2, 4, 2, 16, dtype=I32)),
                dict(new_lens=meta(4, dtype=I32)), dict(scores=meta(4, 2, 48, dtype=torch.float32)),
                dict(extra_refs=meta(8, dtype=I32))):
        with pytest.raises(ValueError):
            ops.xs_kv_evict(**{**good, **bad})
    i = meta(4, dtype=I32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.xs_block_truncate(i, i, bt, lens, i, i[:1], i)
    with pytest.raises(ValueError):
        ops.xs_block_truncate(i, i[:3], bt, lens, i, i[:1], i)


def test_step_refuses_budgets():
    for kw in (dict(budget=0), dict(budget=10, limit=9), dict(budget=10, recent=11), dict(budget=10, first=4, recent=7)):
        with pytest.raises(ValueError):
            BoundedDecodeStep(1, 2, 2, 64, 4, 1, torch.bfloat16, "cpu", **kw)


def test_plain_forms():
    assert plain.seen_by(10, 2, 3) == [0, 1, 7, 8, 9] and plain.seen_by(3, 5, 1) == [0, 1, 2]
    assert plain.seen_by(4, 0, 0) == [0, 1, 2, 3] and plain.seen_by(0, 3, 3) == []
    s = [9.0, 1.0, 5.0, float("nan"), 5.0, 5.0, -float("inf"), 0.0]
    assert plain.keep(s, 8, 1, 1, 4) == [0, 2, 4, 7] and plain.keep(s, 7, 0, 0, 6) == [0, 1, 2, 3, 4, 5]
    # Weights: of a uniform query, 1 / n each; the output their mean.
    q, k, v = torch.zeros(2, 8), torch.randn(5, 1, 8), torch.randn(5, 1, 8)
    o, p, _, _ = plain.attend(q, k, v, 1.0)
    assert torch.allclose(p, torch.full((2, 5), 0.2, dtype=torch.float64)) and torch.allclose(o[0], v[:, 0].double().mean(0))
