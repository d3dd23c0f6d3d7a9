"""Refusals of the cache-side operators, on the host before any CUDA call."""
import ctypes

import pytest
import torch

from paged_kv_cache_230_gb300 import build


@pytest.fixture(scope="module")
def pa():
    build.build()
    from paged_kv_cache_230_gb300 import pagedattn
    return pagedattn


F = ctypes.c_void_p(0x100000)  # never dereferenced
ODD = ctypes.c_void_p(0x100008)
N = ctypes.c_void_p(0)
nan, inf = float("nan"), float("inf")


def desc(pa, NB=4, bs=16, Hkv=2, D=128, dt=2):
    return ctypes.byref(pa.CacheDesc(NB, bs, Hkv, D, dt))


def test_reshape_and_cache_rows_refusals(pa):
    f = pa.lib.pa_reshape_and_cache_rows
    d = desc(pa)
    assert f(F, F, 1, 0, F, F, F, F, d, N, N) == 0  # nothing to do
    assert f(N, F, 1, 1, F, F, F, F, d, F, N) == -1
    assert f(ODD, F, 1, 1, F, F, F, F, d, F, N) == -1
    assert f(F, F, 1, -1, F, F, F, F, d, F, N) == -1
    assert f(F, F, 2, 1, F, F, F, F, d, F, N) == -2
    assert f(F, F, 1, 1, F, F, N, F, d, F, N) == -1
    assert f(F, F, 1, 1, F, F, F, ODD, d, F, N) == -1
    for bad in (desc(pa, dt=1), desc(pa, D=96), desc(pa, bs=12)):
        assert f(F, F, 1, 1, F, F, F, F, bad, F, N) == -2


def test_gather_blocks_rows_refusals(pa):
    f = pa.lib.pa_gather_blocks_rows
    d = desc(pa)
    assert f(F, F, 1, F, F, F, F, d, F, 0, N) == 0
    assert f(F, F, 2, F, F, F, F, d, F, 1, N) == -2
    assert f(N, F, 1, F, F, F, F, d, F, 1, N) == -1
    assert f(F, ODD, 1, F, F, F, F, d, F, 1, N) == -1
    assert f(F, F, 1, F, F, F, F, d, F, -1, N) == -1
    assert f(F, F, 1, F, F, F, F, desc(pa, dt=0), F, 1, N) == -2


def test_block_scales_refusals(pa):
    d, bad = desc(pa), desc(pa, dt=1)
    copy, gather, scatter = pa.lib.pa_copy_block_scales, pa.lib.pa_gather_block_scales, pa.lib.pa_scatter_block_scales
    assert copy(F, F, d, N, 0, N) == 0 and gather(N, F, F, d, N, 0, N) == 0 and scatter(F, F, d, N, N, 0, N) == 0
    assert copy(F, F, bad, F, 1, N) == -2 and gather(F, F, F, bad, F, 1, N) == -2 and scatter(F, F, bad, F, F, 1, N) == -2
    assert copy(N, F, d, F, 1, N) == -1 and copy(F, ODD, d, F, 1, N) == -1 and copy(F, F, d, F, -1, N) == -1
    assert gather(ODD, F, F, d, F, 1, N) == -1 and gather(F, F, F, d, N, 1, N) == -1
    assert scatter(F, F, d, N, F, 1, N) == -1 and scatter(F, F, None, F, F, 1, N) == -1


def test_decode_rows_refusals(pa):
    f = pa.lib.pa_decode_rows

    def call(out=F, q=F, qd=1, S=1, k=1, Hq=4, kc=F, ks=F, d=None, bt=F, maxB=4, cl=F, scale=0.1, most=64, P=0, ws=N, nws=0):
        return f(out, q, qd, S, k, Hq, kc, F, ks, F, d or desc(pa), bt, maxB, cl, scale, most, P, ws, nws, N)

    assert call(S=0, out=N, q=N, bt=N, cl=N) == 0
    assert call(kc=N) == -1 and call(ks=N) == -1 and call(ks=ODD) == -1 and call(out=ODD) == -1 and call(q=N) == -1
    assert call(bt=N) == -1 and call(cl=N) == -1
    assert call(d=desc(pa, dt=1)) == -2 and call(qd=2) == -2 and call(d=desc(pa, D=32)) == -2
    assert call(Hq=5) == -1 and call(Hq=0) == -1 and call(k=0) == -1 and call(maxB=0) == -1 and call(S=-1) == -1
    assert call(k=17) == -2 and call(Hq=2 * 129) == -2
    assert call(scale=nan) == -1 and call(scale=inf) == -1
    assert call(P=100) == -1 and call(P=-64) == -1 and call(P=64, most=-1) == -1
    assert call(P=64) == -3 and call(P=64, ws=F, nws=16) == -3
    need = pa.decode_multi_split_workspace_size(1, 1, 4, 128, 64, 64)
    assert call(P=64, ws=ODD, nws=need) == -3
    assert call(maxB=1 << 30) == -1


def test_norm_rope_cache_refusals(pa):
    f = pa.lib.pa_norm_rope_cache
    far = lambda i: ctypes.c_void_p(0x10000000 * (i + 1))  # noqa: E731

    def call(out=far(0), q=far(1), qs=512, key=far(2), ks=256, val=far(3), vs=256, dt=1, T=2, Hq=4, qw=F, kw=F, eps=1e-6,
             pos=F, tab=F, P=10, rot=128, inter=0, ksc=N, vsc=N, d=None, slots=F, kvs=1.0):
        return f(out, q, qs, key, ks, val, vs, dt, T, Hq, qw, kw, eps, pos, tab, P, rot, inter, F, F, ksc, vsc,
                 d or desc(pa, dt=1), slots, kvs, N)

    assert call(T=0, slots=N) == 0
    assert call(T=-1) == -1 and call(Hq=0) == -1 and call(q=N) == -1 and call(slots=N) == -1 and call(key=ODD) == -1
    assert call(qs=516) == -1 and call(ks=-8) == -1 and call(vs=3) == -1 and call(qs=1 << 31) == -1
    assert call(qw=N) == -1 and call(kw=N) == -1 and call(qw=ODD) == -1
    assert call(eps=-1.0) == -1 and call(eps=nan) == -1
    assert call(rot=130) == -1 and call(rot=-2) == -1 and call(rot=7, inter=1) == -1 and call(inter=2) == -1
    assert call(rot=20) == -2  # pairs a half apart: multiples of 8
    assert call(pos=N) == -1 and call(tab=N) == -1 and call(P=0) == -1
    assert call(dt=2) == -2 and call(dt=0) == -2 and call(d=desc(pa, dt=1, D=80)) == -2
    assert call(kvs=0.5) == -1
    d8 = desc(pa, dt=2)
    assert call(d=d8, kvs=0.0) == -1 and call(d=d8, kvs=inf) == -1
    assert call(d=d8, ksc=F, vsc=N) == -1 and call(d=d8, ksc=F, vsc=F, kvs=0.5) == -1
    assert call(ksc=F, vsc=F) == -2  # row scales with a 16-bit cache
    # q_out over q (but not q itself, contiguous), key or value
    assert call(out=far(1), qs=1024) == -1
    assert call(out=ctypes.c_void_p(far(1).value + 16)) == -1
    assert call(out=far(2)) == -1 and call(out=ctypes.c_void_p(far(3).value - 16)) == -1


def test_block_choice_refusals(pa):
    d = desc(pa, dt=1)
    f = pa.lib.pa_block_bounds
    assert f(N, F, d, N, 4, N, 0, 1, N) == 0
    assert f(N, F, d, F, 4, F, 1, 1, N) == -1 and f(ODD, F, d, F, 4, F, 1, 1, N) == -1
    assert f(F, F, d, F, 4, F, 1, 0, N) == -1 and f(F, F, d, F, 0, F, 1, 1, N) == -1 and f(F, F, d, F, 4, F, -1, 1, N) == -1
    assert f(F, F, d, F, 1 << 26, F, 1 << 10, 2 ** 31 - 1, N) == -1  # 2^36 blocks touched
    assert f(F, N, d, F, 4, F, 1, 1, N) == -1 and f(F, F, desc(pa, D=96), F, 4, F, 1, 1, N) == -2
    f = pa.lib.pa_block_scores
    assert f(N, N, 1, 0, 4, F, d, N, 4, N, N) == 0
    assert f(F, F, 0, 1, 4, F, d, F, 4, F, N) == -2 and f(F, F, 1, 1, 5, F, d, F, 4, F, N) == -1
    assert f(F, F, 1, 1, 2 * 129, F, d, F, 4, F, N) == -2 and f(N, F, 1, 1, 4, F, d, F, 4, F, N) == -1
    assert f(F, F, 1, 1 << 20, 4, F, d, F, 1 << 20, F, N) == -1  # 2^41 scores
    assert f(F, ODD, 1, 1, 4, F, d, F, 4, F, N) == -1 and f(F, F, 1, 1, 4, N, d, F, 4, F, N) == -1
    f = pa.lib.pa_select_blocks
    assert f(N, N, 4, N, N, 4, N, 0, 2, 16, 1, 1, N) == 0
    assert f(F, F, 0, F, F, 4, F, 1, 2, 16, 0, 0, N) == -1 and f(F, F, 4, F, F, 4, F, 1, 2, 16, 3, 2, N) == -1
    assert f(F, F, 4, F, F, 4, F, 1, 2, 16, -1, 2, N) == -1 and f(F, F, 4, F, F, 4, F, 1, 0, 16, 1, 1, N) == -1
    assert f(F, F, 4, F, F, 4, F, 1, 2, 12, 1, 1, N) == -2 and f(N, F, 4, F, F, 4, F, 1, 2, 16, 1, 1, N) == -1
    assert f(F, F, 4, F, F, 4, F, 1, 2, 16, 2 ** 31 - 1, 2 ** 31 - 1, N) == -1
    assert f(F, F, 1 << 30, F, F, 4, F, 1, 2, 16, 1, 1, N) == -1


def test_decode_selected_refusals(pa):
    f = pa.lib.pa_decode_selected

    def call(out=F, q=F, qd=1, S=1, Hq=4, kc=F, d=None, tab=F, n=4, lens=F, scale=0.1, kvs=1.0, P=0, ws=N, nws=0):
        return f(out, q, qd, S, Hq, kc, F, d or desc(pa, dt=1), tab, n, lens, scale, kvs, P, ws, nws, N)

    assert call(S=0, out=N, q=N, tab=N, lens=N) == 0
    assert call(kc=N) == -1 and call(tab=N) == -1 and call(lens=N) == -1 and call(q=ODD) == -1
    assert call(n=0) == -1 and call(n=1 << 30) == -1 and call(Hq=3) == -1
    assert call(qd=0) == -2 and call(Hq=2 * 129) == -2 and call(kvs=2.0) == -1 and call(d=desc(pa), kvs=nan) == -1
    assert call(scale=nan) == -1 and call(P=32) == -1 and call(P=64) == -3


def test_binding_refusals(pa):
    """Tensors of the wrong place, type or shape, before the library is called."""
    t = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    i32, i64 = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    s = torch.ones(4, 2, 16)
    with pytest.raises(ValueError):
        pa.reshape_and_cache_rows(t, t, t, t, s, s, i64)
    with pytest.raises(ValueError):
        pa.gather_blocks_rows(t, t, t, t, s, s, i64)
    with pytest.raises(ValueError):
        pa.decode_rows(t, t, t, t, s, s, i32, i32[:, 0], 1.0)
    with pytest.raises(ValueError):
        pa.norm_rope_cache(t, t, t, t, i64, None, t, t, i64)
    with pytest.raises(ValueError):
        pa.block_bounds(t, t, i32, i32[:, 0])
    with pytest.raises(ValueError):
        pa.block_scores(s, t, t, i32, i32[:, 0], 16)
    with pytest.raises(ValueError):
        pa.select_blocks(i32, i32, s, i32, i32[:, 0], 16)
    with pytest.raises(ValueError):
        pa.decode_selected(t, t, t, t, i32, i32, 1.0)
