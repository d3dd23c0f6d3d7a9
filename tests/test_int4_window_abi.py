"""4-bit caches and windows on the host: refusals before any CUDA call, and the code layout of the references."""
import ctypes

import pytest
import torch

from paged_kv_cache_230_gb300 import build
from tests import _ref_stream as R


@pytest.fixture(scope="module")
def pa():
    build.build()
    from paged_kv_cache_230_gb300 import pagedattn
    return pagedattn


F = ctypes.c_void_p(0x100000)  # never dereferenced
ODD = ctypes.c_void_p(0x100008)
N = ctypes.c_void_p(0)
nan, inf = float("nan"), float("inf")
BIG = 1 << 40


def desc(pa, NB=4, bs=16, Hkv=2, D=128, dt=3):
    return ctypes.byref(pa.CacheDesc(NB, bs, Hkv, D, dt))


def test_reshape_and_cache_int4_refusals(pa):
    f = pa.lib.pa_reshape_and_cache_int4
    d = desc(pa)
    assert f(F, F, 1, 0, F, F, F, F, d, N, N) == 0  # nothing to do
    assert f(N, F, 1, 1, F, F, F, F, d, F, N) == -1 and f(ODD, F, 1, 1, F, F, F, F, d, F, N) == -1
    assert f(F, F, 1, -1, F, F, F, F, d, F, N) == -1 and f(F, F, 1, 1, F, F, F, F, d, N, N) == -1
    assert f(F, F, 2, 1, F, F, F, F, d, F, N) == -2 and f(F, F, 3, 1, F, F, F, F, d, F, N) == -2
    assert f(F, F, 1, 1, F, F, N, F, d, F, N) == -1 and f(F, F, 1, 1, F, F, F, ODD, d, F, N) == -1
    assert f(F, F, 1, 1, ODD, F, F, F, d, F, N) == -1 and f(F, F, 1, 1, F, F, F, F, None, F, N) == -1
    for bad in (desc(pa, dt=2), desc(pa, dt=1), desc(pa, D=96), desc(pa, D=32), desc(pa, bs=12)):
        assert f(F, F, 1, 1, F, F, F, F, bad, F, N) == -2


def test_gather_blocks_int4_refusals(pa):
    f = pa.lib.pa_gather_blocks_int4
    d = desc(pa)
    assert f(F, F, 1, F, F, F, F, d, F, 0, N) == 0
    assert f(F, F, 2, F, F, F, F, d, F, 1, N) == -2 and f(F, F, 1, F, F, F, F, desc(pa, dt=2), F, 1, N) == -2
    assert f(N, F, 1, F, F, F, F, d, F, 1, N) == -1 and f(F, ODD, 1, F, F, F, F, d, F, 1, N) == -1
    assert f(F, F, 1, F, F, F, F, d, F, -1, N) == -1 and f(F, F, 1, F, F, N, F, d, F, 1, N) == -1


def test_other_calls_refuse_four_bit_caches(pa):
    d = desc(pa)
    assert pa.lib.pa_decode(F, F, 1, 1, 4, F, F, d, F, 4, F, 0.1, 1.0, N) == -2
    assert pa.lib.pa_reshape_and_cache(F, F, 1, 1, F, F, d, F, 1.0, N) == -2
    assert pa.lib.pa_prefill(F, F, 1, 1, 4, 4, F, F, d, F, 4, F, 0.1, 1.0, N, 0, N) == -2
    assert pa.lib.pa_decode_window(F, F, 1, 1, 1, 4, F, F, d, F, 4, F, 0.1, 1.0, 8, 0, F, BIG, N) == -2
    assert pa.lib.pa_prefill_window(F, F, 1, 1, 4, 4, F, F, d, F, 4, F, 0.1, 1.0, 8, 0, N) == -2


def test_block_moves_take_four_bit_caches(pa):
    for D in (64, 128):
        d = desc(pa, D=D)
        for f in (pa.lib.pa_copy_blocks, pa.lib.pa_copy_block_scales):
            assert f(F, F, d, N, 0, N) == 0 and f(N, F, d, F, 1, N) == -1 and f(F, F, d, F, -1, N) == -1
            assert f(F, F, desc(pa, D=96), F, 1, N) == -2


def test_decode_int4_refusals(pa):
    f = pa.lib.pa_decode_int4

    def call(out=F, q=F, qd=1, S=1, k=1, Hq=4, kc=F, kp=F, d=None, bt=F, maxB=4, cl=F, scale=0.1, win=0, sinks=0, ws=F, nws=BIG):
        return f(out, q, qd, S, k, Hq, kc, F, kp, F, d or desc(pa), bt, maxB, cl, scale, win, sinks, ws, nws, N)

    assert call(S=0, out=N, q=N, bt=N, cl=N, ws=N, nws=0) == 0
    assert call(kc=N) == -1 and call(kc=ODD) == -1 and call(kp=N) == -1 and call(kp=ODD) == -1
    assert call(out=ODD) == -1 and call(q=N) == -1 and call(bt=N) == -1 and call(cl=N) == -1
    assert call(d=desc(pa, dt=2)) == -2 and call(d=desc(pa, D=32)) == -2 and call(qd=2) == -2 and call(qd=3) == -2
    assert call(Hq=5) == -1 and call(Hq=0) == -1 and call(k=0) == -1 and call(maxB=0) == -1 and call(S=-1) == -1
    assert call(k=17) == -2 and call(Hq=2 * 129) == -2
    assert call(scale=nan) == -1 and call(scale=inf) == -1 and call(win=-1) == -1 and call(sinks=-1) == -1
    assert call(maxB=1 << 27) == -1 and call(S=1 << 30) == -1
    assert call(ws=N) == -3 and call(ws=ODD) == -3 and call(nws=16) == -3
    assert call(nws=pa.decode_flat_workspace_size(128) - 1) == -3


def test_decode_window_refusals(pa):
    f = pa.lib.pa_decode_window

    def call(qd=1, S=1, k=1, Hq=4, d=None, maxB=4, scale=0.1, kvs=1.0, win=8, sinks=0, ws=F, nws=BIG, q=F):
        return f(F, q, qd, S, k, Hq, F, F, d or desc(pa, dt=1), F, maxB, F, scale, kvs, win, sinks, ws, nws, N)

    assert call(S=0, ws=N) == 0
    assert call(win=0) == -1 and call(win=-3) == -1 and call(sinks=-1) == -1 and call(q=ODD) == -1
    assert call(qd=0) == -2 and call(d=desc(pa, dt=0)) == -2 and call(qd=2, d=desc(pa, dt=2)) == -2
    assert call(kvs=0.5) == -1 and call(kvs=0.0, d=desc(pa, dt=2)) == -1 and call(kvs=nan, d=desc(pa, dt=2)) == -1
    assert call(k=17) == -2 and call(Hq=2 * 129) == -2 and call(Hq=3) == -1
    assert call(ws=N) == -3 and call(nws=100) == -3


def test_prefill_window_refusals(pa):
    f = pa.lib.pa_prefill_window

    def call(out=F, qd=1, S=1, C=4, Hq=4, d=None, maxB=4, scale=0.1, kvs=1.0, win=8, sinks=0):
        return f(out, F, qd, S, C, Hq, F, F, d or desc(pa, dt=1), F, maxB, F, scale, kvs, win, sinks, N)

    assert call(S=0, out=N) == 0
    assert call(win=0) == -1 and call(sinks=-1) == -1 and call(out=ODD) == -1 and call(out=N) == -1
    assert call(scale=0.0) == -1 and call(scale=-0.1) == -1 and call(scale=nan) == -1 and call(C=0) == -1
    assert call(qd=0) == -2 and call(kvs=0.5) == -1 and call(Hq=2 * 129) == -2 and call(Hq=3) == -1


def test_workspace_size(pa):
    for D in (64, 128):
        n = pa.decode_flat_workspace_size(D)
        assert n > 0 and n % 16 == 0
    assert pa.decode_flat_workspace_size(96) == 0


def test_binding_refuses_tensors_that_do_not_belong(pa):
    t = torch.zeros(2, 2, 16, 64, dtype=torch.uint8)  # not on a GPU
    par = torch.zeros(2, 2, 16, 2, 2, dtype=torch.bfloat16)
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16)
    bt, cl = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.decode_int4(q, q, t, t, par, par, bt, cl, 0.1)
    with pytest.raises(ValueError):
        pa.decode_window(q, q, t, t, bt, cl, 0.1, 4)
    with pytest.raises(ValueError):
        pa.prefill_window(q[None], q[None], t, t, bt, cl, 0.1, 4)
    with pytest.raises(ValueError):
        pa.reshape_and_cache_int4(q, q, t, t, par, par, cl.long())
    with pytest.raises(ValueError):
        pa.gather_blocks_int4(t, t, t, t, par, par, cl.long())


def test_packing_and_rounding_of_the_reference():
    codes = torch.randint(0, 16, (5, 128), generator=torch.Generator().manual_seed(1)).float()
    assert torch.equal(R.codes_of(R.pack_int4(codes)).float(), codes)
    one = torch.zeros(64)
    one[2] = 5.0
    assert R.pack_int4(one)[0] == 0x50  # channel 2 is the word's nibble 1
    x = torch.randn(7, 128, generator=torch.Generator().manual_seed(2)) * 3 + 50
    c, p = R.quantise_int4(x)
    value, scale, _ = R.wide_int4(R.pack_int4(c), p)
    assert bool(((value - x.double()).abs() <= scale * (0.5 + 1 / 30) + 1e-5).all())
    assert bool((p[..., 1].float() <= x.unflatten(-1, (-1, 64)).amin(-1)).all())


def test_only_bytes_move_as_four_bit_rows(pa):
    """A pool of 32 E4M3 channels is no cache of the library's: the block moves refuse it, as they do 96 channels."""
    desc_of = pa._blocks_desc
    d = desc_of(torch.zeros(4, 2, 8, 32, dtype=torch.uint8))
    assert (d.head_dim, d.kv_dtype) == (64, pa.PA_INT4)
    d = desc_of(torch.zeros(4, 2, 8, 64, dtype=torch.uint8))
    assert (d.head_dim, d.kv_dtype) == (64, pa.PA_FP8_E4M3)
    d = desc_of(torch.zeros(4, 2, 8, 32, dtype=torch.uint8).view(torch.float8_e4m3fn))
    assert (d.head_dim, d.kv_dtype) == (32, pa.PA_FP8_E4M3)
    for f in (pa.lib.pa_copy_blocks, pa.lib.pa_copy_block_scales):
        assert f(F, F, ctypes.byref(d), F, 1, N) == -2
