"""4-bit caches on the GPU: the write and the reading back against the definition bit by bit, the decode against 64-bit
references.  Tolerances are derived in _ref_stream.bound; a weight times its scale enters the second product in f16
(eleven significant bits: half a step is 2^-11 of it)."""
import math

import pytest
import torch

from tests import _ref_stream as R
from tests._gpu import lib
from tests._ref64 import DT, block_table

pytestmark = pytest.mark.gpu

WEIGHT = 2.0 ** -11


def _rows(gen, *shape):
    """Rows with a few wide and off-centre channels."""
    wide = torch.exp(0.6 * torch.randn(shape[-1], generator=gen))
    return torch.randn(*shape, generator=gen) * wide + 0.5 * torch.randn(shape[-1], generator=gen)


def make_pool(gen, NB, Hkv, bs, D):
    """A cache on the GPU written by the reference, and its tensors on the CPU."""
    host = {}
    for x in "kv":
        codes, params = R.quantise_int4(_rows(gen, NB, Hkv, bs, D))
        host[x] = (R.pack_int4(codes), params)
    return host, [host["k"][0].cuda(), host["v"][0].cuda(), host["k"][1].cuda(), host["v"][1].cuda()]


def rows_of(host, bt, lens, bs):
    def rows(s):
        pos = torch.arange(lens[s])
        ids = bt[s, pos // bs].clamp_min(0).long()
        out, sizes = [], []
        for x in "kv":
            data, params = host[x]
            value, scale, low = R.wide_int4(data[ids, :, pos % bs], params[ids, :, pos % bs])
            out.append(value)
            # the products' sizes: q code scale and q low of K; weights times code scale (15 - code where codes are
            # counted from the top) and times low (low + 15 scale) of V
            sizes.append(15 * scale + low if x == "k" else 30 * scale + low)
        return out[0], out[1], sizes[0], sizes[1]
    return rows


def check(pa, lens, k, Hq, Hkv, D, bs, dt, window, sinks, seed=0, scale=None, ws=None, spread=0):
    gen = torch.Generator().manual_seed(seed)
    S, NB = len(lens), sum(-(-n // bs) for n in lens) + 3
    host, pool = make_pool(gen, NB, Hkv, bs, D)
    if spread:  # V rows of very different sizes
        size = torch.exp2(torch.randint(-spread, spread, (NB, Hkv, bs, 1, 1), generator=gen).float()).to(torch.bfloat16)
        host["v"] = (host["v"][0], host["v"][1] * size)
        pool[3] = host["v"][1].cuda()
    bt = block_table(lens, bs, NB, gen)
    q = torch.randn(S, k, Hq, D, generator=gen).to(DT[dt])
    qg = (q if k > 1 else q[:, 0]).cuda()
    out = torch.full_like(qg, 7.0)
    scale = D ** -0.5 if scale is None else scale
    pa.decode_int4(out, qg, *pool, bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scale, window, sinks, ws)
    assert pa.get_device_error() == 0
    want, tol = R.reference(q, rows_of(host, bt, lens, bs), lens, k, Hkv, scale, window, sinks, DT[dt], WEIGHT)
    got = out.cpu().double().view(want.shape)
    worst = ((got - want).abs() / tol.clamp_min(1e-300)).max()
    assert float(worst) <= 1.0, "error %g of the bound" % worst


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,bs,Hkv", [(64, 8, 1), (128, 16, 2), (64, 32, 5), (128, 8, 3)])
@pytest.mark.parametrize("T", [1, 5, 33])
def test_write_is_the_definition(dt, D, bs, Hkv, T):
    pa = lib()
    gen = torch.Generator().manual_seed(T)
    NB = -(-T // bs) + 2
    x = {r: _rows(gen, T, Hkv, D).to(DT[dt]) for r in ("key", "value")}
    slots = torch.randperm(NB * bs, generator=gen)[:T]
    if T > 4:
        slots[2] = -1
        x["key"][0] = 0.25  # one value
        x["key"][1] = 0.0
        x["value"][0] = x["value"][0] * 2.0 ** -12 + 100
        x["value"][3, :, ::2] = torch.finfo(DT[dt]).max
        x["value"][3, :, 1::2] = -torch.finfo(DT[dt]).max
        x["key"][4] = torch.finfo(DT[dt]).tiny * torch.randn(Hkv, D, generator=gen).to(DT[dt])
    cache = [torch.full((NB, Hkv, bs, D // 2), 0xA5, dtype=torch.uint8).cuda() for _ in range(2)]
    params = [torch.full((NB, Hkv, bs, D // 64, 2), 3.0, dtype=torch.bfloat16).cuda() for _ in range(2)]
    pa.reshape_and_cache_int4(x["key"].cuda(), x["value"].cuda(), *cache, *params, slots.cuda())
    assert pa.get_device_error() == 0
    for row, c, p in zip(("key", "value"), cache, params):
        want_c = torch.full((NB, Hkv, bs, D // 2), 0xA5, dtype=torch.uint8)
        want_p = torch.full((NB, Hkv, bs, D // 64, 2), 3.0, dtype=torch.bfloat16)
        codes, par = R.quantise_int4(x[row])
        keep = slots >= 0
        want_c[slots[keep] // bs, :, slots[keep] % bs] = R.pack_int4(codes)[keep]
        want_p[slots[keep] // bs, :, slots[keep] % bs] = par[keep]
        assert torch.equal(p.cpu(), want_p)
        assert torch.equal(c.cpu(), want_c)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_write_of_values_that_are_not_finite(dt):
    pa = lib()
    D, bs = 128, 16
    x = _rows(torch.Generator().manual_seed(3), 6, 1, D).to(DT[dt])
    x[0, 0, 5], x[0, 0, 9] = math.inf, -math.inf  # count as the largest and least finite values
    x[1, 0, 70] = math.nan  # the second group reads as NaN, the first does not
    x[2] = math.inf
    x[3, 0, :64], x[3, 0, 64:] = -math.inf, math.nan
    x[4, 0, 0], x[4, 0, 1] = math.nan, math.inf
    cache = [torch.zeros(1, 1, bs, D // 2, dtype=torch.uint8).cuda() for _ in range(2)]
    params = [torch.zeros(1, 1, bs, 2, 2, dtype=torch.bfloat16).cuda() for _ in range(2)]
    pa.reshape_and_cache_int4(x.cuda(), x.cuda(), *cache, *params, torch.arange(6).cuda())
    codes, par = R.quantise_int4(x)
    for c, p in zip(cache, params):
        got = p.cpu()[0, 0, :6]
        assert torch.equal(torch.isnan(got), torch.isnan(par[:, 0]))
        assert torch.equal(got.nan_to_num(nan=9.0), par[:, 0].nan_to_num(nan=9.0))
        assert torch.equal(R.codes_of(c[0, 0, :6]).float(), codes[:, 0])
    dst = [torch.empty(1, 1, bs, D, dtype=DT[dt]).cuda() for _ in range(2)]
    pa.gather_blocks_int4(*dst, *cache, *params, torch.zeros(1, dtype=torch.int64).cuda())
    back = dst[0].cpu()[0, 0]
    assert bool(torch.isfinite(back[0]).all()) and bool(torch.isfinite(back[1, :64]).all())
    assert bool(torch.isnan(back[1, 64:]).all()) and bool(torch.isnan(back[3, 64:]).all())
    assert back[0, 5] == back[0, :64].max() and back[0, 9] == back[0, :64].min()


def test_slots_outside_the_pool_are_recorded():
    pa = lib()
    x = torch.randn(2, 1, 64, dtype=torch.bfloat16).cuda()
    cache = [torch.zeros(1, 1, 8, 32, dtype=torch.uint8).cuda() for _ in range(2)]
    params = [torch.zeros(1, 1, 8, 1, 2, dtype=torch.bfloat16).cuda() for _ in range(2)]
    pa.reshape_and_cache_int4(x, x, *cache, *params, torch.tensor([8, -5]).cuda())
    assert pa.get_device_error() == pa.DEVERR_SLOT
    assert not cache[0].any() and not params[1].any()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,bs,Hkv,n", [(64, 8, 1, 1), (128, 16, 3, 5), (64, 32, 2, 4)])
def test_reading_back(dt, D, bs, Hkv, n):
    pa = lib()
    gen = torch.Generator().manual_seed(n)
    host, pool = make_pool(gen, n + 2, Hkv, bs, D)
    ids = torch.randperm(n + 2, generator=gen)[:n]
    for pinned in (False, True):
        dst = [torch.zeros(n, Hkv, bs, D, dtype=DT[dt]) for _ in range(2)]
        dst = [t.pin_memory() if pinned else t.cuda() for t in dst]
        pa.gather_blocks_int4(*dst, *pool, ids.cuda())
        assert pa.get_device_error() == 0  # synchronises
        for x, got in zip("kv", dst):
            value = R.wide_int4(*host[x])[0][ids]
            assert torch.equal(got.cpu(), value.float().to(DT[dt]))  # one float32 step, as a fused multiply-add


def test_a_block_id_outside_the_pool_leaves_its_destination():
    pa = lib()
    _, pool = make_pool(torch.Generator().manual_seed(1), 2, 1, 8, 64)
    dst = [torch.full((2, 1, 8, 64), 5.0, dtype=torch.float16).cuda() for _ in range(2)]
    pa.gather_blocks_int4(*dst, *pool, torch.tensor([2, 1]).cuda())
    assert pa.get_device_error() == pa.DEVERR_BLOCK_ID
    assert bool((dst[0][0] == 5).all()) and not bool((dst[0][1] == 5).all())


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 130, 700]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("k,Hq,Hkv,D,bs", [(1, 1, 1, 64, 8), (1, 8, 2, 128, 16), (1, 16, 1, 64, 32), (2, 12, 4, 128, 8),
                                           (3, 6, 2, 64, 16), (1, 40, 2, 128, 32), (16, 2, 1, 128, 16), (5, 9, 3, 64, 8)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 3), (130, 200)])
def test_decode(dt, k, Hq, Hkv, D, bs, window, sinks):
    check(lib(), LENS, k, Hq, Hkv, D, bs, dt, window, sinks, seed=k + Hq)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_decode_of_one_long_context(dt):
    check(lib(), [5003], 1, 8, 2, 128, 16, dt, 0, 0)
    check(lib(), [9001], 2, 4, 1, 64, 8, dt, 3000, 5)


def test_decode_with_another_scale_and_a_workspace_full_of_nan():
    pa = lib()
    ws = torch.full((pa.decode_flat_workspace_size(128),), 0xFF, dtype=torch.uint8).cuda()
    for scale in (-0.3, 0.0, 2.0):
        check(pa, [700, 3], 1, 8, 2, 128, 16, "f16", 0, 0, scale=scale, ws=ws)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("spread,scale", [(12, 0.1), (12, 3.0), (100, 0.1), (100, 3.0)])
def test_values_of_very_different_sizes(dt, spread, scale):
    """Weights times scales that leave f16's range on both sides; outputs past f16's range are infinite in the reference
    too, so f16 stays with the narrower spread."""
    if dt == "f16" and spread > 12:
        spread = 9
    check(lib(), [700, 65, 16], 2, 8, 2, 128, 16, dt, 0, 0, seed=spread, scale=scale, spread=spread)


def test_a_nan_shows_where_it_is_seen_and_nowhere_else():
    pa = lib()
    gen = torch.Generator().manual_seed(9)
    lens, bs, Hkv, D = [200, 200], 16, 2, 128
    host, pool = make_pool(gen, 30, Hkv, bs, D)
    bt = block_table(lens, bs, 30, gen)
    q = torch.randn(2, 2, 4, D, generator=gen).to(torch.bfloat16).cuda()
    cl = torch.tensor(lens, dtype=torch.int32).cuda()

    def run(window, sinks):
        out = torch.empty_like(q)
        pa.decode_int4(out, q, *pool, bt.cuda(), cl, 0.1, window, sinks)
        return out.cpu()

    clean = run(50, 4)
    for which in (2, 3):  # K's parameters, V's
        for pos, affected in ((100, []), (3, [0, 1]), (199, [1]), (149, [0])):
            b, o = int(bt[0, pos // bs]), pos % bs
            kept = pool[which][b, 1, o].clone()
            pool[which][b, 1, o, 1, 0] = math.nan
            out = run(50, 4)
            pool[which][b, 1, o] = kept
            for j in range(2):
                bad = torch.isnan(out[0, j, 2:])
                if j in affected:
                    assert bool(bad.all() if which == 2 else (bad[:, 64:].all() and not bad[:, :64].any())), (which, pos, j)
                else:
                    assert torch.equal(out[0, j], clean[0, j]), (which, pos, j)
            assert torch.equal(out[1], clean[1]) and torch.equal(out[0, :, :2], clean[0, :, :2])


def test_rows_far_into_a_large_pool():
    pa = lib()
    NB, Hkv, bs, D = (1 << 32) // (8 * 16 * 64) + 9, 8, 16, 128  # codes pass 4 GiB
    k, v = (torch.zeros(NB, Hkv, bs, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    kp, vp = (torch.zeros(NB, Hkv, bs, 2, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gen = torch.Generator().manual_seed(4)
    lens = [50]
    bt = torch.tensor([[NB - 1, NB - 4, 0, NB - 2]], dtype=torch.int32)
    pos = torch.arange(50)
    slots = bt[0, pos // bs].long() * bs + pos % bs
    key, value = (_rows(gen, 50, Hkv, D).to(torch.bfloat16) for _ in range(2))
    pa.reshape_and_cache_int4(key.cuda(), value.cuda(), k, v, kp, vp, slots.cuda())
    host = {}
    for x, r in (("k", key), ("v", value)):
        codes, par = R.quantise_int4(r)
        host[x] = (R.pack_int4(codes)[:, :, None], par[:, :, None])  # blocks of one token
    q = torch.randn(1, 1, 8, D, generator=gen).to(torch.bfloat16)
    out = torch.empty(1, 8, D, dtype=torch.bfloat16).cuda()
    pa.decode_int4(out, q[:, 0].cuda(), k, v, kp, vp, bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.1)
    want, tol = R.reference(q, rows_of(host, pos[None].int(), lens, 1), lens, 1, Hkv, 0.1, 0, 0, torch.bfloat16, WEIGHT)
    assert bool(((out.cpu().double() - want[:, 0]).abs() <= tol[:, 0]).all())
    assert pa.get_device_error() == 0


def test_blocks_move_with_their_parameters():
    pa = lib()
    for D in (64, 128):
        _, pool = make_pool(torch.Generator().manual_seed(D), 6, 2, 8, D)
        pairs = torch.tensor([[0, 4], [3, 5]]).cuda()
        before = [t.clone() for t in pool]
        pa.copy_blocks(pool[0], pool[1], pairs)
        pa.copy_block_scales(pool[2], pool[3], pairs)
        for t, b in zip(pool, before):
            assert torch.equal(t[4], b[0]) and torch.equal(t[5], b[3]) and torch.equal(t[:4], b[:4])
        ids = torch.tensor([2, 1]).cuda()
        codes = torch.empty(2, 2, *pool[0].shape[1:], dtype=torch.uint8).pin_memory()
        params = torch.empty(2, 2, *pool[2].shape[1:], dtype=torch.bfloat16).pin_memory()
        pa.gather_blocks(codes, pool[0], pool[1], ids)
        pa.gather_block_scales(params, pool[2], pool[3], ids)
        back = torch.tensor([5, 0]).cuda()
        pa.scatter_blocks(pool[0], pool[1], codes, back)
        pa.scatter_block_scales(pool[2], pool[3], params, back)
        assert pa.get_device_error() == 0
        for t, b in zip(pool, before):
            assert torch.equal(t[5], b[2]) and torch.equal(t[0], b[1])


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("k,Hq,Hkv,D,bs", [(1, 4, 1, 64, 8), (1, 16, 1, 128, 16), (3, 2, 1, 128, 32)])
@pytest.mark.parametrize("reps,window,sinks", [(8, 0, 0), (16, 130, 200), (33, 0, 0), (70, 0, 0), (70, 40, 3), (70, 130, 200)])
def test_decode_of_batches_from_clusters_to_the_line(dt, k, Hq, Hkv, D, bs, reps, window, sinks):
    """Clusters of four, two and one CTA per context, and more contexts than there is room for, which lie on a line."""
    check(lib(), LENS * reps, k, Hq, Hkv, D, bs, dt, window, sinks, seed=reps)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("lens,k", [([5003], 1), ([700, 0, 65, 1], 2)])
def test_a_table_far_wider_than_its_contexts(dt, lens, k):
    """What a context could hold decides between clusters and the line: the same batch by both, within two bounds of
    one another, and captured and replayed over other lengths as it runs without."""
    pa = lib()
    gen = torch.Generator().manual_seed(3)
    Hq, Hkv, D, bs = 8, 2, 128, 16
    NB = sum(-(-n // bs) for n in lens) + 3
    host, pool = make_pool(gen, NB, Hkv, bs, D)
    bt = block_table(lens, bs, NB, gen)
    wide = torch.full((len(lens), 40000), -1, dtype=torch.int32)
    wide[:, :bt.shape[1]] = bt
    q = torch.randn(len(lens), k, Hq, D, generator=gen).to(DT[dt])
    qg = (q if k > 1 else q[:, 0]).cuda()
    cl = torch.tensor(lens, dtype=torch.int32).cuda()
    ws = torch.empty(pa.decode_flat_workspace_size(D), dtype=torch.uint8).cuda()
    want, tol = R.reference(q, rows_of(host, bt, lens, bs), lens, k, Hkv, 0.1, 0, 0, DT[dt], WEIGHT)
    wide = wide.cuda()

    def run(out, table):
        pa.decode_int4(out, qg, *pool, table, cl, 0.1, workspace=ws)

    for table in (bt.cuda(), wide):
        out = torch.full_like(qg, 7.0)
        run(out, table)
        worst = ((out.cpu().double().view(want.shape) - want).abs() / tol.clamp_min(1e-300)).max()
        assert float(worst) <= 1.0, "error %g of the bound" % worst
    held = torch.empty_like(qg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(held, wide)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(held, wide)
    for shorter in (0, 1, 300):
        cl.copy_(torch.tensor([max(n - shorter, 0) for n in lens], dtype=torch.int32))
        g.replay()
        out = torch.empty_like(qg)
        run(out, wide)
        assert torch.equal(held, out)
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("k,Hq", [(1, 1), (5, 1), (1, 7), (3, 3), (1, 11), (5, 3)])
@pytest.mark.parametrize("S", [1, 100, 250])
def test_clusters_join_odd_numbers_of_columns(S, k, Hq, dt):
    """64 channels and an odd number of query columns: half a warp has nothing to join."""
    check(lib(), [(397 * i + 1203) % 1600 for i in range(S)], k, Hq, 1, 64, 16, dt, 0, 0, seed=S + k)


@pytest.mark.parametrize("Hkv", [700, 2500])
@pytest.mark.parametrize("S", [1, 2])
def test_contexts_that_are_not_cut_leave_the_workspace(S, Hkv):
    """With more heads than a part has warps each context lies within one part: there are no pieces to join, and a
    workspace is not written, whatever the number of heads."""
    pa = lib()
    gen = torch.Generator().manual_seed(Hkv)
    D, bs = 64, 8
    host, pool = make_pool(gen, 12, Hkv, bs, D)
    lens = [40, 9][:S]
    bt = block_table(lens, bs, 12, gen)
    q = torch.randn(S, 1, Hkv, D, generator=gen).half()
    out = torch.empty(S, Hkv, D, dtype=torch.half).cuda()
    ws = torch.full((pa.decode_flat_workspace_size(D),), 0x5A, dtype=torch.uint8).cuda()
    pa.decode_int4(out, q[:, 0].cuda(), *pool, bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.1, workspace=ws)
    assert pa.get_device_error() == 0
    want, tol = R.reference(q, rows_of(host, bt, lens, bs), lens, 1, Hkv, 0.1, 0, 0, torch.half, WEIGHT)
    assert bool(((out.cpu().double() - want[:, 0]).abs() <= tol[:, 0]).all())
    if Hkv > 4 * 4 * torch.cuda.get_device_properties(0).multi_processor_count:
        assert bool((ws == 0x5A).all())


def test_pools_of_32_e4m3_channels_are_not_moved():
    pa = lib()
    pool = torch.zeros(4, 2, 8, 32, dtype=torch.uint8).cuda().view(torch.float8_e4m3fn)
    pairs, ids = torch.tensor([[0, 1]]).cuda(), torch.tensor([0]).cuda()
    buf = torch.zeros(1, 2, 2, 8, 32, dtype=torch.uint8).cuda()
    for call in (lambda: pa.copy_blocks(pool, pool, pairs), lambda: pa.gather_blocks(buf, pool, pool, ids),
                 lambda: pa.scatter_blocks(pool, pool, buf, ids)):
        with pytest.raises(pa.PagedAttnError):
            call()


@pytest.mark.parametrize("D,Hq,Hkv,new,lens,window,sinks", [
    (128, 8, 2, 1, [69, 130, 701], 0, 0),
    (64, 16, 2, 1, [69, 130, 701], 0, 0),
    (128, 8, 2, 1, [69, 333, 701], 59, 3),   # unseen rows also behind the sinks and before the window
    (64, 8, 1, 3, [69, 333, 701], 59, 3),
    (128, 6, 2, 2, [69, 130, 701] * 60, 0, 0),  # the line
])
def test_rows_that_a_token_does_not_see_leave_its_bits(D, Hq, Hkv, new, lens, window, sinks):
    """What a block holds in rows that no new token sees (behind a context's end, say, where an earlier owner wrote) does
    not move an output by a bit, nor does a row that only later new tokens see.  V's scales grow along the contexts, so
    that a look at an unseen row's scale would change what the seen rows' weights are rounded against."""
    pa = lib()
    gen = torch.Generator().manual_seed(D + new)
    bs, S = 16, len(lens)
    NB = sum(-(-n // bs) for n in lens) + 1
    _, pool = make_pool(gen, NB, Hkv, bs, D)
    bt = block_table(lens, bs, NB, gen)
    pos = torch.arange(max(lens))
    for s, n in enumerate(lens):  # the newest eight tokens' V is 30 times the others'
        p = pos[max(0, n - 8):n]
        pool[3][bt[s, p // bs].long().cuda(), :, (p % bs).cuda()] *= 30
    q = torch.randn(S, new, Hq, D, generator=gen).half().cuda()
    cl = torch.tensor(lens, dtype=torch.int32).cuda()

    def run():
        out = torch.empty_like(q)
        pa.decode_int4(out, q, *pool, bt.cuda(), cl, 0.02, window, sinks)
        assert pa.get_device_error() == 0
        return out.cpu()

    clean = run()
    kept = [t.clone() for t in pool]
    unseen = torch.ones(NB, bs, dtype=torch.bool)
    for s, n in enumerate(lens):
        seen = torch.zeros(n, dtype=torch.bool)
        for j in range(new):
            seen |= R.sees(n - new + j, n, window, sinks)
        p = pos[:n][seen]
        unseen[bt[s, p // bs].long(), p % bs] = False
    b, o = (i.cuda() for i in unseen.nonzero(as_tuple=True))
    for junk in (2.0 ** 20, 2.0 ** 120, math.inf, math.nan):
        for t in pool[2:]:
            t[b, :, o] = junk
        assert torch.equal(run(), clean), junk
    for t, k in zip(pool, kept):
        t.copy_(k)
    for j in range(1, new):  # the row of the new token j
        for s, n in enumerate(lens):
            pool[3][int(bt[s, (n - new + j) // bs]), :, (n - new + j) % bs] *= 2.0 ** 20
        got = run()
        assert torch.equal(got[:, :j], clean[:, :j])
        for t, k in zip(pool, kept):
            t.copy_(k)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_the_largest_values_are_read_back_finite(dt, D):
    """Values up to the type's largest come back within half a scale of themselves: a least value that bfloat16 rounds
    down, or fifteen scales rounded up, may pass the largest number of 16 bits, which then stands for them.  (bfloat16
    rounds the scale by 2^-8 of itself at most: fifteen of them end within a seventeenth of a scale of the largest value.)"""
    pa = lib()
    gen = torch.Generator().manual_seed(D)
    bs, top = 16, torch.finfo(DT[dt]).max
    x = (2 * torch.rand(bs, 1, D, generator=gen, dtype=torch.float64) - 1) * top * 0.45
    x[:, :, 3] = torch.linspace(0.46, 1.0, bs, dtype=torch.float64)[:, None] * top / (1 if dt == "f16" else 2)
    x[1::2] *= -1
    x[4, 0] = x[4, 0].abs()
    x[5, 0] = -x[5, 0].abs()
    x[6, 0] = top / 2 * (1 + 0.9 * torch.rand(D, generator=gen, dtype=torch.float64))
    x[7, 0] = -x[6, 0]
    x[8, 0], x[9, 0] = top, -top  # scales of a step of bfloat16, and the least
    x = x.to(DT[dt])
    cache = [torch.zeros(1, 1, bs, D // 2, dtype=torch.uint8).cuda() for _ in range(2)]
    params = [torch.zeros(1, 1, bs, D // 64, 2, dtype=torch.bfloat16).cuda() for _ in range(2)]
    pa.reshape_and_cache_int4(x.cuda(), -x.cuda(), *cache, *params, torch.arange(bs).cuda())
    dst = [torch.empty(1, 1, bs, D, dtype=DT[dt]).cuda() for _ in range(2)]
    pa.gather_blocks_int4(*dst, *cache, *params, torch.zeros(1, dtype=torch.int64).cuda())
    assert pa.get_device_error() == 0
    for back, par, want in zip(dst, params, (x, -x)):
        got, want = back.cpu()[0, 0].double(), want[:, 0].double()
        assert bool(torch.isfinite(got).all())
        scale = par.cpu()[0, 0, :, :, 0].double().repeat_interleave(64, -1)
        # float32 steps of the quotient (2^-24 of fifteen scales, twice) and of the multiply-add, and the last rounding
        slack = 2.0 ** -19 * scale + (want.abs() + 0.5 * scale) * (torch.finfo(DT[dt]).eps / 2 + 2.0 ** -23)
        assert bool(((got - want).abs() <= 0.5 * scale + slack).all())
