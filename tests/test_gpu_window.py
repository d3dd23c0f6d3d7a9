"""Attention through a window with sinks on the GPU, decode and prefill, against 64-bit references (tolerances:
_ref_stream.bound; a weight rounds to the MMA's 16-bit type, bf16 on bf16 caches, f16 on the others)."""
import math

import pytest
import torch

from tests import _ref_stream as R
from tests._gpu import lib
from tests._ref64 import DT, E4M3, block_table, wide

pytestmark = pytest.mark.gpu

LENS = [0, 1, 15, 16, 17, 64, 65, 130, 700]


def weight_eps(kv):
    # bf16 holds 8 significant bits: numbers in [1, 2) lie 2^-7 apart, half a step is 2^-8; f16 holds 11
    return 2.0 ** -8 if kv == "bf16" else 2.0 ** -11


def make_pool(gen, NB, Hkv, bs, D, kv):
    pool = [torch.randn(NB, Hkv, bs, D, generator=gen) for _ in range(2)]
    return [t.to(E4M3) if kv == "e4m3" else t.to(DT[kv]) for t in pool]


def hide(bt, lens, new, bs, window, sinks, NB):
    """The table with entries of blocks that no new token sees replaced by ids outside the pool."""
    bt = bt.clone()
    for s, L in enumerate(lens):
        seen = torch.zeros(max(L, 1), dtype=torch.bool)
        for P in range(max(0, L - new), L):
            seen[:L] |= R.sees(P, L, window, sinks)
        for j in range(bt.shape[1]):
            if not seen[j * bs:(j + 1) * bs].any():
                bt[s, j] = NB + 77 if j % 2 else -3
    return bt


def rows_of(pool, bt, lens, bs, kv_scale):
    def rows(s):
        pos = torch.arange(lens[s])
        ids = bt[s, pos // bs].clamp_min(0).long()
        k, v = ((wide(t.view(torch.uint8)[ids, :, pos % bs].view(E4M3) if t.dtype == E4M3 else t[ids, :, pos % bs]) * kv_scale)
                for t in pool)
        return k, v, k.abs(), v.abs()
    return rows


def check(call, pa, lens, k, Hq, Hkv, D, bs, dt, kv, window, sinks, seed=0, hidden=True):
    gen = torch.Generator().manual_seed(seed)
    S, NB = len(lens), sum(-(-n // bs) for n in lens) + 3
    kv_scale = float(torch.tensor(0.7)) if kv == "e4m3" else 1.0
    pool = make_pool(gen, NB, Hkv, bs, D, kv)
    bt = block_table(lens, bs, NB, gen)
    q = torch.randn(S, k, Hq, D, generator=gen).to(DT[dt])
    qg = (q if k > 1 or call == "prefill" else q[:, 0]).cuda()
    out = torch.full_like(qg, 7.0)
    table = hide(bt, lens, k, bs, window, sinks, NB) if hidden else bt
    fn = pa.prefill_window if call == "prefill" else pa.decode_window
    fn(out, qg, pool[0].cuda(), pool[1].cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), D ** -0.5, window,
       num_sinks=sinks, kv_scale=kv_scale)
    assert pa.get_device_error() == 0
    want, tol = R.reference(q, rows_of(pool, bt, lens, bs, kv_scale), lens, k, Hkv, D ** -0.5, window, sinks, DT[dt], weight_eps(kv))
    got = out.cpu().double().view(want.shape)
    worst = ((got - want).abs() / tol.clamp_min(1e-300)).max()
    assert float(worst) <= 1.0, "error %g of the bound" % worst


@pytest.mark.parametrize("dt,kv", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("k,Hq,Hkv,D,bs", [(1, 1, 1, 64, 8), (1, 8, 2, 128, 16), (1, 16, 1, 64, 32), (2, 12, 4, 128, 8),
                                           (3, 6, 2, 64, 16), (1, 40, 2, 128, 32), (16, 2, 1, 128, 16)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (40, 3), (130, 200), (100000, 4)])
def test_decode(dt, kv, k, Hq, Hkv, D, bs, window, sinks):
    check("decode", lib(), LENS, k, Hq, Hkv, D, bs, dt, kv, window, sinks, seed=k + Hq)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_of_one_long_context(kv):
    check("decode", lib(), [9001], 1, 8, 2, 128, 16, "bf16", kv, 5003, 4)


def test_decode_of_many_contexts():
    lens = [(37 * i) % 1500 for i in range(130)]
    check("decode", lib(), lens, 1, 8, 8, 64, 16, "f16", "f16", 600, 4)


@pytest.mark.parametrize("dt,kv", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("C,Hq,Hkv,D,bs", [(1, 4, 2, 128, 16), (7, 6, 2, 64, 8), (150, 4, 2, 128, 32), (300, 3, 1, 64, 16),
                                           (130, 16, 1, 128, 8)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 3), (140, 4), (130, 300), (100000, 4)])
def test_prefill(dt, kv, C, Hq, Hkv, D, bs, window, sinks):
    check("prefill", lib(), [0, 1, 65, 150, 300, 700], C, Hq, Hkv, D, bs, dt, kv, window, sinks, seed=C)


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
def test_values_that_only_some_tokens_see(kv):
    """A NaN or an infinity in a V or K row that a new token does not see leaves that token's output as it was."""
    pa = lib()
    gen = torch.Generator().manual_seed(5)
    lens, bs, Hkv, D, k, window, sinks = [200], 16, 1, 128, 3, 50, 4
    dt = "f16" if kv == "e4m3" else kv
    pool = [t.cuda() for t in make_pool(gen, 16, Hkv, bs, D, kv)]
    bt = block_table(lens, bs, 16, gen)
    q = torch.randn(1, k, 2, D, generator=gen).to(DT[dt]).cuda()
    cl = torch.tensor(lens, dtype=torch.int32).cuda()

    def run():
        out = torch.empty_like(q)
        pa.decode_window(out, q, *pool, bt.cuda(), cl, 0.1, window, num_sinks=sinks)
        return out.cpu()

    clean = run()
    for which in range(2):
        for value in (math.nan, math.inf):
            if kv == "e4m3" and value == math.inf:
                continue
            # positions 197, 198, 199 see from 148, 149, 150 on; and 0 .. 3
            for pos, see in ((100, ()), (147, ()), (148, (0,)), (149, (0, 1)), (199, (2,)), (198, (1, 2)), (2, (0, 1, 2)), (4, ())):
                t = pool[which]
                at = (int(bt[0, pos // bs]), 0, pos % bs, 3)
                kept = t.view(torch.uint8)[at].clone() if kv == "e4m3" else t[at].clone()
                if kv == "e4m3":
                    t.view(torch.uint8)[at] = 0x7F
                else:
                    t[at] = value
                out = run()
                if kv == "e4m3":
                    t.view(torch.uint8)[at] = kept
                else:
                    t[at] = kept
                for j in range(k):
                    if j not in see:
                        assert torch.equal(out[0, j], clean[0, j]), (which, value, pos, j)
                    elif value != value:
                        assert bool(torch.isnan(out[0, j]).all() if which == 0 else torch.isnan(out[0, j, :, 3]).all()), (which, pos, j)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("L,hidden", [(300, (3, 31, 100, 239)), (70, (3, 5, 9)), (90, (3, 20, 29)), (110, (3, 31, 32, 49))])
def test_prefill_ignores_rows_that_no_token_sees(kv, L, hidden):
    pa = lib()
    gen = torch.Generator().manual_seed(6)
    lens, bs, Hkv, D, C, window, sinks = [L], 32, 1, 128, 20, 41, 3
    dt = "f16" if kv == "e4m3" else kv
    pool = [t.cuda() for t in make_pool(gen, 12, Hkv, bs, D, kv)]
    bt = block_table(lens, bs, 12, gen)
    q = torch.randn(1, C, 2, D, generator=gen).to(DT[dt]).cuda()
    cl = torch.tensor(lens, dtype=torch.int32).cuda()

    def run():
        out = torch.empty_like(q)
        pa.prefill_window(out, q, *pool, bt.cuda(), cl, 0.1, window, num_sinks=sinks)
        return out.cpu()

    clean = run()
    for pos in hidden:  # the first new token, at L - 20, sees from L - 60 on
        at = (int(bt[0, pos // bs]), 0, pos % bs)
        for t in pool:
            if kv == "e4m3":
                t.view(torch.uint8)[at] = 0x7F
            else:
                t[at] = math.nan
    assert torch.equal(run(), clean)


def test_rows_behind_the_batch_stay_as_they_were():
    pa = lib()
    gen = torch.Generator().manual_seed(7)
    pool = [t.cuda() for t in make_pool(gen, 8, 2, 16, 64, "bf16")]
    bt = block_table([40, 70], 16, 8, gen).cuda()
    cl = torch.tensor([40, 70], dtype=torch.int32).cuda()
    big = torch.full((5, 4, 64), 3.0, dtype=torch.bfloat16).cuda()
    q = torch.randn(2, 4, 64, generator=gen).to(torch.bfloat16).cuda()
    pa.decode_window(big[1:3], q, *pool, bt, cl, 0.1, 20, num_sinks=2)
    assert bool((big[0] == 3).all()) and bool((big[3:] == 3).all()) and not bool((big[1:3] == 3).any())


def test_lengths_and_ids_out_of_range_are_recorded():
    pa = lib()
    gen = torch.Generator().manual_seed(8)
    pool = [t.cuda() for t in make_pool(gen, 8, 1, 16, 64, "f16")]
    q = torch.randn(2, 2, 64, generator=gen).half().cuda()
    out = torch.empty_like(q)
    bt = torch.tensor([[0, 1], [2, 9]], dtype=torch.int32).cuda()
    pa.decode_window(out, q, *pool, bt, torch.tensor([32, 16], dtype=torch.int32).cuda(), 0.1, 20)
    assert pa.get_device_error() == 0
    pa.decode_window(out, q, *pool, bt, torch.tensor([33, 16], dtype=torch.int32).cuda(), 0.1, 20)
    assert pa.get_device_error() == pa.DEVERR_CONTEXT_LEN
    pa.decode_window(out, q, *pool, bt, torch.tensor([-1, 16], dtype=torch.int32).cuda(), 0.1, 20)
    assert pa.get_device_error() == pa.DEVERR_CONTEXT_LEN and not out[0].any()
    pa.decode_window(out, q, *pool, bt, torch.tensor([32, 20], dtype=torch.int32).cuda(), 0.1, 20)
    assert pa.get_device_error() == pa.DEVERR_BLOCK_ID
    pa.prefill_window(out[:, None], q[:, None], *pool, bt, torch.tensor([32, 20], dtype=torch.int32).cuda(), 0.1, 20)
    assert pa.get_device_error() == pa.DEVERR_BLOCK_ID


def test_a_captured_step_follows_its_inputs_and_two_share_a_workspace():
    pa = lib()
    gen = torch.Generator().manual_seed(10)
    Hkv, bs, D, dt = 2, 16, 128, torch.bfloat16
    S, NB = 3, 40
    codes = [torch.zeros(NB, Hkv, bs, D // 2, dtype=torch.uint8).cuda() for _ in range(2)]
    params = [torch.zeros(NB, Hkv, bs, 2, 2, dtype=torch.bfloat16).cuda() for _ in range(2)]
    bt = torch.randperm(NB, generator=gen)[:36].view(S, 12).int().cuda()
    cl = torch.tensor([5, 100, 180], dtype=torch.int32).cuda()
    q, key, value = (torch.randn(S, h, D, generator=gen).to(dt).cuda() for h in (8, Hkv, Hkv))
    slots = torch.zeros(S, dtype=torch.int64).cuda()
    out = [torch.zeros_like(q) for _ in range(2)]
    ws = torch.empty(pa.decode_flat_workspace_size(D), dtype=torch.uint8).cuda()
    fill = torch.randn(NB * bs, Hkv, D, generator=gen).to(dt).cuda()
    pa.reshape_and_cache_int4(fill, fill, *codes, *params, torch.arange(NB * bs).cuda())

    def step(i):
        pa.reshape_and_cache_int4(key, value, *codes, *params, slots)
        pa.decode_int4(out[i], q, *codes, *params, bt, cl, 0.1, window=(0, 60)[i], num_sinks=4, workspace=ws)

    def place():
        pos = (cl - 1).long()
        slots.copy_(bt.gather(1, (pos // bs)[:, None]).squeeze(1).long() * bs + pos % bs)

    place()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for i in range(2):
            step(i)
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                step(i)
            graphs.append(g)
    torch.cuda.synchronize()
    for n in range(3):
        cl.add_(torch.tensor([40, 3, 1], dtype=torch.int32).cuda())
        q.mul_(-1.1)
        key.add_(0.5)
        place()
        for g in graphs:
            g.replay()
        got = [t.clone() for t in out]
        for i in range(2):
            out[i].zero_()
            step(i)
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(got[i], out[i])  # the same bits, replayed or called
    assert pa.get_device_error() == 0


def test_a_stream_from_its_prompt_to_decoding_over_four_bits():
    """Rows of a prompt written in 4 bits, the chunk prefilled over the blocks read back, then steps of decoding: the
    window of the 4-bit decode, that of the decode over the values read back and the prefill's last token agree."""
    pa = lib()
    gen = torch.Generator().manual_seed(11)
    Hq, Hkv, bs, D, dt, window, sinks = 8, 2, 16, 128, torch.bfloat16, 70, 4
    n, NB = 200, 16
    codes = [torch.zeros(NB, Hkv, bs, D // 2, dtype=torch.uint8).cuda() for _ in range(2)]
    params = [torch.zeros(NB, Hkv, bs, 2, 2, dtype=torch.bfloat16).cuda() for _ in range(2)]
    order = torch.randperm(NB, generator=gen)
    pos = torch.arange(n)
    slots = (order[pos // bs] * bs + pos % bs).cuda()
    rows = [torch.randn(n, Hkv, D, generator=gen).to(dt).cuda() for _ in range(2)]
    pa.reshape_and_cache_int4(*rows, *codes, *params, slots)
    blocks = -(-n // bs)
    back = [torch.zeros(blocks, Hkv, bs, D, dtype=dt).cuda() for _ in range(2)]
    pa.gather_blocks_int4(*back, *codes, *params, order[:blocks].cuda())
    own = torch.arange(blocks, dtype=torch.int32)[None].cuda()
    bt = order[:blocks].int()[None].cuda()
    q = torch.randn(1, n, Hq, D, generator=gen).to(dt).cuda()
    prompt = torch.empty_like(q)
    cl = torch.tensor([n], dtype=torch.int32).cuda()
    pa.prefill_window(prompt, q, *back, own, cl, D ** -0.5, window, num_sinks=sinks)
    for new in (1, 4):
        a, b = (torch.empty(1, new, Hq, D, dtype=dt).cuda() for _ in range(2))
        last = q[:, n - new:].contiguous()
        pa.decode_int4(a, last, *codes, *params, bt, cl, D ** -0.5, window=window, num_sinks=sinks)
        pa.decode_window(b, last, *back, own, cl, D ** -0.5, window, num_sinks=sinks)
        # values below 4, averaged: each side is off by half a step of the output (2^-8 of it) and of each
        # weight (2^-8 of the largest value), the values read back besides by theirs, which K's carry into
        # the scores as well: at most three halves of a step on each side
        assert float((a.double() - b.double()).abs().max()) <= 4 * 6 * 2.0 ** -8
        assert float((b.double() - prompt[:, n - new:].double()).abs().max()) <= 4 * 4 * 2.0 ** -8
    assert pa.get_device_error() == 0


def test_another_stream_and_empty_batches():
    pa = lib()
    gen = torch.Generator().manual_seed(12)
    pool = [t.cuda() for t in make_pool(gen, 8, 2, 16, 64, "bf16")]
    bt = block_table([40, 70], 16, 8, gen).cuda()
    cl = torch.tensor([40, 70], dtype=torch.int32).cuda()
    q = torch.randn(2, 4, 64, generator=gen).to(torch.bfloat16).cuda()
    a, b = torch.empty_like(q), torch.empty_like(q)
    pa.decode_window(a, q, *pool, bt, cl, 0.1, 20)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        pa.decode_window(b, q, *pool, bt, cl, 0.1, 20)
    side.synchronize()
    assert torch.equal(a, b)
    pa.decode_window(a[:0], q[:0], *pool, bt[:0], cl[:0], 0.1, 20)
    pa.prefill_window(a[:0, None], q[:0, None], *pool, bt[:0], cl[:0], 0.1, 20)
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("S,C,Hq,Hkv,D,bs,sinks", [(20, 128, 8, 2, 128, 16, 4), (21, 120, 8, 2, 64, 32, 200), (40, 128, 4, 2, 128, 8, 0)])
def test_prefill_of_chunks_that_pairs_of_heads_take(dt, S, C, Hq, Hkv, D, bs, sinks):
    lens = [0, 60, 1024, 1300] + [1000 + 13 * i for i in range(S - 4)]
    check("prefill", lib(), lens, C, Hq, Hkv, D, bs, dt, dt, 1000, sinks, seed=C)


def test_a_row_of_many_pieces_and_rows_of_one():
    """One context that most warps share beside many that lie within one warp's part."""
    lens = [30000] + [40 + i for i in range(60)]
    check("decode", lib(), lens, 1, 8, 2, 64, 16, "bf16", "bf16", 25000, 3)


@pytest.mark.parametrize("Hkv", [700, 2500])
def test_decode_of_more_heads_than_warps_of_a_part(Hkv):
    check("decode", lib(), [70, 9], 1, Hkv, Hkv, 64, 8, "f16", "f16", 40, 2)


@pytest.mark.parametrize("dt,kv", [("bf16", "bf16"), ("f16", "f16"), ("f16", "e4m3")])
@pytest.mark.parametrize("k,Hq,Hkv,D,bs", [(1, 4, 1, 64, 8), (1, 16, 1, 128, 16), (3, 2, 1, 128, 32)])
@pytest.mark.parametrize("reps,window,sinks", [(8, 40, 3), (16, 130, 200), (33, 40, 0), (70, 1, 1), (70, 40, 3), (70, 130, 200)])
def test_decode_of_batches_from_clusters_to_the_line(dt, kv, k, Hq, Hkv, D, bs, reps, window, sinks):
    """Clusters of four, two and one CTA per context, and more contexts than there is room for, which lie on a line."""
    check("decode", lib(), LENS * reps, k, Hq, Hkv, D, bs, dt, kv, window, sinks, seed=reps)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 8)])
def test_wide_windows_of_many_streams(dt, D, bs):
    """A CTA per context where there are more contexts than places, some shorter than the window, some empty."""
    lens = [0, 1, 1039, 1040, 1041] + [(53 * i) % 1700 for i in range(170)]
    check("decode", lib(), lens, 1, 8, 4, D, bs, dt, dt, 1040, 3)


def test_pieces_of_clusters_hold_extreme_scores():
    """Warps of a cluster whose maxima lie so far apart that all but one piece's weights vanish, and equal ones."""
    pa = lib()
    gen = torch.Generator().manual_seed(12)
    lens, bs, Hkv, D = [1000, 1000, 33], 16, 2, 128
    pool = [t.cuda() for t in make_pool(gen, 140, Hkv, bs, D, "f16")]
    bt = block_table(lens, bs, 140, gen).cuda()
    q = torch.randn(3, 4, D, generator=gen).half().cuda()
    q[1] = 0  # equal weights
    cl = torch.tensor(lens, dtype=torch.int32).cuda()
    for scale in (20.0, -20.0, 0.0):
        out = torch.empty_like(q)
        pa.decode_window(out, q, *pool, bt, cl, scale, 900, num_sinks=2)
        want, tol = R.reference(q[:, None].cpu(), rows_of([t.cpu() for t in pool], bt.cpu(), lens, bs, 1.0), lens, 1, Hkv, scale, 900, 2,
                                torch.float16, weight_eps("f16"))
        worst = ((out.cpu().double().view(want.shape) - want).abs() / tol.clamp_min(1e-300)).max()
        assert float(worst) <= 1.0, "error %g of the bound" % worst
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("kv", ["f16", "e4m3"])
def test_lengths_and_ids_out_of_range_on_the_line(kv):
    """More contexts than there is room for: a bad length is recorded and taken as the nearest good one, a bad block
    id is recorded, and the other contexts' outputs stay."""
    pa = lib()
    gen = torch.Generator().manual_seed(9)
    S, bs, D = 700, 16, 64
    pool = [t.cuda() for t in make_pool(gen, 8, 1, bs, D, kv)]
    q = torch.randn(S, 2, D, generator=gen).half().cuda()
    bt = torch.randint(0, 8, (S, 3), generator=gen, dtype=torch.int32).cuda()
    lens = torch.randint(0, 3 * bs + 1, (S,), generator=gen, dtype=torch.int32)
    lens[[3, 350, 699]] = 40

    def run(cl, table):
        out = torch.full_like(q, 5.0)
        pa.decode_window(out, q, *pool, table, cl.cuda(), 0.1, 20, num_sinks=1)
        return out, pa.get_device_error()

    want, err = run(lens, bt)
    assert err == 0
    others = [s for s in range(S) if s not in (3, 350, 699)]
    for bad, at_most in ((-5, 0), (3 * bs + 7, 3 * bs)):
        cl = lens.clone()
        cl[[3, 350, 699]] = bad
        got, err = run(cl, bt)
        assert err == pa.DEVERR_CONTEXT_LEN
        cl[[3, 350, 699]] = at_most  # the same cuts of the line, so the same bits, the others' too
        clamped, err = run(cl, bt)
        assert err == 0 and torch.equal(got, clamped)
    table = bt.clone()
    table[[3, 350, 699], 2] = 8
    got, err = run(lens, table)
    assert err == pa.DEVERR_BLOCK_ID and torch.equal(got[others], want[others])


@pytest.mark.parametrize("form,S,C,Hq,Hkv,D,kv,L,window", [
    ("prefill", 1, 37, 8, 2, 128, "bf16", 900, 500),    # an item's tiles shared by a cluster
    ("prefill", 20, 40, 6, 6, 64, "bf16", 300, 120),    # packed groups
    ("prefill", 3, 50, 6, 2, 64, "e4m3", 300, 120),
    ("prefill", 20, 128, 8, 2, 128, "bf16", 900, 500),  # pairs of heads
    ("prefill", 20, 128, 8, 2, 64, "bf16", 900, 500),
    ("decode", 3, 1, 8, 2, 128, "bf16", 900, 500),      # clusters
    ("decode", 400, 2, 4, 2, 64, "e4m3", 90, 40),       # the line
    ("decode", 230, 1, 8, 4, 64, "bf16", 1300, 1100),   # a CTA each
])
def test_inputs_rewritten_right_before(form, S, C, Hq, Hkv, D, kv, L, window):
    """Queries, rows, tables and lengths that the kernels before rewrite in place, called and from a graph."""
    pa = lib()
    gen = torch.Generator().manual_seed(S + D)
    bs, NB, nb = 16, 120, -(-L // 16)
    sets = []
    for _ in range(3):
        pool = [t.view(torch.uint8) if kv == "e4m3" else t for t in make_pool(gen, NB, Hkv, bs, D, kv)]
        sets.append([t.cuda() for t in (torch.randn(S, C, Hq, D, generator=gen).bfloat16(), *pool,
                                        torch.randint(0, NB, (S, nb), generator=gen, dtype=torch.int32),
                                        torch.randint(L // 2, L + 1, (S,), generator=gen, dtype=torch.int32))])
    ws = torch.empty(pa.decode_flat_workspace_size(D), dtype=torch.uint8).cuda()

    def call(out, q, k, v, bt, cl):
        if form == "prefill":
            pa.prefill_window(out, q, k, v, bt, cl, 0.1, window, num_sinks=3)
        else:
            pa.decode_window(out, q, k, v, bt, cl, 0.1, window, num_sinks=3, workspace=ws)

    def typed(args):
        return [a.view(E4M3) if a.dtype == torch.uint8 else a for a in args]

    want = []
    for args in sets:
        want.append(torch.full_like(args[0], 7.0))
        call(want[-1], *typed(args))
        torch.cuda.synchronize()
    held = [torch.empty_like(t) for t in sets[0]]
    outs = [torch.full_like(held[0], 7.0) for _ in range(12)]
    for i, out in enumerate(outs):
        for t, new in zip(held, sets[i % 3]):
            t.copy_(new)
        call(out, *typed(held))
    assert all(torch.equal(out, want[i % 3]) for i, out in enumerate(outs))
    graph, i = torch.cuda.CUDAGraph(), torch.zeros(1, dtype=torch.int64, device="cuda")
    stacks = [torch.stack(x) for x in zip(*sets)]
    out = torch.full_like(held[0], 7.0)
    with torch.cuda.graph(graph):
        for t, stack in zip(held, stacks):
            t.copy_(stack.index_select(0, i)[0])
        call(out, *typed(held))
        call(out, *typed(held))
    for n in (2, 0, 1, 1, 2):
        i.fill_(n)
        graph.replay()
        assert torch.equal(out, want[n])
    assert pa.get_device_error() == 0


def test_streams_at_the_same_time():
    """Prefill and decode calls of two streams that run beside one another, each with a workspace of its own."""
    pa = lib()
    gen = torch.Generator().manual_seed(13)
    bs, Hkv, Hq, D, NB, L = 16, 2, 8, 128, 130, 1000
    pool = [t.cuda() for t in make_pool(gen, NB, Hkv, bs, D, "bf16")]
    bt = torch.randint(0, NB, (2, -(-L // bs)), generator=gen, dtype=torch.int32).cuda()
    cl = torch.tensor([L, L - 77], dtype=torch.int32).cuda()
    q = torch.randn(2, 37, Hq, D, generator=gen).bfloat16().cuda()
    last = q[:, -1].contiguous()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(pa.decode_flat_workspace_size(D), dtype=torch.uint8).cuda() for _ in streams]
    pre, dec = torch.empty_like(q), torch.empty_like(last)
    pa.prefill_window(pre, q, *pool, bt, cl, 0.1, 600, num_sinks=2)
    pa.decode_window(dec, last, *pool, bt, cl, 0.1, 600, num_sinks=2, workspace=ws[0])
    outs = [[(torch.empty_like(q), torch.empty_like(last)) for _ in range(20)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for n, st in enumerate(streams):
            with torch.cuda.stream(st):
                pa.prefill_window(outs[n][i][0], q, *pool, bt, cl, 0.1, 600, num_sinks=2)
                pa.decode_window(outs[n][i][1], last, *pool, bt, cl, 0.1, 600, num_sinks=2, workspace=ws[n])
    torch.cuda.synchronize()
    assert all(torch.equal(a, pre) and torch.equal(b, dec) for o in outs for a, b in o)
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("k,Hq", [(1, 1), (5, 1), (1, 7), (3, 3), (1, 11), (5, 3)])
@pytest.mark.parametrize("S", [1, 40, 90, 250])
def test_clusters_join_odd_numbers_of_columns(S, k, Hq, kv):
    """64 channels and an odd number of query columns: half a warp has nothing to join.  By clusters of eight, four and
    two CTAs, by one CTA each and by the line; contexts of all of a cluster's warps, of some and of one."""
    lens = [(397 * i + 1203) % 1600 for i in range(S)]
    dt = "f16" if kv == "e4m3" else kv
    check("decode", lib(), lens, k, Hq, 1, 64, 16, dt, kv, 1100, 3, seed=S + k)


@pytest.mark.parametrize("pairs,S,C,Hq,Hkv,D,kv,window", [
    (False, 8, 300, 18, 6, 128, "e4m3", 40),    # groups of three: 42 tokens an item, one tile and several
    (False, 8, 300, 18, 6, 128, "e4m3", 600),
    (False, 8, 300, 18, 6, 64, "e4m3", 40),
    (False, 8, 300, 18, 6, 64, "e4m3", 600),
    (False, 8, 300, 24, 6, 128, "e4m3", 600),   # groups of four
    (False, 8, 300, 24, 6, 64, "e4m3", 40),
    (False, 8, 300, 18, 6, 128, "16", 40),
    (False, 8, 300, 18, 6, 64, "16", 600),
    (False, 8, 300, 24, 6, 128, "16", 40),
    (True, 10, 380, 24, 6, 128, "16", 200),     # clusters of two, three query tiles
    (True, 10, 380, 24, 6, 128, "16", 600),
    (True, 14, 380, 12, 6, 128, "16", 200),     # a CTA each
    (True, 14, 380, 12, 6, 64, "16", 600),
])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_prefill_of_more_items_than_there_are_places(dt, pairs, S, C, Hq, Hkv, D, kv, window):
    """Each CTA (or cluster) has several work items, of different lengths and some with nothing to attend to: rings,
    barriers and accumulators go on from one item to the next."""
    G, sms = Hq // Hkv, torch.cuda.get_device_properties(0).multi_processor_count
    if pairs:
        in_clusters = D == 128 and G % 4 == 0
        items = S * Hkv * (G // 2) * -(-C // 128) // (2 if in_clusters else 1)
        assert items > (sms // 2 if in_clusters else sms)
    else:
        items = S * Hkv * -(-C // (128 // G))
        assert items > 2 * sms
    lens = [700, 0, 1, 65, C, C + 1, C - 1, 1000, 512, 3, 0, 841, 140, 250][:S]
    check("prefill", lib(), lens, C, Hq, Hkv, D, 16, dt, dt if kv == "16" else kv, window, 3, seed=C + window)
