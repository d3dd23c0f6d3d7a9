"""What a query row does not attend to leaves its output alone, whatever its size: V rows of large scales that a
causal mask hides, and rows whose weight is 0 beside a dominant row of zeros (row-scaled caches)."""
import pytest
import torch

from tests import _gpu
from tests import _ref64 as R
from tests.test_gpu_cache_ops import close, decode_rows_reference, gen, lost, randn, rows_pool

pytestmark = pytest.mark.gpu


def flushed(v, vs, bt, lens, bs):
    """Weights below 2^-126 of the largest are 0: with a sum of weights of 1 at least, each takes up to 2^-126 |v|."""
    wide, most = R.wide(v).abs(), torch.zeros(len(lens), 1, 1, 1, dtype=torch.float64)
    for s, L in enumerate(lens):
        ids = bt[s, : -(-L // bs)].long()
        most[s] = (wide[ids].amax(-1) * vs[ids].double()).amax() * L if L else 0.0
    return most * 2.0 ** -126


def check(pa, q, k, v, ks, vs, bt, lens, scale, bs, P):
    D = q.shape[-1]
    ref, A, d = decode_rows_reference(q, k, v, ks, vs, bt, lens, scale, bs)
    qd = (q if q.shape[1] > 1 else q[:, 0]).contiguous().cuda()
    out = torch.full_like(qd, float("nan"))
    pa.decode_rows(out, qd, k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), bt.cuda(),
                   torch.tensor(lens, dtype=torch.int32).cuda(), scale, max_context_len=max(lens), partition_size=P)
    assert pa.get_device_error() == 0
    bound = R.attention_bound(ref, A, d, D, torch.bfloat16, torch.float16) + lost(lens, A) + flushed(v, vs, bt, lens, bs)
    close(out.view(ref.shape), ref, bound)


@pytest.mark.parametrize("P", [0, 64])
@pytest.mark.parametrize("n,Hq,Hkv,D", [(2, 2, 2, 128), (2, 8, 2, 64), (4, 8, 2, 128), (16, 2, 2, 64)])
def test_new_tokens_of_large_v_scales_are_masked_for_the_others(n, Hq, Hkv, D, P):
    """Slices of 16 (8 columns) and 32 tokens (16 columns) that hold new tokens only: the earlier of these see nothing
    in them."""
    pa = _gpu.lib()
    bs = 16
    lens = [n, 17, 18, 33, 34, 65, 81, 97, 113, 129, 200]
    for e in (3, 20, 60):
        g = gen(e + n)
        NB = sum(-(-x // bs) for x in lens) + 2
        k, v, ks, vs = rows_pool(g, NB, Hkv, bs, D)
        bt = R.block_table(lens, bs, NB, g)
        for s, L in enumerate(lens):
            for t in range(max(L - n + 1, 0), L):
                vs[bt[s, t // bs], :, t % bs] *= 2.0 ** e
        q = randn(g, len(lens), n, Hq, D).bfloat16()
        check(pa, q, k, v, ks, vs, bt, lens, D ** -0.5, bs, P)


@pytest.mark.parametrize("P", [0, 64])
@pytest.mark.parametrize("Hq,n", [(8, 1), (32, 1), (8, 2)])
@pytest.mark.parametrize("gap", [60, 80, 86, 100, 150])
def test_a_dominant_row_of_zeros(Hq, n, gap, P):
    """The token with the weight has a V row of zeros (the least scale); the others score `gap` below it."""
    pa = _gpu.lib()
    g = gen(gap + Hq)
    D, bs, Hkv, lens = 128, 16, 2, [200, 64, 17, 90]
    NB = sum(-(-x // bs) for x in lens) + 2
    k, v, ks, vs = rows_pool(g, NB, Hkv, bs, D)
    bt = R.block_table(lens, bs, NB, g)
    q = torch.ones(len(lens), n, Hq, D).bfloat16()
    ks *= 2.0 ** -12
    vs.clamp_(min=4.0)
    scale = gap / (D * 448.0 / 64)
    for s, t in enumerate([150, 3, 9, 70]):
        b = int(bt[s, t // bs])
        k[b, :, t % bs], ks[b, :, t % bs] = torch.full((Hkv, D), 448.0).to(R.E4M3), 1 / 64
        v[b, :, t % bs], vs[b, :, t % bs] = torch.zeros(Hkv, D).to(R.E4M3), R.LEAST
    check(pa, q, k, v, ks, vs, bt, lens, scale, bs, P)


@pytest.mark.parametrize("n,Hq,Hkv", [(1, 2, 2), (1, 8, 2), (3, 8, 2), (16, 2, 2)])
@pytest.mark.parametrize("shift", [-80, 0, 60])
def test_scales_of_any_size_against_the_weights_they_have(n, Hq, Hkv, shift):
    """V scales by powers of two from 2^-30 to 2^20 around 2^shift, growing, falling and mixed along the context: the
    slack is of the largest weight times scale of each query row, not of the largest scale."""
    pa = _gpu.lib()
    g = gen(9 + n)
    NB, bs, D, L = 32, 16, 64, 500
    k, v, ks, vs = rows_pool(g, NB, Hkv, bs, D)
    bt = torch.arange(NB, dtype=torch.int32)[None]
    e = torch.linspace(-30, 20, NB * bs).round()
    for order in (e, e.flip(0), e[torch.randperm(NB * bs, generator=g)]):
        vs2 = torch.exp2(order + shift).view(NB, 1, bs).expand(NB, Hkv, bs).contiguous()
        q = randn(g, 1, n, Hq, D).bfloat16()
        for P in (0, 128):
            check(pa, q, k, v, ks, vs2, bt, [L], 0.125, bs, P)


@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_an_infinite_query_leaves_the_other_heads(G, bad):
    """E4M3 caches, whose queries share a power of two into f16's range."""
    pa = _gpu.lib()
    g = gen(G)
    bs, D, Hkv, lens = 16, 128, 2, [200, 64, 17]
    NB = sum(-(-x // bs) for x in lens) + 2
    k, v, ks, vs = rows_pool(g, NB, Hkv, bs, D)
    bt = R.block_table(lens, bs, NB, g)
    q = randn(g, 3, 1, G * Hkv, D).bfloat16()
    q[:, 0, 1, 7] = bad
    others = [h for h in range(G * Hkv) if h != 1]
    cl = torch.tensor(lens, dtype=torch.int32).cuda()
    qd, kd, vd, one = q[:, 0].contiguous().cuda(), k.cuda(), v.cuda(), torch.ones(NB, Hkv, bs)
    rows = decode_rows_reference(q, k, v, ks, vs, bt, lens, 0.05, bs)
    plain = decode_rows_reference(q, k, v, one, one, bt, lens, 0.05 / 64, bs)
    tables, tl = bt[:, None].expand(-1, Hkv, -1).contiguous().cuda(), cl[:, None].expand(-1, Hkv).contiguous()
    for P in (0, 64):
        outs = [torch.full_like(qd, float("nan")) for _ in range(3)]
        pa.decode_rows(outs[0], qd, kd, vd, ks.cuda(), vs.cuda(), bt.cuda(), cl, 0.05, 200, P)
        pa.decode_selected(outs[1], qd, kd, vd, tables, tl, 0.05 / 64, 1.0, P)
        args = (outs[2], qd, kd, vd, bt.cuda(), cl, 0.05 / 64, 1.0)
        pa.decode_split(*args, 200, P) if P else pa.decode(*args)
        assert pa.get_device_error() == 0
        for out, (ref, A, d), slack in zip(outs, (rows, plain, plain), (lost(lens, rows[1]), 0.0, 0.0)):
            bound = R.attention_bound(ref, A, d, D, torch.bfloat16, torch.float16) + slack
            close(out.view(ref.shape)[:, :, others], ref[:, :, others], bound[:, :, others])


@pytest.mark.parametrize("P", [0, 64])
@pytest.mark.parametrize("n,Hq,Hkv,D", [(2, 2, 2, 128), (3, 6, 2, 64), (2, 16, 2, 128), (4, 4, 1, 64), (16, 2, 2, 64), (5, 3, 1, 128)])
def test_a_nan_in_a_new_tokens_v_row_shows_where_it_is_seen(n, Hq, Hkv, D, P):
    """In its channel, for this new token and those after it; the NaN keys of later tokens do not show either."""
    pa = _gpu.lib()
    g = gen(n + D)
    bs, lens = 16, [n, 16, 17, 33, 64, 66, 79, 130, 200]
    NB = sum(-(-x // bs) for x in lens) + 2
    k, v, ks, vs = rows_pool(g, NB, Hkv, bs, D)
    bt = R.block_table(lens, bs, NB, g)
    kb, vb = k.view(torch.uint8), v.view(torch.uint8)
    for s, L in enumerate(lens):
        for j, d in ((n - 1, 5), (s % n, 9 + s)):  # the last new token, and another
            t = L - n + j
            vb[bt[s, t // bs], :, t % bs, d] = 0x7F if s % 2 else 0xFF
        if s == 4:
            kb[bt[s, (L - 1) // bs], 0, (L - 1) % bs, 3] = 0x7F
    q = randn(g, len(lens), n, Hq, D).bfloat16()
    ref, A, d = decode_rows_reference(q, k, v, ks, vs, bt, lens, D ** -0.5, bs)
    out = torch.full_like(q, 7.0).cuda()
    pa.decode_rows(out, q.cuda(), k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), bt.cuda(),
                   torch.tensor(lens, dtype=torch.int32).cuda(), D ** -0.5, max_context_len=max(lens), partition_size=P)
    assert pa.get_device_error() == 0
    got = out.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    A = torch.nan_to_num(A)
    bound = R.attention_bound(torch.nan_to_num(ref), A, torch.nan_to_num(d), D, torch.bfloat16, torch.float16) + lost(lens, A)
    assert (((got - ref).abs() <= bound) | torch.isnan(ref)).all()
