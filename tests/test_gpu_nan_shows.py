"""A NaN among the keys or in a query row, and scores that are infinite, come out as NaN rows, as the formulas have
them, in every form of the decode; the other rows are those of the reference, and rows that see no token are 0."""
import pytest
import torch

from tests import _gpu
from tests import _ref64 as R
from tests.test_gpu_cache_ops import decode_rows_reference, gen, lost, pool16, randn, rows_pool

pytestmark = pytest.mark.gpu
nan = float("nan")


def agree(got, ref, bound):
    got = got.cpu().double().view(ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    live = ~torch.isnan(ref)
    assert ((got - ref).abs()[live] <= bound.expand(ref.shape)[live]).all()


def batch(g, lens, bs, extra=0):
    NB = sum(-(-x // bs) for x in lens) + 2
    bt = R.block_table(lens, bs, NB, g)
    if extra > bt.shape[1]:  # room for long contexts in the table, none used
        bt = torch.cat([bt, bt.new_full((len(lens), extra - bt.shape[1]), -1)], 1)
    return NB, bt


# contexts of one NaN key, of only NaN keys (a warp's, a CTA's, a partition's, all of them), and without any
LENS = [1, 0, 70, 300, 300, 300, 64, 40]


def spoil_key(k, b, o):
    k[b, 0, o, 3:4] = torch.tensor([nan]).to(k.dtype)


def spoil(put, bt, bs):
    """put(block, offset) for the NaN tokens of LENS."""
    spoilt = [(0, 0), (2, 69), (4, 200)] + [(3, t) for t in range(128, 192)] + [(5, t) for t in range(300)] + \
        [(6, t) for t in range(16, 32)]
    for s, t in spoilt:
        put(int(bt[s, t // bs]), t % bs)


@pytest.mark.parametrize("P", [0, 64])
@pytest.mark.parametrize("n,Hq,Hkv,D", [(1, 2, 2, 128), (1, 8, 2, 128), (1, 16, 1, 64), (3, 8, 2, 64), (2, 16, 1, 128)])
def test_decode_rows(n, Hq, Hkv, D, P):
    pa = _gpu.lib()
    g = gen(n + Hq)
    bs = 16
    NB, bt = batch(g, LENS, bs)
    k, v, ks, vs = rows_pool(g, NB, Hkv, bs, D)
    q = randn(g, len(LENS), n, Hq, D).bfloat16()
    q[7, 0, 1, 5] = nan  # one query row

    spoil(lambda b, o: spoil_key(k, b, o), bt, bs)
    ref, A, d = decode_rows_reference(q, k, v, ks, vs, bt, LENS, D ** -0.5, bs)
    assert torch.isnan(ref[[0, 2, 3, 4, 5, 6], -1, 0]).all() and torch.isnan(ref[7, 0, 1]).all()
    qd = (q if n > 1 else q[:, 0]).contiguous().cuda()
    out = torch.full_like(qd, 7.0)
    pa.decode_rows(out, qd, k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), bt.cuda(),
                   torch.tensor(LENS, dtype=torch.int32).cuda(), D ** -0.5, max_context_len=300, partition_size=P)
    assert pa.get_device_error() == 0
    A, d = torch.nan_to_num(A), torch.nan_to_num(d)
    agree(out, ref, R.attention_bound(ref, A, d, D, torch.bfloat16, torch.float16) + lost(LENS, A))


def reference16(q, k, v, bt, lens, scale, bs, factor=1.0):
    """(out, A, d) of [S, k, Hq] rows over a pool without row scales."""
    NB, Hkv = k.shape[:2]
    one = torch.full((NB, Hkv, bs), factor)
    return decode_rows_reference(q, k, v, one, one, bt, lens, scale, bs)


@pytest.mark.parametrize("P", [0, 64])
@pytest.mark.parametrize("Hq,Hkv,D,kv", [(2, 2, 128, "bf16"), (6, 2, 64, "f16"), (8, 2, 128, "e4m3"), (16, 1, 64, "bf16")])
def test_decode_selected(Hq, Hkv, D, kv, P):
    pa = _gpu.lib()
    g = gen(Hq + D)
    bs, dt = 16, "f16" if kv == "f16" else "bf16"
    NB, bt = batch(g, LENS, bs)
    k, v = (pool16(g, NB, Hkv, bs, D, dt, kv) for _ in range(2))
    q = randn(g, len(LENS), 1, Hq, D).to(R.DT[dt])
    q[7, 0, 1, 5] = nan
    spoil(lambda b, o: spoil_key(k, b, o), bt, bs)
    ref, A, d = reference16(q, k, v, bt, LENS, D ** -0.5, bs, 0.5 if kv == "e4m3" else 1.0)
    out = torch.full_like(q[:, 0], 7.0).cuda()
    pa.decode_selected(out, q[:, 0].cuda(), k.cuda(), v.cuda(), bt[:, None].expand(-1, Hkv, -1).contiguous().cuda(),
                       torch.tensor(LENS, dtype=torch.int32)[:, None].expand(-1, Hkv).contiguous().cuda(), D ** -0.5,
                       0.5 if kv == "e4m3" else 1.0, P)
    assert pa.get_device_error() == 0
    A, d = torch.nan_to_num(A), torch.nan_to_num(d)
    agree(out, ref, R.attention_bound(ref, A, d, D, R.DT[dt], torch.bfloat16 if kv == "bf16" else torch.float16))


def test_a_nan_key_is_chosen_and_shows():
    """From the write of the key to the output of the decode over the chosen blocks."""
    pa = _gpu.lib()
    g = gen(3)
    Hkv, Hq, D, bs, L, n = 2, 8, 64, 16, 900, 4
    NB, bt = batch(g, [L], bs)
    k, v = (pool16(g, NB, Hkv, bs, D, "bf16", "bf16").cuda() for _ in range(2))
    key, val = randn(g, 1, Hkv, D).bfloat16(), randn(g, 1, Hkv, D).bfloat16()
    key[0, 1, 9] = nan
    q = randn(g, 1, Hq, D).bfloat16().cuda()
    q_out = torch.empty_like(q)
    slot = int(bt[0, 300 // bs]) * bs + 300 % bs
    pa.norm_rope_cache(q_out, q, key.cuda(), val.cuda(), None, None, k, v, torch.tensor([slot]).cuda())
    bounds = torch.zeros((NB, Hkv, 2, D), dtype=torch.bfloat16, device="cuda")
    bt, cl = bt.cuda(), torch.tensor([L], dtype=torch.int32).cuda()
    pa.block_bounds(bounds, k, bt, cl, L)
    scores = torch.empty((1, Hkv, bt.shape[1]), device="cuda")
    pa.block_scores(scores, q_out, bounds, bt, cl, bs)
    tables, lens = torch.empty((1, Hkv, n), dtype=torch.int32).cuda(), torch.empty((1, Hkv), dtype=torch.int32).cuda()
    pa.select_blocks(tables, lens, scores, bt, cl, bs)
    assert int(bt[0, 300 // bs]) in tables[0, 1].tolist()
    out = torch.zeros_like(q)
    pa.decode_selected(out, q_out, k, v, tables, lens, 0.125)
    assert torch.isnan(out[0, 4:]).all() and torch.isfinite(out[0, :4]).all()
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("P", [0, 64])
@pytest.mark.parametrize("n,Hq,Hkv,D,kv", [(1, 2, 2, 128, "bf16"), (1, 6, 2, 64, "f16"), (1, 8, 2, 128, "e4m3"),
                                           (3, 8, 2, 128, "bf16"), (1, 32, 1, 128, "bf16"), (4, 16, 2, 64, "e4m3"),
                                           (20, 2, 2, 128, "f16")])
def test_the_decodes_over_one_table(n, Hq, Hkv, D, kv, P):
    """pa_decode, pa_decode_split and their forms for several new tokens, on the warp-MMA and the tensor-core kernel."""
    pa = _gpu.lib()
    g = gen(n + Hq + D)
    bs, dt = 16, "f16" if kv == "f16" else "bf16"
    lens = [max(L, n) if L else 0 for L in LENS]
    NB, bt = batch(g, lens, bs)
    k, v = (pool16(g, NB, Hkv, bs, D, dt, kv) for _ in range(2))
    q = randn(g, len(lens), n, Hq, D).to(R.DT[dt])
    q[7, 0, 1, 5] = nan
    spoil(lambda b, o: spoil_key(k, b, o), bt, bs)
    f = 0.5 if kv == "e4m3" else 1.0
    ref, A, d = reference16(q, k, v, bt, lens, D ** -0.5, bs, f)
    cl = torch.tensor(lens, dtype=torch.int32).cuda()
    qd = (q if n > 1 else q[:, 0]).contiguous().cuda()
    out = torch.full_like(qd, 7.0)
    args = (out, qd, k.cuda(), v.cuda(), bt.cuda(), cl, D ** -0.5)
    if n == 1:
        pa.decode_split(*args, f, 300, P) if P else pa.decode(*args, f)
    else:
        pa.decode_multi_split(*args, f, 300, P) if P else pa.decode_multi(*args, f)
    assert pa.get_device_error() == 0
    A, d = torch.nan_to_num(A), torch.nan_to_num(d)
    agree(out, ref, R.attention_bound(ref, A, d, D, R.DT[dt], torch.bfloat16 if kv == "bf16" else torch.float16))


@pytest.mark.parametrize("Hq,D,kv", [(8, 128, "bf16"), (4, 64, "f16"), (6, 128, "e4m3")])
def test_prefill(Hq, D, kv):
    pa = _gpu.lib()
    g = gen(Hq + D)
    bs, dt, Hkv, C = 16, "f16" if kv == "f16" else "bf16", 2, 150
    lens = [150, 300]
    NB, bt = batch(g, lens, bs)
    k, v = (pool16(g, NB, Hkv, bs, D, dt, kv) for _ in range(2))
    q = randn(g, 2, C, Hq, D).to(R.DT[dt])
    q[1, 7, 1, 5] = nan
    spoil_key(k, int(bt[0, 100 // bs]), 100 % bs)  # new tokens 100 on see it
    f = 0.5 if kv == "e4m3" else 1.0
    ref, A, d = reference16(q, k, v, bt, lens, D ** -0.5, bs, f)
    out = torch.full_like(q, 7.0).cuda()
    pa.prefill(out, q.cuda(), k.cuda(), v.cuda(), bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), D ** -0.5, f)
    assert pa.get_device_error() == 0
    A, d = torch.nan_to_num(A), torch.nan_to_num(d)
    agree(out, ref, R.attention_bound(ref, A, d, D, R.DT[dt], R.DT[dt]))  # E4M3 blocks are widened to q's type, in which the weights are, too


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("P", [0, 64])
def test_infinite_scores(sign, P):
    """A query of an infinite channel over keys that are positive there: every score is +inf or every one -inf, whose
    softmax is not a number."""
    pa = _gpu.lib()
    g = gen(2)
    Hkv, Hq, D, bs, lens = 2, 8, 64, 16, [200, 5, 0]
    NB, bt = batch(g, lens, bs)
    k, v, ks, vs = rows_pool(g, NB, Hkv, bs, D)
    k16, v16 = (pool16(g, NB, Hkv, bs, D, "bf16", "bf16") for _ in range(2))
    k[..., 11:12], k16[..., 11] = torch.ones(NB, Hkv, bs, 1).to(R.E4M3), 1.0
    q = randn(g, 3, Hq, D).bfloat16()
    q[:, 2, 11] = sign * float("inf")
    cl = torch.tensor(lens, dtype=torch.int32).cuda()
    outs = [torch.full_like(q, 7.0).cuda() for _ in range(3)]
    pa.decode_rows(outs[0], q.cuda(), k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), bt.cuda(), cl, 0.1, 200, P)
    pa.decode_selected(outs[1], q.cuda(), k16.cuda(), v16.cuda(), bt[:, None].expand(-1, Hkv, -1).contiguous().cuda(),
                       cl[:, None].expand(-1, Hkv).contiguous(), 0.1, 1.0, P)
    args = (outs[2], q.cuda(), k16.cuda(), v16.cuda(), bt.cuda(), cl, 0.1)
    pa.decode_split(*args, 1.0, 200, P) if P else pa.decode(*args)
    for out in outs:
        assert torch.isnan(out[:2, 2]).all()
        assert (out[2] == 0).all()
        assert torch.isfinite(out[:2, [0, 1, 3, 4, 5, 6, 7]]).all()
    assert pa.get_device_error() == 0
