"""The cache-side operators on the GPU against plain 64-bit references
(tests/_ref64.py): row-scaled caches, norm + rotation + cache write, block
bounds, scores and selection, and the decode over the chosen blocks; alone,
together as a serving step uses them, and captured in a graph."""
import pytest
import torch

from tests import _gpu
from tests import _ref64 as R

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g)


def close(got, want, bound):
    got = got.cpu().double()
    assert torch.isfinite(got).all()
    over = (got - want).abs() - bound
    assert float(over.max()) <= 0, "off by %g more than the bound" % float(over.max())


def rows_pool(g, NB, Hkv, bs, D):
    """A row-scaled K and V pool with rows of very different size."""
    pool = []
    for _ in range(2):
        codes, s = R.quantise_rows(randn(g, NB, Hkv, bs, D) * torch.exp(1.5 * randn(g, NB, Hkv, bs, 1)))
        pool += [codes, s]
    return pool[0], pool[2], pool[1], pool[3]  # k, v, k scales, v scales


# ---- row-scaled caches ------------------------------------------------------

@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,Hkv,D,bs", [(1, 1, 64, 8), (7, 3, 128, 16), (130, 8, 64, 32), (513, 2, 128, 8)])
def test_rows_written_and_read_back_bit_exact(dt, T, Hkv, D, bs):
    pa = _gpu.lib()
    g = gen(T)
    NB = T // bs + 4
    x = [(randn(g, T, Hkv, D) * torch.exp(2 * randn(g, T, Hkv, 1))).to(R.DT[dt]) for _ in range(2)]
    x[0][0] = 0.0  # a row of zeros
    if T > 6:
        x[0][1, 0, 3], x[0][2, 0, 5], x[0][3, 0] = float("inf"), float("nan"), float("nan")
        x[1][4, 0, :] = torch.finfo(R.DT[dt]).tiny  # rows of tiny values
        x[1][5, 0, :] = torch.finfo(R.DT[dt]).max
    slots = torch.randperm(NB * bs, generator=g)[:T]
    if T > 6:
        slots[6] = -1
    caches = [torch.full((NB, Hkv, bs, D), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((NB, Hkv, bs), 7.0, device="cuda") for _ in range(2)]
    pa.reshape_and_cache_rows(x[0].cuda(), x[1].cuda(), *caches, *scales, slots.cuda())
    live = slots >= 0
    ids = torch.randperm(NB, generator=g)[: NB - 1]
    dst = [torch.full((len(ids), Hkv, bs, D), 3.0, dtype=R.DT[dt], device="cuda") for _ in range(2)]
    pa.gather_blocks_rows(*dst, *caches, *scales, ids.cuda())
    for i in range(2):
        codes, s = R.quantise_rows(x[i][live])
        want = torch.full((NB, Hkv, bs, D), 0x55, dtype=torch.uint8)
        want[slots[live] // bs, :, slots[live] % bs] = codes.view(torch.uint8)
        ws = torch.full((NB, Hkv, bs), 7.0)
        ws[slots[live] // bs, :, slots[live] % bs] = s
        assert R.same_codes(caches[i], want)
        assert torch.equal(scales[i].cpu(), ws)
        back = (want.view(R.E4M3).float()[ids] * ws[ids][..., None]).to(R.DT[dt])
        assert torch.equal(torch.nan_to_num(dst[i].cpu(), nan=123.0), torch.nan_to_num(back, nan=123.0))
    assert pa.get_device_error() == 0


def test_rows_outside_the_pool_are_skipped_and_recorded():
    pa = _gpu.lib()
    g = gen(1)
    x = randn(g, 3, 2, 64).half().cuda()
    caches = [torch.zeros((2, 2, 8, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((2, 2, 8), device="cuda") for _ in range(2)]
    pa.reshape_and_cache_rows(x, x, *caches, *scales, torch.tensor([16, 1 << 40, -5], device="cuda"))
    assert pa.get_device_error() == pa.DEVERR_SLOT
    assert not caches[0].any() and not scales[1].any()
    dst = [torch.full((2, 2, 8, 64), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pa.gather_blocks_rows(*dst, *caches, *scales, torch.tensor([2, -1], device="cuda"))
    assert pa.get_device_error() == pa.DEVERR_BLOCK_ID
    assert (dst[0] == 3).all() and (dst[1] == 3).all()


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 130, 513, 1025]


def decode_rows_reference(q, k, v, ks, vs, bt, lens, scale, bs):
    """(out, A, d) per [S, k, Hq] row, d broadcast over the channels."""
    S, n, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    k, v = R.wide(k) * ks.double()[..., None], R.wide(v) * vs.double()[..., None]
    out, A, d = (torch.zeros(S, n, Hq, D, dtype=torch.float64) for _ in range(3))
    for s in range(S):
        ids = bt[s, : -(-lens[s] // bs)].long()
        for h in range(Hq):
            kk, vv = k[ids, h // G].flatten(0, 1), v[ids, h // G].flatten(0, 1)
            for j in range(n):
                t = max(lens[s] - n + j + 1, 0)
                out[s, j, h], A[s, j, h], d[s, j, h] = R.attend(q[s, j, h].double(), kk[:t], vv[:t], scale)
    return out, A, d


@pytest.mark.parametrize("P", [0, 64, 256])
@pytest.mark.parametrize("Hq,Hkv,D,bs,dt,n", [
    (8, 2, 128, 16, "bf16", 1), (3, 3, 64, 8, "f16", 1), (6, 2, 128, 32, "f16", 1), (4, 4, 128, 16, "bf16", 1),
    (16, 1, 64, 16, "bf16", 1), (8, 1, 128, 16, "f16", 1), (40, 1, 128, 16, "bf16", 1), (17, 1, 64, 16, "f16", 1),
    (8, 2, 128, 16, "bf16", 3), (12, 1, 128, 8, "f16", 2), (2, 2, 64, 16, "bf16", 16)])
def test_decode_rows(Hq, Hkv, D, bs, dt, n, P):
    pa = _gpu.lib()
    g = gen(Hq + n)
    lens = LENS
    NB = sum(-(-x // bs) for x in lens) + 3
    k, v, ks, vs = rows_pool(g, NB, Hkv, bs, D)
    bt = R.block_table(lens, bs, NB, g)
    # what lies behind a context is never read into a result
    dead = torch.ones(NB, bs, dtype=torch.bool)
    for s, L in enumerate(lens):
        for j in range(-(-L // bs)):
            dead[bt[s, j], : min(bs, L - j * bs)] = False
    dead = dead[:, None, :].expand(NB, Hkv, bs)
    for codes, sc in ((k, ks), (v, vs)):
        codes.view(torch.uint8)[dead] = 0x7F
        sc[dead] = float("nan")
    q = randn(g, len(lens), n, Hq, D).to(R.DT[dt])
    scale = D ** -0.5
    ref, A, d = decode_rows_reference(q, k, v, ks, vs, bt, lens, scale, bs)
    qd = q.cuda() if n > 1 else q[:, 0].contiguous().cuda()
    args = (k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scale)
    out = torch.full_like(qd, float("nan"))
    pa.decode_rows(out, qd, *args, max_context_len=max(lens), partition_size=P)
    assert pa.get_device_error() == 0
    close(out.view(ref.shape), ref, R.attention_bound(ref, A, d, D, R.DT[dt], torch.float16))
    again = torch.full_like(qd, float("nan"))
    pa.decode_rows(again, qd, *args, max_context_len=max(lens), partition_size=P)
    assert torch.equal(out, again)


@pytest.mark.parametrize("k_new,Hq", [(1, 8), (1, 2)])
def test_decode_rows_equal_scales_match_the_per_tensor_call(k_new, Hq):
    """Every row scale the same power of two: the codes, scores and weights are those of pa_decode with that
    kv_scale, up to where the scale multiplies; both are within the bound of the same reference."""
    pa = _gpu.lib()
    g = gen(5)
    NB, Hkv, bs, D = 40, 2, 16, 128
    k = randn(g, NB, Hkv, bs, D).to(R.E4M3)
    v = randn(g, NB, Hkv, bs, D).to(R.E4M3)
    sc = torch.full((NB, Hkv, bs), 0.25)
    lens = [200, 33]
    bt = R.block_table(lens, bs, NB, g)
    q = randn(g, 2, 1, Hq, D).bfloat16()
    ref, A, d = decode_rows_reference(q, k, v, sc, sc, bt, lens, 0.1, bs)
    cl = torch.tensor(lens, dtype=torch.int32).cuda()
    a, b = torch.empty_like(q[:, 0]).cuda(), torch.empty_like(q[:, 0]).cuda()
    pa.decode_rows(a, q[:, 0].cuda(), k.cuda(), v.cuda(), sc.cuda(), sc.cuda(), bt.cuda(), cl, 0.1)
    pa.decode(b, q[:, 0].cuda(), k.cuda(), v.cuda(), bt.cuda(), cl, 0.1, 0.25)
    for o in (a, b):
        close(o.view(ref.shape), ref, R.attention_bound(ref, A, d, D, torch.bfloat16, torch.float16))


@pytest.mark.parametrize("Hq", [2, 8])
@pytest.mark.parametrize("shift", [-80, 0, 60])
def test_decode_rows_scales_of_any_size(Hq, shift):
    """V rows scaled by powers of two from 2^-30 to 2^20 around 2^shift, growing, falling and mixed along the
    context; K scales that keep the scores moderate."""
    pa = _gpu.lib()
    g = gen(9)
    NB, Hkv, bs, D, L = 32, 2, 16, 64, 500
    k, v, ks, vs = rows_pool(g, NB, Hkv, bs, D)
    bt = torch.arange(NB, dtype=torch.int32)[None]
    e = torch.linspace(-30, 20, NB * bs).round()
    for order in (e, e.flip(0), e[torch.randperm(NB * bs, generator=g)]):
        vs2 = torch.exp2(order + shift).view(NB, 1, bs).expand(NB, Hkv, bs).contiguous()
        q = randn(g, 1, 1, Hq, D).bfloat16()
        ref, A, d = decode_rows_reference(q, k, v, ks, vs2, bt, [L], 0.125, bs)
        for P in (0, 128):
            out = torch.full_like(q[:, 0], float("nan")).cuda()
            pa.decode_rows(out, q[:, 0].cuda(), k.cuda(), v.cuda(), ks.cuda(), vs2.cuda(), bt.cuda(),
                           torch.tensor([L], dtype=torch.int32).cuda(), 0.125, L, P)
            # a weight times its scale is rounded against the largest scale: half of f16's least step of it
            least = float(vs2.max()) * 448 * L * 2.0 ** -25
            close(out.view(ref.shape), ref, R.attention_bound(ref, A, d, D, torch.bfloat16, torch.float16) + least)


def test_decode_rows_bad_indexes():
    pa = _gpu.lib()
    g = gen(3)
    NB, Hkv, bs, D, Hq = 8, 2, 16, 128, 8
    k, v, ks, vs = rows_pool(g, NB, Hkv, bs, D)
    lens = [40, 100, 64]
    bt = torch.tensor([[0, 8, 2, -1], [3, 4, 5, 6], [-7, 1, 7, 2]], dtype=torch.int32)  # 8 and -7 lie outside
    q = randn(g, 3, 1, Hq, D).bfloat16()
    out = torch.full_like(q[:, 0], float("nan")).cuda()
    cl = torch.tensor(lens, dtype=torch.int32).cuda()
    args = (q[:, 0].cuda(), k.cuda(), v.cuda(), ks.cuda(), vs.cuda())
    for P in (0, 64):
        pa.decode_rows(out, *args, bt.cuda(), cl, 0.1, max_context_len=64, partition_size=P)
        assert pa.get_device_error() == pa.DEVERR_BLOCK_ID | pa.DEVERR_CONTEXT_LEN  # 100 tokens in 4 blocks of 16
        # a block outside the pool reads as zeros
        kz, vz = torch.cat([k, k[:1]]), torch.cat([v, v[:1]])
        sz = torch.zeros(1, Hkv, bs)
        bz = torch.where((bt < 0) | (bt >= NB), NB, bt)
        ref, A, d = decode_rows_reference(q, kz, vz, torch.cat([ks, sz]), torch.cat([vs, sz]), bz, [40, 64, 64], 0.1, bs)
        close(out.view(ref.shape), ref, R.attention_bound(ref, A, d, D, torch.bfloat16, torch.float16))


# ---- norm, rotation, cache write --------------------------------------------

def rope_table(P, rot):
    i = torch.arange(rot // 2, dtype=torch.float64)
    a = torch.arange(P, dtype=torch.float64)[:, None] * 10000.0 ** (-2 * i / max(rot, 1))
    return torch.cat([a.cos(), a.sin()], 1).float()


def rope_bound(want, dtype, x):
    """float32: the sum of squares and the four operations after it are below 16 roundings of the normed value,
    and a rotation adds three roundings of both channels; then half a step of the stored value."""
    return R.half_step(dtype, want) + 24 * R.U * x.abs().amax(-1, keepdim=True) * 2


@pytest.mark.parametrize("kind", ["16", "tensor", "rows"])
@pytest.mark.parametrize("T,Hq,Hkv,D,bs,dt,rot,inter,norm", [
    (1, 1, 1, 64, 8, "bf16", 64, False, True), (5, 8, 2, 128, 16, "bf16", 128, False, True),
    (33, 6, 3, 64, 32, "f16", 32, False, True), (70, 40, 8, 128, 16, "f16", 48, False, False),
    (9, 4, 4, 128, 16, "bf16", 128, True, True), (20, 7, 1, 64, 16, "f16", 50, True, True),
    (3, 5, 5, 128, 8, "bf16", 0, False, True), (6, 3, 2, 64, 16, "bf16", 24, False, True), (2, 3, 1, 64, 16, "bf16", 2, True, False)])
def test_norm_rope_cache(T, Hq, Hkv, D, bs, dt, rot, inter, norm, kind):
    pa = _gpu.lib()
    g = gen(T + rot)
    dtype = R.DT[dt]
    P, NB, eps = 300, T // bs + 3, 1e-5
    qkv = (randn(g, T, (Hq + 2 * Hkv) * D) * torch.exp(randn(g, T, 1))).to(dtype).cuda()
    q, key, val = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    qw, kw = ((1 + 0.3 * randn(g, D)).to(dtype) for _ in range(2)) if norm else (None, None)
    tab = rope_table(P, rot) if rot else None
    pos = torch.randint(0, P, (T,), generator=g)
    slots = torch.randperm(NB * bs, generator=g)[:T]
    if T > 4:
        slots[3] = -1
    live = slots >= 0
    kv_scale = 0.03 if kind == "tensor" else 1.0
    ct = dtype if kind == "16" else torch.uint8
    caches = [torch.full((NB, Hkv, bs, D), 1, dtype=ct, device="cuda") for _ in range(2)]
    scales = [torch.full((NB, Hkv, bs), 7.0, device="cuda") for _ in range(2)] if kind == "rows" else [None, None]
    q_out = torch.full((T, Hq, D), 5.0, dtype=dtype, device="cuda")
    pa.norm_rope_cache(q_out, q, key, val, pos.cuda() if rot else None, tab.cuda() if rot else None, *caches, slots.cuda(),
                       q_weight=qw.cuda() if norm else None, k_weight=kw.cuda() if norm else None, eps=eps,
                       interleaved=inter, kv_scale=kv_scale, k_scales=scales[0], v_scales=scales[1])
    assert pa.get_device_error() == 0
    q64 = R.norm_rope(q.cpu(), qw, eps, tab, pos, inter)
    close(q_out[live.cuda()], q64[live], rope_bound(q64, dtype, q64)[live])
    assert (q_out[~live.cuda()] == 5.0).all()
    blk, off = slots[live] // bs, slots[live] % bs
    for i, (raw, w) in enumerate(((key, kw), (val, None))):
        x = R.norm_rope(raw.cpu(), w, eps, tab, pos, inter)[live] if i == 0 else raw.cpu().double()[live]
        cache = caches[i].cpu()
        untouched = torch.ones(NB, bs, dtype=torch.bool)
        untouched[blk, off] = False
        assert (cache.transpose(1, 2)[untouched] == 1).all()
        got = cache[blk, :, off]
        slack = 48 * R.U * x.abs().amax(-1, keepdim=True) if i == 0 else torch.zeros(())
        if kind == "16":
            if i == 1:
                assert torch.equal(got, raw.cpu()[live])
            else:
                close(got, x, rope_bound(x, dtype, x))
            continue
        s = torch.full(x.shape[:-1], kv_scale, dtype=torch.float32).double()
        if kind == "rows":
            s = scales[i].cpu()[blk, :, off]
            assert (scales[i].cpu()[untouched[:, None, :].expand(NB, Hkv, bs)] == 7.0).all()
            want = (x.abs().amax(-1) / 448).clamp_min(R.LEAST)
            assert ((s.double() - want).abs() <= want * 50 * R.U).all()
            s = s.double()
        if i == 1:  # no arithmetic before the division: bit-exact
            want = R.quantise_rows(raw.cpu()[live])[0] if kind == "rows" else \
                (raw.cpu()[live].float() / torch.tensor(kv_scale)).clamp(-448, 448).to(R.E4M3)
            assert R.same_codes(got, want)
        clamped = x.clamp(-448 * s[..., None], 448 * s[..., None])
        # half a step of E4M3 (2^-4 of a normal value, 2^-10 below), in units of the scale
        half = torch.maximum(clamped.abs() * 2.0 ** -4, s[..., None] * 2.0 ** -10)
        close(R.wide(got.view(R.E4M3)) * s[..., None], clamped, half + slack + clamped.abs() * 4 * R.U)


@pytest.mark.parametrize("T,Hq,Hkv,D", [(300, 20, 4, 128), (305, 17, 2, 64), (1217, 9, 1, 128), (2433, 3, 2, 64), (2434, 1, 1, 128)])
def test_norm_rope_cache_many_tokens(T, Hq, Hkv, D):
    """Each number of threads per token, the last CTA not full, some tokens padding."""
    test_norm_rope_cache(T, Hq, Hkv, D, 16, "bf16", D, False, True, "16")
    test_norm_rope_cache(T, Hq, Hkv, D, 16, "f16", 16, True, True, "rows")


def test_norm_rope_cache_in_place_and_bad_indexes():
    pa = _gpu.lib()
    g = gen(2)
    T, Hq, Hkv, D, bs, NB, P = 6, 4, 2, 128, 16, 2, 10
    q = randn(g, T, Hq, D).bfloat16().cuda()
    kv = [randn(g, T, Hkv, D).bfloat16().cuda() for _ in range(2)]
    tab = rope_table(P, D).cuda()
    pos = torch.tensor([0, 9, 10, -3, 4, 1 << 40]).cuda()
    slots = torch.tensor([0, 31, 32, 5, -1, 1 << 40]).cuda()
    caches = [torch.zeros((NB, Hkv, bs, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    out = torch.zeros_like(q)
    pa.norm_rope_cache(out, q, *kv, pos, tab, *caches, slots)
    assert pa.get_device_error() == pa.DEVERR_SLOT | pa.DEVERR_POSITION
    want = R.norm_rope(q.cpu(), None, 0, tab.cpu(), pos.cpu().clamp(0, P - 1), False)
    want[4] = 0
    close(out, want, rope_bound(want, torch.bfloat16, want))
    assert int((caches[1] != 0).any(-1).sum()) == 3 * Hkv
    with pytest.raises(pa.PagedAttnError):
        pa.norm_rope_cache(out, q, *kv, pos, tab[:, :20].contiguous(), *caches, slots)  # 20 channels, pairs a half apart
    slots[2] = slots[5] = -1
    same = q.clone()
    pa.norm_rope_cache(same, same, *kv, pos.clamp(0, P - 1), tab, *caches, slots)
    keep = slots >= 0
    assert torch.equal(same[keep], out[keep]) and torch.equal(same[~keep], q[~keep])
    assert pa.get_device_error() == 0


# ---- bounds, scores, selection ----------------------------------------------

def pool16(g, NB, Hkv, bs, D, dt, kv):
    x = (randn(g, NB, Hkv, bs, D) * 1.5).to(R.DT[dt])
    return x if kv == dt else x.to(R.E4M3)


def numbers(t):
    """Bits apart from the sign of zero."""
    return (t.float() if t.dtype == R.E4M3 else t) + 0.0


def live_bounds(k, bt, lens, bs, base):
    want = base.clone().float()
    kf = k.float()
    for s, L in enumerate(lens):
        for j in range(-(-L // bs)):
            rows = kf[bt[s, j]][:, : min(bs, L - j * bs)]
            want[bt[s, j], :, 0], want[bt[s, j], :, 1] = rows.amin(1), rows.amax(1)
    return want


@pytest.mark.parametrize("Hq,Hkv,D,bs,dt,kv", [
    (8, 2, 128, 16, "bf16", "bf16"), (3, 3, 64, 8, "f16", "f16"), (6, 1, 64, 32, "f16", "e4m3"), (16, 1, 128, 16, "bf16", "e4m3"),
    (34, 2, 128, 16, "bf16", "bf16"), (128, 1, 64, 16, "f16", "f16"), (9, 1, 128, 8, "bf16", "e4m3")])
def test_block_bounds_and_scores(Hq, Hkv, D, bs, dt, kv):
    pa = _gpu.lib()
    g = gen(D + Hq)
    lens = [0, 1, 7, 8, 9, 31, 32, 33, 100, 1111]
    NB = sum(-(-x // bs) for x in lens) + 2
    k = pool16(g, NB, Hkv, bs, D, dt, kv)
    bt = R.block_table(lens, bs, NB, g)
    base = torch.full((NB, Hkv, 2, D), 3.0).to(k.dtype)
    bounds = base.cuda()
    cl = torch.tensor(lens, dtype=torch.int32).cuda()
    pa.block_bounds(bounds, k.cuda(), bt.cuda(), cl, max(lens))
    want = live_bounds(k, bt, lens, bs, base)
    assert torch.equal(numbers(bounds).float().cpu(), want + 0.0)
    # one step on: only the newest token's block is read again
    k2 = pool16(g, NB, Hkv, bs, D, dt, kv)
    pa.block_bounds(bounds, k2.cuda(), bt.cuda(), cl, 1)
    for s, L in enumerate(lens):
        if L:
            j = (L - 1) // bs
            rows = k2.float()[bt[s, j]][:, : L - j * bs]
            want[bt[s, j], :, 0], want[bt[s, j], :, 1] = rows.amin(1), rows.amax(1)
    assert torch.equal(numbers(bounds).float().cpu(), want + 0.0)

    q = (randn(g, len(lens), Hq, D) * 2).to(R.DT[dt])
    scores = torch.full((len(lens), Hkv, bt.shape[1]), 9.0, device="cuda")
    pa.block_scores(scores, q.cuda(), bounds, bt.cuda(), cl, bs)
    assert pa.get_device_error() == 0
    got = scores.cpu().double()
    lo, hi = want[:, :, 0].double(), want[:, :, 1].double()
    for s, L in enumerate(lens):
        nb = -(-L // bs)
        assert (got[s, :, nb:] == float("-inf")).all()
        ids = bt[s, :nb].long()
        for h in range(Hkv):
            qq = q[s, h * (Hq // Hkv): (h + 1) * (Hq // Hkv)].double()
            ref = (qq.clamp(min=0) @ hi[ids, h].T + qq.clamp(max=0) @ lo[ids, h].T).amax(0) if nb else torch.zeros(0)
            size = (qq.abs() @ torch.maximum(lo[ids, h].abs(), hi[ids, h].abs()).T).amax(0) if nb else torch.zeros(0)
            # 2 D products summed in float32, each addition off by at most a whole step
            assert ((got[s, h, :nb] - ref).abs() <= 2 * 2 * D * R.U * size).all()


def test_bounds_are_bounds_and_nan_shows():
    pa = _gpu.lib()
    g = gen(4)
    NB, Hkv, bs, D, Hq, L = 12, 2, 16, 64, 8, 190
    k = pool16(g, NB, Hkv, bs, D, "bf16", "bf16")
    k[5, 1, 3, 7] = float("nan")
    k[6, 0, 0, 0] = float("inf")
    bt = torch.arange(NB, dtype=torch.int32)[None].cuda()
    cl = torch.tensor([L], dtype=torch.int32).cuda()
    bounds = torch.zeros((NB, Hkv, 2, D), dtype=torch.bfloat16, device="cuda")
    pa.block_bounds(bounds, k.cuda(), bt, cl, L)
    q = randn(g, 1, Hq, D).bfloat16()
    q[0, :, 0] = 1.0
    scores = torch.zeros((1, Hkv, NB), device="cuda")
    pa.block_scores(scores, q.cuda(), bounds, bt, cl, bs)
    sc = scores.cpu()[0]
    assert torch.isnan(sc[1, 5]) and not torch.isnan(sc[0, 5]) and sc[0, 6] == float("inf")
    true = torch.einsum("hgd,jhtd->hjgt", q[0].double().view(Hkv, Hq // Hkv, D), k.double())
    ok = torch.isfinite(sc)
    best = true.flatten(2).amax(-1)
    assert (best[ok] <= sc.double()[ok] + 1e-3).all()
    tables = torch.zeros((1, Hkv, 3), dtype=torch.int32, device="cuda")
    lens = torch.zeros((1, Hkv), dtype=torch.int32, device="cuda")
    pa.select_blocks(tables, lens, scores, bt, cl, bs, 0, 0)
    assert 5 in tables.cpu()[0, 1].tolist() and 6 in tables.cpu()[0, 0].tolist()


def check_selection(pa, scores, bt, lens, bs, n, sink, recent):
    S, Hkv, maxB = scores.shape
    tables = torch.full((S, Hkv, n), 77, dtype=torch.int32, device="cuda")
    out = torch.full((S, Hkv), 77, dtype=torch.int32, device="cuda")
    pa.select_blocks(tables, out, scores.cuda(), bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), bs, sink, recent)
    assert pa.get_device_error() == 0
    tables, out = tables.cpu(), out.cpu()
    for s in range(S):
        for h in range(Hkv):
            want = R.select(scores[s, h], lens[s], bs, n, sink, recent)
            assert tables[s, h].tolist() == [int(bt[s, j]) for j in want] + [-1] * (n - len(want))
            assert int(out[s, h]) == sum(min(bs, lens[s] - j * bs) for j in want)


@pytest.mark.parametrize("n,sink,recent", [(1, 0, 0), (1, 0, 1), (2, 1, 1), (7, 2, 3), (64, 1, 2), (600, 0, 4), (5, 0, 5)])
def test_select_blocks(n, sink, recent):
    pa = _gpu.lib()
    g = gen(n)
    bs = 16
    lens = [0, 1, 16, 17, 16 * n, 16 * n + 1, 513, 16 * 511, 16 * 512, 16 * 513 - 3, 20000]
    bt = R.block_table(lens, bs, sum(-(-x // bs) for x in lens) + 1, g)
    S, maxB = bt.shape
    scores = torch.stack([randn(g, S, maxB), randn(g, S, maxB).round(), torch.zeros(S, maxB),
                          -torch.rand((S, maxB), generator=g) * 1e-38], 1)
    scores[:, 2, ::2] = -0.0
    check_selection(pa, scores, bt, lens, bs, n, sink, recent)


def test_select_blocks_special_scores():
    pa = _gpu.lib()
    g = gen(8)
    bs, lens = 8, [8 * 100, 8 * 99 + 1]
    bt = R.block_table(lens, bs, 300, g)
    x = randn(g, 2, 5, 100)
    x[:, 0, 10::7], x[:, 0, 3] = float("nan"), float("inf")
    x[:, 1] = float("-inf")
    x[:, 1, 90] = -3e38
    x[:, 2] = float("nan")
    x[:, 3, ::3] = float("inf")
    x[:, 4] = torch.where(x[:, 4] > 0, 1e-45, -1e-45)  # denormals count
    for n in (1, 6, 20, 50):
        check_selection(pa, x, bt, lens, bs, n, 0, 1)
        check_selection(pa, x, bt, lens, bs, n, 0, 0)


@pytest.mark.parametrize("S,Hkv,blocks", [(1, 3, 1000), (77, 2, 900), (77, 2, 2048), (77, 2, 3000), (160, 5, 1024), (160, 4, 40), (160, 4, 1500)])
def test_select_blocks_of_many_rows(S, Hkv, blocks):
    """Each number of threads per row; a score far from the others puts these into one bin."""
    pa = _gpu.lib()
    g = gen(S + blocks)
    bs = 8
    lens = torch.randint(1, blocks * bs + 1, (S,), generator=g).tolist()
    lens[0], lens[S // 2] = blocks * bs, 0
    bt = torch.arange(blocks, dtype=torch.int32).expand(S, -1).contiguous()
    x = randn(g, S, Hkv, blocks)
    x[:, 0] = x[:, 0].round()
    x[: S // 2 + 1, -1, ::5] = 1e30
    x[: S // 3, -1, 1::97] = -1e38
    check_selection(pa, x, bt, lens, bs, 16, 1, 2)
    check_selection(pa, x, bt, lens, bs, blocks // 3, 0, 1)


def test_select_blocks_among_very_many():
    """Contexts of up to 60000 blocks: more keys than shared memory holds, several passes over the ballots."""
    pa = _gpu.lib()
    g = gen(12)
    bs, lens = 8, [8 * 60000 - 3, 8 * 33000, 8 * 51200 + 1, 90]
    bt = torch.stack([torch.randperm(70000, generator=g)[:60000] for _ in lens]).to(torch.int32)
    x = torch.stack([randn(g, 4, 60000), randn(g, 4, 60000).round()], 1)
    for n in (3, 700, 40000):
        check_selection(pa, x, bt, lens, bs, n, 1, 1)
    # one row with fewer blocks: 1024 threads
    check_selection(pa, x[:1, :, :20000].contiguous(), bt[:1, :20000].contiguous(), [8 * 20000 - 1], bs, 600, 2, 1)


def test_offsets_past_32_bits():
    """Pools whose elements pass 2^32: rows written to, read from, bounded, scored and attended over in their last
    blocks."""
    pa = _gpu.lib()
    g = gen(13)
    Hkv, bs, D, Hq, L = 8, 32, 128, 8, 70
    NB = (1 << 32) // (Hkv * bs * D) + 9
    assert NB * Hkv * bs * D > 1 << 32
    k8, v8 = (torch.zeros((NB, Hkv, bs, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((NB, Hkv, bs), device="cuda") for _ in range(2))
    bt = torch.tensor([[NB - 1, NB - 7, NB - 3]], dtype=torch.int32)
    pos = torch.arange(L)
    slots = bt[0].long()[pos // bs] * bs + pos % bs
    key, val = (randn(g, L, Hkv, D).bfloat16() for _ in range(2))
    pa.reshape_and_cache_rows(key.cuda(), val.cuda(), k8, v8, ks, vs, slots.cuda())
    kc, kss = R.quantise_rows(key)
    vc, vss = R.quantise_rows(val)
    blk, off = slots // bs, slots % bs
    assert R.same_codes(k8[blk.cuda(), :, off.cuda()], kc) and torch.equal(vs[blk.cuda(), :, off.cuda()].cpu(), vss)
    assert int(torch.count_nonzero(k8[: NB - 8])) == 0
    dst = [torch.zeros((3, Hkv, bs, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pa.gather_blocks_rows(*dst, k8, v8, ks, vs, bt[0].long().cuda())
    assert torch.equal(dst[0].cpu().transpose(1, 2).flatten(0, 1)[:L], (kc.float() * kss[..., None]).bfloat16())
    q = randn(g, 1, Hq, D).bfloat16()
    cl = torch.tensor([L], dtype=torch.int32).cuda()
    out = torch.empty_like(q).cuda()
    pa.decode_rows(out, q.cuda(), k8, v8, ks, vs, bt.cuda(), cl, 0.1)
    kd, vd = R.wide(kc) * kss.double()[..., None], R.wide(vc) * vss.double()[..., None]
    for h in range(Hq):
        ref, A, d = R.attend(q[0, h].double(), kd[:, h], vd[:, h], 0.1)
        close(out[0, h], ref, R.attention_bound(ref, A, d, D, torch.bfloat16, torch.float16))
    # the same pool read per tensor: bounds, scores, selection and decode of chosen blocks
    bounds = torch.zeros((NB, Hkv, 2, D), dtype=torch.uint8, device="cuda")
    pa.block_bounds(bounds, k8, bt.cuda(), cl, L)
    kf = R.wide(kc)
    last = bounds[NB - 3].view(R.E4M3).float().cpu().double()
    assert torch.equal(last[:, 0] + 0.0, kf[64:].amin(0) + 0.0) and torch.equal(last[:, 1] + 0.0, kf[64:].amax(0) + 0.0)
    scores = torch.zeros((1, Hkv, 3), device="cuda")
    pa.block_scores(scores, q.cuda(), bounds, bt.cuda(), cl, bs)
    tables = torch.zeros((1, Hkv, 2), dtype=torch.int32, device="cuda")
    lens = torch.zeros((1, Hkv), dtype=torch.int32, device="cuda")
    pa.select_blocks(tables, lens, scores, bt.cuda(), cl, bs, 0, 1)
    pa.decode_selected(out, q.cuda(), k8, v8, tables, lens, 0.001, 0.5)
    for h in range(Hq):
        want = R.select(scores[0, h].cpu(), L, bs, 2, 0, 1)
        rows = torch.cat([pos[j * bs: min(L, (j + 1) * bs)] for j in want])
        ref, A, d = R.attend(q[0, h].double(), kf[rows, h] * 0.5, R.wide(vc)[rows, h] * 0.5, 0.001)
        close(out[0, h], ref, R.attention_bound(ref, A, d, D, torch.bfloat16, torch.float16))
    assert pa.get_device_error() == 0


def test_block_choice_bad_indexes():
    pa = _gpu.lib()
    g = gen(11)
    NB, Hkv, bs, D, Hq = 6, 1, 8, 64, 2
    k = pool16(g, NB, Hkv, bs, D, "f16", "f16").cuda()
    bt = torch.tensor([[0, 6, 1], [2, 3, 4], [-2, 5, 0]], dtype=torch.int32).cuda()
    cl = torch.tensor([20, 99, -4], dtype=torch.int32).cuda()  # 99 > 24, -4 < 0
    bounds = torch.zeros((NB, Hkv, 2, D), dtype=torch.float16, device="cuda")
    pa.block_bounds(bounds, k, bt, cl, 24)
    assert pa.get_device_error() == pa.DEVERR_BLOCK_ID | pa.DEVERR_CONTEXT_LEN
    scores = torch.full((3, Hkv, 3), 5.0, device="cuda")
    pa.block_scores(scores, randn(g, 3, Hq, D).half().cuda(), bounds, bt, cl, bs)
    assert pa.get_device_error() == pa.DEVERR_BLOCK_ID | pa.DEVERR_CONTEXT_LEN
    assert scores[0, 0, 1] == 0 and torch.isinf(scores[2]).all() and torch.isfinite(scores[1]).all()
    tables = torch.zeros((3, Hkv, 2), dtype=torch.int32, device="cuda")
    lens = torch.zeros((3, Hkv), dtype=torch.int32, device="cuda")
    pa.select_blocks(tables, lens, scores, bt, cl, bs, 0, 1)
    assert pa.get_device_error() == pa.DEVERR_CONTEXT_LEN
    assert lens.cpu().tolist() == [[12], [16], [0]] and tables[2].cpu().tolist() == [[-1, -1]]


# ---- decode over the chosen blocks ------------------------------------------

@pytest.mark.parametrize("P", [0, 64])
@pytest.mark.parametrize("Hq,Hkv,D,bs,dt,kv", [
    (8, 2, 128, 16, "bf16", "bf16"), (3, 3, 64, 8, "f16", "f16"), (6, 2, 128, 32, "f16", "f16"), (32, 2, 64, 16, "bf16", "e4m3"),
    (33, 1, 128, 16, "bf16", "bf16"), (8, 1, 128, 8, "f16", "e4m3"), (2, 2, 128, 16, "bf16", "e4m3"), (128, 1, 64, 16, "f16", "f16")])
def test_decode_selected(Hq, Hkv, D, bs, dt, kv, P):
    pa = _gpu.lib()
    g = gen(Hq)
    S, n = 5, 19
    NB = 64
    k, v = (pool16(g, NB, Hkv, bs, D, dt, kv) for _ in range(2))
    kvs = 0.7 if kv == "e4m3" else 1.0
    lens = torch.randint(1, n * bs + 1, (S, Hkv), generator=g).to(torch.int32)
    lens[0, 0], lens[1, 0], lens[2, 0] = 0, 1, n * bs
    tables = torch.full((S, Hkv, n), -1, dtype=torch.int32)
    for s in range(S):
        for h in range(Hkv):
            m = -(-int(lens[s, h]) // bs)
            tables[s, h, :m] = torch.randperm(NB, generator=g)[:m].to(torch.int32)
    q = randn(g, S, Hq, D).to(R.DT[dt])
    out = torch.full_like(q, float("nan")).cuda()
    scale = D ** -0.5
    pa.decode_selected(out, q.cuda(), k.cuda(), v.cuda(), tables.cuda(), lens.cuda(), scale, kvs, P)
    assert pa.get_device_error() == 0
    ref, A, d = (torch.zeros(S, Hq, D, dtype=torch.float64) for _ in range(3))
    factor, k64, v64 = float(torch.tensor(kvs)), R.wide(k), R.wide(v)
    for s in range(S):
        for hq in range(Hq):
            h = hq // (Hq // Hkv)
            L = int(lens[s, h])
            ids = tables[s, h, : -(-L // bs)].long()
            kk, vv = (x[ids, h].flatten(0, 1)[:L] * factor for x in (k64, v64))
            ref[s, hq], A[s, hq], d[s, hq] = R.attend(q[s, hq].double(), kk, vv, scale)
    weights = torch.bfloat16 if kv == "bf16" else torch.float16
    close(out, ref, R.attention_bound(ref, A, d, D, R.DT[dt], weights))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_all_blocks_chosen_equals_decode_bit_for_bit(kv):
    """336 contexts: enough that each has one CTA, too few for a second wave, so the sums run in the same order."""
    pa = _gpu.lib()
    g = gen(6)
    NB, Hkv, bs, D, Hq, lens = 80, 2, 16, 128, 8, [1, 100, 515, 48]
    k, v = (pool16(g, NB, Hkv, bs, D, "bf16", kv).cuda() for _ in range(2))
    bt = R.block_table(lens, bs, NB, g).cuda()
    bt, cl = bt.repeat(42, 1), torch.tensor(lens * 42, dtype=torch.int32).cuda()
    q = randn(g, 168, Hq, D).bfloat16().cuda()
    a, b = torch.empty_like(q), torch.empty_like(q)
    pa.decode(a, q, k, v, bt, cl, 0.09)
    pa.decode_selected(b, q, k, v, bt[:, None].expand(-1, Hkv, -1).contiguous(), cl[:, None].expand(-1, Hkv).contiguous(), 0.09)
    assert torch.equal(a, b)


@pytest.mark.parametrize("S,Hkv,kv", [(1, 1, "bf16"), (3, 2, "e4m3"), (15, 4, "bf16"), (60, 4, "bf16"), (121, 4, "f16"), (160, 4, "e4m3")])
def test_decode_selected_over_few_and_many_contexts(S, Hkv, kv):
    """Contexts shared by clusters of 8, 4, 2 and 1 CTAs, and last waves split over clusters, some contexts empty
    or shorter than the cluster's tiles."""
    pa = _gpu.lib()
    g = gen(S)
    D, bs, n, NB, Hq = 64, 16, 70, 100, 4 * Hkv
    dt = "f16" if kv == "f16" else "bf16"
    k, v = (pool16(g, NB, Hkv, bs, D, dt, kv) for _ in range(2))
    tables = torch.rand((S, Hkv, NB), generator=g).argsort(-1)[..., :n].to(torch.int32).contiguous()
    lens = torch.randint(0, n * bs + 1, (S, Hkv), generator=g).to(torch.int32)
    lens.view(-1)[::5], lens.view(-1)[1::7], lens.view(-1)[-1] = 0, 3, n * bs
    q = randn(g, S, Hq, D).to(R.DT[dt])
    out = torch.full_like(q, float("nan")).cuda()
    pa.decode_selected(out, q.cuda(), k.cuda(), v.cuda(), tables.cuda(), lens.cuda(), 0.125, 0.5 if kv == "e4m3" else 1.0)
    assert pa.get_device_error() == 0
    f = 0.5 if kv == "e4m3" else 1.0
    heads = torch.arange(Hkv)[None, :, None]
    kk, vv = (R.wide(x)[tables.long(), heads].flatten(2, 3) * f for x in (k, v))  # [S, Hkv, tokens, D]
    qq = q.double().view(S, Hkv, 4, D)
    seen = torch.arange(n * bs) < lens[:, :, None, None]
    w = torch.softmax((qq @ kk.transpose(-1, -2) * 0.125).masked_fill(~seen, -1e300), -1) * seen.any(-1, keepdim=True)
    ref, A = (w @ vv).view(S, Hq, D), (w @ vv.abs()).view(S, Hq, D)
    d = (qq.abs() @ kk.abs().transpose(-1, -2)).amax(-1, keepdim=True).expand(S, Hkv, 4, D).reshape(S, Hq, D) * 0.125
    close(out, ref, R.attention_bound(ref, A, d, D, R.DT[dt], torch.bfloat16 if kv == "bf16" else torch.float16))


@pytest.mark.parametrize("S,Hkv", [(1, 1), (5, 2), (40, 4)])
def test_decode_rows_over_few_contexts(S, Hkv):
    pa = _gpu.lib()
    g = gen(S + 100)
    D, bs, Hq = 128, 16, 4 * Hkv
    lens = [int(x) for x in torch.randint(0, 900, (S,), generator=g)]
    lens[0] = 1111
    NB = sum(-(-x // bs) for x in lens) + 2
    k, v, ks, vs = rows_pool(g, NB, Hkv, bs, D)
    bt = R.block_table(lens, bs, NB, g)
    q = randn(g, S, 1, Hq, D).half()
    ref, A, d = decode_rows_reference(q, k, v, ks, vs, bt, lens, 0.1, bs)
    out = torch.full_like(q[:, 0], float("nan")).cuda()
    pa.decode_rows(out, q[:, 0].cuda(), k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), bt.cuda(),
                   torch.tensor(lens, dtype=torch.int32).cuda(), 0.1)
    assert pa.get_device_error() == 0
    close(out.view(ref.shape), ref, R.attention_bound(ref, A, d, D, torch.float16, torch.float16))


def lost(lens, A):
    """What weights below f16's normal range lose: each is off by 2^-25 R, where R is a quarter of the largest weight
    times scale at most, times a code of 448 at most.  Some channel of that token's row has the code 448, so the largest A
    of a query row is that weight times 448 at least."""
    return max(lens) * 2.0 ** -27 * A.amax(-1, keepdim=True)


@pytest.mark.parametrize("Hq,n", [(2, 1), (8, 2), (32, 1)])
@pytest.mark.parametrize("ratio", [2.0 ** -10, 2.0 ** -20, 2.0 ** -40, 2.0 ** 30])
def test_the_token_with_the_weight_has_the_smallest_scale(Hq, n, ratio):
    """One token takes nearly all of the weight, before or after tokens whose V rows are far larger; its own V row is
    what comes out."""
    pa = _gpu.lib()
    g = gen(Hq)
    D, bs, Hkv, lens = 128, 16, 2, [200, 200, 64, 17]
    NB = sum(-(-x // bs) for x in lens) + 2
    k, v, ks, vs = rows_pool(g, NB, Hkv, bs, D)
    bt = R.block_table(lens, bs, NB, g)
    q = torch.randn(len(lens), 1, Hq, D, generator=g).abs().half().expand(-1, n, -1, -1).contiguous()
    ks *= 0.02
    for s, t in enumerate([3, 150, 40, 9]):  # a score near 36, the others' near 0
        b = int(bt[s, t // bs])
        k[b, :, t % bs], ks[b, :, t % bs] = torch.full((Hkv, D), 448.0).to(R.E4M3), 1 / 64
        vs[b, :, t % bs] *= ratio
    ref, A, d = decode_rows_reference(q, k, v, ks, vs, bt, lens, 0.05, bs)
    for P in (0, 64):
        qd = (q if n > 1 else q[:, 0]).contiguous().cuda()
        out = torch.full_like(qd, float("nan"))
        pa.decode_rows(out, qd, k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), bt.cuda(),
                       torch.tensor(lens, dtype=torch.int32).cuda(), 0.05, max_context_len=max(lens), partition_size=P)
        assert pa.get_device_error() == 0
        got, bound = out.view(ref.shape).cpu(), R.attention_bound(ref, A, d, D, torch.float16, torch.float16) + lost(lens, A)
        big = ref.abs() - bound > 65520  # 2^30 times a row passes f16's largest number, 65504: infinity is the rounding
        assert torch.equal(got[big].float(), torch.full_like(ref[big], float("inf")).copysign(ref[big]).float())
        small = ref.abs() + bound < 65520
        if small.any():
            close(got[small], ref[small], bound[small])


@pytest.mark.parametrize("S,Hkv,G,long", [(100, 8, 4, 3), (100, 8, 4, 0), (230, 4, 2, 40), (100, 8, 4, 100), (31, 32, 8, 1)])
def test_decode_rows_of_mixed_lengths(S, Hkv, G, long):
    """More CTAs than run at once and fewer than three times as many: contexts much longer than the others, none of
    them, only them; from a replayed graph the same again."""
    pa = _gpu.lib()
    g = gen(S + long)
    D, bs, Hq = 64, 16, G * Hkv
    lens = [int(x) for x in torch.randint(0, 40, (S,), generator=g)]
    for s in torch.randperm(S, generator=g)[:long].tolist():
        lens[s] = 2000 + s % 49 if long < S else 200 + s
    NB = sum(-(-x // bs) for x in lens) + 2
    k, v, ks, vs = rows_pool(g, NB, Hkv, bs, D)
    bt = R.block_table(lens, bs, NB, g)
    bt = torch.cat([bt, bt.new_full((S, max(0, 130 - bt.shape[1])), -1)], 1)
    q = randn(g, S, 1, Hq, D).half()
    ref, A, d = decode_rows_reference(q, k, v, ks, vs, bt, lens, 0.1, bs)
    out = torch.full_like(q[:, 0], float("nan")).cuda()
    args = [t.cuda() for t in (q[:, 0], k, v, ks, vs, bt, torch.tensor(lens, dtype=torch.int32))]
    pa.decode_rows(out, *args, 0.1)
    assert pa.get_device_error() == 0
    close(out.view(ref.shape), ref, R.attention_bound(ref, A, d, D, torch.float16, torch.float16) + lost(lens, A))
    again, graph = torch.full_like(out, float("nan")), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.decode_rows(again, *args, 0.1)
    graph.replay()
    assert torch.equal(again, out)


# ---- together ---------------------------------------------------------------

class Step:
    """A layer's decode step: norm + rotation + cache write, bounds, scores, selection, decode over the choice."""

    def __init__(self, pa, g, lens, n=6, P=64, Hq=8, Hkv=2, D=128, bs=16, device="cuda"):
        self.pa, self.n, self.P, self.bs, self.D = pa, n, P, bs, D
        S = len(lens)
        NB = sum(-(-x // bs) for x in lens) + 2
        bt = R.block_table(lens, bs, NB, g)
        slot = [int(bt[s, (L - 1) // bs]) * bs + (L - 1) % bs for s, L in enumerate(lens)]
        self.k, self.v = (pool16(g, NB, Hkv, bs, D, "bf16", "bf16").to(device) for _ in range(2))
        self.bt, self.cl = bt.to(device), torch.tensor(lens, dtype=torch.int32, device=device)
        self.slots, self.pos = torch.tensor(slot, device=device), torch.tensor([x - 1 for x in lens], device=device)
        self.qkv = randn(g, S, (Hq + 2 * Hkv) * D).bfloat16().to(device)
        self.q, self.key, self.val = (t.unflatten(1, (-1, D)) for t in self.qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
        self.w = [(1 + 0.1 * randn(g, D)).bfloat16().to(device) for _ in range(2)]
        self.tab = rope_table(max(lens), D).to(device)
        self.bounds = torch.zeros((NB, Hkv, 2, D), dtype=torch.bfloat16, device=device)
        pa.block_bounds(self.bounds, self.k, self.bt, self.cl, max(lens))
        self.q_out = torch.zeros((S, Hq, D), dtype=torch.bfloat16, device=device)
        self.scores = torch.zeros((S, Hkv, bt.shape[1]), device=device)
        self.tables = torch.zeros((S, Hkv, n), dtype=torch.int32, device=device)
        self.lens = torch.zeros((S, Hkv), dtype=torch.int32, device=device)
        self.out = torch.zeros_like(self.q_out)
        self.ws = torch.empty(pa.decode_split_workspace_size(S, Hq, D, n * bs, P), dtype=torch.uint8, device=device)

    def run(self):
        pa = self.pa
        pa.norm_rope_cache(self.q_out, self.q, self.key, self.val, self.pos, self.tab, self.k, self.v, self.slots,
                           q_weight=self.w[0], k_weight=self.w[1])
        pa.block_bounds(self.bounds, self.k, self.bt, self.cl, 1)
        pa.block_scores(self.scores, self.q_out, self.bounds, self.bt, self.cl, self.bs)
        pa.select_blocks(self.tables, self.lens, self.scores, self.bt, self.cl, self.bs)
        pa.decode_selected(self.out, self.q_out, self.k, self.v, self.tables, self.lens, self.D ** -0.5,
                           partition_size=self.P, workspace=self.ws)
        return self.out


def test_a_decode_step_through_all_of_them():
    pa = _gpu.lib()
    lens = [3, 700, 96, 1500]
    st = Step(pa, gen(21), lens)
    out = st.run()
    assert pa.get_device_error() == 0
    S, Hq, D = out.shape
    Hkv = st.k.shape[1]
    k, v, q = R.wide(st.k), R.wide(st.v), st.q_out.cpu().double()
    bounds = live_bounds(st.k.cpu(), st.bt.cpu(), lens, st.bs, st.bounds.cpu())
    assert torch.equal(numbers(st.bounds).float().cpu(), bounds + 0.0)
    for s, L in enumerate(lens):
        for h in range(Hkv):
            want = R.select(st.scores[s, h].cpu(), L, st.bs, st.n, 1, 1)
            ids = st.bt[s].cpu().long()[want]
            assert st.tables[s, h].cpu().tolist()[: len(want)] == ids.tolist()
            t = int(st.lens[s, h])
            kk, vv = k[ids, h].flatten(0, 1)[:t], v[ids, h].flatten(0, 1)[:t]
            for g in range(Hq // Hkv):
                row = h * (Hq // Hkv) + g
                ref, A, d = R.attend(q[s, row], kk, vv, D ** -0.5)
                close(out[s, row], ref, R.attention_bound(ref, A, d, D, torch.bfloat16, torch.bfloat16))


def test_the_step_captured_replays_with_new_inputs():
    pa = _gpu.lib()
    a, b = Step(pa, gen(31), [40, 900, 333]), Step(pa, gen(31), [40, 900, 333])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    for seed in (1, 2):
        new = randn(gen(seed), *a.qkv.shape).bfloat16().cuda()
        a.qkv.copy_(new)
        b.qkv.copy_(new)
        graph.replay()
        b.run()
        torch.cuda.synchronize()
        for x in ("out", "q_out", "k", "v", "bounds", "scores", "tables", "lens"):
            assert torch.equal(getattr(a, x), getattr(b, x)), x
    assert pa.get_device_error() == 0


def test_row_scaled_chunk_written_read_back_and_prefilled():
    """A prompt's rows written row-scaled by norm_rope_cache, read back for pa_prefill of the chunk, and decoded
    over as they are."""
    pa = _gpu.lib()
    g = gen(41)
    T, Hq, Hkv, D, bs, NB = 150, 8, 2, 128, 16, 14
    q, key, val = (randn(g, T, H, D).bfloat16().cuda() for H in (Hq, Hkv, Hkv))
    bt = R.block_table([T], bs, NB, g)
    slots = (bt[0].long()[torch.arange(T) // bs] * bs + torch.arange(T) % bs).cuda()
    caches = [torch.zeros((NB, Hkv, bs, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones((NB, Hkv, bs), device="cuda") for _ in range(2)]
    q_out = torch.empty_like(q)
    pa.norm_rope_cache(q_out, q, key, val, torch.arange(T).cuda(), rope_table(T, D).cuda(), *caches, slots,
                       k_scales=scales[0], v_scales=scales[1])
    nb = bt.shape[1]
    wide = [torch.empty((nb, Hkv, bs, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pa.gather_blocks_rows(*wide, *caches, *scales, bt[0].long().cuda())
    out = torch.empty((1, T, Hq, D), dtype=torch.bfloat16, device="cuda")
    cl = torch.tensor([T], dtype=torch.int32).cuda()
    pa.prefill(out, q_out[None], *wide, torch.arange(nb, dtype=torch.int32).cuda()[None], cl, D ** -0.5)
    last = torch.empty((1, Hq, D), dtype=torch.bfloat16, device="cuda")
    pa.decode_rows(last, q_out[-1:], *caches, *scales, bt.cuda(), cl, D ** -0.5)
    assert pa.get_device_error() == 0
    k, v = (R.wide(c.view(R.E4M3)) * s.cpu().double()[..., None] for c, s in zip(caches, scales))
    for h in range(Hq):
        kk, vv = (x[bt[0].long(), h // 4].flatten(0, 1)[:T] for x in (k, v))
        ref, A, d = R.attend(q_out[-1, h].cpu().double(), kk, vv, D ** -0.5)
        close(last[0, h], ref, R.attention_bound(ref, A, d, D, torch.bfloat16, torch.float16))
        # the prefill reads values rounded to bf16 once more: each score and each v moves by half a step
        eps = torch.finfo(torch.bfloat16).eps / 2
        close(out[0, -1, h], ref, R.attention_bound(ref, A, d, D, torch.bfloat16, torch.bfloat16) + A * (eps + 2 * eps * d))


@pytest.mark.parametrize("Hkv,bs,pinned", [(1, 8, False), (2, 16, True), (5, 32, True)])
def test_row_scaled_blocks_copied_and_swapped(Hkv, bs, pinned):
    """A shared last block copied before it is written to, and a sequence swapped out and back to other blocks: the
    decode reads the same values."""
    pa = _gpu.lib()
    g = gen(Hkv)
    D, L, NB = 64, 3 * bs + 5, 20
    k, v, ks, vs = (t.cuda() for t in rows_pool(g, NB, Hkv, bs, D))
    bt = torch.tensor([[3, 9, 14, 6], [3, 9, 14, 11]], dtype=torch.int32)
    old = [t.clone() for t in (k, v, ks, vs)]
    pairs = torch.tensor([[6, 11]]).cuda()
    pa.copy_blocks(k, v, pairs)
    pa.copy_block_scales(ks, vs, pairs)
    for t, o in zip((k, v, ks, vs), old):
        keep = [i for i in range(NB) if i != 11]
        t, o = t.view(torch.uint8).cpu(), o.view(torch.uint8).cpu()
        assert torch.equal(t[keep], o[keep]) and torch.equal(t[11], o[6])
    q = randn(g, 2, 4 * Hkv, D).half()
    q[1] = q[0]
    lens = torch.full((2,), L, dtype=torch.int32).cuda()
    out = torch.full_like(q, float("nan")).cuda()
    pa.decode_rows(out, q.cuda(), k, v, ks, vs, bt.cuda(), lens, 0.1)
    assert torch.equal(out[0], out[1]) and torch.isfinite(out).all()
    # out to a buffer, back to other blocks, an id outside the pool among them
    ids = torch.tensor([3, 9, 14, 11, NB])
    codes = torch.full((5, 2, Hkv, bs, D), 7, dtype=torch.uint8, pin_memory=pinned, device=None if pinned else "cuda")
    scales = torch.full((5, 2, Hkv, bs), 7.0, pin_memory=pinned, device=None if pinned else "cuda")
    pa.gather_blocks(codes, k, v, ids.cuda())
    pa.gather_block_scales(scales, ks, vs, ids.cuda())
    torch.cuda.synchronize()
    assert pa.get_device_error() == pa.DEVERR_BLOCK_ID
    assert torch.equal(scales[:4, 0].cpu(), ks[ids[:4]].cpu()) and torch.equal(scales[:4, 1].cpu(), vs[ids[:4]].cpu())
    assert (scales[4] == 7.0).all()
    to = torch.tensor([0, 19, 2, 18, -1])
    pa.scatter_blocks(k, v, codes, to.cuda())
    pa.scatter_block_scales(ks, vs, scales, to.cuda())
    assert pa.get_device_error() == pa.DEVERR_BLOCK_ID
    again = torch.full_like(out, float("nan"))
    pa.decode_rows(again, q.cuda(), k, v, ks, vs, torch.stack([to[:4], to[:4]]).to(torch.int32).cuda(), lens, 0.1)
    assert torch.equal(out, again) and pa.get_device_error() == 0


def test_empty_batches_do_nothing():
    pa = _gpu.lib()
    k = torch.zeros((2, 2, 16, 64), dtype=torch.float16, device="cuda")
    k8, s = torch.zeros((2, 2, 16, 64), dtype=torch.uint8, device="cuda"), torch.ones((2, 2, 16), device="cuda")
    q, kv, i = (torch.zeros((0, h, 64), dtype=torch.float16, device="cuda") for h in (4, 2, 1))
    i64, i32 = torch.zeros(0, dtype=torch.int64, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    bt = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    pa.reshape_and_cache_rows(kv, kv, k8, k8, s, s, i64)
    pa.gather_blocks_rows(k[:0], k[:0], k8, k8, s, s, i64)
    pa.decode_rows(q, q, k8, k8, s, s, bt, i32, 1.0)
    pa.norm_rope_cache(q, q, kv, kv, i64, torch.zeros((4, 64), device="cuda"), k, k, i64)
    bounds = torch.zeros((2, 2, 2, 64), dtype=torch.float16, device="cuda")
    pa.block_bounds(bounds, k, bt, i32, 1)
    sc, tab = torch.zeros((0, 2, 3), device="cuda"), torch.zeros((0, 2, 3), dtype=torch.int32, device="cuda")
    pa.block_scores(sc, q, bounds, bt, i32, 16)
    pa.select_blocks(tab, i32.view(0, 1).expand(0, 2).contiguous(), sc, bt, i32, 16)
    pa.decode_selected(q, q, k, k, tab, torch.zeros((0, 2), dtype=torch.int32, device="cuda"), 1.0)
    assert pa.get_device_error() == 0


def test_two_streams_at_once():
    """Two steps side by side, each on its own stream and host thread, with its own buffers."""
    import threading
    pa = _gpu.lib()
    steps = [Step(pa, gen(61 + i), [600, 50 + i, 1400]) for i in range(2)]
    want = [s.run().clone() for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(20):
                steps[i].out.zero_()
                steps[i].run()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(s.out, w) for s, w in zip(steps, want))
    assert pa.get_device_error() == 0


def test_check_mode_reports_bad_indexes():
    pa = _gpu.lib()
    k = torch.zeros((4, 2, 16, 64), dtype=torch.float16, device="cuda")
    q, kv = torch.zeros((1, 4, 64), dtype=torch.float16, device="cuda"), torch.zeros((1, 2, 64), dtype=torch.float16, device="cuda")
    prev = pa.set_check_mode(True)
    try:
        with pytest.raises(pa.PagedAttnError) as e:
            pa.norm_rope_cache(torch.empty_like(q), q, kv, kv, None, None, k, k.clone(), torch.tensor([64], device="cuda"))
        assert e.value.status == -5
        with pytest.raises(pa.PagedAttnError) as e:
            pa.decode_selected(torch.empty_like(q), q, k, k, torch.tensor([[[9], [0]]], dtype=torch.int32, device="cuda"),
                               torch.tensor([[5, 5]], dtype=torch.int32, device="cuda"), 1.0)
        assert e.value.status == -5
        pa.norm_rope_cache(torch.empty_like(q), q, kv, kv, None, None, k, k.clone(), torch.tensor([63], device="cuda"))
    finally:
        pa.set_check_mode(prev)
    assert pa.get_device_error() == 0


def test_another_stream_than_the_tensors_own():
    pa = _gpu.lib()
    a = Step(pa, gen(51), [70, 300])
    torch.cuda.synchronize()
    want = a.run().clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.run()
    side.synchronize()
    assert torch.equal(a.out, want)
