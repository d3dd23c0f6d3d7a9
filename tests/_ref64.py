"""Plain 64-bit references of the cache-side operators (torch on the CPU), and
the error bounds their tests use.

Rounding: a value stored in a 16-bit type is off by at most half a step,
eps / 2 of it (or half the least subnormal); float32 arithmetic by 2^-24 of
each intermediate result."""
import torch

U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
LEAST = 2.0 ** -126


def half_step(dtype, want):
    """Largest rounding error of storing `want` in `dtype`."""
    info = torch.finfo(dtype)
    return torch.maximum(want.abs() * (info.eps / 2), torch.full_like(want, info.tiny * info.eps / 2))


def wide(t):
    t = t.cpu()
    return t.float().double() if t.dtype == E4M3 else t.double()


def quantise_rows(x):
    """(codes, scales) of rows x in float32, as the library defines them."""
    x = x.float().cpu()
    finite = torch.where(torch.isfinite(x), x.abs(), torch.zeros(()))
    s = (finite.amax(-1) / torch.tensor(448.0)).clamp_min(LEAST)
    y = x / s[..., None]
    return torch.where(torch.isnan(y), y, y.clamp(-448.0, 448.0)).to(E4M3), s


def same_codes(a, b):
    """Equal E4M3 codes; any NaN code equals any other."""
    a, b = a.cpu().view(torch.uint8), b.cpu().view(torch.uint8)
    nan = (a & 0x7F) == 0x7F
    return bool(torch.equal(nan, (b & 0x7F) == 0x7F) and torch.equal(a[~nan], b[~nan]))


def norm_rope(x, w, eps, cos_sin, positions, interleaved):
    """x [T, H, D] in 64 bits -> normed and rotated."""
    x = x.double()
    D = x.shape[-1]
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + eps) * w.double()
    if cos_sin is None:
        return x
    rot = cos_sin.shape[1]
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    cs = cos_sin.double()[positions]
    c, s = cs[:, None, : rot // 2], cs[:, None, rot // 2:]
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def attend(q, k, v, scale):
    """One query row q [D] over k, v [t, D] in 64 bits: the output, and per
    channel A = sum p |v| and d = the largest |q|.|k| scale over the tokens,
    which the error bounds use."""
    if k.shape[0] == 0:
        z = torch.zeros(q.shape[0], dtype=torch.float64)
        return z, z, 0.0
    w = torch.softmax(k @ q * scale, 0)
    return w @ v, w @ v.abs(), float((k.abs() @ q.abs()).max() * abs(scale))


def attention_bound(out, A, d, D, out_dtype, weight_dtype):
    """|error| of a decode output: half a step of the stored output; each
    weight rounded to the MMA's 16-bit type; each score off by D + 8 float32
    roundings of d, which moves its weight, and the sum of the weights, by that
    relative amount each (twice that, as log2 e scales them); running sums,
    rescalings and exponentials below 2^-14 in all."""
    return half_step(out_dtype, out) + A * (torch.finfo(weight_dtype).eps / 2 + 4 * (D + 8) * U * d + 2.0 ** -14)


def block_table(lens, bs, NB, gen):
    nb = [-(-n // bs) for n in lens]
    perm = torch.randperm(NB, generator=gen)
    bt = torch.full((len(lens), max(nb + [1])), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(nb):
        bt[s, :n] = perm[at:at + n].to(torch.int32)
        at += n
    return bt


def select(scores, lens, bs, n, sink, recent):
    """Logical blocks chosen for one (sequence, kv head)."""
    nb = -(-lens // bs)
    if nb <= n:
        return list(range(nb))
    forced = set(range(min(sink, nb))) | set(range(max(nb - recent, 0), nb))
    rest = [j for j in range(nb) if j not in forced]
    x = [float(scores[j]) for j in range(nb)]
    rest.sort(key=lambda j: (0 if x[j] != x[j] else 1, 0.0 if x[j] != x[j] else -x[j], j))
    return sorted(forced | set(rest[:n - len(forced)]))
