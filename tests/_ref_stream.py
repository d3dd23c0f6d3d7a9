"""Plain 64-bit references of 4-bit caches and of attention through a window (torch on the CPU), with the error
bounds that their tests use."""
import math

import torch

from tests._ref64 import U, half_step

GROUP = 64
LEAST = 2.0 ** -126
F32_MAX = torch.finfo(torch.float32).max
BF16_MAX = torch.finfo(torch.bfloat16).max


def quantise_int4(x):
    """(codes [..., D] as numbers, params bf16 [..., D / 64, 2]) of rows x, in float32 as the library defines them."""
    g = x.float().cpu().unflatten(-1, (-1, GROUP))
    nan = torch.isnan(g).any(-1)
    finite = torch.isfinite(g)
    least = torch.where(finite, g, math.inf).amin(-1)
    most = torch.where(finite, g, -math.inf).amax(-1)
    none = least > most
    least, most = (torch.where(none, 0.0, t) for t in (least, most))
    low = least.to(torch.bfloat16)
    low = torch.where(low.float() > least, torch.nextafter(low, torch.full_like(low, -math.inf)), low).clamp_min(-BF16_MAX)
    spread = (most - low.float()).clamp_max(F32_MAX)
    scale = (spread / torch.tensor(15.0)).clamp_min(LEAST).to(torch.bfloat16)
    q = (g - low.float()[..., None]) / scale.float()[..., None]
    codes = torch.nan_to_num(q, nan=0.0, posinf=15.0, neginf=0.0).clamp(0, 15).round()
    scale = torch.where(nan, torch.tensor(math.nan, dtype=torch.bfloat16), scale)
    return codes.flatten(-2), torch.stack([scale, low], -1)


def pack_int4(codes):
    """Bytes [..., D / 2]: of every eight channels, 2 p and 2 p + 1 are nibbles p and p + 4 of a word."""
    c = codes.to(torch.int64).unflatten(-1, (-1, 8))
    word = torch.zeros(c.shape[:-1], dtype=torch.int64)
    for d in range(8):
        word |= c[..., d] << (4 * (d // 2 + 4 * (d % 2)))
    return torch.stack([(word >> (8 * b)) & 255 for b in range(4)], -1).flatten(-2).to(torch.uint8)


def codes_of(data):
    """Codes [..., D] of bytes [..., D / 2]."""
    b = data.cpu().to(torch.int64).unflatten(-1, (-1, 4))
    word = sum(b[..., i] << (8 * i) for i in range(4))
    return torch.stack([(word >> (4 * (d // 2 + 4 * (d % 2)))) & 15 for d in range(8)], -1).flatten(-2)


def wide_int4(data, params):
    """Values [..., D] in 64 bits, and of each the |scale| and |low|."""
    scale, low = (params.cpu().double()[..., i].repeat_interleave(GROUP, -1) for i in (0, 1))
    return codes_of(data).double() * scale + low, scale.abs(), low.abs()


def sees(P, n, window, sinks):
    """Which of tokens 0 .. n - 1 the token at position P attends to."""
    i = torch.arange(n)
    m = i <= P
    return m & ((i < sinks) | (i > P - window)) if window else m


def attend_rows(q, k, v, seen, scale):
    """Queries q [n, D] over k, v [t, D] where seen [n, t], in 64 bits -> outputs [n, D]; rows that see nothing are 0."""
    x = (q @ k.T * scale).masked_fill(~seen, -math.inf)
    w = torch.softmax(x, -1)
    w = torch.where(seen.any(-1, keepdim=True), w, torch.zeros((), dtype=w.dtype)).masked_fill(~seen, 0.0)
    vv = torch.where(seen.any(0)[:, None], v, torch.zeros((), dtype=v.dtype))
    return w @ vv, w


def bound(out, w, v_size, d, D, dtype, weight_eps):
    """|error| of outputs: half a step of the stored output; each weight off by weight_eps of itself (with it up to
    v_size of the output); each score by 2 (D + 8) float32 steps of d, the largest sum of its products' sizes, which
    moves a weight, and their sum, by that each; running sums, rescalings and exponentials below 2^-14 in all."""
    A = w @ v_size
    return half_step(dtype, out) + A * (weight_eps + 8 * (D + 8) * U * d + 2.0 ** -14)


def reference(q, rows, lens, k_new, Hkv, scale, window, sinks, dtype, weight_eps):
    """Outputs [S, k, Hq, D] in 64 bits and their bounds.  rows(s) gives (k, v, k_size, v_size) [L, Hkv, D]."""
    S, n, Hq, D = q.shape
    G = Hq // Hkv
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    for s in range(S):
        L = lens[s]
        if L == 0:
            continue
        k, v, ks, vs = rows(s)
        seen = torch.stack([sees(L - n + j, L, window, sinks) for j in range(n)])
        any_seen = seen.any(0)
        for h in range(Hkv):
            x = q[s, :, h * G:(h + 1) * G].double().cpu().reshape(n * G, D)
            m = seen.repeat_interleave(G, 0)
            kk = torch.where(any_seen[:, None], k[:, h], 0.0)
            o, w = attend_rows(x, kk, v[:, h], m, scale)
            d = float((x.abs() @ torch.where(any_seen[:, None], ks[:, h], 0.0).T).max() * abs(scale))
            t = bound(o, w, torch.where(any_seen[:, None], vs[:, h], 0.0), d, D, dtype, weight_eps)
            out[s, :, h * G:(h + 1) * G] = o.view(n, G, D)
            tol[s, :, h * G:(h + 1) * G] = t.view(n, G, D)
    return out, tol
