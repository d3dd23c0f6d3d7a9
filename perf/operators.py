"""The cache-side operators of a decode or prefill step, as measured cases.

  rope    norm_rope_cache: RMS norm of each q and k head, rotation by position, K/V rows into the paged cache
  rowsio  reshape_and_cache_rows, then gather_blocks_rows: an E4M3 cache with one scale per (token, head) row
  rows    decode_rows: attention of the new tokens over a row-scaled cache
  score   block_bounds of the newest tokens' blocks, then block_scores of every block of the contexts
  select  select_blocks: the blocks each (sequence, kv head) attends to
  chosen  decode_selected: attention of one new token over the chosen blocks

``own`` false: elementary torch operations in 32 bits; true: the library's calls on the same state.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # a decode step of four short sequences: what one small launch costs
        {"name": "rope_step", "op": "rope", "T": 4, "Hq": 8, "Hkv": 8, "D": 64, "bs": 16, "dt": "f16", "kv": "f16",
         "rot": 64, "inter": False, "pad": 0, "maxpos": 4096},
        # a prefill chunk of 16 x 2048 tokens with 32/8 heads: the largest rows written in one call
        {"name": "rope_chunk", "op": "rope", "T": 32768, "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "dt": "bf16",
         "kv": "bf16", "rot": 128, "inter": False, "pad": 0, "maxpos": 8192},
        # one new token of 64 sequences written, and a preempted sequence's 37 blocks read back
        {"name": "rowsio_step", "op": "rowsio", "T": 64, "Hkv": 8, "D": 64, "bs": 8, "dt": "f16", "nread": 37},
        # a prefill chunk written, and all its blocks read back for the next chunk's attention
        {"name": "rowsio_chunk", "op": "rowsio", "T": 32768, "Hkv": 8, "D": 128, "bs": 16, "dt": "bf16", "nread": 2048},
        # a decode step of 256 sequences of mixed lengths, 32/8 heads
        {"name": "rows_batch", "op": "rows", "S": 256, "k": 1, "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "dt": "bf16",
         "lens": "lognormal", "lo": 16, "hi": 8192, "lens_seed": 2, "P": 0},
        # eight long contexts, 64/8 heads, split into 512-token partitions
        {"name": "rows_long", "op": "rows", "S": 8, "k": 1, "Hq": 64, "Hkv": 8, "D": 128, "bs": 16, "dt": "bf16",
         "lens": "uniform", "lo": 32768, "hi": 131072, "lens_seed": 3, "P": 512},
        # one sequence's step with narrow heads and wide blocks: latency
        {"name": "score_one", "op": "score", "S": 1, "new": 1, "Hq": 8, "Hkv": 8, "D": 64, "bs": 32, "dt": "f16",
         "kv": "f16", "lens": "uniform", "lo": 20011, "hi": 20011, "lens_seed": 4},
        # the blocks of eight long contexts, 64/8 heads
        {"name": "score_long", "op": "score", "S": 8, "new": 1, "Hq": 64, "Hkv": 8, "D": 128, "bs": 16, "dt": "bf16",
         "kv": "bf16", "lens": "uniform", "lo": 32768, "hi": 131072, "lens_seed": 3},
        # 64 of one sequence's 1251 blocks
        {"name": "select_one", "op": "select", "S": 1, "Hkv": 8, "bs": 16, "n": 64, "sink": 1, "recent": 2,
         "lens": "uniform", "lo": 20011, "hi": 20011, "lens_seed": 4, "ties": False},
        # 256 of up to 8192 blocks each, scores with many ties
        {"name": "select_long", "op": "select", "S": 32, "Hkv": 8, "bs": 16, "n": 256, "sink": 1, "recent": 2,
         "lens": "uniform", "lo": 32768, "hi": 131072, "lens_seed": 5, "ties": True},
        # one sequence over 64 chosen blocks: latency
        {"name": "chosen_one", "op": "chosen", "S": 1, "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "dt": "bf16",
         "kv": "bf16", "n": 64, "blocks": 1251, "P": 64},
        # 64 sequences over 128 chosen blocks each
        {"name": "chosen_batch", "op": "chosen", "S": 64, "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "dt": "bf16",
         "kv": "bf16", "n": 128, "blocks": 512, "P": 0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rowsio", "rows", "score", "select", "chosen"])
    dt = rng.choice(["bf16", "f16"])
    D, bs = rng.choice([64, 128]), rng.choice([8, 16, 32])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    if op == "rope":
        inter, Hkv, G = rng.choice([False, True]), min(Hkv, 8), min(G, 8)
        return {"op": op, "T": _log_int(rng, 1, min(12000, (1 << 20) // (Hkv * (G + 2)))), "Hq": Hkv * G, "Hkv": Hkv, "D": D,
                "bs": bs, "dt": dt, "kv": rng.choice([dt, "e4m3", "rows"]),
                "rot": rng.choice([D, D // 2, 24, 50] if inter else [D, D // 2, 32, 48]), "inter": inter,
                "pad": rng.choice([0, 1, 3]), "maxpos": rng.choice([4096, 131072])}
    if op == "rowsio":
        T = _log_int(rng, 1, 20000)
        return {"op": op, "T": T, "Hkv": min(Hkv, 8), "D": D, "bs": bs, "dt": dt, "nread": max(1, T // (bs * rng.choice([1, 2, 5])))}
    if op == "rows":
        k = rng.choice([1, 1, 1, 2, 4])
        G = max(1, min(G, 16 // k))
        S = _log_int(rng, 1, 128)
        hi = max(64, min(65536, (1 << 20) // (S * Hkv)))
        lo = max(1, hi // rng.choice([1, 3, 9]))
        return {"op": op, "S": S, "k": k, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "bs": bs, "dt": dt, "lens": "uniform", "lo": lo,
                "hi": hi, "lens_seed": rng.randrange(1 << 20), "P": rng.choice([0, 256, 512]) if hi < 8192 else 512}
    if op == "chosen":
        S, n = _log_int(rng, 1, 48), _log_int(rng, 3, 160)
        return {"op": op, "S": S, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "bs": bs, "dt": dt, "kv": rng.choice([dt, "e4m3"]), "n": n,
                "blocks": n + _log_int(rng, 1, 256), "P": rng.choice([0, 64, 128, 256])} if S * Hkv * n * bs <= 1 << 20 else draw(rng)
    S = _log_int(rng, 1, 48)
    hi = max(64, min(100000, (3 << 20) // (S * Hkv)))
    lo = max(1, hi // rng.choice([1, 3, 9]))
    lens = {"lens": "uniform", "lo": lo, "hi": hi, "lens_seed": rng.randrange(1 << 20)}
    if op == "score":
        return {"op": op, "S": S, "new": rng.choice([1, 1, 2, 40]), "Hq": Hkv * G, "Hkv": Hkv, "D": D, "bs": bs, "dt": dt,
                "kv": rng.choice([dt, "e4m3"]), **lens}
    return {"op": op, "S": S, "Hkv": Hkv, "bs": bs, "n": _log_int(rng, 4, 512), "sink": rng.choice([0, 1, 2]),
            "recent": rng.choice([0, 1, 2]), **lens, "ties": rng.choice([False, True])}


def _lengths(case):
    r = random.Random(case["lens_seed"])
    if case["lens"] == "lognormal":  # median 1000
        return [min(case["hi"], max(case["lo"], int(round(math.exp(r.gauss(math.log(1000.0), 1.0)))))) for _ in range(case["S"])]
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["S"])]


def _blocks_of(lens, bs):
    return [-(-n // bs) for n in lens]


def _bytes_of(kv):
    return 1 if kv in ("e4m3", "rows") else 2


def work(case):
    op = case["op"]
    if op == "rope":
        T, Hq, Hkv, D = (case[x] for x in ("T", "Hq", "Hkv", "D"))
        live = T - case["pad"] if T > case["pad"] else T
        out = 2 * live * Hkv * (D * _bytes_of(case["kv"]) + (4 if case["kv"] == "rows" else 0))
        return {"bytes": live * ((Hq + 2 * Hkv) * D * 2 + Hq * D * 2 + case["rot"] * 4 + 16) + out + D * 4,
                "flops": live * (Hq + Hkv) * D * 8}
    if op == "rowsio":
        T, Hkv, D, bs, n = (case[x] for x in ("T", "Hkv", "D", "bs", "nread"))
        return {"bytes": 2 * T * Hkv * (3 * D + 4) + 8 * T + 2 * n * Hkv * bs * (3 * D + 4) + 8 * n,
                "flops": 2 * T * Hkv * D * 2 + 2 * n * Hkv * bs * D}
    if op == "rows":
        lens = _lengths(case)
        tok, nb = sum(lens), sum(_blocks_of(lens, case["bs"]))
        q = case["S"] * case["k"] * case["Hq"] * case["D"]
        return {"bytes": tok * case["Hkv"] * (2 * case["D"] + 8) + 4 * q + 4 * nb + 4 * case["S"],
                "flops": 4 * tok * case["k"] * case["Hq"] * case["D"]}
    if op == "score":
        lens = _lengths(case)
        nb, e = sum(_blocks_of(lens, case["bs"])), _bytes_of(case["kv"])
        new = sum(min(case["new"], n) for n in lens)
        return {"bytes": nb * case["Hkv"] * (2 * case["D"] * e + 4) + 4 * nb + new * case["Hkv"] * case["D"] * e
                + case["S"] * case["Hq"] * case["D"] * 2, "flops": 4 * nb * case["Hq"] * case["D"]}
    if op == "select":
        nb = _blocks_of(_lengths(case), case["bs"])
        return {"bytes": sum(nb) * (case["Hkv"] + 1) * 4 + sum(min(x, case["n"]) for x in nb) * case["Hkv"] * 4 + 8 * case["S"],
                "flops": sum(nb) * case["Hkv"]}
    tok = case["S"] * case["Hkv"] * case["n"] * case["bs"]
    return {"bytes": tok * 2 * case["D"] * _bytes_of(case["kv"]) + 4 * case["S"] * case["Hq"] * case["D"] + tok // case["bs"] * 4,
            "flops": 4 * tok * case["Hq"] // case["Hkv"] * case["D"]}


# ---- inputs ---------------------------------------------------------------


def _quantised(x):
    """E4M3 codes and the scale of each row (last dimension) of x, in 32 bits."""
    s = (x.abs().amax(-1) / torch.full((), E4M3_MAX, device=x.device)).clamp_min(TINY)
    return (x / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s


def _tables(lens, bs, NB, gen):
    """int32 [S, max blocks], -1 past each context, blocks placed at random in a pool of NB."""
    nb = torch.tensor(_blocks_of(lens, bs), device="cuda")
    most = max(1, int(max(_blocks_of(lens, bs))))
    at = torch.arange(most, device="cuda")[None, :]
    first = nb.cumsum(0) - nb
    perm = torch.randperm(NB, generator=gen, device="cuda")
    bt = perm[(first[:, None] + at).clamp(max=NB - 1)]
    return torch.where(at < nb[:, None], bt, -1).to(torch.int32)


def _pool(case, NB, gen):
    """K and V pools [NB, Hkv, bs, D] of the cache's type, standard normal values."""
    shape = (NB, case["Hkv"], case["bs"], case["D"])
    dt = DT[case["dt"]]
    k, v = (torch.randn(shape, generator=gen, device="cuda", dtype=dt) for _ in range(2))
    return (k, v) if case["kv"] == case["dt"] else (k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn))


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op, st = case["op"], {"case": case}
    randn = lambda *shape, dtype=torch.float32: torch.randn(shape, generator=gen, device="cuda", dtype=dtype)  # noqa: E731
    if op in ("rope", "rowsio"):
        T, Hkv, D, bs, dt = case["T"], case["Hkv"], case["D"], case["bs"], DT[case["dt"]]
        kv = "rows" if op == "rowsio" else case["kv"]
        NB = max(-(-T // bs), case.get("nread", 0)) + 3
        # whole blocks of consecutive tokens, blocks in random places
        perm = torch.randperm(NB, generator=gen, device="cuda")
        t = torch.arange(T, device="cuda")
        st["slots"] = perm[t // bs] * bs + t % bs
        shape = (NB, Hkv, bs, D)
        ct = torch.float8_e4m3fn if kv in ("e4m3", "rows") else dt
        st["k_cache"], st["v_cache"] = (torch.zeros(shape, device="cuda", dtype=ct) for _ in range(2))
        if kv == "rows":
            st["k_scales"], st["v_scales"] = (torch.ones(shape[:3], device="cuda") for _ in range(2))
        if op == "rowsio":  # a pool that other sequences have written to
            for x in "kv":
                st[x + "_cache"], st[x + "_scales"] = _quantised(randn(*shape) * torch.exp(0.5 * randn(*shape[:3], 1)))
            st["key"], st["value"] = ((randn(T, Hkv, D) * torch.exp(randn(T, Hkv, 1))).to(dt) for _ in range(2))
            st["ids"] = perm[: case["nread"]].clone()
            st["k16"], st["v16"] = (torch.zeros((case["nread"],) + shape[1:], device="cuda", dtype=dt) for _ in range(2))
            return st
        Hq, rot = case["Hq"], case["rot"]
        # q, k and v are views of one projection's rows, the heads' widths as trained models have them
        qkv = (randn(T, (Hq + 2 * Hkv) * D) * torch.exp(0.5 * randn(T, 1))).to(dt)
        st["q"] = qkv[:, : Hq * D].unflatten(1, (Hq, D))
        st["key"] = qkv[:, Hq * D : (Hq + Hkv) * D].unflatten(1, (Hkv, D))
        st["value"] = qkv[:, (Hq + Hkv) * D :].unflatten(1, (Hkv, D))
        st["q_out"] = torch.zeros((T, Hq, D), device="cuda", dtype=dt)
        st["q_weight"], st["k_weight"] = ((1 + 0.2 * randn(D)).to(dt) for _ in range(2))
        i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
        angle = torch.arange(case["maxpos"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2 * i / rot)
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        start = torch.randint(0, case["maxpos"], (1,), generator=gen, device="cuda")
        st["positions"] = (start + t) % case["maxpos"]
        if 0 < case["pad"] < T:  # a batch padded to a captured size
            st["slots"][-case["pad"]:] = -1
        st["kv_scale"] = 0.02 if kv == "e4m3" else 1.0
        return st
    if op == "select":
        lens, bs, Hkv = _lengths(case), case["bs"], case["Hkv"]
        nb = _blocks_of(lens, bs)
        st["bt"] = _tables(lens, bs, sum(nb) + 5, gen)
        st["cl"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        x = randn(case["S"], Hkv, st["bt"].shape[1]) * 3 + 12
        x = (x * 2).round() / 2 if case["ties"] else x
        st["scores"] = torch.where((st["bt"] >= 0)[:, None, :], x, -math.inf)
        st["tables"] = torch.full((case["S"], Hkv, case["n"]), -1, device="cuda", dtype=torch.int32)
        st["sel_lens"] = torch.zeros((case["S"], Hkv), device="cuda", dtype=torch.int32)
        return st
    S, Hq, Hkv, D, bs, dt = case["S"], case["Hq"], case["Hkv"], case["D"], case["bs"], DT[case["dt"]]
    st["scale"] = D ** -0.5
    if op == "chosen":
        n, most = case["n"], case["blocks"]
        NB = S * most
        st["k_cache"], st["v_cache"] = _pool(case, NB, gen)
        own_blocks = torch.randperm(NB, generator=gen, device="cuda").view(S, 1, most).expand(S, Hkv, most)
        pick = torch.rand((S, Hkv, most), generator=gen, device="cuda").argsort(-1)[..., :n].sort(-1).values
        st["tables"] = own_blocks.gather(2, pick).to(torch.int32)
        tail = torch.randint(1, bs + 1, (S, 1), generator=gen, device="cuda").expand(S, Hkv)
        st["sel_lens"] = ((n - 1) * bs + tail).to(torch.int32).contiguous()
        st["q"] = randn(S, Hq, D, dtype=dt)
        st["kv_scale"] = 0.9 if case["kv"] == "e4m3" else 1.0
        st["out"] = torch.empty_like(st["q"])
        most_tokens = n * bs
        rows = S
    else:
        lens = _lengths(case)
        NB = sum(_blocks_of(lens, bs)) + 5
        st["bt"] = _tables(lens, bs, NB, gen)
        st["cl"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        if op == "score":
            k_cache, _ = _pool(case, NB, gen)
            st["k_cache"] = k_cache
            st["q"] = randn(S, Hq, D, dtype=dt)
            x = k_cache.float()
            st["bounds"] = torch.stack([x.amin(2), x.amax(2)], 2).to(k_cache.dtype)
            st["scores"] = torch.empty((S, Hkv, st["bt"].shape[1]), device="cuda")
            return st
        for name in ("k", "v"):
            x = randn(NB, Hkv, bs, D, dtype=dt).float().mul_(torch.exp(0.5 * randn(NB, Hkv, bs, 1)))
            st[name + "_cache"], st[name + "_scales"] = _quantised(x)
            del x
        st["q"] = randn(*((S, Hq, D) if case["k"] == 1 else (S, case["k"], Hq, D)), dtype=dt)
        st["out"] = torch.empty_like(st["q"])
        most_tokens = max(lens)
        rows = S * case["k"]
    st["most"] = most_tokens
    if case["P"]:  # one float row and its (m, l) per partition of each query head
        st["workspace"] = torch.empty(rows * Hq * -(-most_tokens // case["P"]) * (D + 2) * 4, device="cuda", dtype=torch.uint8)
    return st


# ---- the library's calls --------------------------------------------------


def _run_own(st):
    from paged_kv_cache_230_gb300 import pagedattn as pa
    c = st["case"]
    op = c["op"]
    if op == "rope":
        pa.norm_rope_cache(st["q_out"], st["q"], st["key"], st["value"], st["positions"], st["cos_sin"], st["k_cache"], st["v_cache"],
                           st["slots"], q_weight=st["q_weight"], k_weight=st["k_weight"], eps=1e-6, interleaved=c["inter"],
                           kv_scale=st["kv_scale"], k_scales=st.get("k_scales"), v_scales=st.get("v_scales"))
    elif op == "rowsio":
        pa.reshape_and_cache_rows(st["key"], st["value"], st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"], st["slots"])
        pa.gather_blocks_rows(st["k16"], st["v16"], st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"], st["ids"])
    elif op == "rows":
        pa.decode_rows(st["out"], st["q"], st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"], st["bt"], st["cl"], st["scale"],
                       max_context_len=st["most"], partition_size=c["P"], workspace=st.get("workspace"))
    elif op == "score":
        pa.block_bounds(st["bounds"], st["k_cache"], st["bt"], st["cl"], c["new"])
        pa.block_scores(st["scores"], st["q"], st["bounds"], st["bt"], st["cl"], c["bs"])
    elif op == "select":
        pa.select_blocks(st["tables"], st["sel_lens"], st["scores"], st["bt"], st["cl"], c["bs"], sink_blocks=c["sink"],
                         recent_blocks=c["recent"])
    else:
        pa.decode_selected(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["sel_lens"], st["scale"],
                           kv_scale=st["kv_scale"], partition_size=c["P"], workspace=st.get("workspace"))


# ---- the plain forms ------------------------------------------------------


def _put(cache, slots, src, rows):
    """cache[block, :, offset] = rows[src] at each slot; 8-bit types through their bytes."""
    bs = cache.shape[2]
    if cache.dtype == torch.float8_e4m3fn:
        cache, rows = cache.view(torch.uint8), rows.view(torch.uint8)
    cache[slots // bs, :, slots % bs] = rows[src]


def _take(cache, ids):
    """Blocks `ids` of a cache, as 32-bit values."""
    if cache.dtype == torch.float8_e4m3fn:
        return cache.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
    return cache[ids].float()


def _rotated(x, cos_sin, rot, inter):
    cos, sin = cos_sin[:, None, : rot // 2], cos_sin[:, None, rot // 2:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., : rot // 2], x[..., rot // 2: rot])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y, z], -1).flatten(-2) if inter else torch.cat([y, z], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _normed(x, w, eps):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()


def _plain_rope(st):
    c = st["case"]
    dt = st["q"].dtype
    live = st["slots"] >= 0
    src = torch.where(live, torch.arange(c["T"], device="cuda"), 0)  # a padding token repeats token 0's write
    slots = st["slots"][src]
    table = st["cos_sin"][st["positions"]]
    q = _rotated(_normed(st["q"], st["q_weight"], 1e-6), table, c["rot"], c["inter"]).to(dt)
    st["q_out"].copy_(torch.where(live[:, None, None], q, st["q_out"]))
    k, v = _rotated(_normed(st["key"], st["k_weight"], 1e-6), table, c["rot"], c["inter"]), st["value"].float()
    for name, x in (("k", k), ("v", v)):
        if c["kv"] == "rows":
            codes, s = _quantised(x)
            st[name + "_scales"][slots // c["bs"], :, slots % c["bs"]] = s[src]
        elif c["kv"] == "e4m3":
            codes = (x / torch.full((), st["kv_scale"], device="cuda")).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        else:
            codes = x.to(dt)
        _put(st[name + "_cache"], slots, src, codes)


def _plain_rowsio(st):
    bs, src = st["case"]["bs"], torch.arange(st["case"]["T"], device="cuda")
    for x, name in ((st["key"], "k"), (st["value"], "v")):
        codes, s = _quantised(x.float())
        _put(st[name + "_cache"], st["slots"], src, codes)
        st[name + "_scales"][st["slots"] // bs, :, st["slots"] % bs] = s
        st[name + "16"].copy_(_take(st[name + "_cache"], st["ids"]) * st[name + "_scales"][st["ids"]][..., None])


def _attend(q, k, v, seen, scale):
    """q [..., n, D], k and v [..., t, D], seen [..., n, t] -> softmax(scale q k') v."""
    w = (q @ k.transpose(-1, -2) * scale).masked_fill(~seen, -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True).clamp_min(-1e30))
    return (w @ v) / w.sum(-1, keepdim=True).clamp_min(TINY)


def _plain_rows(st):
    c = st["case"]
    S, n, Hkv, D, G = c["S"], c["k"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    ids = st["bt"].clamp_min(0).long()
    k, v = ((_take(st[x + "_cache"], ids) * st[x + "_scales"][ids][..., None]).transpose(1, 2).reshape(S, Hkv, -1, D) for x in "kv")
    q = st["q"].float().view(S, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, n * G, D)
    at = torch.arange(k.shape[2], device="cuda")
    last = st["cl"][:, None] - n + torch.arange(n, device="cuda")  # position of each new token
    seen = (at <= last[..., None]).repeat_interleave(G, 1)[:, None]
    out = _attend(q, k, v, seen, st["scale"]).view(S, Hkv, n, G, D).permute(0, 2, 1, 3, 4)
    st["out"].copy_(out.reshape(st["out"].shape))


def _plain_score(st):
    c = st["case"]
    bs, S, Hkv, G = c["bs"], c["S"], c["Hkv"], c["Hq"] // c["Hkv"]
    L = st["cl"].long()[:, None]
    nb = (L + bs - 1) // bs
    j = ((L - c["new"]).clamp_min(0) // bs + torch.arange((c["new"] + bs - 2) // bs + 1, device="cuda")).minimum(nb - 1)
    ids = st["bt"].long().gather(1, j)
    x = _take(st["k_cache"], ids)
    live = (j[..., None] * bs + torch.arange(bs, device="cuda") < L[..., None])[:, :, None, :, None]
    lohi = torch.stack([x.masked_fill(~live, math.inf).amin(3), x.masked_fill(~live, -math.inf).amax(3)], 3).to(st["bounds"].dtype)
    if lohi.dtype == torch.float8_e4m3fn:
        st["bounds"].view(torch.uint8)[ids] = lohi.view(torch.uint8)
    else:
        st["bounds"][ids] = lohi
    every = _take(st["bounds"], st["bt"].clamp_min(0).long())  # [S, blocks, Hkv, 2, D]
    q = st["q"].float().view(S, Hkv, G, c["D"])
    q = torch.cat([q.clamp(max=0), q.clamp(min=0)], -1)
    score = (q @ every.permute(0, 2, 3, 4, 1).reshape(S, Hkv, 2 * c["D"], -1)).amax(2)
    st["scores"].copy_(score.masked_fill((torch.arange(score.shape[-1], device="cuda") >= nb)[:, None], -math.inf))


def _plain_select(st):
    c = st["case"]
    bs, n = c["bs"], c["n"]
    most = st["bt"].shape[1]
    L = st["cl"].long()[:, None, None]
    nb = (L + bs - 1) // bs
    at = torch.arange(most, device="cuda")
    rank = torch.where((at < c["sink"]) | (at >= nb - c["recent"]), 2, 1)
    rank = torch.where(at < nb, rank, 0).expand(st["scores"].shape)
    best = (st["scores"] + 0.0).sort(dim=-1, descending=True, stable=True).indices
    best = best.gather(-1, rank.gather(-1, best).sort(dim=-1, descending=True, stable=True).indices)[..., :n]
    best = torch.where(best < nb, best, most).sort(-1).values
    count = (best < most).sum(-1, keepdim=True)
    phys = st["bt"].long()[:, None, :].expand(-1, c["Hkv"], -1).gather(-1, best.clamp(max=most - 1))
    st["tables"].fill_(-1)
    st["tables"][..., : best.shape[-1]] = torch.where(best < most, phys, -1).to(torch.int32)
    has_last = (best == nb - 1).any(-1, keepdim=True)
    st["sel_lens"].copy_((count * bs - torch.where(has_last, nb * bs - L, 0)).squeeze(-1))


def _plain_chosen(st):
    c = st["case"]
    S, Hkv, D, G = c["S"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    heads = torch.arange(Hkv, device="cuda")[None, :, None]
    ids = st["tables"].long()
    if st["k_cache"].dtype == torch.float8_e4m3fn:
        k, v = (st[x].view(torch.uint8)[ids, heads].view(torch.float8_e4m3fn).float() * st["kv_scale"] for x in ("k_cache", "v_cache"))
    else:
        k, v = (st[x][ids, heads].float() for x in ("k_cache", "v_cache"))
    k, v = k.reshape(S, Hkv, -1, D), v.reshape(S, Hkv, -1, D)
    seen = torch.arange(k.shape[2], device="cuda") < st["sel_lens"][:, :, None, None]
    st["out"].copy_(_attend(st["q"].float().view(S, Hkv, G, D), k, v, seen, st["scale"]).reshape(st["out"].shape))


PLAIN = {"rope": _plain_rope, "rowsio": _plain_rowsio, "rows": _plain_rows, "score": _plain_score, "select": _plain_select,
         "chosen": _plain_chosen}
OUTPUTS = {"rope": ("q_out", "k_cache", "v_cache", "k_scales", "v_scales"),
           "rowsio": ("k_cache", "v_cache", "k_scales", "v_scales", "k16", "v16"),
           "rows": ("out",), "score": ("bounds", "scores"), "select": ("tables", "sel_lens"), "chosen": ("out",)}


def run(state):
    if own:
        _run_own(state)
    else:
        PLAIN[state["case"]["op"]](state)
    return {x: state[x] for x in OUTPUTS[state["case"]["op"]] if x in state}


# ---- the definitions in 64 bits -------------------------------------------


def _wide(x):
    """Any cache or input tensor in 64 bits."""
    return x.float().double() if x.dtype == torch.float8_e4m3fn else x.double()


def _codes64(x, s):
    """The E4M3 value nearest x / s (ties to even), by its exponent and three bits of fraction."""
    y = (x / s).clamp(-E4M3_MAX, E4M3_MAX)
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (y / step).round() * step


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "select":
        return None
    if op in ("rope", "rowsio"):
        key, value = st["key"].double(), st["value"].double()
        res = {}
        if op == "rope":
            rot, D = case["rot"], case["D"]
            i = torch.arange(rot // 2, device="cuda")
            left, right = (2 * i, 2 * i + 1) if case["inter"] else (i, i + rot // 2)
            cs = st["cos_sin"].double()[st["positions"]]

            def turned(x, w):
                x = x.double()
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + 1e-6) * w.double()
                y = x.clone()
                c, s = cs[:, None, : rot // 2], cs[:, None, rot // 2:]
                y[..., left] = x[..., left] * c - x[..., right] * s
                y[..., right] = x[..., right] * c + x[..., left] * s
                return y

            res["q_out"] = turned(st["q"], st["q_weight"])
            res["q_out"][st["slots"] < 0] = 0.0
            key = turned(st["key"], st["k_weight"])
        keep = st["slots"] >= 0
        blk, off = st["slots"][keep] // case["bs"], st["slots"][keep] % case["bs"]
        kv = "rows" if op == "rowsio" else case["kv"]
        for name, x in (("k", key), ("v", value)):
            x = x[keep]
            pool = _wide(st[name + "_cache"])
            if kv == "rows":
                s = (x.abs().amax(-1) / E4M3_MAX).clamp_min(TINY)
                scales = st[name + "_scales"].double()
                scales[blk, :, off] = s
                res[name + "_scales"] = scales
                pool[blk, :, off] = _codes64(x, s[..., None])
                if op == "rowsio":
                    res[name + "16"] = pool[st["ids"]] * scales[st["ids"]][..., None]
            else:
                pool[blk, :, off] = _codes64(x, float(torch.tensor(st["kv_scale"]))) if kv == "e4m3" else x
            res[name + "_cache"] = pool
        return {x: res[x] for x in OUTPUTS[op] if x in res}
    S, Hkv, G = case["S"], case["Hkv"], case["Hq"] // case["Hkv"]
    if op == "score":
        scores = torch.full(st["scores"].shape, -math.inf, device="cuda", dtype=torch.float64)
        bounds = _wide(st["bounds"])
        for s, L in enumerate(_lengths(case)):
            nb = -(-L // case["bs"])
            ids = st["bt"][s, :nb].long()
            for j in range(max(0, L - case["new"]) // case["bs"], nb):
                keys = _wide(st["k_cache"][ids[j]])[:, : L - j * case["bs"]]
                bounds[ids[j], :, 0], bounds[ids[j], :, 1] = keys.min(1).values, keys.max(1).values
            for h in range(Hkv):
                q = st["q"][s, h * G: (h + 1) * G].double()
                lo, hi = bounds[ids, h, 0], bounds[ids, h, 1]
                scores[s, h, :nb] = (q.clamp(min=0) @ hi.T + q.clamp(max=0) @ lo.T).max(0).values
        return {"bounds": bounds, "scores": scores}
    out = torch.zeros(st["out"].shape, device="cuda", dtype=torch.float64)
    k_new = case.get("k", 1)
    flat = out.view(S, k_new, case["Hq"], case["D"])
    q = st["q"].double().view(flat.shape)
    lens = _lengths(case) if op == "rows" else None
    for s in range(S):
        for h in range(Hkv):
            if op == "rows":
                L, ids = lens[s], st["bt"][s].long()
                ids = ids[: -(-L // case["bs"])]
            else:
                L, ids = int(st["sel_lens"][s, h]), st["tables"][s, h].long()
            k, v = (st[x + "_cache"].view(torch.uint8)[ids, h].view(st[x + "_cache"].dtype) for x in "kv")
            k, v = _wide(k), _wide(v)
            if op == "rows":
                k, v = k * st["k_scales"][ids, h].double()[..., None], v * st["v_scales"][ids, h].double()[..., None]
            else:
                k, v = k * float(torch.tensor(st["kv_scale"])), v * float(torch.tensor(st["kv_scale"]))
            k, v = k.flatten(0, 1), v.flatten(0, 1)
            for j in range(k_new):
                t = L - k_new + j + 1
                if t > 0:
                    w = torch.softmax(q[s, j, h * G: (h + 1) * G] @ k[:t].T * st["scale"], -1)
                    flat[s, j, h * G: (h + 1) * G] = w @ v[:t]
    return {"out": out}
