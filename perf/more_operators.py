"""Attention over long streams in little memory, as measured cases.

  int4io  reshape_and_cache_int4, then gather_blocks_int4: a cache of 4-bit codes with a scale and a least value per 64 channels
  int4    decode_int4: attention of the new tokens over a 4-bit cache, over whole contexts or through a window
  window  decode_window: attention of the new tokens over the last `win` tokens and the first `sinks` ones
  prompt  prefill_window: the same for the tokens of a prompt's chunk

``own`` false: elementary torch operations in 32 bits; true: the library's calls on the same state.
"""
import math
import random

import torch

own = False

GROUP = 64  # channels that share a scale and a least value
LEAST_SCALE = 2.0 ** -126
BF16_MAX = torch.finfo(torch.bfloat16).max
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one new token of 48 sequences written, and a preempted sequence's 29 blocks read back
        {"name": "int4io_step", "op": "int4io", "T": 48, "Hkv": 8, "D": 64, "bs": 8, "dt": "f16", "nread": 29},
        # a prefill chunk of 16 x 2048 tokens written, and all its blocks read back for the next chunk's attention
        {"name": "int4io_chunk", "op": "int4io", "T": 32768, "Hkv": 8, "D": 128, "bs": 16, "dt": "bf16", "nread": 2048},
        # one sequence's step over its whole context, 32/8 heads: latency
        {"name": "int4_one", "op": "int4", "S": 1, "k": 1, "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "dt": "bf16",
         "lens": "uniform", "lo": 1999, "hi": 1999, "lens_seed": 11, "win": 0, "sinks": 0},
        # a decode step of 256 sequences of mixed lengths, 32/8 heads
        {"name": "int4_batch", "op": "int4", "S": 256, "k": 1, "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "dt": "bf16",
         "lens": "lognormal", "lo": 16, "hi": 8192, "lens_seed": 2, "win": 0, "sinks": 0},
        # eight long contexts, 64/8 heads
        {"name": "int4_long", "op": "int4", "S": 8, "k": 1, "Hq": 64, "Hkv": 8, "D": 128, "bs": 16, "dt": "f16",
         "lens": "uniform", "lo": 32768, "hi": 131072, "lens_seed": 3, "win": 0, "sinks": 0},
        # two new tokens of 75 long streams, narrow heads, through a window
        {"name": "int4_window", "op": "int4", "S": 75, "k": 2, "Hq": 32, "Hkv": 8, "D": 64, "bs": 32, "dt": "bf16",
         "lens": "uniform", "lo": 5000, "hi": 30000, "lens_seed": 7, "win": 4096, "sinks": 4},
        # one stream's step through a window of 1024, 32/8 heads: latency
        {"name": "window_one", "op": "window", "S": 1, "k": 1, "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "dt": "bf16",
         "kv": "bf16", "lens": "uniform", "lo": 50021, "hi": 50021, "lens_seed": 4, "win": 1024, "sinks": 4},
        # a decode step of 256 streams through a window of 4096; some are shorter than it
        {"name": "window_batch", "op": "window", "S": 256, "k": 1, "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "dt": "bf16",
         "kv": "bf16", "lens": "uniform", "lo": 100, "hi": 16000, "lens_seed": 5, "win": 4096, "sinks": 4},
        # four draft tokens of 33 streams verified over an E4M3 cache
        {"name": "window_verify", "op": "window", "S": 33, "k": 4, "Hq": 16, "Hkv": 4, "D": 128, "bs": 16, "dt": "f16",
         "kv": "e4m3", "lens": "uniform", "lo": 3, "hi": 20000, "lens_seed": 6, "win": 2000, "sinks": 1},
        # a short question after one stream's context
        {"name": "prompt_one", "op": "prompt", "S": 1, "C": 37, "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "dt": "bf16",
         "kv": "bf16", "lens": "uniform", "lo": 9001, "hi": 9001, "lens_seed": 8, "win": 1024, "sinks": 4},
        # a chunk of 16 x 2048 prompt tokens, 32/8 heads
        {"name": "prompt_chunk", "op": "prompt", "S": 16, "C": 2048, "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "dt": "bf16",
         "kv": "bf16", "lens": "uniform", "lo": 4096, "hi": 12000, "lens_seed": 9, "win": 1024, "sinks": 4},
        # chunks of narrow heads over an E4M3 cache
        {"name": "prompt_e4m3", "op": "prompt", "S": 5, "C": 1000, "Hq": 24, "Hkv": 8, "D": 64, "bs": 32, "dt": "f16",
         "kv": "e4m3", "lens": "uniform", "lo": 900, "hi": 9000, "lens_seed": 10, "win": 512, "sinks": 32},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["int4io", "int4", "int4", "window", "window", "prompt"])
    dt = rng.choice(["bf16", "f16"])
    D, bs = rng.choice([64, 128]), rng.choice([8, 16, 32])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    if op == "int4io":
        T = _log_int(rng, 1, 20000)
        return {"op": op, "T": T, "Hkv": min(Hkv, 8), "D": D, "bs": bs, "dt": dt, "nread": -(-T // bs) * rng.choice([1, 1, 2])}
    sinks = rng.choice([0, 1, 4, 4, 16, 33, 100])
    base = {"op": op, "Hkv": Hkv, "Hq": Hkv * G, "D": D, "bs": bs, "dt": dt, "lens": "uniform", "lens_seed": rng.randrange(1 << 20),
            "sinks": sinks}
    if op == "prompt":
        S = _log_int(rng, 1, 12)
        C = _log_int(rng, 2, max(2, min(2048, (1 << 19) // (S * Hkv * G))))
        hi = _log_int(rng, 64, 9000)
        return {**base, "S": S, "C": C, "kv": rng.choice([dt, dt, "e4m3"]), "lo": max(0, hi // rng.choice([1, 3, 9])), "hi": hi,
                "win": _log_int(rng, 1, 3000)}
    S, k = _log_int(rng, 1, 128), rng.choice([1, 1, 1, 2, 3, 5])
    hi = max(64, min(65536, (3 << 20) // (S * Hkv)))
    span = {"S": S, "k": k, "lo": hi // rng.choice([1, 3, 9, hi + 1]), "hi": hi, "win": _log_int(rng, 1, min(hi, 8192))}
    if op == "window":
        return {**base, **span, "kv": rng.choice([dt, "e4m3"])}
    if rng.random() < 0.6:
        span.update(win=0, sinks=0)
    return {**base, **span}


def _lengths(case):
    r = random.Random(case["lens_seed"])
    if case["lens"] == "lognormal":  # median 1000
        return [min(case["hi"], max(case["lo"], int(round(math.exp(r.gauss(math.log(1000.0), 1.0)))))) for _ in range(case["S"])]
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["S"])]


def _blocks_of(lens, bs):
    return [-(-n // bs) for n in lens]


def _seen_by(pos, win, sinks):
    """How many tokens the token at `pos` attends to."""
    if pos < 0:
        return 0
    first = max(0, pos - win + 1) if win else 0
    return pos + 1 - first + min(sinks, first)


def _seen_by_any(L, new, win, sinks):
    """How many tokens any of the last `new` tokens of a context of L attends to."""
    if L == 0:
        return 0
    first = max(0, max(0, L - new) - win + 1) if win else 0
    return L - first + min(sinks, first)


def work(case):
    op = case["op"]
    if op == "int4io":
        T, Hkv, D, bs, n = (case[x] for x in ("T", "Hkv", "D", "bs", "nread"))
        row = D // 2 + 4 * (D // GROUP)
        return {"bytes": 2 * T * Hkv * (2 * D + row) + 8 * T + 2 * n * Hkv * bs * (2 * D + row) + 8 * n,
                "flops": 2 * T * Hkv * D * 4 + 2 * n * Hkv * bs * D * 2}
    lens, Hq, Hkv, D, win, sinks = _lengths(case), case["Hq"], case["Hkv"], case["D"], case["win"], case["sinks"]
    new = case["C"] if op == "prompt" else case["k"]
    tok = sum(_seen_by_any(n, new, win, sinks) for n in lens)
    pairs = sum(sum(_seen_by(n - new + j, win, sinks) for j in range(new)) for n in lens)
    row = D // 2 + 4 * (D // GROUP) if op == "int4" else D * (1 if case["kv"] == "e4m3" else 2)
    return {"bytes": 2 * tok * Hkv * row + 4 * case["S"] * new * Hq * D + 4 * (tok // case["bs"]) + 4 * case["S"],
            "flops": 4 * pairs * Hq * D}


# ---- 4-bit codes ------------------------------------------------------------


def _quantised(x):
    """Codes 0..15 [..., D] and parameters bf16 [..., D / 64, 2] (scale, least value) of rows x, finite, in 32 bits.

    The least value is the group's smallest, rounded down to bf16, so that every value lies at or above it."""
    g = x.unflatten(-1, (-1, GROUP))
    least = g.amin(-1)
    low = least.to(torch.bfloat16)
    down = torch.nextafter(low, torch.full_like(low, -math.inf))
    low = torch.where(low.float() > least, down, low).clamp_min(-BF16_MAX)
    spread = (g.amax(-1) - low.float()).clamp_max(torch.finfo(torch.float32).max)
    scale = (spread / torch.full((), 15.0, device=x.device)).to(torch.bfloat16).clamp_min(LEAST_SCALE)
    codes = ((g - low.float()[..., None]) / scale.float()[..., None]).round().clamp(0, 15)
    return codes.flatten(-2), torch.stack([scale, low], -1)


def _packed(codes):
    """Bytes [..., D / 2]: channels 2p and 2p + 1 of eight are nibbles p and p + 4 of a word, lowest first."""
    c = codes.to(torch.uint8).unflatten(-1, (-1, 8))
    c = c[..., [0, 2, 4, 6, 1, 3, 5, 7]]
    return (c[..., 0::2] | c[..., 1::2] << 4).flatten(-2)


def _values(data, params):
    """The values that bytes [..., D / 2] with params [..., D / 64, 2] stand for, in 32 bits."""
    b = data.unflatten(-1, (-1, 4))
    low, high = b & 15, b >> 4
    c = torch.stack([low[..., 0], low[..., 2], high[..., 0], high[..., 2], low[..., 1], low[..., 3], high[..., 1], high[..., 3]], -1)
    c = c.flatten(-2).unflatten(-1, (-1, GROUP)).float()
    return (c * params[..., 0:1].float() + params[..., 1:2].float()).flatten(-2)


# ---- inputs -----------------------------------------------------------------


def _tables(lens, bs, NB, gen):
    """int32 [S, max blocks], -1 past each context, blocks placed at random in a pool of NB."""
    nb = torch.tensor(_blocks_of(lens, bs), device="cuda")
    most = max(1, max(_blocks_of(lens, bs)))
    at = torch.arange(most, device="cuda")[None, :]
    first = nb.cumsum(0) - nb
    perm = torch.randperm(NB, generator=gen, device="cuda")
    bt = perm[(first[:, None] + at).clamp(max=NB - 1)]
    return torch.where(at < nb[:, None], bt, -1).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op, st = case["op"], {"case": case}
    Hkv, D, bs, dt = case["Hkv"], case["D"], case["bs"], DT[case["dt"]]
    randn = lambda *shape, dtype=torch.float32: torch.randn(shape, generator=gen, device="cuda", dtype=dtype)  # noqa: E731

    def channels(x):  # a few channels of keys and values are several times as wide as the others, and off centre
        wide = torch.exp(0.6 * randn(Hkv, 1, D)).to(x.dtype)
        return x * wide + (0.5 * randn(Hkv, 1, D)).to(x.dtype)

    if op == "int4io":
        T, n = case["T"], case["nread"]
        NB = max(-(-T // bs), n) + 3
        # whole blocks of consecutive tokens, blocks in random places
        perm = torch.randperm(NB, generator=gen, device="cuda")
        t = torch.arange(T, device="cuda")
        st["slots"] = perm[t // bs] * bs + t % bs
        st["ids"] = perm[:n].clone()
        for x, row in (("k", "key"), ("v", "value")):  # a pool that other sequences have written to
            codes, params = _quantised(channels(randn(NB, Hkv, bs, D)))
            st[x + "_cache"], st[x + "_params"] = _packed(codes), params
            st[row] = channels(randn(T, Hkv, 1, D)).squeeze(2).to(dt)
            st[x + "16"] = torch.zeros((n, Hkv, bs, D), device="cuda", dtype=dt)
        return st
    lens, S, Hq = _lengths(case), case["S"], case["Hq"]
    NB = sum(_blocks_of(lens, bs)) + 5
    st["bt"] = _tables(lens, bs, NB, gen)
    st["cl"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    st["scale"] = D ** -0.5
    for x in "kv":
        pool = channels(randn(NB, Hkv, bs, D, dtype=dt))
        if op == "int4":
            codes, params = _quantised(pool.float())
            st[x + "_cache"], st[x + "_params"] = _packed(codes), params
            del codes
        else:
            st[x + "_cache"] = pool if case["kv"] == case["dt"] else pool.to(torch.float8_e4m3fn)
        del pool
    new = case["C"] if op == "prompt" else case["k"]
    st["q"] = randn(*((S, Hq, D) if op != "prompt" and new == 1 else (S, new, Hq, D)), dtype=dt)
    st["out"] = torch.empty_like(st["q"])
    if op != "int4":
        st["kv_scale"] = 0.9 if case["kv"] == "e4m3" else 1.0
    if own and op != "prompt":
        from paged_kv_cache_230_gb300 import pagedattn as pa
        st["workspace"] = torch.empty(pa.decode_flat_workspace_size(D), device="cuda", dtype=torch.uint8)
    return st


# ---- the library's calls ----------------------------------------------------


def _run_own(st):
    from paged_kv_cache_230_gb300 import pagedattn as pa
    c = st["case"]
    op = c["op"]
    if op == "int4io":
        pa.reshape_and_cache_int4(st["key"], st["value"], st["k_cache"], st["v_cache"], st["k_params"], st["v_params"], st["slots"])
        pa.gather_blocks_int4(st["k16"], st["v16"], st["k_cache"], st["v_cache"], st["k_params"], st["v_params"], st["ids"])
    elif op == "int4":
        pa.decode_int4(st["out"], st["q"], st["k_cache"], st["v_cache"], st["k_params"], st["v_params"], st["bt"], st["cl"], st["scale"],
                       window=c["win"], num_sinks=c["sinks"], workspace=st["workspace"])
    elif op == "window":
        pa.decode_window(st["out"], st["q"], st["k_cache"], st["v_cache"], st["bt"], st["cl"], st["scale"], c["win"],
                         num_sinks=c["sinks"], kv_scale=st["kv_scale"], workspace=st["workspace"])
    else:
        pa.prefill_window(st["out"], st["q"], st["k_cache"], st["v_cache"], st["bt"], st["cl"], st["scale"], c["win"],
                          num_sinks=c["sinks"], kv_scale=st["kv_scale"])


# ---- the plain forms --------------------------------------------------------


def _plain_int4io(st):
    bs = st["case"]["bs"]
    block, offset = st["slots"] // bs, st["slots"] % bs
    for x, row in (("k", "key"), ("v", "value")):
        codes, params = _quantised(st[row].float())
        st[x + "_cache"][block, :, offset] = _packed(codes)
        st[x + "_params"][block, :, offset] = params
        st[x + "16"].copy_(_values(st[x + "_cache"][st["ids"]], st[x + "_params"][st["ids"]]))


def _tokens(st, x, block, offset):
    """K or V rows at (block, offset) [...], as 32-bit values [..., Hkv, D]."""
    cache = st[x + "_cache"]
    if st["case"]["op"] == "int4":
        return _values(cache[block, :, offset], st[x + "_params"][block, :, offset])
    if cache.dtype == torch.float8_e4m3fn:
        return cache.view(torch.uint8)[block, :, offset].view(cache.dtype).float() * st["kv_scale"]
    return cache[block, :, offset].float()


def _attend(q, k, v, seen, scale):
    """q [..., n, D], k and v [..., t, D], seen [..., n, t] -> softmax(scale q k') v, zeros where nothing is seen."""
    w = (q @ k.transpose(-1, -2) * scale).masked_fill(~seen, -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True).clamp_min(-1e30))
    return (w @ v) / w.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain_decode(st):
    c = st["case"]
    S, n, Hkv, D, G, bs, win, sinks = c["S"], c["k"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"], c["bs"], c["win"], c["sinks"]
    L = st["cl"].long()[:, None]
    if win:  # the first tokens, then those of the window of any new token
        first = (L - n).clamp_min(0) - win + 1
        at = torch.arange(min(win + n - 1, c["hi"]), device="cuda") + first.clamp_min(0)
        pos = torch.cat([torch.arange(sinks, device="cuda").expand(S, -1), torch.where(at < sinks, -1, at)], 1)
    else:
        pos = torch.arange(st["bt"].shape[1] * bs, device="cuda").expand(S, -1)
    live = (pos >= 0) & (pos < L)
    block = st["bt"].long().gather(1, torch.where(live, pos, 0) // bs).clamp_min(0)
    k, v = (_tokens(st, x, block, pos.clamp_min(0) % bs).transpose(1, 2) for x in "kv")
    q = st["q"].float().view(S, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, n * G, D)
    me = (L - n + torch.arange(n, device="cuda"))[..., None]  # position of each new token
    seen = live[:, None] & (pos[:, None] <= me)
    if win:
        seen &= (pos[:, None] < sinks) | (pos[:, None] > me - win)
    out = _attend(q, k, v, seen.repeat_interleave(G, 1)[:, None], st["scale"]).view(S, Hkv, n, G, D).permute(0, 2, 1, 3, 4)
    st["out"].copy_(out.reshape(st["out"].shape))


def _plain_prompt(st):
    c = st["case"]
    C, Hkv, D, G, bs, win, sinks = c["C"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"], c["bs"], c["win"], c["sinks"]
    for s, L in enumerate(_lengths(c)):
        for i in range(0, C, 512):  # pieces of the chunk, each with the tokens that its windows reach
            n = min(512, C - i)
            me = torch.arange(L - C + i, L - C + i + n, device="cuda")
            first = max(0, L - C + i - win + 1)
            pos = torch.cat([torch.arange(min(sinks, first), device="cuda"), torch.arange(first, max(first, L - C + i + n), device="cuda")])
            if len(pos) == 0:
                st["out"][s, i: i + n] = 0
                continue
            block = st["bt"][s].long()[pos // bs]
            k, v = (_tokens(st, x, block, pos % bs).transpose(0, 1) for x in "kv")
            q = st["q"][s, i: i + n].float().view(n, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, n * G, D)
            seen = (pos <= me[:, None]) & ((pos < sinks) | (pos > me[:, None] - win))
            out = _attend(q, k, v, seen.repeat_interleave(G, 0), st["scale"])
            st["out"][s, i: i + n] = out.view(Hkv, n, G, D).permute(1, 0, 2, 3).reshape(n, Hkv * G, D).to(st["out"].dtype)


PLAIN = {"int4io": _plain_int4io, "int4": _plain_decode, "window": _plain_decode, "prompt": _plain_prompt}


def run(state):
    op = state["case"]["op"]
    if own:
        _run_own(state)
    else:
        PLAIN[op](state)
    if op == "int4io":
        # every block written is read back: what its codes stand for
        return {x: state[x] for x in ("k_params", "v_params", "k16", "v16")}
    return {"out": state["out"]}


# ---- the definitions in 64 bits ---------------------------------------------


def _rows64(case, st, s, x, pos):
    """Rows of sequence s at positions pos, in 64 bits [t, Hkv, D]."""
    ids = st["bt"][s, pos // case["bs"]].long()
    off = pos % case["bs"]
    data = st[x + "_cache"].view(torch.uint8)[ids, :, off] if st[x + "_cache"].element_size() == 1 else st[x + "_cache"][ids, :, off]
    if case["op"] != "int4":
        if data.dtype == torch.uint8:
            return data.view(torch.float8_e4m3fn).float().double() * float(torch.tensor(st["kv_scale"]))
        return data.double()
    scale, low = (st[x + "_params"][ids, :, off][..., i].double().repeat_interleave(GROUP, -1) for i in (0, 1))
    res = torch.empty(low.shape, device="cuda", dtype=torch.float64)
    for d in range(8):  # channel d of every eight: its nibble's byte and half
        nibble = d // 2 + 4 * (d % 2)
        byte = data[..., nibble // 2:: 4]
        res[..., d:: 8] = (byte // 16 if nibble % 2 else byte % 16).double()
    return res * scale + low


def exact(case, seed):
    st = prepare(case, seed)
    op, bs, Hkv = case["op"], case["bs"], case["Hkv"]
    if op == "int4io":
        res = {}
        at = (st["slots"] // bs, slice(None), st["slots"] % bs)
        for x, row in (("k", "key"), ("v", "value")):
            pool = {"op": "int4", "bs": bs}
            flat = {"bt": st["ids"][None, :], x + "_cache": st[x + "_cache"], x + "_params": st[x + "_params"]}
            pos = torch.arange(case["nread"] * bs, device="cuda")
            now = _rows64(pool, flat, 0, x, pos).view(case["nread"], bs, Hkv, -1).transpose(1, 2).clone()
            # the rows written: the group's least value at most, in eight bits, and a fifteenth of the spread above it
            g = st[row].double().unflatten(-1, (-1, GROUP))
            least, most = g.amin(-1), g.amax(-1)
            step = torch.exp2(torch.floor(torch.log2(least.abs().clamp_min(1e-300))) - 7)
            low = torch.where(least == 0, 0.0, torch.floor(least / step) * step)
            scale = ((most - low) / 15).clamp_min(LEAST_SCALE)
            step = torch.exp2(torch.floor(torch.log2(scale)) - 7)
            scale = (scale / step).round() * step
            value = (((g - low[..., None]) / scale[..., None]).round().clamp(0, 15) * scale[..., None] + low[..., None]).flatten(-2)
            params = st[x + "_params"].double()
            params[at] = torch.stack([scale, low], -1)
            place = torch.full((int(st[x + "_cache"].shape[0]),), -1, device="cuda", dtype=torch.long)
            place[st["ids"]] = torch.arange(case["nread"], device="cuda")
            where = place[st["slots"] // bs]
            now[where[where >= 0], :, (st["slots"] % bs)[where >= 0]] = value[where >= 0]
            res.update({x + "_params": params, x + "16": now})
        return {x: res[x] for x in ("k_params", "v_params", "k16", "v16")}
    new = case["C"] if op == "prompt" else case["k"]
    G, D, win, sinks = case["Hq"] // Hkv, case["D"], case["win"], case["sinks"]
    out = torch.zeros((case["S"], new, case["Hq"], D), device="cuda", dtype=torch.float64)
    q = st["q"].double().view(out.shape)
    for s, L in enumerate(_lengths(case)):
        for i in range(0, new, 128):
            me = torch.arange(max(0, L - new + i), max(0, L - new + min(new, i + 128)), device="cuda")
            n = len(me)
            if n == 0:
                continue
            j = min(new, i + 128) - n  # the first of the piece that has a position
            first = max(0, int(me[0]) - win + 1) if win else 0
            pos = torch.cat([torch.arange(min(sinks, first), device="cuda"), torch.arange(first, int(me[-1]) + 1, device="cuda")])
            hidden = pos[None, :] > me[:, None]
            if win:
                hidden |= (pos[None, :] <= me[:, None] - win) & (pos[None, :] >= sinks)
            k, v = (_rows64(case, st, s, x, pos) for x in "kv")
            for h in range(Hkv):
                x = torch.einsum("ngd,td->gnt", q[s, j: j + n, h * G: (h + 1) * G], k[:, h]) * st["scale"]
                w = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
                out[s, j: j + n, h * G: (h + 1) * G] = torch.einsum("gnt,td->ngd", w, v[:, h])
    return {"out": out.view(st["out"].shape)}
