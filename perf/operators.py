"""The operators for several new tokens over an OTT cache, and their workloads.

Kinds of cases:

* ``rope``: rotary positions with one to four axes, applied to the queries and
  keys of a decode step or of a prompt chunk (``rope``);
* ``chunk``: attention of n new tokens per sequence over a filled cache and,
  causally, over one another (``OTTCache.chunk_attn``): chunks of long prompts,
  and the few tokens of a draft that is verified;
* ``window``: the decode step of one query per sequence that sees the last
  ``window`` tokens and the first ``sinks`` (``OTTCache.decode_attn_window``);
* ``prompt``: a prompt taken in chunks, each attended and then appended
  (``chunk_attn`` and ``OTTCache.append_chunk``), and one decode afterwards.

Where ``own`` is false the cache is kept as plain tensors (unpacked 2-bit codes,
their scales and zeros, the fp16 tokens, token indices) and everything is
elementary torch arithmetic in 32 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
OUTLIER_CHANNELS, OUTLIER_SCALE, LOW_NORM = 4, 15.0, 0.03


# ---------------------------------------------------------------- cases
def _rope(name, B, Hq, Hkv, n, d, sect, base=10000.0, interleaved=False, restart=False, far=0):
    s = list(sect) + [0] * (4 - len(sect))
    return dict(name=name, kind="rope", B=B, Hq=Hq, Hkv=Hkv, n=n, d=d, axes=len(sect), s0=s[0], s1=s[1], s2=s[2],
                s3=s[3], base=base, interleaved=interleaved, restart=restart, far=far)


def _cache(name, kind, B, Hq, Hkv, d, T, n, G=128, R=32, P=32, rate=0.005, window=0, sinks=0, T_lo=0, n_lo=0,
           paged=False, chunk=0, lens_seed=0):
    return dict(name=name, kind=kind, B=B, Hq=Hq, Hkv=Hkv, d=d, T=T, n=n, G=G, R=R, P=P, rate=rate, window=window,
                sinks=sinks, T_lo=T_lo, n_lo=n_lo, paged=paged, chunk=chunk, lens_seed=lens_seed)


def listed():
    return [
        # the rotation of one decode step of the 32-sequence batch: launch latency
        _rope("rope_step", 32, 32, 32, 1, 128, (16, 24, 24), far=4096),
        # a long video prompt (time, height, width) with grouped kv heads
        _rope("rope_video", 1, 32, 8, 32767, 128, (16, 24, 24), base=1000000.0),
        # image patches, two axes with a ladder of frequencies each, adjacent pairs, odd token count, half of the
        # channels left alone
        _rope("rope_image", 3, 12, 12, 1021, 64, (8, 8), interleaved=True, restart=True, far=100000),
        # four draft tokens verified over the 32-sequence batch's 4K contexts
        _cache("verify_b32", "chunk", 32, 32, 32, 128, 4096, 4),
        # the next 512 tokens of four 32K prompts (grouped kv heads, larger groups)
        _cache("chunk_32k", "chunk", 4, 32, 8, 128, 32768, 512, G=256, R=64),
        # a long document's chunk over 131K tokens
        _cache("chunk_131k", "chunk", 1, 32, 8, 128, 131072, 2048, P=64, rate=0.002),
        # a serving batch of mixed lengths from a paged pool: long chunks, short ones and sequences without new tokens
        _cache("chunk_paged", "chunk", 16, 32, 32, 128, 7168, 257, T_lo=1024, n_lo=0, paged=True, lens_seed=5),
        # a chunk that sees a window of 4096 tokens and four sinks
        _cache("chunk_window", "chunk", 4, 32, 8, 128, 32768, 512, window=4096, sinks=4),
        # decode steps with a window: the 32-sequence batch, and one long sequence (latency)
        _cache("window_b32", "window", 32, 32, 32, 128, 4096, 1, window=1024, sinks=4),
        _cache("window_131k", "window", 1, 32, 8, 128, 131072, 1, P=64, rate=0.002, window=4096, sinks=16),
        # a prompt taken in chunks of 1024, and a ragged batch of short ones with 64-wide heads
        _cache("prompt_8k", "prompt", 1, 32, 8, 128, 8192, 0, chunk=1024),
        _cache("prompt_ragged", "prompt", 5, 14, 2, 64, 1500, 0, T_lo=77, chunk=333, lens_seed=9),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    while True:
        c = _draw(rng)
        w = work(c)
        if w["flops"] <= 2e12 and w["bytes"] <= 4e8:
            return c


def _draw(rng):
    kind = rng.choice(["rope", "chunk", "chunk", "chunk", "window", "prompt"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 32])
    g = rng.choice([1, 1, 2, 3, 4, 4, 5, 7, 8]) if Hkv < 32 else 1
    if kind == "rope":
        B = _logint(rng, 1, 32)
        n = _logint(rng, 1, 32768)
        while B * n * (g + 1) * Hkv * d > 32767 * 40 * 128:
            B, n = (B + 1) // 2, (n + 1) // 2
        axes = rng.randint(1, 4)
        half = d // 2 if rng.random() < 0.7 else d // 4
        cuts = sorted(rng.sample(range(1, half), axes - 1))
        sect = [b - a for a, b in zip([0] + cuts, cuts + [half])]
        c = _rope(None, B, Hkv * g, Hkv, n, d, sect, base=rng.choice([10000.0, 500000.0, 1000000.0]),
                  interleaved=rng.random() < 0.5, restart=rng.random() < 0.5, far=rng.choice([0, 4096, 1000000]))
    else:
        B = _logint(rng, 1, 32)
        T = _logint(rng, 1, 65536)
        while B * T * Hkv > 32 * 4096 * 16:
            B, T = (B + 1) // 2, max(1, T * 3 // 4)
        n = _logint(rng, 1, 2048)
        while B * Hkv * g * n * (T + n) > 4 * 32 * 512 * 32768:
            n = (n + 1) // 2
        G, R = rng.choice([(128, 32), (128, 32), (256, 64), (64, 0), (48, 17)])
        P = rng.choice([0, 17, 32, 32, 64])
        window = 0 if kind == "chunk" and rng.random() < 0.5 else _logint(rng, 1, 8192)
        sinks = rng.choice([0, 1, 4, 4, 16, 130]) if window else 0
        ragged = rng.random() < 0.5
        c = _cache(None, kind, B, Hkv * g, Hkv, d, T, n, G=G, R=R, P=P, window=window, sinks=sinks,
                   T_lo=max(1, T // rng.randint(2, 9)) if ragged else 0, n_lo=rng.choice([0, 1, n]) if ragged else n,
                   paged=rng.random() < 0.5, lens_seed=rng.randint(0, 1 << 30))
        if kind == "window":
            c["n"] = c["n_lo"] = 1
        if kind == "prompt":
            T = min(T, 4096)
            c["T"], c["n"], c["n_lo"] = T, 0, 0
            c["T_lo"] = max(1, T // rng.randint(2, 9)) if ragged else 0
            c["chunk"] = max(T // 24 + 1, _logint(rng, 16, 1024))
    del c["name"]
    return c


def _lens(c):
    """(tokens in the cache, new tokens) of every sequence."""
    r = random.Random(c["lens_seed"])
    B, T, n = c["B"], c["T"], c["n"]
    Ts = [r.randint(c["T_lo"], T) for _ in range(B)] if c["T_lo"] else [T] * B
    ns = [r.randint(c["n_lo"], n) if c["T_lo"] else n for _ in range(B)]
    if c["T_lo"]:
        Ts[r.randrange(B)] = T
        ns[r.randrange(B)] = n
    return Ts, ns


def _nf(c, T):
    return (T - c["R"]) // c["G"] if T >= c["G"] + c["R"] else 0


def _seen(T, n, window, sinks, decode):
    """Keys that the queries of one sequence see, and the cache tokens that any of them sees."""
    pos0 = T - 1 if decode else T
    if window <= 0:
        return sum(pos0 + 1 + i for i in range(n)) if n < 64 else n * (pos0 + 1) + n * (n - 1) // 2, T if n else 0
    keys = 0
    for i in range(n):
        p = pos0 + i
        lo = max(0, p - window + 1)
        keys += p + 1 - lo + min(sinks, lo)
    lo = max(0, pos0 - window + 1)
    return keys, max(0, T - lo) + min(sinks, lo, T) if n else 0


def _store_bytes(c, T, seen):
    """Bytes of the stores that hold `seen` of a unit's T tokens."""
    d, G, P = c["d"], c["G"], c["P"]
    nf = _nf(c, T)
    full = min(seen, T - nf * G + min(P, nf * G))
    quant = max(0, seen - full)
    return full * 4 * d + quant * (d // 2 + d // 32 * 4) + -(-quant // G) * 4 * d


def work(case):
    c = case
    if c["kind"] == "rope":
        e = c["B"] * (c["Hq"] + c["Hkv"]) * c["n"] * c["d"]
        return {"bytes": 4 * e + 4 * c["axes"] * c["B"] * c["n"], "flops": 3 * e}
    Ts, ns = _lens(c)
    by = fl = 0
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    for T, n in zip(Ts, ns):
        if c["kind"] == "prompt":
            for a in range(0, T, c["chunk"]):
                m = min(c["chunk"], T - a)
                keys, seen = _seen(a, m, c["window"], c["sinks"], False)
                fl += 4 * d * Hq * keys
                by += Hkv * _store_bytes(c, a, seen) + 4 * d * m * (Hq + Hkv)
            # the cache as it is written, and the decode over it
            by += Hkv * _store_bytes(c, T, T) * 2 + 4 * d * Hq
            fl += 4 * d * Hq * T
        else:
            decode = c["kind"] == "window"
            keys, seen = _seen(T, n, c["window"], c["sinks"], decode)
            fl += 4 * d * Hq * keys
            by += Hkv * _store_bytes(c, T, seen) + 4 * d * n * Hq + (0 if decode else 4 * d * n * Hkv)
    return {"bytes": by, "flops": fl}


# ---------------------------------------------------------------- inputs
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _keys(g, shape, rate):
    """Keys with four large channels per kv head (dim 1) and a few tokens of small norm."""
    Hkv, d = shape[1], shape[-1]
    k = torch.randn(shape, generator=g, device=DEV)
    sc = torch.ones(Hkv, d, device=DEV)
    ch = torch.rand(Hkv, d, generator=g, device=DEV).argsort(1)[:, :OUTLIER_CHANNELS]
    sc.scatter_(1, ch, OUTLIER_SCALE)
    k.mul_(sc.view(1, Hkv, *([1] * (len(shape) - 3)), d))
    low = torch.rand(shape[:-1], generator=g, device=DEV) < rate
    return torch.where(low.unsqueeze(-1), k * LOW_NORM, k).half()


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).half()


def _inputs(c, seed):
    """Everything that is drawn, the same for both sides."""
    g = _gen(seed, 17)
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    if c["kind"] == "rope":
        n, axes = c["n"], c["axes"]
        q, k = _rand(g, B, Hq, n, d), _rand(g, B, Hkv, n, d)
        # a raster over the axes (time slowest), from a random start
        ext = max(1, round(n ** (1.0 / axes)))
        t = torch.arange(n, device=DEV)
        pos = []
        for a in range(axes):
            step = ext ** (axes - 1 - a)
            v = t // step if a == 0 else (t // step) % ext
            start = torch.randint(0, c["far"] + 1, (B, 1), generator=g, device=DEV)
            pos.append(v.view(1, n) + start)
        return dict(q=q, k=k, pos=torch.stack(pos).int().contiguous())
    Ts, ns = _lens(c)
    T = max(Ts)
    x = dict(Ts=Ts, ns=ns)
    if c["kind"] == "prompt":
        n = c["chunk"]
        K, V, Q = _keys(g, (B, Hkv, T, d), c["rate"]), _rand(g, B, Hkv, T, d), _rand(g, B, Hq, T, d)
        cut = range(0, T, n)
        x.update(K=[K[:, :, a:a + n].contiguous() for a in cut], V=[V[:, :, a:a + n].contiguous() for a in cut],
                 Q=[Q[:, :, a:a + n].contiguous() for a in cut],
                 lens=[[max(0, min(n, t - a)) for t in Ts] for a in cut], q=_rand(g, B, Hq, d))
        return x
    x.update(K=_keys(g, (B, Hkv, T, d), c["rate"]), V=_rand(g, B, Hkv, T, d))
    if c["kind"] == "window":
        x["q"] = _rand(g, B, Hq, d)
    else:
        n = c["n"]
        x.update(q=_rand(g, B, Hq, n, d), k=_keys(g, (B, Hkv, n, d), c["rate"]), v=_rand(g, B, Hkv, n, d))
    return x


def prepare(case, seed):
    c = case
    x = _inputs(c, seed)
    st = dict(c=c, **x)
    if c["kind"] == "rope":
        return st
    B, Hq = c["B"], c["Hq"]
    if c["kind"] == "prompt":
        # rows behind a sequence's last new token stay as they are: zero
        st["outs"] = [torch.zeros_like(q) for q in st["Q"]]
    elif c["kind"] == "chunk":
        st["out"] = torch.zeros_like(st["q"])
        st["lens"] = x["ns"] if c["T_lo"] else None
    if not own:
        if c["kind"] != "prompt":
            st["stores"] = _quantized_batch(c, st.pop("K"), st.pop("V"), x["Ts"])
        return st
    import bit_kv_cache_ott_gb300 as ott
    room = max(x["Ts"]) + c["n"]
    kw = dict(ragged=True)
    if c["paged"]:
        kw["pool_blocks"] = max(1, sum(_nf(c, t + c["n"]) for t in x["Ts"]) * c["Hkv"])
    elif not c["T_lo"] and c["kind"] != "prompt":
        kw = {}
    st["cache"] = cache = ott.OTTCache(B, Hq, c["Hkv"], c["d"], c["G"], c["R"], c["P"], max_tokens=room, **kw)
    if c["kind"] != "prompt":
        K, V = st.pop("K"), st.pop("V")
        if c["T_lo"]:
            cache.prefill_lens(K, V, x["Ts"])
        else:
            cache.prefill(K, V)
        torch.cuda.synchronize()   # K and V are dropped here
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["c"]
    return {"rope": _run_rope, "chunk": _run_chunk, "window": _run_window, "prompt": _run_prompt}[c["kind"]](c, state)


def _sections(c):
    return [c["s0"], c["s1"], c["s2"], c["s3"]][:c["axes"]]


def _run_rope(c, s):
    if own:
        import bit_kv_cache_ott_gb300 as ott
        return ott.rope(s["q"], s["k"], s["pos"], _sections(c), base=c["base"], interleaved=c["interleaved"],
                        restart=c["restart"])
    sect = _sections(c)
    half = sum(sect)
    ang = []
    for a, m in enumerate(sect):
        i = torch.arange(m, device=DEV, dtype=torch.float64)
        e = i / m if c["restart"] else (i + sum(sect[:a])) / half
        # angles of far positions: 64 bits
        ang.append(s["pos"][a].double().unsqueeze(-1) * torch.exp(-math.log(c["base"]) * e))
    ang = torch.cat(ang, -1).unsqueeze(1)              # [B][1][n][half]
    co, si = torch.cos(ang).float(), torch.sin(ang).float()
    res = []
    for x in (s["q"], s["k"]):
        f = x.float()
        y = f.clone()
        i0, i1 = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c["interleaved"] else (slice(0, half),
                                                                                         slice(half, 2 * half))
        y[..., i0] = f[..., i0] * co - f[..., i1] * si
        y[..., i1] = f[..., i0] * si + f[..., i1] * co
        res.append(y.half())
    return tuple(res)


def _run_chunk(c, s):
    if own:
        return s["cache"].chunk_attn(s["q"], s["k"], s["v"], lens=s["lens"], window=c["window"], sinks=c["sinks"],
                                     out=s["out"])
    out = torch.zeros_like(s["q"])
    for b in range(c["B"]):
        n = s["ns"][b]
        if n:
            out[b, :, :n] = _attend(c, s["q"][b, :, :n], s["stores"][b], s["Ts"][b], s["k"][b, :, :n], s["v"][b, :, :n])
    return out


def _run_window(c, s):
    if own:
        return s["cache"].decode_attn_window(s["q"], c["window"], c["sinks"])
    out = torch.empty_like(s["q"])
    for b in range(c["B"]):
        out[b] = _attend(c, s["q"][b].unsqueeze(1), s["stores"][b], s["Ts"][b] - 1).squeeze(1)
    return out


def _run_prompt(c, s):
    if own:
        cache = s["cache"]
        for b in range(c["B"]):
            if cache.seq_counts(b)[0]:
                cache.release_seq(b)
        for q, k, v, lens, out in zip(s["Q"], s["K"], s["V"], s["lens"], s["outs"]):
            cache.chunk_attn(q, k, v, lens=lens, window=c["window"], sinks=c["sinks"], out=out)
            cache.append_chunk(k, v, lens=lens)
        return s["outs"], cache.decode_attn(s["q"])
    outs = [torch.zeros_like(q) for q in s["Q"]]
    dec = torch.empty_like(s["q"])
    for b, T in enumerate(s["Ts"]):
        K = torch.cat([k[b] for k in s["K"]], 1)[:, :T]
        V = torch.cat([v[b] for v in s["V"]], 1)[:, :T]
        hist = _history(c, K, V)
        a = 0
        for i, out in enumerate(outs):
            n = s["lens"][i][b]
            if n:
                out[b, :, :n] = _attend(c, s["Q"][i][b, :, :n], _stores_at(c, K, V, hist, a), a, s["K"][i][b, :, :n],
                                        s["V"][i][b, :, :n])
                a += n
        full = dict(c, window=0, sinks=0)
        dec[b] = _attend(full, s["q"][b].unsqueeze(1), _stores_at(c, K, V, hist, T), T - 1).squeeze(1)
    return outs, dec


# ---------------------------------------------------------------- the plain cache
# A sequence's stores: "parts", a list of (token indices [Hkv][m], -1 for none; then either fp16 keys and values
# [Hkv][m][d], or codes with scales and zeros).
def _key_norms(K):
    """Squared norms, 32 bits, summed in channel order: [U][T][d] -> [U][T]."""
    Kt = K.permute(2, 0, 1).float().contiguous()
    acc = torch.zeros_like(Kt[0])
    for ch in range(Kt.shape[0]):
        acc = acc + Kt[ch] * Kt[ch]
    return acc


def _history(c, K, V, nf=None):
    """Every flush of units with the same length, in turn: the quantized blocks and the pool after each."""
    G, P, U, T, d = c["G"], c["P"], K.shape[0], K.shape[1], K.shape[2]
    nf = _nf(c, T) if nf is None else nf
    norms = _key_norms(K[:, :nf * G]) if nf else None
    pool = torch.empty(U, 0, dtype=torch.int64, device=DEV)
    pools, rests = [pool], []
    for j in range(nf):
        cand = torch.cat([pool, torch.arange(j * G, (j + 1) * G, device=DEV).expand(U, G)], 1)   # ascending
        order = norms.gather(1, cand).argsort(dim=1, stable=True)   # ties to the lower index
        pool = cand.gather(1, order[:, :P]).sort(1).values
        rest = cand.gather(1, order[:, P:]).sort(1).values
        rests.append(torch.nn.functional.pad(rest, (0, G - rest.shape[1]), value=-1))
        pools.append(pool)
    blocks = None
    if nf:
        idx = torch.stack(rests, 1)                              # [U][nf][G]
        at = idx.clamp(min=0).reshape(U, nf * G, 1).expand(U, nf * G, d)
        ok = (idx >= 0).unsqueeze(-1)
        Kb = K.gather(1, at).view(U, nf, G, d).float()
        kc, ks, kz = _two_bits(Kb, ok, 2)
        del Kb
        Vb = V.gather(1, at).view(U, nf, G, d // 32, 32).float()
        vc, vs, vz = _two_bits(Vb, ok.unsqueeze(-1), 4)
        blocks = dict(idx=idx, kc=kc, ks=ks, kz=kz, vc=vc, vs=vs, vz=vz)
    return dict(pools=pools, blocks=blocks)


def _two_bits(x, ok, dim):
    """Asymmetric 2-bit codes along `dim` over the valid entries: (codes, scale fp16, zero fp16)."""
    inf = float("inf")
    mn = x.masked_fill(~ok, inf).amin(dim, keepdim=True)
    mx = x.masked_fill(~ok, -inf).amax(dim, keepdim=True)
    none = mn > mx                                               # an empty block
    mn, mx = mn.masked_fill(none, 0.0), mx.masked_fill(none, 0.0)
    s = ((mx - mn) / torch.full_like(mx, 3.0)).half()            # tensor by tensor: an IEEE division
    sf = s.float()
    code = ((x - mn) / torch.where(sf == 0, torch.ones_like(sf), sf)).round().clamp(0, 3)
    code = torch.where((sf == 0) | ~ok, torch.zeros_like(code), code)
    return code.to(torch.uint8), s, mn.half()


def _stores_at(c, K, V, hist, T):
    """The stores of [Hkv] units after T tokens, from their history."""
    nf = _nf(c, T)
    U = K.shape[0]
    pool = hist["pools"][nf]
    tail = torch.arange(nf * c["G"], T, device=DEV).expand(U, -1)
    idx = torch.cat([tail, pool], 1)
    at = idx.unsqueeze(-1).expand(-1, -1, K.shape[2])
    st = dict(fidx=idx, fk=K.gather(1, at), fv=V.gather(1, at))
    if nf:
        st["blocks"] = {k: v[:, :nf] for k, v in hist["blocks"].items()}
    return st


def _quantized_batch(c, K, V, Ts):
    """The plain cache of every sequence after its Ts[b] tokens."""
    B, Hkv, d = K.shape[0], K.shape[1], K.shape[3]
    if len(set(Ts)) > 1:
        return [_stores_at(c, K[b, :, :T], V[b, :, :T], _history(c, K[b, :, :T], V[b, :, :T]), T)
                for b, T in enumerate(Ts)]
    Ku, Vu = K.view(B * Hkv, -1, d), V.view(B * Hkv, -1, d)
    st = _stores_at(c, Ku, Vu, _history(c, Ku, Vu), Ts[0])

    def part(x, b):
        return {k: part(v, b) for k, v in x.items()} if isinstance(x, dict) else x[b * Hkv:(b + 1) * Hkv]

    return [part(st, b) for b in range(B)]


def _attend(c, q, st, pos0, k=None, v=None):
    """q [Hq][n][d] at positions pos0 .. pos0+n-1 over a sequence's stores and its new tokens k, v [Hkv][n][d]."""
    Hq, n, d = q.shape
    Hkv = c["Hkv"]
    g = Hq // Hkv
    pos = (pos0 + torch.arange(n, device=DEV)).repeat(g)
    out = torch.empty(Hkv, g * n, d, device=DEV)
    qf = q.reshape(Hkv, g * n, d)
    for h in range(Hkv):
        Ks, Vs, ids = [st["fk"][h].float()], [st["fv"][h].float()], [st["fidx"][h]]
        bl = st.get("blocks")
        if bl is not None:
            Ks.append((bl["kz"][h].float() + bl["ks"][h].float() * bl["kc"][h].float()).view(-1, d))
            Vs.append((bl["vz"][h].float() + bl["vs"][h].float() * bl["vc"][h].float()).view(-1, d))
            ids.append(bl["idx"][h].reshape(-1))
        if k is not None:
            Ks.append(k[h].float())
            Vs.append(v[h].float())
            ids.append(pos0 + torch.arange(n, device=DEV))
        Kh, Vh, idx = torch.cat(Ks), torch.cat(Vs), torch.cat(ids)
        step = max(1, (1 << 28) // Kh.shape[0])
        for r in range(0, g * n, step):
            s = qf[h, r:r + step].float() @ Kh.t() / math.sqrt(d)
            p = pos[r:r + step, None]
            hide = (idx < 0) | (idx > p)
            if c["window"]:
                hide = hide | ((idx <= p - c["window"]) & (idx >= c["sinks"]))
            s.masked_fill_(hide, float("-inf"))
            w = torch.exp(s - s.amax(1, keepdim=True))
            out[h, r:r + step] = (w @ Vh) / w.sum(1, keepdim=True)
    return out.half().view(Hq, n, d)


# ---------------------------------------------------------------- from the definitions, in 64 bits
def exact(case, seed):
    """What ``run`` returns, in 64 bits. The stored codes are part of the operators' definition (32-bit norms and
    divisions), so they are found the same way here, by a selection of its own."""
    c = case
    x = _inputs(c, seed)
    if c["kind"] == "rope":
        sect, half = _sections(c), sum(_sections(c))
        owner = [(a, j) for a, m in enumerate(sect) for j in range(m)]
        res = []
        for t in (x["q"], x["k"]):
            y = t.double().clone()
            for i, (a, j) in enumerate(owner):
                e = j / sect[a] if c["restart"] else i / half
                th = (x["pos"][a].double() * c["base"] ** -e).unsqueeze(1)
                l, r = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
                z = torch.complex(t[..., l].double(), t[..., r].double()) * torch.complex(th.cos(), th.sin())
                y[..., l], y[..., r] = z.real, z.imag
            res.append(y)
        return tuple(res)
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    g = Hq // Hkv
    if c["kind"] == "prompt":
        K, V, Q = (torch.cat(x[k], 2) for k in ("K", "V", "Q"))
        full = torch.zeros(B, Hq, K.shape[2], d, dtype=torch.float64, device=DEV)
        dec = torch.empty(B, Hq, d, dtype=torch.float64, device=DEV)
        for b, T in enumerate(x["Ts"]):
            for h in range(Hkv):
                hs = slice(h * g, (h + 1) * g)
                for a in range(0, T, c["chunk"]):
                    e = min(T, a + c["chunk"])
                    k64, v64, ids = _exact_unit(c, K[b, h, :a], V[b, h, :a])
                    full[b, hs, a:e] = _exact_rows(Q[b, hs, a:e], k64, v64, ids, a, c, K[b, h, a:e], V[b, h, a:e])
                k64, v64, ids = _exact_unit(c, K[b, h, :T], V[b, h, :T])
                dec[b, hs] = _exact_rows(x["q"][b, hs].unsqueeze(1), k64, v64, ids, T - 1, dict(c, window=0)).squeeze(1)
        return [full[:, :, a:a + c["chunk"]].contiguous() for a in range(0, full.shape[2], c["chunk"])], dec
    decode = c["kind"] == "window"
    out = torch.zeros(x["q"].shape, dtype=torch.float64, device=DEV)
    for b, (T, n) in enumerate(zip(x["Ts"], x["ns"])):
        units = _exact_units(c, x["K"][b, :, :T], x["V"][b, :, :T])
        for h in range(Hkv):
            hs = slice(h * g, (h + 1) * g)
            k64, v64, ids = next(units)
            if decode:
                out[b, hs] = _exact_rows(x["q"][b, hs].unsqueeze(1), k64, v64, ids, T - 1, c).squeeze(1)
            elif n:
                out[b, hs, :n] = _exact_rows(x["q"][b, hs, :n], k64, v64, ids, T, c, x["k"][b, h, :n], x["v"][b, h, :n])
    return out


def _exact_unit(c, k, v):
    return next(_exact_units(c, k.unsqueeze(0), v.unsqueeze(0)))


def _exact_units(c, K, V):
    """For each unit of K, V [U][T][d]: what its cache stands for, as (keys, values, token indices), one token a row."""
    G, R, P = c["G"], c["R"], c["P"]
    U, T, d = K.shape
    done = 0
    while T - done * G >= G + R:
        done += 1
    # norms as ordered integers with the token index below: one number decides, ties included
    score = torch.zeros(U, T, device=DEV)
    for ch in range(d):
        col = K[:, :, ch].float()
        score += col * col
    rank = (score.view(torch.int32).long() << 32) | torch.arange(T, device=DEV)
    held = torch.empty(U, 0, dtype=torch.int64, device=DEV)
    member = torch.full((U, T), -1, dtype=torch.int64, device=DEV)   # the block that holds a token, -1: fp16
    for j in range(done):
        now = torch.cat([held, rank[:, j * G:(j + 1) * G]], 1)
        keep = min(P, now.shape[1])
        inner = now.kthvalue(keep, 1, keepdim=True).values if keep else torch.full((U, 1), -1, device=DEV)
        stay = now <= inner
        gone = now.masked_select(~stay).view(U, -1) & 0xFFFFFFFF
        member.scatter_(1, gone, j)
        held = now.masked_select(stay).view(U, -1)
    for u in range(U):
        k64, v64 = K[u].double(), V[u].double()
        if done:
            m = member[u]
            tok = (m >= 0).nonzero().squeeze(1)
            blk = m[tok]
            kf = K[u][tok].float()
            lo = torch.full((done, d), math.inf, device=DEV).scatter_reduce(0, blk[:, None].expand(-1, d), kf, "amin")
            hi = torch.full((done, d), -math.inf, device=DEV).scatter_reduce(0, blk[:, None].expand(-1, d), kf, "amax")
            k64[tok] = _exact_code(kf, lo[blk], hi[blk])
            vf = V[u][tok].float().view(-1, d // 32, 32)
            lo, hi = vf.amin(2, keepdim=True).expand_as(vf), vf.amax(2, keepdim=True).expand_as(vf)
            v64[tok] = _exact_code(vf, lo, hi).view(-1, d)
        yield k64, v64, torch.arange(T, device=DEV)


def _exact_code(x, lo, hi):
    s = torch.div(hi - lo, torch.tensor(3.0, device=DEV).expand_as(hi).contiguous()).half().float()
    r = torch.div(x - lo, s).round()
    r = torch.where(s > 0, r.clamp(0, 3), torch.zeros_like(r))
    return lo.double() + s.double() * r.double()


def _exact_rows(q, k, v, ids, pos0, c, k_new=None, v_new=None):
    """q [g][n][d] of one kv head."""
    g, n, d = q.shape
    if k_new is not None:
        k, v = torch.cat([k, k_new.double()]), torch.cat([v, v_new.double()])
        ids = torch.cat([ids, pos0 + torch.arange(n, device=DEV)])
    out = torch.empty(g, n, d, dtype=torch.float64, device=DEV)
    step = max(1, (1 << 27) // max(1, k.shape[0]))
    for i in range(0, n, step):
        p = pos0 + torch.arange(i, min(n, i + step), device=DEV)[:, None]
        see = ids <= p
        if c["window"]:
            see = see & ((p - ids < c["window"]) | (ids < c["sinks"]))
        for h in range(g):
            logit = (q[h, i:i + step].double() @ k.t()) * d ** -0.5
            logit = torch.where(see, logit, torch.full_like(logit, -math.inf))
            out[h, i:i + step] = torch.softmax(logit, 1) @ v
    return out
