"""The operators of a cache held in 8 bits, and their workloads.

``ByteCache`` keeps the keys and values of complete blocks of G tokens as 8-bit
codes (int8 or e4m3) with one scale for the keys and one for the values of each
block and kv head; the tokens of the block that is still open stay fp16.

Kinds of cases:

* ``store``: prompts written in chunks (``append_chunk``) and read back whole
  (``read``);
* ``read``: a range of tokens of every sequence of a filled cache, read back;
* ``steps``: a short conversation: a prompt, then tokens one by one, each
  appended and attended (``append``, ``decode_attn``), and the cache read back;
* ``decode``: one query per sequence over a filled cache (``decode_attn``);
* ``chunk``: n new tokens per sequence over a filled cache and, causally, one
  another (``chunk_attn``): prompt chunks and drafts to verify;
* ``sparse``: the same, or one query per sequence where ``n`` is 0, over the
  ``topk`` blocks that a bound selects for each query (``chunk_attn_topk``,
  ``decode_attn_topk``).

Where ``own`` is false the cache is kept as plain tensors (codes, scales, the
fp16 tokens, the blocks' channel ranges) and everything is elementary torch
arithmetic in 32 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
OUTLIER_CHANNELS, OUTLIER_SCALE, LOW_NORM = 4, 15.0, 0.03


# ---------------------------------------------------------------- cases
def _case(name, kind, B, Hq, Hkv, d, T, n=0, G=64, fmt="int8", T_lo=0, n_lo=0, paged=False, chunk=0, start=0, topk=0,
          lens_seed=0):
    return dict(name=name, kind=kind, B=B, Hq=Hq, Hkv=Hkv, d=d, T=T, n=n, G=G, fmt=fmt, T_lo=T_lo, n_lo=n_lo,
                paged=paged, chunk=chunk, start=start, topk=topk, lens_seed=lens_seed)


def listed():
    return [
        # the prompts of the 32-sequence batch, written and read back
        _case("store_b32", "store", 32, 32, 32, 128, 4096, chunk=4096),
        # ragged prompts taken in chunks, 64-wide heads, small blocks
        _case("store_ragged", "store", 5, 14, 2, 64, 1500, G=32, fmt="e4m3", T_lo=77, chunk=333, lens_seed=9),
        # the last thousand tokens of four long contexts, handed to another consumer
        _case("read_tail", "read", 4, 32, 8, 128, 32768, n=1021, start=31747),
        # a short conversation: launch latency
        _case("steps_short", "steps", 3, 14, 2, 64, 61, n=8, G=32, fmt="e4m3"),
        # decode steps: the 32-sequence batch, one long sequence, a serving batch of mixed lengths from a paged pool
        _case("decode_b32", "decode", 32, 32, 32, 128, 4096),
        _case("decode_131k", "decode", 1, 32, 8, 128, 131072, fmt="e4m3"),
        _case("decode_paged", "decode", 32, 32, 8, 128, 7168, G=128, T_lo=1024, paged=True, lens_seed=5),
        # four draft tokens verified over the 32-sequence batch's 4K contexts
        _case("verify_b32", "chunk", 32, 32, 32, 128, 4096, n=4, fmt="e4m3"),
        # the next 512 tokens of four 32K prompts (grouped kv heads, larger blocks)
        _case("chunk_32k", "chunk", 4, 32, 8, 128, 32768, n=512, G=128),
        # a long document's chunk over 131K tokens
        _case("chunk_131k", "chunk", 1, 32, 8, 128, 131072, n=2048, fmt="e4m3"),
        # one query over an eighth of the blocks of a long context
        _case("sparse_131k", "sparse", 1, 32, 8, 128, 131071, topk=256),
        # drafts of mixed lengths, seven query heads to a kv head, each token with blocks of its own
        _case("sparse_draft", "sparse", 8, 28, 4, 128, 16384, n=5, G=32, fmt="e4m3", T_lo=3001, n_lo=1, topk=40,
              lens_seed=3),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    while True:
        c = _draw(rng)
        w = work(c)
        if w["flops"] <= 4.4e12 and w["bytes"] <= 5e9:
            return c


def _draw(rng):
    kind = rng.choice(["store", "read", "steps", "decode", "decode", "chunk", "chunk", "sparse", "sparse"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 32])
    g = rng.choice([1, 1, 2, 3, 4, 4, 5, 7, 8, 16]) if Hkv < 32 else 1
    B = _logint(rng, 1, 32)
    T = _logint(rng, 1, 131072)
    while B * T * Hkv > 32 * 4096 * 32:
        B, T = (B + 1) // 2, max(1, T * 3 // 4)
    ragged = rng.random() < 0.5
    c = _case(None, kind, B, Hkv * g, Hkv, d, T, G=rng.choice([32, 64, 64, 128]), fmt=rng.choice(["int8", "e4m3"]),
              T_lo=max(1, T // rng.randint(2, 9)) if ragged else 0, paged=rng.random() < 0.5,
              lens_seed=rng.randint(0, 1 << 30))
    if kind == "store":
        c["chunk"] = max(T // 24 + 1, _logint(rng, 16, 4096))
    elif kind == "read":
        c["start"] = rng.randrange(T)
        c["n"] = rng.randint(1, T - c["start"])
    elif kind == "steps":
        c["T"] = T = min(T, 4096)
        c["T_lo"] = min(c["T_lo"], T)
        c["n"] = rng.randint(2, 16)
    elif kind == "chunk":
        n = _logint(rng, 1, 2048)
        while B * Hkv * g * n * (T + n) > 2048 * 32 * 131072:
            n = (n + 1) // 2
        c["n"], c["n_lo"] = n, rng.choice([0, 1, n]) if ragged else n
    elif kind == "sparse":
        c["n"] = rng.choice([0, 0, 1, 2, 3, 5, 8])
        c["n_lo"] = rng.choice([0, 1, c["n"]]) if ragged else c["n"]
        c["topk"] = _logint(rng, 1, max(2, T // c["G"]))
    del c["name"]
    return c


def _lens(c):
    """(tokens in the cache, new tokens) of every sequence."""
    r = random.Random(c["lens_seed"])
    B, T, n = c["B"], c["T"], c["n"]
    Ts = [r.randint(c["T_lo"], T) for _ in range(B)] if c["T_lo"] else [T] * B
    ns = [r.randint(min(c["n_lo"], n), n) if c["T_lo"] else n for _ in range(B)]
    if c["T_lo"]:
        Ts[r.randrange(B)] = T
        ns[r.randrange(B)] = n
    return Ts, ns


def _held(c, T):
    """Bytes of a unit's T tokens as the cache holds them (channel ranges apart)."""
    nb = T // c["G"]
    return nb * (2 * c["G"] * c["d"] + 8) + (T - nb * c["G"]) * 4 * c["d"]


def work(case):
    c = case
    kind, B, Hq, Hkv, d, G = c["kind"], c["B"], c["Hq"], c["Hkv"], c["d"], c["G"]
    by = fl = 0
    for T, n in zip(*_lens(c)):
        if kind == "store":
            # read, held (with the blocks' channel ranges), read again, given out
            by += Hkv * (4 * d * T + 2 * _held(c, T) + T // G * 4 * d + 4 * d * T)
            fl += Hkv * 6 * d * T
        elif kind == "read":
            m = max(0, min(T, c["start"] + c["n"]) - c["start"])
            by += Hkv * (_held(c, T) * m // T + 4 * d * m)
            fl += Hkv * 2 * d * m
        elif kind == "steps":
            N = c["n"]
            by += Hkv * (4 * d * (T + N) + 3 * _held(c, T + N) + 4 * d * (T + N))
            for i in range(1, N + 1):
                by += Hkv * _held(c, T + i) + 4 * d * Hq
                fl += 4 * d * Hq * (T + i)
        elif kind == "sparse":
            N, nb = max(n, 1 if c["n"] == 0 else 0), T // G
            some = min(nb, c["topk"])
            open_ = T - nb * G
            if N:
                by += Hkv * (nb * 4 * d + min(nb, some * N) * (2 * G * d + 8) + open_ * 4 * d) + 4 * d * Hq * N
                by += 4 * d * n * Hkv + 4 * some * N * Hkv
                fl += N * Hq * (2 * d * nb + 4 * d * (some * G + open_)) + 4 * d * Hq * n * (n + 1) // 2
        else:
            N = n if kind == "chunk" else 1
            if N:
                by += Hkv * _held(c, T) + 4 * d * Hq * N + 4 * d * n * Hkv
                fl += 4 * d * Hq * (N * T + n * (n + 1) // 2)
    return {"bytes": by, "flops": fl}


# ---------------------------------------------------------------- inputs
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _keys(g, shape, rate=0.005):
    """Keys with four large channels per kv head (dim 1) and a few tokens of small norm."""
    Hkv, d = shape[1], shape[-1]
    k = torch.randn(shape, generator=g, device=DEV)
    sc = torch.ones(Hkv, d, device=DEV)
    ch = torch.rand(Hkv, d, generator=g, device=DEV).argsort(1)[:, :OUTLIER_CHANNELS]
    sc.scatter_(1, ch, OUTLIER_SCALE)
    k.mul_(sc.view(1, Hkv, 1, d))
    low = torch.rand(shape[:-1], generator=g, device=DEV) < rate
    return torch.where(low.unsqueeze(-1), k * LOW_NORM, k).half()


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).half()


def _inputs(c, seed):
    """Everything that is drawn, the same for both sides."""
    g = _gen(seed, 23)
    B, Hq, Hkv, d, n = c["B"], c["Hq"], c["Hkv"], c["d"], c["n"]
    Ts, ns = _lens(c)
    T = max(Ts)
    x = dict(Ts=Ts, ns=ns, K=_keys(g, (B, Hkv, T, d)), V=_rand(g, B, Hkv, T, d))
    if c["kind"] == "decode" or (c["kind"] == "sparse" and n == 0):
        x["q"] = _rand(g, B, Hq, d)
    elif c["kind"] in ("chunk", "sparse"):
        x.update(q=_rand(g, B, Hq, n, d), k=_keys(g, (B, Hkv, n, d)), v=_rand(g, B, Hkv, n, d))
    elif c["kind"] == "steps":
        k, v, q = _keys(g, (B, Hkv, n, d)), _rand(g, B, Hkv, n, d), _rand(g, B, Hq, n, d)
        x.update(k=k, v=v, q=q)
    return x


def _cut(c, Ts):
    """The chunks of a prompt: (first token, tokens of each sequence)."""
    step = c["chunk"]
    return [(a, [max(0, min(step, t - a)) for t in Ts]) for a in range(0, max(Ts), step)]


def prepare(case, seed):
    c = case
    x = _inputs(c, seed)
    st = dict(c=c, **x)
    kind, B, Hkv, d, n = c["kind"], c["B"], c["Hkv"], c["d"], c["n"]
    Ts = x["Ts"]
    st["lens"] = x["ns"] if c["T_lo"] and kind in ("chunk", "sparse") and n else None
    # rows behind a sequence's last token stay as they are: zero
    if kind == "chunk" or (kind == "sparse" and n):
        st["out"] = torch.zeros_like(x["q"])
    if kind == "sparse":
        slots = min(c["topk"], max(Ts) // c["G"])
        st["sel"] = torch.full((B, max(n, 1), Hkv, slots), -1, dtype=torch.int32, device=DEV)
    if kind in ("store", "steps", "read"):
        rows = max(Ts) + (n if kind == "steps" else 0) if kind != "read" else n
        st["back"] = [torch.zeros(B, Hkv, rows, d, dtype=torch.float16, device=DEV) for _ in range(2)]
    if kind == "store":
        st["parts"] = [(x["K"][:, :, a:a + c["chunk"]].contiguous(), x["V"][:, :, a:a + c["chunk"]].contiguous(), ln)
                       for a, ln in _cut(c, Ts)]
    if kind == "steps":
        st["rows"] = [tuple(x[i][:, :, s].contiguous() for i in "kvq") for s in range(n)]
    if not own:
        if kind not in ("store", "steps"):
            st["stores"] = [_stores(c, x["K"][b, :, :T], x["V"][b, :, :T]) for b, T in enumerate(Ts)]
            del st["K"], st["V"]
        return st
    import bit_kv_cache_ott_gb300 as ott
    kw = {}
    if c["paged"]:
        kw["pool_blocks"] = max(1, sum((t + (n if kind == "steps" else 0)) // c["G"] for t in Ts) * Hkv)
    room = max(Ts) + (n if kind == "steps" else 0)
    st["cache"] = cache = ott.ByteCache(B, c["Hq"], Hkv, d, c["G"], c["fmt"], max_tokens=room, **kw)
    if kind not in ("store", "steps"):
        cache.append_chunk(st.pop("K"), st.pop("V"), lens=Ts)
        torch.cuda.synchronize()   # K and V are dropped here
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["c"]
    return {"store": _run_store, "read": _run_read, "steps": _run_steps, "decode": _run_decode, "chunk": _run_chunk,
            "sparse": _run_sparse}[c["kind"]](c, state)


def _run_store(c, s):
    K, V = s["back"]
    if own:
        cache = s["cache"]
        cache.reset()
        for k, v, lens in s["parts"]:
            cache.append_chunk(k, v, lens=lens)
        return cache.read(0, K.shape[2], out_k=K, out_v=V)
    for b, T in enumerate(s["Ts"]):
        k = torch.cat([p[0][b] for p in s["parts"]], 1)[:, :T]
        v = torch.cat([p[1][b] for p in s["parts"]], 1)[:, :T]
        st = _stores(c, k, v)
        K[b, :, :T], V[b, :, :T] = _dequantized(st, "k").half(), _dequantized(st, "v").half()
    return K, V


def _run_read(c, s):
    K, V = s["back"]
    if own:
        return s["cache"].read(c["start"], c["n"], out_k=K, out_v=V)
    for b, T in enumerate(s["Ts"]):
        m = min(T, c["start"] + c["n"]) - c["start"]
        if m > 0:
            for x, out in (("k", K), ("v", V)):
                out[b, :, :m] = _dequantized(s["stores"][b], x, c["start"], c["start"] + m).half()
    return K, V


def _run_steps(c, s):
    K, V = s["back"]
    outs = []
    if own:
        cache = s["cache"]
        cache.reset()
        cache.append_chunk(s["K"], s["V"], lens=s["Ts"])
        for k, v, q in s["rows"]:
            cache.append(k, v)
            outs.append(cache.decode_attn(q))
        cache.read(0, K.shape[2], out_k=K, out_v=V)
        return outs, K, V
    seqs = [(s["K"][b, :, :T], s["V"][b, :, :T]) for b, T in enumerate(s["Ts"])]
    for k, v, q in s["rows"]:
        seqs = [(torch.cat([a, k[b].unsqueeze(1)], 1), torch.cat([e, v[b].unsqueeze(1)], 1)) for b, (a, e) in enumerate(seqs)]
        outs.append(torch.stack([_attend(c, q[b].unsqueeze(1), _stores(c, a, e)).squeeze(1) for b, (a, e) in enumerate(seqs)]))
    for b, (a, e) in enumerate(seqs):
        st = _stores(c, a, e)
        K[b, :, :a.shape[1]], V[b, :, :a.shape[1]] = _dequantized(st, "k").half(), _dequantized(st, "v").half()
    return outs, K, V


def _run_decode(c, s):
    if own:
        return s["cache"].decode_attn(s["q"])
    return torch.stack([_attend(c, s["q"][b].unsqueeze(1), s["stores"][b]).squeeze(1) for b in range(c["B"])])


def _run_chunk(c, s):
    if own:
        return s["cache"].chunk_attn(s["q"], s["k"], s["v"], lens=s["lens"], out=s["out"])
    out = torch.zeros_like(s["q"])
    for b, n in enumerate(s["ns"]):
        if n:
            out[b, :, :n] = _attend(c, s["q"][b, :, :n], s["stores"][b], s["k"][b, :, :n], s["v"][b, :, :n])
    return out


def _run_sparse(c, s):
    if own:
        if c["n"] == 0:
            return s["cache"].decode_attn_topk(s["q"], c["topk"], sel=s["sel"]), s["sel"]
        return s["cache"].chunk_attn_topk(s["q"], s["k"], s["v"], c["topk"], lens=s["lens"], out=s["out"],
                                          sel=s["sel"]), s["sel"]
    G, Hkv, g = c["G"], c["Hkv"], c["Hq"] // c["Hkv"]
    out, sel = torch.zeros_like(s["q"]), torch.full_like(s["sel"], -1)
    for b in range(c["B"]):
        st = s["stores"][b]
        nb = s["Ts"][b] // G
        m = min(c["topk"], nb)
        for i in range(s["ns"][b] if c["n"] else 1):
            q = s["q"][b, :, i] if c["n"] else s["q"][b]
            hide = None
            if nb:
                qf = q.float().view(Hkv, g, 1, c["d"])
                lo, hi = (st[x].float().unsqueeze(1) for x in ("lo", "hi"))
                score = torch.zeros(Hkv, g, nb, device=DEV)
                for ch in range(c["d"]):     # 32-bit sums in channel order
                    score = score + torch.maximum(qf[..., ch] * lo[..., ch], qf[..., ch] * hi[..., ch])
                order = score.amax(1).argsort(dim=1, descending=True, stable=True)   # ties to the lower block
                pick = order[:, :m].sort(1).values
                sel[b, i, :, :m] = pick.int()
                hide = torch.ones(Hkv, nb, dtype=torch.bool, device=DEV).scatter_(1, pick, False).repeat_interleave(G, 1)
            if c["n"]:
                new = (s["k"][b, :, :i + 1], s["v"][b, :, :i + 1])
                out[b, :, i] = _attend(c, q.unsqueeze(1), st, *new, hide=hide, last=True).squeeze(1)
            else:
                out[b] = _attend(c, q.unsqueeze(1), st, hide=hide).squeeze(1)
    return out, sel


# ---------------------------------------------------------------- the plain cache
def _codes(c, x):
    """8-bit codes of x [Hkv][nb][G][d] and the scale of each block, [Hkv][nb]."""
    f = x.float()
    a = f.abs().amax((2, 3), keepdim=True)
    top = 127.0 if c["fmt"] == "int8" else 448.0
    r = (f * top) / torch.where(a > 0, a, torch.ones_like(a))     # exact product, one rounding
    code = r.round().to(torch.int8) if c["fmt"] == "int8" else r.to(torch.float8_e4m3fn)
    return code, (a / torch.full_like(a, top)).view(a.shape[:2])


def _stores(c, K, V):
    """A sequence's tokens K, V [Hkv][T][d] as the cache holds them."""
    Hkv, T, d = K.shape
    G = c["G"]
    nb = T // G
    Kb, Vb = (x[:, :nb * G].view(Hkv, nb, G, d) if nb else None for x in (K.contiguous(), V.contiguous()))
    st = dict(nb=nb, G=G, fk=K[:, nb * G:].contiguous(), fv=V[:, nb * G:].contiguous())
    if nb:
        st["kc"], st["ks"] = _codes(c, Kb)
        st["vc"], st["vs"] = _codes(c, Vb)
        st["lo"], st["hi"] = Kb.amin(2), Kb.amax(2)
    return st


def _dequantized(st, x, t0=0, t1=None):
    """Tokens [t0, t1) of the keys ("k") or values ("v") in 32 bits, [Hkv][t1 - t0][d]."""
    G, held = st["G"], st["nb"] * st["G"]
    f = st["f" + x]
    t1 = held + f.shape[1] if t1 is None else t1
    parts = []
    if t0 < held:
        j0, j1 = t0 // G, min(st["nb"], -(-t1 // G))
        full = (st[x + "c"][:, j0:j1].float() * st[x + "s"][:, j0:j1, None, None]).flatten(1, 2)
        parts.append(full[:, t0 - j0 * G:min(t1, held) - j0 * G])
    if t1 > held:
        parts.append(f[:, max(t0, held) - held:t1 - held].float())
    return torch.cat(parts, 1)


def _attend(c, q, st, k=None, v=None, hide=None, last=False):
    """q [Hq][n][d] over a sequence's stores and its new tokens k, v [Hkv][m][d]: causal, or (last) one query that sees
    them all. hide [Hkv][tokens of complete blocks]: those that are not attended."""
    Hq, n, d = q.shape
    Hkv = c["Hkv"]
    g = Hq // Hkv
    out = torch.empty(Hkv, g * n, d, device=DEV)
    qf = q.reshape(Hkv, g * n, d).float()
    m = 0 if k is None else k.shape[1]
    K, V = _dequantized(st, "k"), _dequantized(st, "v")
    T = K.shape[1]
    for h in range(Hkv):
        Kh, Vh = K[h], V[h]
        if m:
            Kh, Vh = torch.cat([Kh, k[h].float()]), torch.cat([Vh, v[h].float()])
        step = max(1, (1 << 28) // Kh.shape[0])
        for r in range(0, g * n, step):
            s = qf[h, r:r + step] @ Kh.t() / math.sqrt(d)
            if m and not last:
                i = torch.arange(r, min(g * n, r + step), device=DEV) % n
                s[:, T:].masked_fill_(torch.arange(m, device=DEV) > i[:, None], float("-inf"))
            if hide is not None:
                s[:, :hide.shape[1]].masked_fill_(hide[h], float("-inf"))
            w = torch.exp(s - s.amax(1, keepdim=True))
            out[h, r:r + step] = (w @ Vh) / w.sum(1, keepdim=True)
    return out.half().view(Hq, n, d)


# ---------------------------------------------------------------- from the definitions, in 64 bits
def _exact_values(c, x):
    """What the cache stands for after tokens x [T][d], 64 bits."""
    T, d = x.shape
    G = c["G"]
    y = x.double()
    whole = T - T % G
    if not whole:
        return y
    t = y[:whole].reshape(-1, G * d)
    peak = t.abs().max(1, keepdim=True).values
    safe = peak.clamp(min=2.0 ** -30)
    if c["fmt"] == "int8":
        val = torch.round(t * 127 / safe) * safe / 127
    else:
        r = t * 448 / safe
        e = torch.frexp(r.abs().clamp(min=2.0 ** -6)).exponent - 1      # 2^e <= |r| < 2^(e+1), not below the subnormals'
        unit = torch.ldexp(torch.ones_like(r), e - 3)
        val = torch.round(r / unit) * unit * safe / 448
    y[:whole] = torch.where(peak > 0, val, torch.zeros_like(val)).view(whole, d)
    return y


def _exact_rows(q, k, v, see):
    """q [rows][d] over tokens k, v [m][d]; see [rows][m]."""
    out = torch.empty(q.shape, dtype=torch.float64, device=DEV)
    step = max(1, (1 << 27) // k.shape[0])
    for i in range(0, q.shape[0], step):
        logit = (q[i:i + step].double() @ k.t()) * q.shape[1] ** -0.5
        out[i:i + step] = torch.softmax(torch.where(see(i, i + step), logit, -math.inf), 1) @ v
    return out


def exact(case, seed):
    """What ``run`` returns, in 64 bits. (A block's bound is a 32-bit number by definition: sums in channel order, each
    rounded, which is done here in 64 bits with a rounding after each.)"""
    c = case
    x = _inputs(c, seed)
    kind, B, Hq, Hkv, d, n, G = c["kind"], c["B"], c["Hq"], c["Hkv"], c["d"], c["n"], c["G"]
    g = Hq // Hkv
    Ts, ns = x["Ts"], x["ns"]
    if kind in ("store", "read"):
        a, rows = (0, max(Ts)) if kind == "store" else (c["start"], n)
        res = []
        for t in (x["K"], x["V"]):
            y = torch.zeros(B, Hkv, rows, d, dtype=torch.float64, device=DEV)
            for b in range(B):
                for h in range(Hkv):
                    e = _exact_values(c, t[b, h, :Ts[b]])[a:a + rows]
                    y[b, h, :e.shape[0]] = e
            res.append(y)
        return tuple(res)
    if kind == "steps":
        K = [torch.cat([x["K"][b, :, :T], x["k"][b]], 1) for b, T in enumerate(Ts)]
        V = [torch.cat([x["V"][b, :, :T], x["v"][b]], 1) for b, T in enumerate(Ts)]
        outs = [torch.empty(B, Hq, d, dtype=torch.float64, device=DEV) for _ in range(n)]
        back = [torch.zeros(B, Hkv, max(Ts) + n, d, dtype=torch.float64, device=DEV) for _ in range(2)]
        for b, T in enumerate(Ts):
            for h in range(Hkv):
                hs = slice(h * g, (h + 1) * g)
                for s in range(n):
                    k, v = (_exact_values(c, t[b][h, :T + s + 1]) for t in (K, V))
                    outs[s][b, hs] = torch.softmax((x["q"][b, hs, s].double() @ k.t()) * d ** -0.5, 1) @ v
                back[0][b, h, :T + n], back[1][b, h, :T + n] = k, v
        return outs, *back
    one = kind == "decode" or n == 0
    out = torch.zeros(x["q"].shape, dtype=torch.float64, device=DEV)
    sel = None
    if kind == "sparse":
        sel = torch.full((B, max(n, 1), Hkv, min(c["topk"], max(Ts) // G)), -1, dtype=torch.int32, device=DEV)
    for b, T in enumerate(Ts):
        m = 0 if one else ns[b]
        if not one and m == 0:
            continue
        nb = T // G
        heads = []
        for h in range(Hkv):
            k, v = _exact_values(c, x["K"][b, h, :T]), _exact_values(c, x["V"][b, h, :T])
            if m:
                k, v = torch.cat([k, x["k"][b, h, :m].double()]), torch.cat([v, x["v"][b, h, :m].double()])
            heads.append((k, v))
        q = x["q"][b].view(Hkv, g, 1, d) if one else x["q"][b, :, :m].reshape(Hkv, g, m, d)
        ids = torch.arange(T + m, device=DEV)
        if kind != "sparse":
            for h, (k, v) in enumerate(heads):
                for i in range(g):
                    y = _exact_rows(q[h, i], k, v, lambda r0, r1: ids <= (T - one) + torch.arange(q.shape[2], device=DEV)[r0:r1, None])
                    out[b, h * g + i] = y[0] if one else torch.nn.functional.pad(y, (0, 0, 0, n - m))
            continue
        keys = x["K"][b, :, :nb * G].reshape(Hkv, nb, G, d)
        lo, hi = (keys.amin(2).double(), keys.amax(2).double()) if nb else (None, None)
        for i in range(q.shape[2]):
            best = None
            if nb:
                acc = torch.zeros(Hkv, g, nb, dtype=torch.float64, device=DEV)
                for ch in range(d):
                    t = q[:, :, i, ch].double()[:, :, None]
                    acc = (acc + torch.where(t > 0, t * hi[:, None, :, ch], t * lo[:, None, :, ch])).float().double()
                best = acc.amax(1).tolist()
            for h, (k, v) in enumerate(heads):
                ok = ids <= T - one + i
                if nb:
                    chosen = sorted(sorted(range(nb), key=lambda j: (-best[h][j], j))[:c["topk"]])
                    sel[b, i, h, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32, device=DEV)
                    mark = torch.zeros(nb, dtype=torch.bool, device=DEV)
                    mark[chosen] = True
                    ok[:nb * G] &= mark.repeat_interleave(G)
                y = torch.softmax(torch.where(ok, (q[h, :, i].double() @ k.t()) * d ** -0.5, -math.inf), 1) @ v
                hs = slice(h * g, (h + 1) * g)
                if one:
                    out[b, hs] = y
                else:
                    out[b, hs, i] = y
    return out if sel is None else (out, sel)
