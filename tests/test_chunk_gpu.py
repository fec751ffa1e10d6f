"""ott_chunk_attn, ott_decode_attn_window and ott_append_chunk: against the
plain 64-bit form over the exported state (tests/chunk_util.py), and appends
of chunks against one-token appends, bit for bit, in every cache variant.
"""
import ctypes as C

import numpy as np
import pytest
import torch

from tests.chunk_util import attend, check, draw

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _cache(ott, kind, B, Hq, Hkv, d, G, R, P, T, room):
    """A cache of the kind with T tokens (a list for kinds with lengths of their own)."""
    kw = {"uniform": {}, "ragged": dict(ragged=True), "cold": dict(cold=5), "pct": dict(pct=(1500, 3))}.get(kind)
    Ts = T if isinstance(T, list) else [T] * B
    if kind == "paged":
        kw = dict(pool_blocks=max(1, sum((t + room) // G + 1 for t in Ts) * Hkv))
    c = ott.OTTCache(B, Hq, Hkv, d, G, R, P, max_tokens=max(Ts) + room, **kw)
    if kind in ("ragged", "paged"):
        K, V = draw(sum(Ts) + G, B, Hkv, max(Ts) + 1, d), draw(sum(Ts) + G + 1, B, Hkv, max(Ts) + 1, d, outliers=False)
        for b, t in enumerate(Ts):
            if t:
                c.prefill_seq(b, K[b, :, :t].contiguous().to(DEV), V[b, :, :t].contiguous().to(DEV))
    elif max(Ts):
        c.prefill(draw(Ts[0] + G, B, Hkv, Ts[0], d).to(DEV), draw(Ts[0] + G + 1, B, Hkv, Ts[0], d, outliers=False).to(DEV))
    return c, Ts


#    kind       B  Hq Hkv d    G    R   P   T              n    window sinks
CHUNKS = [
    ("uniform", 2, 4, 4, 128, 32, 4, 6, 300, 4, 0, 0),           # a draft over several blocks
    ("uniform", 1, 1, 1, 64, 16, 4, 5, 0, 1, 0, 0),              # one token over an empty cache
    ("uniform", 1, 2, 1, 128, 128, 32, 32, 0, 200, 0, 0),        # an empty cache: plain causal attention
    ("uniform", 3, 8, 2, 64, 16, 0, 40, 200, 33, 0, 0),          # R = 0, a pool larger than a group, empty blocks
    ("uniform", 1, 6, 2, 128, 17, 3, 0, 170, 7, 0, 0),           # odd group, no pool, three heads per kv head
    ("uniform", 1, 8, 1, 128, 128, 32, 32, 1000, 65, 0, 0),      # multi-query, rows cross tiles
    ("uniform", 1, 5, 1, 64, 200, 9, 32, 900, 128, 0, 0),        # blocks of four chunks, five heads
    ("ragged", 4, 4, 2, 128, 32, 4, 6, [0, 1, 37, 333], [9, 0, 1, 5], 0, 0),
    ("ragged", 3, 2, 2, 64, 16, 3, 5, [90, 0, 300], [0, 130, 77], 0, 0),
    ("paged", 3, 8, 2, 128, 32, 8, 8, [5, 400, 129], [17, 3, 40], 0, 0),
    ("cold", 2, 4, 2, 128, 32, 4, 8, 400, 6, 0, 0),
    ("cold", 1, 2, 1, 64, 16, 4, 8, 333, 50, 90, 3),
    ("pct", 2, 4, 2, 128, 32, 4, 16, 400, 6, 0, 0),
    ("pct", 1, 2, 1, 64, 32, 4, 16, 333, 50, 100, 2),
    ("uniform", 2, 4, 2, 128, 32, 4, 6, 700, 5, 64, 4),          # window over the ring and some blocks
    ("uniform", 1, 4, 1, 64, 16, 0, 9, 500, 40, 1, 0),           # each query sees itself only
    ("uniform", 1, 2, 2, 128, 32, 4, 12, 600, 33, 7, 1000),      # every token of the past is a first token
    ("uniform", 1, 4, 4, 128, 128, 32, 32, 1500, 300, 200, 130), # sinks over more than a block, window under the chunk
    ("ragged", 4, 4, 2, 128, 32, 4, 6, [2, 80, 37, 533], [9, 21, 1, 40], 50, 4),
    ("paged", 3, 6, 2, 64, 32, 8, 8, [5, 400, 129], [17, 3, 90], 33, 1),
    ("uniform", 1, 4, 2, 128, 256, 64, 32, 3000, 150, 0, 0),
    ("uniform", 1, 4, 2, 128, 64, 16, 32, 2000, 600, 1000, 4),
    ("uniform", 2, 16, 2, 128, 128, 32, 64, 1111, 33, 0, 0),
    ("uniform", 1, 3, 1, 64, 128, 32, 32, 1200, 257, 0, 0),
]


CHUNKS += [
    # up to four rows per kv head: every kind, some sequences with nothing, windows, listed blocks
    ("ragged", 4, 4, 2, 128, 32, 4, 6, [0, 1, 37, 333], [2, 0, 1, 2], 0, 0),
    ("ragged", 4, 3, 1, 64, 16, 3, 5, [90, 0, 300, 7], [1, 1, 1, 0], 40, 3),
    ("paged", 3, 2, 2, 128, 32, 8, 8, [5, 400, 129], [4, 1, 0], 0, 0),
    ("paged", 3, 4, 4, 64, 16, 4, 8, [50, 333, 129], [3, 4, 2], 30, 20),
    ("cold", 2, 4, 2, 128, 32, 4, 8, 400, 2, 0, 0),
    ("cold", 1, 4, 4, 64, 16, 4, 8, 333, 3, 90, 40),
    ("pct", 2, 4, 2, 128, 32, 4, 16, 400, 2, 120, 3),
    ("uniform", 2, 3, 1, 128, 17, 3, 4, 300, 1, 0, 0),           # odd group
    ("uniform", 2, 3, 1, 64, 40, 3, 4, 500, 1, 100, 33),         # first tokens over a tile, not over the block
    ("uniform", 64, 8, 8, 64, 16, 4, 8, 400, 2, 90, 30),         # more blocks than warps
    # five to sixteen
    ("ragged", 4, 4, 2, 64, 32, 4, 6, [2, 80, 37, 533], [8, 0, 1, 5], 50, 4),
    ("paged", 2, 8, 1, 128, 40, 8, 8, [77, 400], [2, 1], 120, 33),
    ("cold", 2, 4, 1, 128, 32, 4, 8, 400, 4, 90, 5),
    ("pct", 1, 10, 2, 64, 32, 4, 16, 333, 3, 0, 0),
    ("uniform", 1, 16, 1, 128, 200, 9, 32, 900, 1, 300, 70),
    # seventeen and more: every kind, heads that do not divide a tile, more heads than a pair of tiles has rows
    ("paged", 2, 6, 2, 128, 40, 8, 8, [77, 400], [90, 6], 120, 33),
    ("cold", 2, 4, 1, 128, 32, 4, 8, 400, 70, 0, 0),
    ("pct", 1, 10, 2, 128, 32, 4, 16, 333, 61, 0, 0),
    ("uniform", 1, 300, 1, 64, 32, 4, 6, 300, 2, 0, 0),
    ("uniform", 1, 17, 1, 128, 100, 4, 6, 700, 1, 0, 0),
    ("uniform", 2, 8, 2, 64, 100, 4, 6, 1500, 130, 500, 90),     # listed blocks of several groups
    ("uniform", 19, 8, 8, 64, 32, 4, 6, 200, 17, 0, 0),          # as many equal tiles as SMs
    ("uniform", 38, 8, 8, 64, 32, 4, 6, 200, 17, 0, 0),          # twice as many
]


@pytest.mark.parametrize("kind,B,Hq,Hkv,d,G,R,P,T,n,window,sinks", CHUNKS)
def test_chunk_attn(ott, kind, B, Hq, Hkv, d, G, R, P, T, n, window, sinks):
    lens = n if isinstance(n, list) else None
    ns = n if lens else [n] * B
    m = max(ns) + (2 if lens else 0)   # rooms with rows that no sequence uses
    c, Ts = _cache(ott, kind, B, Hq, Hkv, d, G, R, P, T, m)
    with c:
        q, k, v = draw(7, B, Hq, m, d, outliers=False), draw(8, B, Hkv, m, d), draw(9, B, Hkv, m, d, outliers=False)
        out = torch.full((B, Hq, m, d), 7.0, dtype=torch.float16, device=DEV)
        nan = float("nan")
        for b in range(B):   # rows behind a sequence's tokens are not read
            q[b, :, ns[b]:], k[b, :, ns[b]:], v[b, :, ns[b]:] = nan, nan, nan
        before = [c.seq_counts(b) for b in range(B)]
        c.chunk_attn(q.to(DEV), k.to(DEV), v.to(DEV), lens=lens, window=window, sinks=sinks, out=out)
        c.check_device()
        assert before == [c.seq_counts(b) for b in range(B)]
        for b in range(B):
            assert bool((out[b, :, ns[b]:] == 7.0).all()), f"rows behind sequence {b}'s tokens were written"
            if ns[b]:
                ref, tol = attend(c, b, q[b, :, :ns[b]], Ts[b], window, sinks, k[b, :, :ns[b]], v[b, :, :ns[b]],
                                  folded=max(ns) * Hq // Hkv <= 4)
                check(out[b, :, :ns[b]], ref, tol, f"sequence {b}")


#    kind       B  Hq Hkv d    G    R   P   T              window sinks
WINDOWS = [
    ("uniform", 2, 4, 4, 128, 32, 4, 6, 700, 64, 4),
    ("uniform", 2, 4, 4, 128, 32, 4, 6, 700, 0, 0),
    ("uniform", 1, 8, 1, 64, 16, 0, 9, 512, 1, 0),               # R = 0, T a whole number of groups
    ("uniform", 1, 8, 1, 64, 16, 0, 0, 512, 3, 2),               # no fp16 token at all
    ("uniform", 1, 5, 1, 128, 32, 4, 12, 600, 100, 1000),
    ("uniform", 1, 12, 1, 128, 128, 32, 32, 2000, 300, 1),       # more rows than one group of columns
    ("uniform", 1, 40, 2, 64, 16, 4, 8, 1, 5, 2),                # one token
    ("ragged", 4, 4, 2, 128, 32, 4, 6, [1, 80, 37, 533], 50, 4),
    ("paged", 3, 6, 2, 64, 32, 8, 8, [5, 400, 129], 33, 1),
    ("cold", 2, 4, 2, 128, 32, 4, 8, 400, 100, 3),
    ("pct", 2, 4, 2, 128, 32, 4, 16, 400, 90, 3),
    ("uniform", 1, 32, 8, 128, 128, 32, 64, 5000, 1024, 16),
    # many blocks before the window
    ("uniform", 2, 4, 4, 64, 16, 4, 8, 900, 100, 20),
    ("cold", 2, 4, 2, 64, 16, 4, 8, 900, 100, 40),
    # more blocks than warps: items of several listed slots
    ("uniform", 64, 8, 8, 64, 16, 4, 8, 900, 100, 40),
    ("uniform", 64, 8, 8, 64, 16, 4, 8, 200, 100, 40),
    ("uniform", 64, 8, 8, 64, 128, 4, 8, 1100, 600, 130),
]


@pytest.mark.parametrize("kind,B,Hq,Hkv,d,G,R,P,T,window,sinks", WINDOWS)
def test_decode_attn_window(ott, kind, B, Hq, Hkv, d, G, R, P, T, window, sinks):
    c, Ts = _cache(ott, kind, B, Hq, Hkv, d, G, R, P, T, 4)
    with c:
        q = draw(11, B, Hq, 1, d, outliers=False)
        out = c.decode_attn_window(q[:, :, 0].contiguous().to(DEV), window, sinks)
        c.check_device()
        for b in range(B):
            ref, tol = attend(c, b, q[b], Ts[b] - 1, window, sinks, folded=Hq // Hkv <= 4)
            check(out[b].unsqueeze(1), ref, tol, f"sequence {b}")


def test_more_sequences_than_one_launch_takes(ott):
    B, d = 300, 64
    c, Ts = _cache(ott, "uniform", B, 2, 1, d, 16, 4, 5, 60, 8)
    with c:
        q, k, v = draw(3, B, 2, 3, d, outliers=False), draw(4, B, 1, 3, d), draw(5, B, 1, 3, d)
        out = c.chunk_attn(q.to(DEV), k.to(DEV), v.to(DEV), window=20, sinks=2)
        c.append_chunk(k.to(DEV), v.to(DEV))
        for b in (0, 255, 256, 299):
            e = c.export_state(b, 1)
            assert e["T"] == 63 and np.array_equal(e["tk"][0, -3:].view(np.float16), k[b, 0].numpy())
        with _cache(ott, "uniform", B, 2, 1, d, 16, 4, 5, 60, 8)[0] as c2:
            for b in (0, 255, 256, 299):
                ref, tol = attend(c2, b, q[b], 60, 20, 2, k[b], v[b])
                check(out[b], ref, tol, f"sequence {b}")


@pytest.mark.parametrize("kind,B,Hq,Hkv,d,G,R,P,T,n", [
    ("uniform", 2, 2, 2, 128, 32, 4, 6, 50, 100),
    ("uniform", 1, 1, 1, 64, 16, 40, 5, 0, 200),        # a ring longer than two groups, from empty
    ("uniform", 2, 2, 1, 64, 16, 0, 9, 47, 1),          # the last token that a flush waits for
    ("uniform", 2, 2, 1, 64, 16, 0, 9, 47, 2),
    ("ragged", 4, 2, 2, 64, 16, 3, 5, [0, 1, 37, 200], [70, 0, 1, 33]),
    ("uniform", 1, 2, 2, 64, 16, 4, 40, 100, 150),      # a pool larger than a group
    ("uniform", 1, 2, 2, 64, 16, 4, 0, 100, 150),       # no pool
    ("uniform", 3, 2, 2, 128, 32, 8, 32, 300, 700),     # the pool as large as a group, many flushes
    ("uniform", 1, 1, 1, 64, 16, 4, 16, 20, 2000),      # a scan over many lists
    ("ragged", 1, 2, 1, 128, 32, 8, 12, [95], [300]),
    ("paged", 2, 2, 2, 64, 16, 3, 8, [0, 333], [260, 80]),
    ("paged", 3, 2, 1, 128, 32, 4, 6, [10, 300, 35], [100, 3, 0]),
    ("paged", 2, 2, 1, 128, 32, 4, 6, 40, 60),
    ("cold", 2, 2, 1, 64, 16, 4, 8, 100, 77),
    ("pct", 2, 2, 1, 64, 32, 4, 16, 100, 77),
])
def test_append_chunk_is_that_many_appends(ott, kind, B, Hq, Hkv, d, G, R, P, T, n):
    lens = n if isinstance(n, list) else None
    ns = n if lens else [n] * B
    m = max(ns) + (1 if lens else 0)
    k, v = draw(21, B, Hkv, m, d).to(DEV), draw(22, B, Hkv, m, d).to(DEV)
    c, Ts = _cache(ott, kind, B, Hq, Hkv, d, G, R, P, T, m)
    with c:
        c.append_chunk(k, v, lens=lens)
        c.check_device()
        for b in range(B):   # the same tokens as one prompt: every variant defines prefill as that many appends
            one_kind = "uniform" if kind in ("ragged", "paged") else kind
            Kp, Vp = _cache_inputs(kind, B, Hkv, d, G, Ts)
            K1 = torch.cat([Kp[b:b + 1, :, :Ts[b]].to(DEV), k[b:b + 1, :, :ns[b]]], 2).contiguous()
            V1 = torch.cat([Vp[b:b + 1, :, :Ts[b]].to(DEV), v[b:b + 1, :, :ns[b]]], 2).contiguous()
            kw = {"cold": dict(cold=5), "pct": dict(pct=(1500, 3))}.get(one_kind, {})
            with ott.OTTCache(1, Hq, Hkv, d, G, R, P, max_tokens=Ts[b] + m, **kw) as c1:
                for t in range(K1.shape[2]):
                    c1.append(K1[:, :, t].contiguous(), V1[:, :, t].contiguous())
                e, f = c.export_state(b * Hkv, Hkv), c1.export_state()
                for key in f:
                    assert np.array_equal(e[key], f[key]), (b, key)


def _cache_inputs(kind, B, Hkv, d, G, Ts):
    if kind in ("ragged", "paged"):
        return draw(sum(Ts) + G, B, Hkv, max(Ts) + 1, d), draw(sum(Ts) + G + 1, B, Hkv, max(Ts) + 1, d, outliers=False)
    return draw(Ts[0] + G, B, Hkv, max(Ts[0], 1), d), draw(Ts[0] + G + 1, B, Hkv, max(Ts[0], 1), d, outliers=False)


def test_append_chunk_feeds_the_other_paths(ott):
    """Chunks, single appends, decodes and host steps in turn, against the same tokens one by one."""
    B, Hq, Hkv, d, G, R, P = 2, 4, 2, 128, 32, 4, 6
    K, V = draw(31, B, Hkv, 400, d).to(DEV), draw(32, B, Hkv, 400, d).to(DEV)
    q = draw(33, B, Hq, 1, d, outliers=False)[:, :, 0].contiguous().to(DEV)
    with ott.OTTCache(B, Hq, Hkv, d, G, R, P, max_tokens=400) as c, ott.OTTCache(B, Hq, Hkv, d, G, R, P, max_tokens=400) as r:
        t = 0
        for n in (1, 35, 1, 64, 3, 128, 100):
            c.append_chunk(K[:, :, t:t + n].contiguous(), V[:, :, t:t + n].contiguous())
            for x in range(t, t + n):
                r.append(K[:, :, x].contiguous(), V[:, :, x].contiguous())
            t += n
            assert c.counts() == r.counts()
            assert torch.equal(c.decode_attn(q), r.decode_attn(q))
            assert torch.equal(c.decode_attn_window(q, 50, 2), r.decode_attn_window(q, 50, 2))
            c.append(K[:, :, t].contiguous(), V[:, :, t].contiguous())
            r.append(K[:, :, t].contiguous(), V[:, :, t].contiguous())
            t += 1
        c.check_device()


def test_the_loop_of_a_serving_step(ott):
    """Rotate, attend, append, chunk by chunk; then rotate, append, windowed decode: together, on a side stream."""
    B, Hq, Hkv, d, G, R, P = 2, 4, 2, 64, 32, 4, 6
    s = torch.cuda.Stream()
    with ott.OTTCache(B, Hq, Hkv, d, G, R, P, max_tokens=400) as c:
        T = 0
        for step, n in enumerate((70, 1, 33, 130)):
            q, k, v = (draw(50 + step + x, B, h, n, d, outliers=False) for x, h in ((0, Hq), (100, Hkv), (200, Hkv)))
            pos = torch.stack([T + torch.arange(n), torch.arange(n) // 7]).int()[:, None].expand(2, B, n).contiguous()
            qd, kd, vd, pd = q.to(DEV), k.to(DEV), v.to(DEV), pos.to(DEV)
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                qr, kr = ott.rope(qd, kd, pd, (20, 12))
                out = c.chunk_attn(qr, kr, vd, window=100, sinks=4)
            s.synchronize()
            for b in range(B):
                ref, tol = attend(c, b, qr[b].cpu(), T, 100, 4, kr[b].cpu(), v[b], folded=n * Hq // Hkv <= 4)
                check(out[b], ref, tol, f"step {step}")
            with torch.cuda.stream(s):
                c.append_chunk(kr, vd)
            T += n
            with torch.cuda.stream(s):
                dec = c.decode_attn_window(qr[:, :, -1].contiguous(), 60, 4)
            s.synchronize()
            for b in range(B):
                ref, tol = attend(c, b, qr[b, :, -1:].cpu(), T - 1, 60, 4, folded=Hq // Hkv <= 4)
                check(dec[b].unsqueeze(1), ref, tol, f"decode {step}")
        c.check_device()


def test_results_repeat_and_replay(ott):
    """The same call twice gives the same bits, and so does its captured graph."""
    c, _ = _cache(ott, "uniform", 2, 8, 2, 128, 32, 4, 6, 700, 64)
    with c:
        for n in (3, 64):
            q, k, v = (draw(60 + x, 2, h, n, 128, outliers=False).to(DEV) for x, h in ((0, 8), (1, 2), (2, 2)))
            out = torch.zeros_like(q)
            ref = c.chunk_attn(q, k, v, window=300, sinks=4)
            assert torch.equal(ref, c.chunk_attn(q, k, v, window=300, sinks=4))
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                c.chunk_attn(q, k, v, window=300, sinks=4, out=out)
            out.zero_()
            for _ in range(3):
                g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
        c.check_device()


def test_refusals(ott):
    B, Hq, Hkv, d = 2, 4, 2, 64
    q, k = torch.zeros(B, Hq, 3, d, dtype=torch.float16, device=DEV), torch.zeros(B, Hkv, 3, d, dtype=torch.float16, device=DEV)
    L = ott.load()

    def code(fn, *a, **kw):
        with pytest.raises(ott.OTTError) as ei:
            fn(*a, **kw)
        return ei.value.code

    with ott.OTTCache(B, Hq, Hkv, d, 16, 4, 5, max_tokens=10) as c:
        assert code(c.decode_attn_window, q[:, :, 0].contiguous(), 4) == ott.OTT_ERR_STATE       # empty
        assert code(c.chunk_attn, q, k, k, lens=[1, 1]) == ott.OTT_ERR_STATE                     # one length for all
        assert code(c.append_chunk, k, k, lens=[1, 1]) == ott.OTT_ERR_STATE
        for bad in (dict(window=-1), dict(window=4, sinks=-1)):
            assert code(c.chunk_attn, q, k, k, **bad) == ott.OTT_ERR_INVALID
        assert code(c.chunk_attn, q, k, k, out=q) == ott.OTT_ERR_INVALID
        for _ in range(3):
            c.append_chunk(k, k)
        assert code(c.append_chunk, k, k) == ott.OTT_ERR_CAPACITY and c.counts()[0] == 9
        assert code(c.decode_attn_window, q[:, :, 0].contiguous(), -1) == ott.OTT_ERR_INVALID
        h, p = c._h, q.data_ptr()
        assert L.ott_chunk_attn(h, p + 2, k.data_ptr(), k.data_ptr(), p, 3, None, 0, 0, None) == ott.OTT_ERR_INVALID
        assert L.ott_chunk_attn(h, None, k.data_ptr(), k.data_ptr(), p, 3, None, 0, 0, None) == ott.OTT_ERR_INVALID
        assert L.ott_chunk_attn(h, None, None, None, None, 0, None, 0, 0, None) == ott.OTT_OK
        assert L.ott_append_chunk(h, None, None, -1, None, None) == ott.OTT_ERR_INVALID
        for wrong in (q.float(), q.cpu(), q[:, :, :2], q.transpose(1, 2)):
            with pytest.raises((TypeError, ValueError)):
                c.chunk_attn(wrong, k, k)
        with pytest.raises(ValueError):
            c.append_chunk(k, k[:, :, :2].contiguous())
        assert c.counts()[0] == 9
        c.decode_attn_window(q[:, :, 0].contiguous(), 4)   # the cache still serves
        c.check_device()
    with ott.OTTCache(B, Hq, Hkv, d, 16, 4, 5, max_tokens=100, pool_blocks=3) as c:
        for bad in ([4, 1], [-1, 1]):
            assert code(c.chunk_attn, q, k, k, lens=bad) == ott.OTT_ERR_INVALID
            assert code(c.append_chunk, k, k, lens=bad) == ott.OTT_ERR_INVALID
        with pytest.raises(ValueError):
            c.append_chunk(k, k, lens=[1])
        big = torch.zeros(B, Hkv, 40, d, dtype=torch.float16, device=DEV)
        assert code(c.append_chunk, big, big) == ott.OTT_ERR_CAPACITY      # four unit flushes each, three blocks
        assert c.free_blocks() == 3 and c.counts()[0] == 0
        c.append_chunk(big, big, lens=[20, 3])
        assert c.free_blocks() == 1 and [c.seq_counts(b)[0] for b in (0, 1)] == [20, 3]
        c.release_seq(1)
        assert code(c.decode_attn_window, q[:, :, 0].contiguous(), 4) == ott.OTT_ERR_STATE
        c.chunk_attn(q, k, k, lens=[0, 0])
        c.check_device()


@pytest.mark.parametrize("value", [48000.0, 1e-3, 6e-8])
def test_range_of_keys_and_values(ott, value):
    """Keys and values at the documented limit, and as small as fp16 goes."""
    B, H, d, n = 1, 2, 64, 5
    K = (torch.rand(B, H, 200, d, generator=torch.Generator().manual_seed(1)) * 2 - 1) * value
    V = (torch.rand(B, H, 200, d, generator=torch.Generator().manual_seed(2)) * 2 - 1) * value
    K[..., 0], V[..., 0] = value, -value
    K, V = K.half(), V.half()
    q = torch.randn(B, H, n, d, generator=torch.Generator().manual_seed(3))
    q = (q / max(1.0, value / 4)).half()
    with ott.OTTCache(B, H, H, d, 32, 4, 6, max_tokens=300) as c:
        c.prefill(K.to(DEV), V.to(DEV))
        out = c.chunk_attn(q.to(DEV), K[:, :, :n].contiguous().to(DEV), V[:, :, :n].contiguous().to(DEV))
        ref, tol = attend(c, 0, q[0], 200, 0, 0, K[0, :, :n], V[0, :, :n])
        check(out[0], ref, tol)
