"""The cache held in 8 bits: writing and reading back number for number, attention of
every kernel and kind of call within derived bounds, selections equal."""
import numpy as np
import pytest
import torch

from tests import byte_util as bu
from tests.chunk_util import check, draw

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _kv(seed, B, Hkv, T, d):
    return draw(seed, B, Hkv, T, d), draw(seed + 1, B, Hkv, T, d, outliers=False)


def _fill(c, K, V, Ts):
    c.append_chunk(K.to(DEV), V.to(DEV), lens=Ts)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d,G", [(128, 32), (128, 64), (128, 128), (64, 32), (64, 64), (64, 128)])
def test_written_and_read_back(ott, fmt, d, G):
    """Every way to cut the tokens into calls gives the same numbers; awkward values; ranges of any alignment."""
    B, Hkv, T = 2, 3, 3 * G + 21
    K, V = _kv(1, B, Hkv, T, d)
    V[0, 0, :G] = 0                                             # a block of zeros
    K[0, 1, :G] = torch.randn(G, d).half() * 2.0 ** -22         # subnormals
    V[1, 0, G:2 * G] = (torch.arange(G * d).reshape(G, d) % 509 - 254).half() / 2   # ties of int8 (a = 127)
    V[1, 0, G, 0] = 127
    K[1, 2, :G] *= 400                                          # up to 65504
    K[1, 2, 3, 5] = -65504
    V[0, 2, 5] = -0.0
    want = [bu.read_back(x, fmt, G) for x in (K, V)]
    Kd, Vd = K.to(DEV), V.to(DEV)
    for cut in ([T], [1] * T, [G, G, G, 21], [G - 1, 2, T - G - 1], [7, 5 * G // 2, T - 7 - 5 * G // 2]):
        with ott.ByteCache(B, Hkv, Hkv, d, G, fmt, max_tokens=T) as c:
            a = 0
            for n in cut:
                part = [x[:, :, a:a + n].contiguous() for x in (Kd, Vd)]
                if n == 1:
                    c.append(part[0][:, :, 0].contiguous(), part[1][:, :, 0].contiguous())
                else:
                    c.append_chunk(*part)
                a += n
            assert c.seq_counts(1) == (T, 3)
            for got, ref in zip(c.read(0, T), want):
                assert bu.same(got, ref), cut
            if cut == [T]:
                for s, n in ((0, 1), (5, 16), (G - 1, 2), (2 * G + 3, G + 18), (3 * G + 20, 1), (1, T - 1)):
                    for got, ref in zip(c.read(s, n), want):
                        assert bu.same(got, ref[:, :, s:s + n]), (s, n)
            c.check_device()


def test_rows_behind_a_sequence_stay(ott):
    B, Hkv, d, G = 4, 2, 64, 32
    Ts = [0, 31, 32, 70]
    K, V = _kv(3, B, Hkv, 80, d)
    for b, t in enumerate(Ts):
        K[b, :, t:] = float("nan")       # never read
        V[b, :, t:] = float("inf")
    with ott.ByteCache(B, 4, Hkv, d, G, "int8", max_tokens=100) as c:
        _fill(c, K, V, Ts)
        outs = [torch.full((B, Hkv, 60, d), 7.0, dtype=torch.float16, device=DEV) for _ in range(2)]
        c.read(20, 60, out_k=outs[0], out_v=outs[1])
        for x, o in ((K, outs[0]), (V, outs[1])):
            for b, t in enumerate(Ts):
                m = max(0, min(t - 20, 60))
                if m:
                    assert bu.same(o[b, :, :m], bu.read_back(x[b, :, :t], "int8", G)[:, 20:20 + m])
                assert (o[b, :, m:] == 7).all()
        # a ragged chunk over it: padded rows hold anything, outputs behind lens stay
        n, ns = 9, [9, 0, 1, 4]
        q = draw(5, B, 4, n, d, outliers=False)
        k, v = _kv(6, B, Hkv, n, d)
        qd, kd, vd = q.clone(), k.clone(), v.clone()
        for b, m in enumerate(ns):
            qd[b, :, m:] = float("nan")
            kd[b, :, m:] = float("inf")
            vd[b, :, m:] = float("nan")
        for topk in (0, 1):
            out = torch.full((B, 4, n, d), 7.0, dtype=torch.float16, device=DEV)
            c.chunk_attn_topk(qd.to(DEV), kd.to(DEV), vd.to(DEV), topk, lens=ns, out=out)
            for b, m in enumerate(ns):
                assert (out[b, :, m:] == 7).all()
                if m:
                    ch = bu.choose(q[b, :, :m], K[b, :, :Ts[b]], G, topk) if topk else None
                    check(out[b, :, :m], *bu.attend(q[b, :, :m], K[b, :, :Ts[b]], V[b, :, :Ts[b]], "int8", G, k[b, :, :m], v[b, :, :m], ch))
        c.check_device()


#   B, Hq, Hkv, d, G, Ts, n
SHAPES = [
    (1, 1, 1, 128, 64, [1], 1), (1, 1, 1, 128, 64, [64], 1), (2, 2, 2, 64, 32, [31, 33], 2),
    (1, 4, 1, 128, 128, [0], 1), (2, 6, 2, 128, 32, [0, 200], 3), (3, 8, 1, 128, 64, [700, 63, 129], 1),
    (2, 10, 2, 64, 64, [333, 500], 3), (1, 16, 1, 128, 32, [260], 1), (2, 14, 2, 128, 64, [511, 64], 2),
    (1, 32, 1, 128, 64, [900], 1), (1, 20, 4, 64, 32, [1111], 5), (2, 4, 4, 128, 128, [900, 1300], 40),
    (1, 2, 2, 128, 32, [0], 300), (1, 8, 2, 64, 128, [260], 77), (3, 3, 1, 128, 64, [5, 1000, 320], 130),
    (1, 7, 1, 128, 64, [2500], 37),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_attention(ott, fmt, case):
    """Chunks and (where every sequence holds a token) decodes: rows kernels of 8 and 16 columns, tiles."""
    B, Hq, Hkv, d, G, Ts, n = SHAPES[case]
    T = max(Ts + [1])
    K, V = _kv(10 + case, B, Hkv, T, d)
    q = draw(50 + case, B, Hq, n, d, outliers=False)
    k, v = _kv(70 + case, B, Hkv, n, d)
    with ott.ByteCache(B, Hq, Hkv, d, G, fmt, max_tokens=T) as c:
        _fill(c, K, V, Ts)
        out = c.chunk_attn(q.to(DEV), k.to(DEV), v.to(DEV))
        for b in range(B):
            check(out[b], *bu.attend(q[b], K[b, :, :Ts[b]], V[b, :, :Ts[b]], fmt, G, k[b], v[b]), f"chunk {b}")
        if min(Ts) > 0:
            out = c.decode_attn(q[:, :, 0].contiguous().to(DEV))
            for b in range(B):
                check(out[b].unsqueeze(1), *bu.attend(q[b, :, :1], K[b, :, :Ts[b]], V[b, :, :Ts[b]], fmt, G), f"decode {b}")
        c.check_device()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("B,Hq,Hkv,d,G,Ts,n,topk", [
    (2, 2, 2, 128, 32, [500, 333], 1, 3), (1, 8, 2, 64, 32, [1999], 4, 1), (3, 9, 1, 128, 64, [10, 64, 700], 2, 4),
    (1, 20, 1, 64, 32, [640], 3, 5), (2, 4, 4, 128, 128, [1280, 127], 2, 100), (1, 4, 1, 128, 32, [4000], 2, 60),
    (2, 4, 2, 64, 32, [700, 90], 100, 3),
])
def test_selected_blocks(ott, fmt, B, Hq, Hkv, d, G, Ts, n, topk):
    K, V = _kv(5, B, Hkv, max(Ts), d)
    K[:, :, G:2 * G] = K[:, :, :G]     # two blocks of equal bounds: the lower one first
    q = draw(6, B, Hq, n, d, outliers=False)
    k, v = _kv(7, B, Hkv, n, d)
    slots = min(topk, max(Ts) // G)
    with ott.ByteCache(B, Hq, Hkv, d, G, fmt, max_tokens=max(Ts)) as c:
        _fill(c, K, V, Ts)
        sel = torch.full((B, n, Hkv, slots), 99, dtype=torch.int32, device=DEV)
        out = c.chunk_attn_topk(q.to(DEV), k.to(DEV), v.to(DEV), topk, sel=sel)
        assert torch.equal(out, c.chunk_attn_topk(q.to(DEV), k.to(DEV), v.to(DEV), topk))   # lists in scratch
        dsel = torch.full((B, Hkv, slots), 99, dtype=torch.int32, device=DEV)
        dout = c.decode_attn_topk(q[:, :, 0].contiguous().to(DEV), topk, sel=dsel)
        for b in range(B):
            Kb, Vb = K[b, :, :Ts[b]], V[b, :, :Ts[b]]
            ch = bu.choose(q[b], Kb, G, topk)
            for i in range(n):
                for h in range(Hkv):
                    want = ch[i][h] + [-1] * (slots - len(ch[i][h]))
                    assert sel[b, i, h].tolist() == want
                    assert i > 0 or dsel[b, h].tolist() == want
            check(out[b], *bu.attend(q[b], Kb, Vb, fmt, G, k[b], v[b], ch))
            check(dout[b].unsqueeze(1), *bu.attend(q[b, :, :1], Kb, Vb, fmt, G, chosen=ch[:1]))
        c.check_device()


@pytest.mark.parametrize("T,K", [(300000, 700), (40000, 1249), (32 * 33, 5), (32 * 2, 1), (32 * 34 + 5, 34)])
def test_selected_among_many_blocks(ott, T, K):
    """More blocks than a cluster's shared memory holds at once, every number of blocks in the last 32, ties throughout
    (keys repeat), selections of nearly all of them."""
    d, G, Hq = 64, 32, 3
    g = torch.Generator().manual_seed(T)
    Kx = torch.randn(1, 1, 997 * G, d, generator=g).half().repeat(1, 1, T // (997 * G) + 1, 1)[:, :, :T].contiguous()
    V = torch.randn(1, 1, T, d, generator=g).half()
    q = torch.randn(1, Hq, d, generator=g).half()
    with ott.ByteCache(1, Hq, 1, d, G, max_tokens=T, pool_blocks=T // G) as c:
        _fill(c, Kx, V, [T])
        sel = torch.full((1, 1, min(K, T // G)), 7, dtype=torch.int32, device=DEV)
        out = c.decode_attn_topk(q.to(DEV), K, sel=sel)
        ch = bu.choose(q[0].unsqueeze(1), Kx[0], G, K)
        assert sel[0, 0].tolist() == ch[0][0]
        see = torch.ones(T, dtype=torch.bool)
        see[:T // G * G] = torch.zeros(T // G, dtype=torch.bool).index_fill_(0, torch.tensor(ch[0][0]), True).repeat_interleave(G)
        Kh, Vh = (bu.held(x[0], "int8", G)[0][0][see] for x in (Kx, V))
        ref = torch.softmax(q[0].double() @ Kh.t() / d ** 0.5, 1) @ Vh
        assert (out[0].double().cpu() - ref).abs().max().item() <= 2e-3   # outputs below 1: two roundings of 2^-11
        c.check_device()


def test_more_blocks_than_there_are_is_every_block(ott):
    B, Hq, Hkv, d, G, T = 2, 4, 2, 128, 32, 500
    K, V = _kv(8, B, Hkv, T, d)
    q = draw(9, B, Hq, 1, d, outliers=False)[:, :, 0].contiguous().to(DEV)
    with ott.ByteCache(B, Hq, Hkv, d, G, max_tokens=T) as c:
        _fill(c, K, V, [T, T])
        assert torch.equal(c.decode_attn_topk(q, 1000), c.decode_attn(q))
        assert torch.equal(c.decode_attn_topk(q, 0), c.decode_attn(q))
        c.check_device()
    with ott.ByteCache(B, Hq, Hkv, d, G, max_tokens=T) as c:      # no complete block: nothing to select
        _fill(c, K, V, [31, 1])
        assert torch.equal(c.decode_attn_topk(q, 3), c.decode_attn(q))
        c.check_device()


def test_blocks_of_very_different_scales(ott):
    """Values from 2^-24 to 65504 side by side: weights follow the products, whatever the blocks' scales."""
    Hq, d, G, T = 4, 128, 32, 200
    K, V = _kv(11, 1, 1, T, d)
    for j, s in enumerate((2.0 ** -10, 900.0, 2.0 ** -21, 1.0, 0.0, 14000.0)):
        V[0, 0, j * G:(j + 1) * G] = (V[0, 0, j * G:(j + 1) * G].float() * s).clamp(-65504, 65504).half()
    for n in (1, 8):            # rows, tiles
        q = draw(12, 1, Hq, n, d, outliers=False)
        q[0, 1] *= 30           # a row of one large weight
        q[0, 2] = 0             # all weights equal
        k, v = _kv(13, 1, 1, n, d)
        with ott.ByteCache(1, Hq, 1, d, G, max_tokens=T) as c:
            _fill(c, K, V, [T])
            for upto in (G, T):   # and a sequence whose only block holds small values
                if upto == G:
                    c.reset()
                    _fill(c, K, V, [G])
                else:
                    c.reset()
                    _fill(c, K, V, [T])
                out = c.chunk_attn(q.to(DEV), k.to(DEV), v.to(DEV))
                check(out[0], *bu.attend(q[0], K[0, :, :upto], V[0, :, :upto], "int8", G, k[0], v[0]))
            c.check_device()


@pytest.mark.parametrize("n", [2, 40])
def test_a_query_that_is_not_finite_spoils_its_own_row(ott, n):
    B, Hq, Hkv, d, G, T = 1, 4, 2, 128, 32, 150
    K, V = _kv(14, B, Hkv, T, d)
    q = draw(15, B, Hq, n, d, outliers=False)
    k, v = _kv(16, B, Hkv, n, d)
    with ott.ByteCache(B, Hq, Hkv, d, G, max_tokens=T) as c:
        _fill(c, K, V, [T])
        ref = c.chunk_attn(q.to(DEV), k.to(DEV), v.to(DEV))
        for bad in (float("nan"), float("inf"), -float("inf")):
            p = q.clone()
            p[0, 1, 1, 7] = bad
            out = c.chunk_attn(p.to(DEV), k.to(DEV), v.to(DEV))
            assert torch.isnan(out[0, 1, 1]).all()
            keep = torch.ones(Hq, n, dtype=torch.bool)
            keep[1, 1] = False
            assert torch.equal(out[0][keep.to(DEV)], ref[0][keep.to(DEV)])
            c.chunk_attn_topk(p.to(DEV), k.to(DEV), v.to(DEV), 2)
        c.check_device()


def test_more_sequences_than_a_launch_holds(ott):
    """70 sequences, two launches; in the second nobody holds a block (its lists are -1)."""
    B, Hq, Hkv, d, G = 70, 2, 1, 64, 32
    Ts = [1 + 7 * b % 90 for b in range(64)] + [5, 31, 1, 30, 2, 9]
    K, V = _kv(17, B, Hkv, 96, d)
    n = 2
    q = draw(18, B, Hq, n, d, outliers=False)
    k, v = _kv(19, B, Hkv, n, d)
    blocks = sum(t // G for t in Ts)
    with ott.ByteCache(B, Hq, Hkv, d, G, "e4m3", max_tokens=100, pool_blocks=blocks) as c:
        _fill(c, K, V, Ts)
        assert c.free_blocks() == 0
        out = c.chunk_attn(q.to(DEV), k.to(DEV), v.to(DEV))
        sel = torch.full((B, n, Hkv, 2), 9, dtype=torch.int32, device=DEV)
        outk = c.chunk_attn_topk(q.to(DEV), k.to(DEV), v.to(DEV), 2, sel=sel)
        back = c.read(0, 96)
        for b, T in enumerate(Ts):
            Kb, Vb = K[b, :, :T], V[b, :, :T]
            check(out[b], *bu.attend(q[b], Kb, Vb, "e4m3", G, k[b], v[b]))
            ch = bu.choose(q[b], Kb, G, 2)
            assert all(sel[b, i, 0].tolist() == (ch[i][0] + [-1, -1])[:2] for i in range(n))
            check(outk[b], *bu.attend(q[b], Kb, Vb, "e4m3", G, k[b], v[b], ch))
            for x, y in zip((Kb, Vb), back):
                assert bu.same(y[b, :, :T], bu.read_back(x, "e4m3", G))
        c.check_device()


@pytest.mark.parametrize("G", [32, 128])
def test_paged_release_and_refill(ott, G):
    """Sequences leave and others take their place and blocks, in any order; the same outputs as without a pool."""
    B, Hq, Hkv, d = 3, 4, 2, 128
    L = 4 * G
    g = torch.Generator().manual_seed(4)
    pool = Hkv * 10
    with ott.ByteCache(B, Hq, Hkv, d, G, max_tokens=L, pool_blocks=pool) as a, ott.ByteCache(B, Hq, Hkv, d, G, max_tokens=L) as c:
        free = pool
        have = [0] * B
        for turn in range(12):
            b = int(torch.randint(0, B, (1,), generator=g))
            n = int(torch.randint(1, L + 1, (1,), generator=g))
            K, V = _kv(100 + turn, 1, Hkv, n, d)
            for x in (a, c):
                x.release_seq(b)
            free += Hkv * (have[b] // G)
            if Hkv * (n // G) > free:
                with pytest.raises(ott.OTTError) as e:
                    a.prefill_seq(b, K[0].to(DEV), V[0].to(DEV))
                assert e.value.code == ott.OTT_ERR_CAPACITY and a.seq_counts(b) == (0, 0)
                n = G - 1
                K, V = K[:, :, :n].contiguous(), V[:, :, :n].contiguous()
            for x in (a, c):
                x.prefill_seq(b, K[0].to(DEV), V[0].to(DEV))
            have[b] = n
            free -= Hkv * (n // G)
            assert a.free_blocks() == free and c.free_blocks() == -1
            for y, z in zip(a.read(0, L), c.read(0, L)):
                assert torch.equal(y, z), turn
            m = 5
            q = draw(200 + turn, B, Hq, m, d, outliers=False).to(DEV)
            k, v = (t.to(DEV) for t in _kv(300 + turn, B, Hkv, m, d))
            assert torch.equal(a.chunk_attn(q, k, v), c.chunk_attn(q, k, v))
            assert torch.equal(a.chunk_attn_topk(q, k, v, 2), c.chunk_attn_topk(q, k, v, 2))
        a.reset()
        assert a.free_blocks() == pool and a.seq_counts(0) == (0, 0)
        a.check_device()
        c.check_device()


def test_capacity_and_refusals(ott):
    B, Hq, Hkv, d, G = 2, 4, 2, 64, 32
    K, V = (x.to(DEV) for x in _kv(20, B, Hkv, 70, d))
    q = torch.zeros(B, Hq, d, dtype=torch.float16, device=DEV)

    def code(f, *a, **kw):
        with pytest.raises(ott.OTTError) as e:
            f(*a, **kw)
        return e.value.code

    with ott.ByteCache(B, Hq, Hkv, d, G, max_tokens=70, pool_blocks=5) as c:
        assert code(c.decode_attn, q) == ott.OTT_ERR_STATE                      # empty
        c.append_chunk(K, V, lens=[40, 0])
        assert code(c.decode_attn, q) == ott.OTT_ERR_STATE                      # one sequence empty
        before = [x.clone() for x in c.read(0, 70)]
        assert code(c.append_chunk, K, V) == ott.OTT_ERR_CAPACITY               # 40 + 70 > 70
        assert code(c.append_chunk, K, V, lens=[0, 70]) == ott.OTT_ERR_CAPACITY   # 4 blocks, 3 free
        assert code(c.append_chunk, K, V, lens=[0, 71]) == ott.OTT_ERR_INVALID
        assert code(c.append_chunk, K, V, lens=[-1, 0]) == ott.OTT_ERR_INVALID
        assert c.seq_counts(0) == c.seq_counts(-1) == (40, 1) and c.seq_counts(1) == (0, 0) and c.free_blocks() == 3
        for b in (-2, 2):
            assert code(c.seq_counts, b) == ott.OTT_ERR_INVALID
        assert all(torch.equal(x, y) for x, y in zip(before, c.read(0, 70)))
        c.append_chunk(K, V, lens=[0, 33])
        assert code(c.decode_attn_topk, q, -1) == ott.OTT_ERR_INVALID
        assert code(c.decode_attn, q, q) == ott.OTT_ERR_INVALID                 # out is q
        assert code(c.read, -1, 4) == ott.OTT_ERR_INVALID
        assert code(c.release_seq, 2) == ott.OTT_ERR_INVALID
        assert code(c.prefill, K, V) == ott.OTT_ERR_STATE
        assert code(c.prefill_seq, 0, K[0], V[0]) == ott.OTT_ERR_STATE
        assert code(c.read, 0, 70, out_k=before[0], out_v=before[0]) == ott.OTT_ERR_INVALID
        buf = torch.zeros(3 * B * Hq * 8 * d, dtype=torch.float16, device=DEV)
        nq, nk = B * Hq * 8 * d, B * Hkv * 8 * d
        qq, kk, vv = buf[:nq].view(B, Hq, 8, d), buf[nq:nq + nk].view(B, Hkv, 8, d), buf[nq + nk:nq + 2 * nk].view(B, Hkv, 8, d)
        for at in (8, nq - 8, nq + nk - 8, nq + 2 * nk - 8):                    # out overlaps an input
            assert code(c.chunk_attn, qq, kk, vv, out=buf[at:at + nq].view(B, Hq, 8, d)) == ott.OTT_ERR_INVALID
        c.chunk_attn(qq, kk, vv, out=buf[nq + 2 * nk:2 * nq + 2 * nk].view(B, Hq, 8, d))
        for bad in ([1], [1, 2 ** 32], [1, -2 ** 31 - 1]):
            with pytest.raises(ValueError):
                c.append_chunk(K, V, lens=bad)
        with pytest.raises(TypeError):
            c.append_chunk(K, V, lens=[1, 1.5])
        with pytest.raises(ValueError):
            c.append_chunk(K, V[:, :, :5])
        with pytest.raises(ValueError):
            c.append_chunk(K.transpose(2, 3).contiguous().transpose(2, 3), V)   # strides
        with pytest.raises(TypeError):
            c.decode_attn(q.float())
        with pytest.raises(ValueError):
            c.decode_attn_topk(q, 1, sel=torch.zeros(B, Hkv, 2, dtype=torch.int32, device=DEV))
        with pytest.raises(TypeError):
            c.decode_attn_topk(q, 1, sel=torch.zeros(B, Hkv, 1, dtype=torch.int64, device=DEV))
        with pytest.raises(ValueError):
            c.chunk_attn_topk(qq, kk, vv, 2 ** 31)
        # nothing to do
        c.append_chunk(K[:, :, :0].contiguous(), V[:, :, :0].contiguous())
        c.append_chunk(K, V, lens=[0, 0])
        c.read(5, 0)
        c.read(69, 3)
        assert c.decode_attn(q).shape == q.shape
        c.check_device()
    with pytest.raises(ValueError):
        ott.ByteCache(1, 1, 1, 64, 32, "int4")
    with pytest.raises(ValueError):
        ott.ByteCache(1, 1, 1, 64, 32, pool_blocks=0)
    assert code(ott.ByteCache, 1, 1, 1, 64, 48) == ott.OTT_ERR_INVALID


def test_a_failed_allocation(ott, monkeypatch):
    monkeypatch.setenv("OTT_FAULT", "alloc")
    with pytest.raises(ott.OTTError) as e:
        ott.ByteCache(1, 1, 1, 64, 32)
    assert e.value.code == ott.OTT_ERR_OOM


@pytest.mark.parametrize("T,n", [(300, 3), (300, 40)])
def test_captured_and_replayed(ott, T, n):
    """A serving step (chunk, append that completes blocks, decode, Top-K, read) in one graph, against plain calls; the
    calls on another stream than the tensors' own."""
    B, Hq, Hkv, d, G = 2, 8, 2, 128, 64
    K, V = (x.to(DEV) for x in _kv(21, B, Hkv, T, d))
    q = draw(22, B, Hq, n, d, outliers=False).to(DEV)
    k, v = (x.to(DEV) for x in _kv(23, B, Hkv, n, d))
    q1 = q[:, :, 0].contiguous()

    def step(c, out, dec, top, back):
        c.chunk_attn(q, k, v, out=out)
        c.append_chunk(k, v)
        c.decode_attn(q1, out=dec)
        c.decode_attn_topk(q1, 2, out=top)
        c.read(T - 50, 50 + n, out_k=back[0], out_v=back[1])

    bufs = [(torch.zeros_like(q), torch.zeros_like(q1), torch.zeros_like(q1),
             [torch.zeros(B, Hkv, 50 + n, d, dtype=torch.float16, device=DEV) for _ in range(2)]) for _ in range(3)]
    with ott.ByteCache(B, Hq, Hkv, d, G, max_tokens=T + n, pool_blocks=40) as a, ott.ByteCache(B, Hq, Hkv, d, G, max_tokens=T + n, pool_blocks=40) as b:
        for c in (a, b):
            c.prefill(K, V)
        step(a, *bufs[0])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(b, *bufs[1])
        g.replay()   # once: it appends
        torch.cuda.synchronize()
        for x, y in zip(bufs[0], bufs[1]):
            for s, t in zip(x if isinstance(x, list) else [x], y if isinstance(y, list) else [y]):
                assert torch.equal(s, t)
        assert a.seq_counts(0) == b.seq_counts(0) and a.free_blocks() == b.free_blocks()
        # attention alone, two graphs of one cache in turn (they share its scratch), new inputs between replays
        graphs = []
        for f in (lambda: a.chunk_attn_topk(q, k, v, 2, out=bufs[1][0]), lambda: a.decode_attn(q1, out=bufs[1][1])):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                f()
            graphs.append(g)
        for turn in range(3):
            q.copy_(draw(30 + turn, B, Hq, n, d, outliers=False))
            q1.copy_(q[:, :, 0])
            want = a.chunk_attn_topk(q, k, v, 2), a.decode_attn(q1)
            for g in graphs:
                g.replay()
            torch.cuda.synchronize()
            assert torch.equal(bufs[1][0], want[0]) and torch.equal(bufs[1][1], want[1])
        a.check_device()
        b.check_device()


def test_two_caches_on_two_streams(ott):
    shapes = [(1, 8, 2, 128, 9000, 200), (2, 4, 4, 64, 3000, 3), (4, 8, 8, 128, 2000, 1)]
    caches, xs = [], []
    for B, Hq, Hkv, d, T, n in shapes:
        c = ott.ByteCache(B, Hq, Hkv, d, 64, "e4m3", max_tokens=T)
        _fill(c, *_kv(24, B, Hkv, T, d), [T] * B)
        caches.append(c)
        xs.append((draw(25, B, Hq, n, d, outliers=False).to(DEV), *(t.to(DEV) for t in _kv(26, B, Hkv, n, d))))
    ref = [(c.chunk_attn(*x), c.chunk_attn_topk(*(t[:, :, :1].contiguous() for t in x), 5)) for c, x in zip(caches, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in shapes]
    outs = [[(torch.zeros_like(r[0]), torch.zeros_like(r[1])) for _ in range(10)] for r in ref]
    one = [tuple(t[:, :, :1].contiguous() for t in x) for x in xs]
    torch.cuda.synchronize()
    for i in range(10):
        for c, x, y, s, o in zip(caches, xs, one, streams, outs):
            c.chunk_attn(*x, out=o[i][0], stream=s)
            c.chunk_attn_topk(*y, 5, out=o[i][1], stream=s)
    torch.cuda.synchronize()
    for c, r, o in zip(caches, ref, outs):
        c.check_device()
        assert all(torch.equal(a, r[0]) and torch.equal(b, r[1]) for a, b in o)
        c.close()


@pytest.mark.parametrize("rows", [1, 40])
def test_long_sums_of_one_sign(ott, rows):
    """200,000 tokens of equal weight and one value: sums on the tensor cores end in time (each loses up to 6e-9 of
    itself per token, 25,088 tokens at most)."""
    d, G, T = 128, 64, 200000
    K = torch.zeros(1, 1, T, d, dtype=torch.float16, device=DEV)
    V = torch.full((1, 1, T, d), 1.0, dtype=torch.float16, device=DEV)
    with ott.ByteCache(1, rows, 1, d, G, max_tokens=T) as c:
        c.prefill(K, V)
        out = c.decode_attn(torch.ones(1, rows, d, dtype=torch.float16, device=DEV))
        # 1.5e-4 and half a step of fp16 below 1
        assert (out.double() - 1).abs().max().item() <= 1.5e-4 + 2.0 ** -12
        c.check_device()


def test_places_beyond_32_bits(ott):
    """A cache of more than 2^32 bytes: its last units, read and attended."""
    B, Hkv, d, G, T = 32, 32, 128, 128, 17000
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device=DEV).manual_seed(2)
    with ott.ByteCache(B, Hkv, Hkv, d, G, max_tokens=T) as c:
        K = torch.randn(B, Hkv, T, d, generator=g, device=DEV, dtype=torch.float16)
        V = torch.randn(B, Hkv, T, d, generator=g, device=DEV, dtype=torch.float16)
        c.prefill(K, V)
        assert B * Hkv * (T // G) * 2 * G * d > 2 ** 32
        bk, bv = c.read(T - 300, 300)
        q = draw(27, B, Hkv, 1, d, outliers=False)
        out = c.decode_attn(q[:, :, 0].contiguous().to(DEV))
        for b, h in ((0, 0), (30, 1), (31, 31)):
            Kx, Vx = K[b, h:h + 1].cpu(), V[b, h:h + 1].cpu()
            for x, y in ((Kx, bk), (Vx, bv)):
                assert bu.same(y[b, h], bu.read_back(x, "int8", G)[0, T - 300:])
            check(out[b, h:h + 1].unsqueeze(1), *bu.attend(q[b, h:h + 1], Kx, Vx, "int8", G))
        c.check_device()
        del K, V, bk, bv
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt,n", [("int8", 1), ("e4m3", 3)])
def test_long_batches_share_their_last_items(ott, fmt, n):
    """Calls long enough that warps claim the last items of every unit: sequences of every length, the same bits every
    time, several units of several sequences against the 64-bit form."""
    B, Hkv, d, G = 20, 32, 128, 64
    Ts = [9000, 1, 70, 5000, 64, 9000, 33, 7777, 3, 8200, 9000, 640, 9000, 129, 6500, 9000, 2, 8888, 9000, 4096]
    g = torch.Generator(device=DEV).manual_seed(5)
    K = torch.randn(B, Hkv, max(Ts), d, generator=g, device=DEV, dtype=torch.float16)
    V = torch.randn(B, Hkv, max(Ts), d, generator=g, device=DEV, dtype=torch.float16)
    q = draw(6, B, Hkv, n, d, outliers=False)
    k, v = _kv(7, B, Hkv, n, d)
    with ott.ByteCache(B, Hkv, Hkv, d, G, fmt, max_tokens=max(Ts)) as c:
        c.append_chunk(K, V, lens=Ts)
        if n == 1:
            outs = [c.decode_attn(q[:, :, 0].contiguous().to(DEV)).unsqueeze(2) for _ in range(3)]
        else:
            outs = [c.chunk_attn(q.to(DEV), k.to(DEV), v.to(DEV)) for _ in range(3)]
        c.check_device()
        assert all(torch.equal(outs[0], o) for o in outs[1:])
        for b in (0, 1, 2, 4, 8, 9, 13, 19):
            for h in (0, 13, 31):
                Kx, Vx = K[b, h:h + 1, :Ts[b]].cpu(), V[b, h:h + 1, :Ts[b]].cpu()
                new = (k[b, h:h + 1], v[b, h:h + 1]) if n > 1 else ()
                check(outs[0][b, h:h + 1], *bu.attend(q[b, h:h + 1], Kx, Vx, fmt, G, *new), f"{b} {h}")
    del K, V, outs
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [1, 40, 1000, 1024, 1025, 1100, 5000])
def test_units_of_a_cta_and_of_several(ott, T):
    """Calls on both sides of the size up to which a CTA serves a unit alone; more warps than items; ragged."""
    B, Hq, Hkv, d, G = 3, 6, 2, 128, 32
    Ts = [T, max(1, T // 3), 1]
    K, V = _kv(31, B, Hkv, T, d)
    q = draw(33, B, Hq, 4, d, outliers=False)
    k, v = _kv(34, B, Hkv, 4, d)
    with ott.ByteCache(B, Hq, Hkv, d, G, "e4m3", max_tokens=T) as c:
        _fill(c, K, V, Ts)
        one = c.decode_attn(q[:, :, 0].contiguous().to(DEV))
        ns = [4, 0, 2]
        out = c.chunk_attn(q.to(DEV), k.to(DEV), v.to(DEV), lens=ns)
        for b in range(B):
            Kb, Vb = K[b, :, :Ts[b]], V[b, :, :Ts[b]]
            check(one[b].unsqueeze(1), *bu.attend(q[b, :, :1], Kb, Vb, "e4m3", G))
            m = ns[b]
            if m:
                check(out[b, :, :m], *bu.attend(q[b, :, :m], Kb, Vb, "e4m3", G, k[b, :, :m], v[b, :, :m]))
        c.check_device()


@pytest.mark.parametrize("fmt,d,G,g,n,topk", [("int8", 128, 64, 4, 1, 0), ("e4m3", 64, 32, 1, 9, 0), ("int8", 128, 32, 5, 3, 30),
                                              ("e4m3", 128, 128, 16, 1, 0)])
@pytest.mark.parametrize("B,Hkv,T", [(12, 5, 1700), (3, 10, 2100), (2, 7, 5000), (1, 3, 9001), (1, 1, 20001)])
def test_units_of_a_cluster(ott, fmt, d, G, g, n, topk, B, Hkv, T):
    """Units that clusters of 2, 4, 8 and 16 CTAs serve, beside short ones and empty ones; rows more and fewer than CTAs;
    the same bits again and from a graph."""
    Ts = [max(1, T - 301 * b) for b in range(B)]
    K, V = _kv(71, B, Hkv, T, d)
    q = draw(73, B, Hkv * g, n, d, outliers=False)
    k, v = _kv(74, B, Hkv, n, d)
    ns = [0 if b % 5 == 2 else n - b % n for b in range(B)]
    with ott.ByteCache(B, Hkv * g, Hkv, d, G, fmt, max_tokens=T) as c:
        _fill(c, K, V, Ts)
        dev = [x.to(DEV) for x in (q, k, v)]
        q1 = dev[0][:, :, 0].contiguous()
        run = lambda: (c.decode_attn_topk(q1, topk), c.chunk_attn_topk(*dev, topk, lens=ns, out=torch.full_like(dev[0], 7)))
        one, out = run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            again = run()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again[0], one) and torch.equal(again[1], out)
        for b in range(B):
            if b and b + 2 < B and b % 5 != 2:
                continue   # the first, the last, an empty and its neighbours
            Kb, Vb, m = K[b, :, :Ts[b]], V[b, :, :Ts[b]], ns[b]
            ch = bu.choose(q[b], Kb, G, topk) if topk else None
            check(one[b].unsqueeze(1), *bu.attend(q[b, :, :1], Kb, Vb, fmt, G, chosen=ch and ch[:1]))
            if m:
                check(out[b, :, :m], *bu.attend(q[b, :, :m], Kb, Vb, fmt, G, k[b, :, :m], v[b, :, :m], ch and ch[:m]))
            assert (out[b, :, m:] == 7).all()
        c.check_device()


def test_beside_an_ott_cache(ott):
    """A model whose first layer is kept in 8 bits and the second in 2: the same loop over both kinds."""
    B, Hq, Hkv, d, T, n = 2, 8, 2, 128, 300, 20
    layers = [ott.ByteCache(B, Hq, Hkv, d, 64, max_tokens=T + 3 * n), ott.OTTCache(B, Hq, Hkv, d, max_tokens=T + 3 * n, ragged=True)]
    K, V = _kv(28, B, Hkv, T, d)
    for c in layers:
        c.prefill_lens(K.to(DEV), V.to(DEV), [T, T - 77])
    seen = [[K[0], K[1, :, :T - 77]], [V[0], V[1, :, :T - 77]]]
    for turn in range(3):
        q = draw(30 + turn, B, Hq, n, d, outliers=False)
        k, v = _kv(40 + turn, B, Hkv, n, d)
        outs = []
        for c in layers:
            outs.append(c.chunk_attn(q.to(DEV), k.to(DEV), v.to(DEV), lens=[n, 5 + turn]))
            c.append_chunk(k.to(DEV), v.to(DEV), lens=[n, 5 + turn])
        for b, m in enumerate((n, 5 + turn)):
            check(outs[0][b, :, :m], *bu.attend(q[b, :, :m], seen[0][b], seen[1][b], "int8", 64, k[b, :, :m], v[b, :, :m]))
            for s, t in zip(seen, (k, v)):
                s[b] = torch.cat([s[b], t[b, :, :m]], 1)
    for c in layers:
        c.check_device()
        c.close()
