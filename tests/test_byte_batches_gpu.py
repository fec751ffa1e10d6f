"""The cache held in 8 bits: batches of unlike sequences, long calls of many rows, queries that are not finite."""
import pytest
import torch

from tests import byte_util as bu
from tests.chunk_util import check, draw

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _kv(seed, B, Hkv, T, d):
    return draw(seed, B, Hkv, T, d), draw(seed + 1, B, Hkv, T, d, outliers=False)


@pytest.mark.parametrize("T", [150, 160])   # with an open block, and without
@pytest.mark.parametrize("Hq,n", [(4, 2), (4, 40), (2, 3), (40, 2)])
def test_a_selection_by_a_query_that_is_not_finite(ott, Hq, n, T):
    """Its own row is NaN; the list of its token and kv head is any ascending list of blocks, which the kv head's other
    query heads attend; lists and rows of every other token and kv head are as with a finite query."""
    B, Hkv, d, G, topk = 2, 2, 128, 32, 2
    g = Hq // Hkv
    K, V = _kv(14, B, Hkv, T, d)
    q = draw(15, B, Hq, n, d, outliers=False)
    k, v = _kv(16, B, Hkv, n, d)
    dev = [x.to(DEV) for x in (k, v)]
    hb, ib = 1, n - 1          # the query's head and token, of sequence 0
    with ott.ByteCache(B, Hq, Hkv, d, G, max_tokens=T) as c:
        c.prefill(K.to(DEV), V.to(DEV))

        def run(x):
            sel = torch.full((B, n, Hkv, topk), 99, dtype=torch.int32, device=DEV)
            out = c.chunk_attn_topk(x.to(DEV), *dev, topk, sel=sel)
            one = torch.full((B, Hkv, topk), 99, dtype=torch.int32, device=DEV)
            dec = c.decode_attn_topk(x[:, :, ib].contiguous().to(DEV), topk, sel=one)
            return out.cpu(), sel.cpu(), dec.cpu(), one.cpu()

        ref = run(q)
        for bad in (float("nan"), float("inf"), -float("inf")):
            p = q.clone()
            p[0, hb, ib, 7] = bad
            out, sel, dec, one = run(p)
            assert torch.isnan(out[0, hb, ib]).all() and torch.isnan(dec[0, hb]).all()
            kv = hb // g
            for got, want, lead in ((sel, ref[1], (0, ib, kv)), (one, ref[3], (0, kv))):
                keep = torch.ones(got.shape[:-1], dtype=torch.bool)
                keep[lead] = False
                assert torch.equal(got[keep], want[keep])
                mine = [j for j in got[lead].tolist() if j >= 0]
                assert mine == sorted(set(mine)) and all(j < T // G for j in mine)
                assert got[lead].tolist() == mine + [-1] * (topk - len(mine))
            keep = torch.ones(B, Hq, n, dtype=torch.bool)
            keep[0, kv * g:(kv + 1) * g, ib] = False
            assert torch.equal(out[keep], ref[0][keep])
            assert torch.equal(dec[keep[:, :, ib]], ref[2][keep[:, :, ib]])
            # the kv head's other query heads, over the blocks that came back
            for got, chosen, new in ((out[0, :, ib:ib + 1], sel[0, ib], True), (dec[0].unsqueeze(1), one[0], False)):
                Kx, Vx = K[0], V[0]
                ch = [[[j for j in row.tolist() if j >= 0] for row in chosen]]
                if new:   # token ib sees the new tokens up to itself: appended here, the open block's among them
                    want, tol = _token(q[0, :, ib:ib + 1], Kx, Vx, k[0, :, :n], v[0, :, :n], ib, G, ch[0])
                else:
                    want, tol = bu.attend(q[0, :, ib:ib + 1], Kx, Vx, "int8", G, chosen=ch)
                for h in range(kv * g, (kv + 1) * g):
                    if h != hb:
                        check(got[h:h + 1], want[h:h + 1], tol[h:h + 1], f"{bad} {h}")
        c.check_device()


def _token(q, K, V, k, v, i, G, chosen):
    """New token i alone: the plain form of a chunk of its tokens, of which only the last is asked for."""
    n = i + 1
    Hq, _, d = q.shape
    full = torch.zeros(Hq, n, d, dtype=torch.float16)
    full[:, i:] = q
    every = [[list(range(K.shape[1] // G))] * K.shape[0]] * i + [chosen]
    out, tol = bu.attend(full, K, V, "int8", G, k[:, :n], v[:, :n], every)
    return out[:, i:], tol[:, i:]


@pytest.mark.parametrize("fmt,d,G,Hkv,g,n,paged", [
    ("int8", 64, 32, 28, 4, 3, True), ("e4m3", 128, 64, 24, 16, 1, False), ("int8", 128, 128, 24, 1, 13, True),
    ("e4m3", 64, 64, 24, 3, 2, True),
])
def test_long_batches_of_many_rows(ott, fmt, d, G, Hkv, g, n, paged):
    """Calls long enough that warps claim the last items of every unit: 6 to 16 rows per kv head, sequences without new
    tokens between long ones, a pool; the same bits every time and from a graph."""
    B = 24
    Ts = [9000, 1, 9001, 5000, 64, 9000, 33, 8777, 3, 9000, 9000, 640, 9000, 129, 8500, 9000, 2, 8888, 9000, 4096, 9000, 8999, 9000, 7000]
    ns = [n - b % n for b in range(B)]
    for b in (3, 4, 7, 16, 23):
        ns[b] = 0
    gen = torch.Generator(device=DEV).manual_seed(5)
    K, V = (torch.randn(B, Hkv, max(Ts), d, generator=gen, device=DEV, dtype=torch.float16) for _ in range(2))
    q = draw(6, B, Hkv * g, n, d, outliers=False)
    k, v = _kv(7, B, Hkv, n, d)
    dev = [x.to(DEV) for x in (q, k, v)]
    q1 = dev[0][:, :, 0].contiguous()
    pool = Hkv * sum(t // G for t in Ts) if paged else None
    with ott.ByteCache(B, Hkv * g, Hkv, d, G, fmt, max_tokens=max(Ts), pool_blocks=pool) as c:
        c.append_chunk(K, V, lens=Ts)
        run = lambda: (c.decode_attn(q1), c.chunk_attn(*dev, lens=ns, out=torch.full_like(dev[0], 7)))
        one, out = run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            again = run()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again[0], one) and torch.equal(again[1], out)
        assert all(torch.equal(x, y) for x, y in zip(run(), (one, out)))
        c.check_device()
        for b in (0, 1, 2, 3, 7, 8, 13, 20, 23):
            for h in (0, Hkv // 2 + 1, Hkv - 1):
                Kx, Vx = K[b, h:h + 1, :Ts[b]].cpu(), V[b, h:h + 1, :Ts[b]].cpu()
                rows, m = slice(h * g, (h + 1) * g), ns[b]
                check(one[b, rows].unsqueeze(1), *bu.attend(q[b, rows, :1], Kx, Vx, fmt, G), f"decode {b} {h}")
                if m:
                    check(out[b, rows, :m], *bu.attend(q[b, rows, :m], Kx, Vx, fmt, G, k[b, h:h + 1, :m], v[b, h:h + 1, :m]), f"chunk {b} {h}")
            assert (out[b, :, ns[b]:] == 7).all()
    del K, V
    torch.cuda.empty_cache()


@pytest.mark.parametrize("B,n,long,fmt,d,G,Hkv,g", [
    (32, 512, (5,), "int8", 128, 64, 2, 4), (70, 300, (0, 69), "e4m3", 64, 32, 1, 8), (9, 130, (3, 4), "int8", 128, 128, 3, 1),
    (66, 33, (2,), "e4m3", 128, 32, 1, 3),
])
@pytest.mark.parametrize("paged", [False, True])
def test_a_prompt_beside_single_tokens(ott, B, n, long, fmt, d, G, Hkv, g, paged):
    """One sequence takes a chunk of its prompt while the others take a token each, or none: attention, and writing."""
    Ts = [(37 * b * b) % 1900 for b in range(B)]
    Ts[long[0]] = 1111
    ns = [n if b in long else (0 if b % 7 == 6 else 1) for b in range(B)]
    K, V = _kv(81, B, Hkv, max(Ts), d)
    q = draw(83, B, Hkv * g, n, d, outliers=False)
    k, v = _kv(84, B, Hkv, n, d)
    dirty = [x.clone() for x in (q, k, v)]
    for b, m in enumerate(ns):
        for x in dirty:
            x[b, :, m:] = float("nan")   # never read
    dev = [x.to(DEV) for x in dirty]
    pool = Hkv * sum((t + m) // G for t, m in zip(Ts, ns)) if paged else None
    with ott.ByteCache(B, Hkv * g, Hkv, d, G, fmt, max_tokens=max(Ts) + n, pool_blocks=pool) as c:
        c.append_chunk(K.to(DEV), V.to(DEV), lens=Ts)
        out = c.chunk_attn(*dev, lens=ns, out=torch.full_like(dev[0], 7))
        assert torch.equal(out, c.chunk_attn(*dev, lens=ns, out=torch.full_like(dev[0], 7)))
        c.append_chunk(*dev[1:], lens=ns)
        back = c.read(0, max(Ts) + n)
        assert not paged or c.free_blocks() == 0
        c.check_device()
        for b in range(B):
            T, m = Ts[b], ns[b]
            for x, new, y in ((K, k, back[0]), (V, v, back[1])):
                assert bu.same(y[b, :, :T + m], bu.read_back(torch.cat([x[b, :, :T], new[b, :, :m]], 1), fmt, G)), b
            assert (out[b, :, m:] == 7).all()
            if m and (b in long or b % 5 == 0):
                check(out[b, :, :m], *bu.attend(q[b, :, :m], K[b, :, :T], V[b, :, :T], fmt, G, k[b, :, :m], v[b, :, :m]), f"{b}")


@pytest.mark.parametrize("fmt,d,G,Hkv,g", [("int8", 128, 64, 8, 4), ("e4m3", 64, 32, 2, 7), ("e4m3", 128, 32, 1, 1), ("int8", 64, 128, 3, 2)])
@pytest.mark.parametrize("rows", [17, 24, 32, 63, 100, 127, 128, 129, 255, 257])
def test_row_counts_of_one_and_two_tiles(ott, fmt, d, G, Hkv, g, rows):
    n = -(-rows // g)
    Ts, ns = [700, 2050, 0], [n, max(1, n // 3), n]
    B = len(Ts)
    K, V = _kv(91, B, Hkv, max(Ts), d)
    q = draw(93, B, Hkv * g, n, d, outliers=False)
    k, v = _kv(94, B, Hkv, n, d)
    with ott.ByteCache(B, Hkv * g, Hkv, d, G, fmt, max_tokens=max(Ts)) as c:
        c.append_chunk(K.to(DEV), V.to(DEV), lens=Ts)
        out = c.chunk_attn(*(x.to(DEV) for x in (q, k, v)), lens=ns)
        c.check_device()
        for b in range(B):
            m = ns[b]
            for h in {0, Hkv - 1}:
                s = slice(h * g, (h + 1) * g)
                check(out[b, s, :m], *bu.attend(q[b, s, :m], K[b, h:h + 1, :Ts[b]], V[b, h:h + 1, :Ts[b]], fmt, G, k[b, h:h + 1, :m], v[b, h:h + 1, :m]), f"{b} {h}")
