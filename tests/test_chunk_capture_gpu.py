"""The chunk calls captured and replayed (with scratch of their own, several
graphs of one cache, a whole serving step in one graph), and two caches at
work on two streams at once: the bits of the plain calls.
"""
import numpy as np
import pytest
import torch

from tests.chunk_util import draw
from tests.test_chunk_gpu import _cache

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _chunk(seed, B, Hq, Hkv, n, d):
    return (draw(seed, B, Hq, n, d, outliers=False).to(DEV), draw(seed + 1, B, Hkv, n, d).to(DEV),
            draw(seed + 2, B, Hkv, n, d, outliers=False).to(DEV))


def test_graphs_of_one_cache(ott):
    """Tiles cut between CTAs (their parts need more than the cache's own scratch), few rows, a windowed step; new inputs
    in place between replays, in turn on one stream."""
    B, Hq, Hkv, d, T = 1, 8, 1, 128, 40000
    c, _ = _cache(ott, "uniform", B, Hq, Hkv, d, 128, 32, 32, T, 300)
    with c:
        calls = []
        for n in (300, 2, 0):
            if n:
                x = _chunk(3, B, Hq, Hkv, n, d)
                calls.append((x, lambda out, x=x: c.chunk_attn(*x, window=30000, sinks=5, out=out), torch.zeros_like(x[0])))
            else:
                x = (draw(4, B, Hq, 1, d, outliers=False)[:, :, 0].contiguous().to(DEV),)
                calls.append((x, lambda out, x=x: c.decode_attn_window(x[0], 20000, 5, out=out), torch.zeros_like(x[0])))
        graphs = []
        for x, f, out in calls:
            f(out)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                f(out)
            graphs.append(g)
        for turn in range(3):
            want = []
            for x, f, out in calls:
                for t in x:
                    t.copy_(draw(10 * turn + t.shape[-2], *t.shape[:2], t.shape[-2] if t.dim() == 4 else 1, d, outliers=False)
                            .view(t.shape))
                want.append(f(None).clone())
                out.zero_()
            for g in graphs:
                g.replay()
            torch.cuda.synchronize()
            for (x, f, out), ref in zip(calls, want):
                assert torch.equal(out, ref), turn
        c.check_device()


@pytest.mark.parametrize("kind,T,n", [("uniform", 300, 70), ("uniform", 0, 500), ("paged", [40, 300], 90), ("cold", 200, 70)])
def test_a_serving_step_in_one_graph(ott, kind, T, n):
    B, Hq, Hkv, d, G = 2, 4, 2, 64, 32
    a, Ts = _cache(ott, kind, B, Hq, Hkv, d, G, 4, 6, T, n)
    b, _ = _cache(ott, kind, B, Hq, Hkv, d, G, 4, 6, T, n)
    q, k, v = _chunk(5, B, Hq, Hkv, n, d)
    pos = torch.arange(n, dtype=torch.int32, device=DEV).expand(1, B, n).contiguous()

    def step(c, qr, kr, out, dec):
        ott.rope(q, k, pos, (d // 2,), out_q=qr, out_k=kr)
        c.chunk_attn(qr, kr, v, out=out)
        c.append_chunk(kr, v)
        c.decode_attn_window(q[:, :, 0].contiguous(), 40, 3, out=dec)

    bufs = [[torch.zeros_like(t) for t in (q, k, q, q[:, :, 0].contiguous())] for _ in range(2)]
    with a, b:
        step(a, *bufs[0])
        a.check_device()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(b, *bufs[1])
        g.replay()
        torch.cuda.synchronize()
        b.check_device()
        for x, y in zip(*bufs):
            assert torch.equal(x, y)
        for s in range(B):
            e, f = a.export_state(s * Hkv, Hkv), b.export_state(s * Hkv, Hkv)
            for key in f:
                assert np.array_equal(e[key], f[key]), key


def test_two_caches_on_two_streams(ott):
    shapes = [(1, 8, 2, 128, 9000, 200), (2, 4, 4, 64, 3000, 150), (4, 8, 8, 128, 2000, 3)]
    caches = [_cache(ott, "uniform", B, Hq, Hkv, d, 64, 16, 8, T, n)[0] for B, Hq, Hkv, d, T, n in shapes]
    xs = [_chunk(7, B, Hq, Hkv, n, d) for B, Hq, Hkv, d, T, n in shapes]
    ref = [c.chunk_attn(*x) for c, x in zip(caches, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in shapes]
    outs = [[torch.zeros_like(x[0]) for _ in range(20)] for x in xs]
    torch.cuda.synchronize()
    for i in range(20):
        for c, x, s, o in zip(caches, xs, streams, outs):
            c.chunk_attn(*x, out=o[i], stream=s)
    torch.cuda.synchronize()
    for c, r, o in zip(caches, ref, outs):
        c.check_device()
        assert all(torch.equal(y, r) for y in o)
        c.close()
