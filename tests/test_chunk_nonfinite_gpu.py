"""A query that is not finite: NaN in its own rows of the output, as
ott_decode_attn gives it, and nothing changed in any other row, whichever
kernel serves the call and however its work is cut.
"""
import pytest
import torch

from tests.chunk_util import draw
from tests.test_chunk_gpu import _cache

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
NAN, INF = float("nan"), float("inf")

#   B  Hq Hkv d    G    T     n   window sinks
CALLS = [
    (2, 2, 2, 128, 32, 300, 1, 0, 0),       # up to four rows: the decode kernel
    (1, 8, 2, 64, 16, 300, 1, 90, 20),
    (1, 2, 2, 128, 32, 0, 4, 0, 0),         # an empty cache
    (1, 1, 1, 64, 16, 3000, 2, 0, 0),       # one unit over many warps
    (2, 8, 2, 128, 32, 300, 2, 0, 0),       # 5 to 16 rows
    (1, 4, 1, 64, 16, 900, 4, 90, 20),
    (1, 2, 2, 64, 16, 0, 9, 0, 0),
    (1, 8, 1, 128, 128, 5000, 2, 0, 0),
    (2, 2, 1, 64, 32, 300, 40, 0, 0),       # more: tiles, whole
    (1, 2, 2, 128, 32, 0, 70, 0, 0),
    (1, 4, 2, 128, 128, 9000, 33, 0, 0),    # tiles cut between CTAs
    (1, 4, 2, 64, 32, 3000, 33, 500, 40),
]


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("B,Hq,Hkv,d,G,T,n,window,sinks", CALLS)
def test_a_query_that_is_not_finite(ott, B, Hq, Hkv, d, G, T, n, window, sinks, bad):
    c, _ = _cache(ott, "uniform", B, Hq, Hkv, d, G, 4, 6, T, n)
    with c:
        q, k, v = draw(7, B, Hq, n, d, outliers=False), draw(8, B, Hkv, n, d), draw(9, B, Hkv, n, d, outliers=False)
        k[..., 3] = k[..., 3].abs() + 1   # on an empty cache, an infinity there makes every score +inf or -inf
        kd, vd = k.to(DEV), v.to(DEV)
        ref = c.chunk_attn(q.to(DEV), kd, vd, window=window, sinks=sinks).cpu()
        hit = torch.zeros(B, Hq, n, dtype=torch.bool)
        hit[B - 1, Hq - 1, n - 1] = hit[0, 0, n // 2] = True
        qb = q.clone()
        qb[..., 3][hit] = bad
        out = c.chunk_attn(qb.to(DEV), kd, vd, window=window, sinks=sinks).cpu()
        c.check_device()
        assert bool(out[hit].isnan().all()), "finite values for a query that is not"
        assert torch.equal(out[~hit], ref[~hit]), "another row changed"


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("Hq,Hkv,T,window", [(2, 2, 300, 0), (2, 2, 300, 64), (8, 2, 20, 7), (12, 1, 2000, 300), (40, 1, 20, 0),
                                             (40, 1, 2000, 300), (1, 1, 3, 1)])
def test_a_windowed_step(ott, Hq, Hkv, T, window, bad):
    c, _ = _cache(ott, "uniform", 2, Hq, Hkv, 64, 32, 4, 6, T, 1)
    with c:
        q = draw(11, 2, Hq, 1, 64, outliers=False)[:, :, 0].contiguous()
        ref = c.decode_attn_window(q.to(DEV), window).cpu()
        qb = q.clone()
        qb[1, Hq - 1, 3] = bad
        out = c.decode_attn_window(qb.to(DEV), window).cpu()
        full = c.decode_attn(qb.to(DEV)).cpu()
        c.check_device()
        assert bool(full[1, Hq - 1].isnan().all())
        assert bool(out[1, Hq - 1].isnan().all()), "finite values for a query that is not"
        out[1, Hq - 1] = ref[1, Hq - 1]
        assert torch.equal(out, ref), "another row changed"


@pytest.mark.parametrize("Hq,n", [(1, 3), (3, 3), (4, 20)])
def test_every_score_minus_infinity(ott, Hq, n):
    """Queries of which every score is -inf (no finite key can cause it): NaN, in chunks and in windowed steps."""
    with ott.OTTCache(1, Hq, 1, 64, 32, 4, 6, max_tokens=100) as c:
        q, k = torch.ones(1, Hq, n, 64, dtype=torch.float16), torch.ones(1, 1, n, 64, dtype=torch.float16)
        q[..., 5] = -INF
        assert bool(c.chunk_attn(q.to(DEV), k.to(DEV), k.to(DEV)).isnan().all())
        c.append_chunk(k.to(DEV), k.to(DEV))
        q1 = q[:, :, 0].contiguous().to(DEV)
        assert bool(c.decode_attn(q1).isnan().all())
        assert bool(c.decode_attn_window(q1, 2).isnan().all())
        assert bool(c.decode_attn_window(torch.ones_like(q1), 2).eq(1.0).all())
        c.check_device()
