"""Chunk attention over caches so long that the sums themselves can go wrong."""
import math

import pytest
import torch

from tests.chunk_util import unit_tokens

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def test_sums_over_a_million_tokens_do_not_shrink(ott):
    """8,192 new tokens of eight heads over 2^20: 256 pairs of row tiles, each of 9,400 steps of 112 tokens.

    The tensor cores truncate as they add, so a long sum of values of one sign comes out too small; sums have to be
    short enough, and joined in fp32. Required: the outputs of a call are too small by a third of their own largest
    rounding (2^-11) at most. Each output's rounding is uniform over +-2^-11 at most: 2,048 rows of 64 channels, whose
    outputs differ by far more than a rounding, leave 2^-11 / sqrt(3 * 131072) of it, 1e-6."""
    T, n, Hq, d = 1 << 20, 8192, 8, 64
    g = torch.Generator(device=DEV).manual_seed(5)
    K = torch.randn(1, 1, T, d, generator=g, device=DEV).half()
    V = (2 + K).half()   # a query's output is about 2 + q / 8, so rows differ
    q = torch.randn(1, Hq, n, d, generator=g, device=DEV).half()
    k = torch.randn(1, 1, n, d, generator=g, device=DEV).half()
    v = (2 + k).half()
    with ott.OTTCache(1, Hq, 1, d, 128, 32, 32, max_tokens=T) as c:
        c.prefill(K, V)
        out = c.chunk_attn(q, k, v)
        c.check_device()
        (Kc, Vc, idx, _), = unit_tokens(c, 0)[0]
    Kc, Vc = torch.cat([Kc.to(DEV), k[0, 0].double()]), torch.cat([Vc.to(DEV), v[0, 0].double()])
    idx = torch.cat([idx, T + torch.arange(n)]).to(DEV)
    num = den = 0.0
    for i in range(0, n, 32):   # eight rows at a time
        lg = (q[0, :, i].double() @ Kc.t() / math.sqrt(d)).masked_fill(idx > T + i, -math.inf)
        ref = torch.softmax(lg, 1) @ Vc
        o = out[0, :, i].double()
        num += float((o * ref).sum())
        den += float((ref * ref).sum())
    shrink = 1 - num / den
    assert abs(shrink) <= 2.0 ** -11 / 3, f"outputs are {shrink:.2e} too small"


def test_sums_of_few_rows_over_many_long_caches(ott):
    """76 x 32 units of 131,072 tokens: a unit each for the warps of up to 16 rows per kv head. The same requirement."""
    B, H, d, T = 76, 32, 64, 131072
    g = torch.Generator(device=DEV).manual_seed(5)
    K = torch.randn(1, H, T, d, generator=g, device=DEV).half()
    with ott.OTTCache(B, H, H, d, 128, 32, 32, max_tokens=T, ragged=True) as c:
        for b in range(B):
            c.prefill_seq(b, K[0], 2 + K[0])
        del K
        units, _ = unit_tokens(c, 0)
        units = [tuple(x.to(DEV) for x in units[h][:3]) for h in range(0, H, 4)]
        for n in (1, 4, 8, 16):
            q, k = (torch.randn(B, H, n, d, generator=g, device=DEV).half() for _ in range(2))
            v = 2 + k
            out = c.chunk_attn(q, k, v)
            c.check_device()
            num = den = 0.0
            for h in range(0, H, 4):
                Kd, Vd = torch.cat([units[h // 4][0], k[0, h].double()]), torch.cat([units[h // 4][1], v[0, h].double()])
                idx = torch.cat([units[h // 4][2], T + torch.arange(n, device=DEV)])
                hide = idx > (T + torch.arange(n, device=DEV))[:, None]
                ref = torch.softmax((q[0, h].double() @ Kd.t() / math.sqrt(d)).masked_fill(hide, -math.inf), 1) @ Vd
                num += float((out[0, h].double() * ref).sum())
                den += float((ref * ref).sum())
            # 8 n rows of 64 channels: their roundings leave 2^-11 / sqrt(3 * 512 n), 5e-6 at n = 4 and 1.3e-5 at 1
            assert abs(1 - num / den) <= 2.0 ** -11 / 3, f"{n} rows: outputs are {1 - num / den:.2e} too small"


#    B  Hq  Hkv d    G    T       n     window  sinks
LONG = [
    (1, 8, 1, 64, 128, 131072, 1100, 0, 0),         # more than 32 pairs per head, tiles over several CTAs and sums
    (1, 8, 1, 64, 128, 131072, 1100, 100000, 200),
    (1, 32, 32, 64, 128, 131072, 100, 0, 0),        # one tile of rows
    (1, 16, 4, 128, 256, 60000, 700, 0, 0),
]


@pytest.mark.parametrize("B,Hq,Hkv,d,G,T,n,window,sinks", LONG)
def test_rows_over_long_caches(ott, B, Hq, Hkv, d, G, T, n, window, sinks):
    """Sampled rows, element by element: the bound of tests/chunk_util.py, but 2^-32 of the row's largest weight per token
    (twice that allowed), and the sums' 2^-11 / 3 (above); one query is NaN."""
    g = torch.Generator(device=DEV).manual_seed(9)
    K, V = (torch.randn(B, Hkv, T, d, generator=g, device=DEV).half() for _ in range(2))
    K[:, :, 17::5000] *= 0.03
    q, k, v = (torch.randn(B, h, n, d, generator=g, device=DEV).half() for h in (Hq, Hkv, Hkv))
    q[:, Hq - 1, n // 2, 1] = float("nan")
    with ott.OTTCache(B, Hq, Hkv, d, G, 32, 32, max_tokens=T) as c:
        c.prefill(K, V)
        del K, V
        out = c.chunk_attn(q, k, v, window=window, sinks=sinks)
        c.check_device()
        units, _ = unit_tokens(c, 0)
    rep = Hq // Hkv
    assert bool(out[0, Hq - 1, n // 2].isnan().all())
    for h in sorted({0, Hkv // 2, Hkv - 1}):
        Kd, Vd = torch.cat([units[h][0].to(DEV), k[0, h].double()]), torch.cat([units[h][1].to(DEV), v[0, h].double()])
        idx = torch.cat([units[h][2], T + torch.arange(n)]).to(DEV)
        for hh in (h * rep, h * rep + rep - 1):
            rows = torch.tensor(sorted({0, 1, 31, 32, 97, n // 3, n // 2 + 1, n - 2, n - 1}), device=DEV)
            p = (T + rows)[:, None]
            see = idx <= p
            if window:
                see &= (idx > p - window) | (idx < sinks)
            qd = q[0, hh, rows].double()
            mag = ((qd.abs() @ Kd.abs().t()) / d ** 0.5).masked_fill(~see, 0).amax(1, keepdim=True)
            w = torch.softmax((qd @ Kd.t() / d ** 0.5).masked_fill(~see, -math.inf), 1)
            ref, A = w @ Vd, w @ Vd.abs()
            e = (d / 16 + 4) * 2.0 ** -22 * 2 * mag + 3 * 2.0 ** -23 * mag + 2.0 ** -21
            tol = 2.0 ** -11 * (2 * A + ref.abs() + A / 3) * 1.01 + 2 * e * A + 2.0 ** -31 * (see.double() @ Vd.abs()) + 2.0 ** -24
            got = out[0, hh, rows].double()
            assert bool(got.isfinite().all()), (h, hh)
            assert bool(((got - ref).abs() <= tol).all()), (h, hh, ((got - ref).abs() - tol).max().item())
