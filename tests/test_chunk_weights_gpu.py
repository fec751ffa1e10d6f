"""Chunk attention with weights far below a row's largest."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


#                    B   Hkv g  n
@pytest.mark.parametrize("B,Hkv,g,n,T", [(38, 64, 1, 8, 1024), (38, 32, 2, 8, 1024), (1, 1, 8, 4864, 16384)])
def test_small_weights_beside_a_large_one(ott, B, Hkv, g, n, T):
    """Token 0 has the largest weight, every other token 2^-25.5 of it; a unit's tokens are one warp's or CTA's.

    Keys 12, 0, 0 .. in one channel dequantize exactly, values are 0 for token 0 and 1 for the others, so with N others
    in sight the output is N w / (1 + N w). Weights are held in steps of 2^-24 where the row's largest is at least 2^7:
    2^-32 per token. The sums' and roundings' part: two roundings of 2^-11; a logit of 17.7 off by
    (d / 16 + 4) 2^-22 * 2 of it and 2^-21, twice; subnormal outputs in steps of 2^-24."""
    d = 64
    K = torch.zeros(B, Hkv, T, d, dtype=torch.float16, device=DEV)
    V = torch.ones(B, Hkv, T, d, dtype=torch.float16, device=DEV)
    K[:, :, 0, 7], V[:, :, 0] = 12.0, 0.0
    q = torch.zeros(B, Hkv * g, n, d, dtype=torch.float16, device=DEV)
    q[..., 7] = 25.5 * math.log(2) * 8 / 12
    k, v = torch.zeros(B, Hkv, n, d, dtype=torch.float16, device=DEV), torch.ones(B, Hkv, n, d, dtype=torch.float16, device=DEV)
    with ott.OTTCache(B, Hkv * g, Hkv, d, 128, 0, 0, max_tokens=T) as c:
        c.prefill(K, V)
        del K, V
        out = c.chunk_attn(q, k, v).double()
        c.check_device()
    lg = float(q[0, 0, 0, 7]) * 12 / 8
    N = T + torch.arange(n, device=DEV, dtype=torch.float64)
    w = math.exp(-lg)
    ref = (N * w / (1 + N * w))[None, None, :, None].expand_as(out)
    e = (d / 16 + 4) * 2.0 ** -22 * 2 * lg + 2.0 ** -21
    tol = (2 * 2.0 ** -11 + 2 * e) * 1.01 * ref + 2.0 ** -32 * N[None, None, :, None] * 1.01 + 2.0 ** -25
    over = ((out - ref).abs() - tol).max().item()
    assert over <= 0, f"{over:.3e} over the bound; {out.flatten()[0].item():.4e} for {ref.flatten()[0].item():.4e}"
