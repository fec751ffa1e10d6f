"""Chunk attention over the whole range of keys that a cache takes."""
import pytest
import torch

from tests.chunk_util import attend, check

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.mark.parametrize("n,Hq", [(1, 2), (5, 2), (40, 2), (16, 32)])
def test_the_largest_keys(ott, n, Hq):
    """Keys over the whole of fp16 (a channel from -65,504 to 65,504: a scale of 43,680) on every path, values up to 65,440."""
    B, H, d = 1, 2, 64
    K = (torch.rand(B, H, 200, d, generator=torch.Generator().manual_seed(1)) * 2 - 1) * 65504
    V = (torch.rand(B, H, 200, d, generator=torch.Generator().manual_seed(2)) * 2 - 1) * 65440
    K[:, :, 0::7, ::3], K[:, :, 3::7, ::3] = 65504, -65504
    V[..., 0], V[..., 1] = 65440, -65440
    K[..., 2] = torch.randn(B, H, 200, generator=torch.Generator().manual_seed(4))   # beside small ones
    K, V = K.half(), V.half()
    q = (torch.randn(B, Hq, n, d, generator=torch.Generator().manual_seed(3)) / 16384).half()
    with ott.OTTCache(B, Hq, H, d, 32, 4, 6, max_tokens=300) as c:
        c.prefill(K.to(DEV), V.to(DEV))
        k, v = K[:, :, 2:2 + n].contiguous(), V[:, :, 2:2 + n].contiguous()
        for window, sinks in ((0, 0), (150, 3)):
            out = c.chunk_attn(q.to(DEV), k.to(DEV), v.to(DEV), window=window, sinks=sinks)
            ref, tol = attend(c, 0, q[0], 200, window, sinks, k[0], v[0], folded=n * Hq // H <= 4)
            check(out[0], ref, tol)
        q1 = q[:, :, 0].contiguous()
        out = c.decode_attn_window(q1.to(DEV), 150, 3)
        ref, tol = attend(c, 0, q[0, :, :1], 199, 150, 3, folded=Hq // H <= 4)
        check(out[0].unsqueeze(1), ref, tol)
        c.check_device()
