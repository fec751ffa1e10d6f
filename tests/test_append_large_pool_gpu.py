"""Prompts of many groups beside a pool that is large for the scan's lists:
in one call, the same state as in many.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.mark.parametrize("how", ["prefill", "append_chunk"])
@pytest.mark.parametrize("P", [460, 700])
def test_many_groups_and_a_large_pool(ott, P, how):
    G, R, d, T = 16, 3, 64, 1030 * 16 + 5
    g = torch.Generator(device=DEV).manual_seed(3)
    K, V = (torch.randn(1, 1, T, d, generator=g, device=DEV).half() for _ in range(2))
    with ott.OTTCache(1, 1, 1, d, G, R, P, max_tokens=T) as a, ott.OTTCache(1, 1, 1, d, G, R, P, max_tokens=T) as b:
        getattr(a, how)(K, V)
        a.check_device()
        for t in range(0, T, 700):
            b.append_chunk(K[:, :, t:t + 700].contiguous(), V[:, :, t:t + 700].contiguous())
        b.check_device()
        e, f = a.export_state(), b.export_state()
        for key in f:
            assert np.array_equal(e[key], f[key]), key
