"""Whole numbers of the chunk calls that do not fit the C ABI's 32 bits are
refused, not wrapped (ctypes would drop their upper bits).
"""
import types

import pytest

import bit_kv_cache_ott_gb300 as pkg


@pytest.mark.parametrize("x", [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1, 2 ** 63])
def test_lengths(x):
    with pytest.raises(ValueError):
        pkg.OTTCache._lens(types.SimpleNamespace(B=2), [1, x])


@pytest.mark.parametrize("x", [2 ** 32 + 5, -2 ** 32 + 16])
def test_rope_sections(x):
    with pytest.raises(ValueError):
        pkg._rope_plan((16, x), 10000.0, False, False)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(window=2 ** 32 + 1), dict(window=2 ** 31), dict(window=3, sinks=2 ** 32)])
def test_windows(ott, kw):
    import torch
    q = torch.zeros(1, 1, 1, 64, dtype=torch.float16, device="cuda")
    with ott.OTTCache(1, 1, 1, 64, 16, 4, 5, max_tokens=10) as c:
        c.append_chunk(q, q)
        with pytest.raises(ValueError):
            c.chunk_attn(q, q, q, **kw)
        with pytest.raises(ValueError):
            c.decode_attn_window(q[:, :, 0].contiguous(), **kw)
        c.decode_attn_window(q[:, :, 0].contiguous(), window=2 ** 31 - 1)
        c.check_device()
