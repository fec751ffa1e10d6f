"""Outputs of the chunk calls that share memory with their inputs, in part or
whole, are refused; outputs that end where an input begins are not.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
B, Hq, Hkv, n, d = 2, 4, 2, 9, 64
NQ, NK = B * Hq * n * d, B * Hkv * n * d


def _view(buf, at, heads, rows=n):
    shape = (B, heads, rows, d) if rows else (B, heads, d)
    return buf[at:at + B * heads * max(rows, 1) * d].view(shape)


#   q, k, v, out: first elements in one buffer
@pytest.mark.parametrize("at,ok", [
    ((0, NQ, NQ + NK, NQ + 2 * NK), True),              # one behind the other
    ((NQ, 2 * NQ, 2 * NQ + NK, 0), True),               # the output first, up to the queries
    ((0, NQ, NQ + NK, 0), False),
    ((0, 2 * NQ, 2 * NQ + NK, NQ - 8), False),          # the queries' last 16 bytes
    ((NQ - 8, 2 * NQ, 2 * NQ + NK, 0), False),
    ((0, NQ, 3 * NQ, NQ + NK - 8), False),              # the keys' last
    ((0, 2 * NQ - 8, 3 * NQ, NQ), False),               # the keys' first
    ((0, NQ, NQ + NK, NQ + 2 * NK - 8), False),         # the values' last
    ((0, 3 * NQ, 2 * NQ - 8, NQ), False),               # the values' first
])
def test_chunk_attn(ott, at, ok):
    buf = torch.zeros(5 * NQ, dtype=torch.float16, device=DEV)
    q, k, v, out = (_view(buf, a, h) for a, h in zip(at, (Hq, Hkv, Hkv, Hq)))
    with ott.OTTCache(B, Hq, Hkv, d, 16, 4, 5, max_tokens=10) as c:
        if ok:
            c.chunk_attn(q, k, v, out=out)
        else:
            with pytest.raises(ott.OTTError) as e:
                c.chunk_attn(q, k, v, out=out)
            assert e.value.code == ott.OTT_ERR_INVALID
        c.append_chunk(k, v)   # the cache still serves
        c.check_device()


@pytest.mark.parametrize("off,ok", [(0, False), (8, False), (B * Hq * d - 8, False), (B * Hq * d, True)])
@pytest.mark.parametrize("swap", [False, True])
def test_decode_attn_window(ott, off, ok, swap):
    buf = torch.zeros(2 * B * Hq * d, dtype=torch.float16, device=DEV)
    q, out = _view(buf, 0, Hq, 0), _view(buf, off, Hq, 0)
    if swap:
        q, out = out, q
    kv = torch.zeros(B, Hkv, 3, d, dtype=torch.float16, device=DEV)
    with ott.OTTCache(B, Hq, Hkv, d, 16, 4, 5, max_tokens=10) as c:
        c.append_chunk(kv, kv)
        if ok:
            c.decode_attn_window(q, 2, out=out)
        else:
            with pytest.raises(ott.OTTError) as e:
                c.decode_attn_window(q, 2, out=out)
            assert e.value.code == ott.OTT_ERR_INVALID
        c.check_device()
