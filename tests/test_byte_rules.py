"""The 8-bit rules on the CPU: the plain form against brute force, the division
that decides a code, calls without a device."""
import ctypes as C
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests import byte_util as bu


def _e4m3():
    """Every finite e4m3 number, from its definition."""
    out = []
    for b in range(128):
        e, m = b >> 3, b & 7
        if b < 127:
            out.append(Fraction(m, 512) if e == 0 else Fraction(8 + m, 8) * Fraction(2) ** (e - 7))
    return out


def _nearest(r, grid):
    """Nearest number of an ascending grid, ties to the even position."""
    best = min(range(len(grid)), key=lambda i: (abs(grid[i] - r), i % 2))
    return grid[best]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_codes_against_fractions(fmt):
    grid = [Fraction(i) for i in range(128)] if fmt == "int8" else _e4m3()
    g = torch.Generator().manual_seed(1)
    for a in (1.0, 0.33349609375, 65504.0, 2.0 ** -24, 3 * 2.0 ** -24, 127.0, 254.0, 448.0):
        x = (torch.randn(1, 32, 64, generator=g) * a / 3).clamp(-a, a).half()
        x[0, 0, 0] = a
        if a in (127.0, 254.0):   # ties
            x[0, 1:9] = (torch.arange(512).reshape(8, 64) / 4).clamp(max=a).half()
        c, peak = bu.codes(x, fmt, 32)
        assert float(peak) == a
        for v, got in zip(x.reshape(-1).tolist()[:900], c.reshape(-1).tolist()):
            want = _nearest(abs(Fraction(v)) * Fraction(bu.TOP[fmt]) / Fraction(a), grid)
            assert abs(Fraction(got)) == want and (got >= 0 or v < 0), (fmt, a, v)


@pytest.mark.parametrize("top", [127.0, 448.0])
def test_a_32_bit_quotient_decides_as_the_exact_one(top):
    """The kernel's quotient (a reciprocal, one correction) against the exact one, near and on every tie of many a."""
    rng = np.random.default_rng(3)
    a = np.concatenate([rng.integers(1024, 2048, 400) * 2.0 ** rng.integers(-24, 5, 400), [65504.0, 2.0 ** -24]])
    n = 0
    for peak in a:
        ks = np.arange(0.5, top if top == 127.0 else 16.0, 1.0)
        if top == 448.0:
            ks = np.concatenate([(ks + 16) * 2.0 ** e for e in range(-9, 4)] + [ks * 2.0 ** -9])
        x = np.float16(ks * peak / top)
        x = np.unique(np.concatenate([x, np.nextafter(x, np.float16(0)), np.nextafter(x, np.float16(np.inf))]))
        x = x[x <= peak]
        f, A = x.astype(np.float32), np.float32(peak)
        p = f * np.float32(top)
        inv = np.float32(1) / A
        q = p * inv
        e = (p.astype(np.float64) - q.astype(np.float64) * np.float64(A)).astype(np.float32)        # an fma's residual
        r = (q.astype(np.float64) + e.astype(np.float64) * np.float64(inv)).astype(np.float32)
        exact = x.astype(np.float64) * top / float(peak)
        if top == 127.0:
            assert np.array_equal(np.rint(r), np.rint(exact))
        else:
            rnd = lambda z: np.rint(z / 2.0 ** (np.floor(np.log2(np.maximum(np.abs(z), 2.0 ** -6))) - 3))
            assert np.array_equal(rnd(r.astype(np.float64)), rnd(exact))
        n += len(x)
    assert n > 10000


def test_calls_without_a_handle():
    from bit_kv_cache_ott_gb300 import build
    L = C.CDLL(build.build())
    L.ott_byte_free_blocks.restype = L.ott_byte_bytes.restype = C.c_longlong
    out = C.c_void_p(1)
    big = C.c_longlong(0)
    assert L.ott_byte_create(1, 1, 1, 128, 64, 0, 100, big, None) == -1
    for bad in ((0, 1, 1, 128, 64, 0, 100), (257, 1, 1, 128, 64, 0, 100), (1, 3, 2, 128, 64, 0, 100), (1, 1, 1, 96, 64, 0, 100),
                (1, 1, 1, 128, 48, 0, 100), (1, 1, 1, 128, 64, 2, 100), (1, 1, 1, 128, 64, 0, -1), (256, 2 ** 20, 1, 128, 64, 0, 1)):
        assert L.ott_byte_create(*bad, big, C.byref(out)) == -1, bad
        assert out.value is None
    assert L.ott_byte_create(1, 1, 1, 128, 64, 0, 100, C.c_longlong(-1), C.byref(out)) == -1
    assert L.ott_byte_append(None, None, None, 1, None, None) == -1
    assert L.ott_byte_append_seq(None, 0, None, None, 1, None) == -1
    assert L.ott_byte_read(None, None, None, 0, 1, None) == -1
    assert L.ott_byte_decode(None, None, None, 0, None, None) == -1
    assert L.ott_byte_attn(None, None, None, None, None, 1, None, 0, None, None) == -1
    assert L.ott_byte_release(None, 0, None) == -1 and L.ott_byte_reset(None, None) == -1
    assert L.ott_byte_counts(None, 0, None, None) == -1 and L.ott_byte_check(None) == -1
    assert L.ott_byte_free_blocks(None) == -1 and L.ott_byte_bytes(None) == 0 and L.ott_byte_destroy(None) == 0
