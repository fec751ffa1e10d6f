"""ott_rope against the rotation in 64 bits, and its refusals.

Bound: the reduced angle is off by pos * 2^-53 of its turns (the 53-bit
frequency) and 2^-25 of half a turn (32 bits as a float), 2^-20 at most here;
sine and cosine by two units of fp32; the products and the sum add three fp32
roundings of the pair's size; the result is rounded once to fp16 (half a step,
2^-11 relative, 2^-25 below the normal range).
"""
import ctypes as C
import math

import pytest
import torch

import bit_kv_cache_ott_gb300 as pkg

DEV = "cuda"


def plain(x, pos, sections, base, interleaved, restart):
    half = sum(sections)
    y = x.double().clone()
    i = 0
    for a, m in enumerate(sections):
        for j in range(m):
            e = j / m if restart else i / half
            th = (pos[a].double() * base ** -e).unsqueeze(1)
            l, r = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
            x0, x1 = x[..., l].double(), x[..., r].double()
            y[..., l], y[..., r] = x0 * th.cos() - x1 * th.sin(), x0 * th.sin() + x1 * th.cos()
            i += 1
    size = torch.zeros_like(y)
    for i in range(half):
        l, r = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        size[..., l] = size[..., r] = x[..., l].double().abs() + x[..., r].double().abs()
    return y, 2.0 ** -11 * y.abs() * 1.001 + 2.0 ** -25 + 2.0 ** -20 * size


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,n,d,sections,base,interleaved,restart,far", [
    (1, 1, 1, 1, 128, (64,), 10000.0, False, False, 0),
    (32, 32, 32, 1, 128, (16, 24, 24), 10000.0, False, False, 100000),
    (2, 8, 2, 333, 128, (16, 24, 24), 1e6, False, False, 2 ** 31 - 1),
    (2, 5, 1, 77, 64, (16, 16), 10000.0, True, True, 1000),
    (1, 3, 3, 50, 64, (8, 8), 10000.0, True, True, 100000),       # half of the channels copied
    (1, 3, 3, 50, 64, (8, 8), 10000.0, False, False, 100000),
    (3, 2, 2, 19, 64, (5, 7, 1, 2), 500000.0, False, True, 10),   # 15 pairs: no whole vectors
    (3, 2, 2, 19, 80, (5, 7, 1, 2), 500000.0, True, False, 10),
    (1, 2, 1, 4097, 256, (128,), 10000.0, False, False, 5000),
    (2, 7, 0, 9, 16, (4, 4), 1.0, False, False, 3),               # queries only; base 1
    (2, 0, 7, 9, 32, (16,), 10000.0, True, False, 3),
])
def test_rope(ott, B, Hq, Hkv, n, d, sections, base, interleaved, restart, far):
    g = torch.Generator().manual_seed(n + d)
    q = torch.randn(B, Hq, n, d, generator=g).half() if Hq else None
    k = torch.randn(B, Hkv, n, d, generator=g).half() if Hkv else None
    pos = torch.randint(-far, far + 1, (len(sections), B, n), generator=g, dtype=torch.int64).int()
    dev = [None if t is None else t.to(DEV) for t in (q, k)]
    outs = ott.rope(*dev, pos.to(DEV), sections, base, interleaved, restart)
    for x, xd, o in zip((q, k), dev, outs):
        if x is None:
            assert o is None
            continue
        ref, tol = plain(x, pos, sections, base, interleaved, restart)
        d_ = (o.double().cpu() - ref).abs()
        assert bool((d_ <= tol).all()), f"{(d_ - tol).max().item():.3e} over the bound"
        assert torch.equal(xd.cpu(), x)
        if 2 * sum(sections) < d:
            assert torch.equal(o[..., 2 * sum(sections):].cpu(), x[..., 2 * sum(sections):])
    # in place
    res = ott.rope(*dev, pos.to(DEV), sections, base, interleaved, restart, out_q=dev[0], out_k=dev[1])
    for o, r in zip(outs, res):
        assert o is r or torch.equal(o, r)


def _plan(sections=(32,), axes=None, base=10000.0):
    return pkg.RopePlan(len(sections) if axes is None else axes, (C.c_int * 4)(*sections), base, 0, 0)


def test_refusals():
    """Every refusal comes before the device is touched, so a host has them all."""
    L = pkg.load(build_if_missing=True)
    a, b, p = 1 << 20, 1 << 24, 1 << 28   # addresses that nothing reads

    def call(q=a, qo=a, Hq=2, k=b, ko=b, Hkv=1, pos=p, B=1, n=4, d=64, plan=_plan()):
        return L.ott_rope(q, qo, Hq, k, ko, Hkv, pos, B, n, d, None if plan is None else C.byref(plan), None)

    assert call(n=0) == pkg.OTT_OK
    bad = [dict(plan=None), dict(B=0), dict(n=-1), dict(Hq=0, Hkv=0), dict(Hq=-1), dict(d=24), dict(d=272), dict(d=0),
           dict(q=None), dict(qo=None), dict(k=None), dict(pos=None), dict(pos=p + 2), dict(q=a + 8), dict(qo=a + 16),
           dict(ko=b - 32), dict(plan=_plan((33,))), dict(plan=_plan((20, 20))), dict(plan=_plan((0, 32))),
           dict(plan=_plan((32,), axes=0)), dict(plan=_plan((8, 8, 8, 8), axes=5)), dict(plan=_plan(base=0.5)),
           dict(plan=_plan(base=math.inf)), dict(plan=_plan(base=math.nan))]
    for kw in bad:
        assert call(**kw) == pkg.OTT_ERR_INVALID, kw


def test_outputs_apart_from_everything_else():
    """An output on the other operand, on the other output or on the positions is refused; neighbours are not."""
    L = pkg.load(build_if_missing=True)
    a, nq, nk = 1 << 20, 2 * 4 * 64 * 2, 4 * 64 * 2   # two heads of four tokens, one head
    o, pos = 1 << 24, 1 << 28
    plan = _plan()

    def call(q, qo, k, ko, pos, n=4):
        return L.ott_rope(q, qo, 2, k, ko, 1, pos, 1, n, 64, C.byref(plan), None)

    for q, qo, k, ko, ps in [(a, o, o, o, pos), (a, o, o + nq - 16, o + nq - 16, pos), (a, o, o + (1 << 20), o + nq - 16, pos),
                             (a, a, o, a + 16, pos), (a, a, o, a + nq - 16, pos), (a, o, a + (1 << 19), a - nk + 16, pos),
                             (a, o, o + nq, o + nq, o), (a, o, o + nq, o + nq, o + nq + nk - 4)]:
        assert call(q, qo, k, ko, ps) == pkg.OTT_ERR_INVALID, (q, qo, k, ko, ps)


def test_null_caches_are_refused():
    L = pkg.load(build_if_missing=True)
    assert L.ott_chunk_attn(None, None, None, None, None, 1, None, 0, 0, None) == pkg.OTT_ERR_INVALID
    assert L.ott_append_chunk(None, None, None, 1, None, None) == pkg.OTT_ERR_INVALID
    assert L.ott_decode_attn_window(None, None, None, 1, 0, None) == pkg.OTT_ERR_INVALID


def test_binding_refuses_before_the_library():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.float16)
    pos = torch.zeros(1, 1, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkg.rope(None, None, pos, (32,))
    with pytest.raises(TypeError):
        pkg.rope(x, None, pos, (32,))          # CPU tensors
    with pytest.raises(ValueError):
        pkg.rope(x, None, pos, ())
