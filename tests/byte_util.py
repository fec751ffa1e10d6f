"""The cache held in 8 bits in plain 64-bit form, and the error bounds that its
kernels' arithmetic allows."""
from __future__ import annotations

import torch

TOP = {"int8": 127.0, "e4m3": 448.0}


def codes(x, fmt, G):
    """Complete blocks of x [..][T][d] (fp16): (codes, as the numbers they are, [..][nb][G][d]; a = max |x| of each
    block [..][nb][1][1]), 64 bits."""
    *lead, T, d = x.shape
    nb = T // G
    t = x[..., :nb * G, :].double().reshape(*lead, nb, G, d)
    a = t.abs().amax((-2, -1), keepdim=True) if nb else t.new_zeros(*lead, 0, 1, 1)
    r = t * TOP[fmt] / torch.where(a > 0, a, torch.ones_like(a))   # products exact, one rounding far below a tie's distance
    if fmt == "int8":
        return r.round(), a
    e = torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return (r / step).round() * step, a


def held(x, fmt, G):
    """What the cache stands for after tokens x [..][T][d], 64 bits, and per token the value scale (0: fp16)."""
    c, a = codes(x, fmt, G)
    y = x.double().clone()
    n = c.shape[-3] * G
    y[..., :n, :] = (c * a / TOP[fmt]).reshape(*x.shape[:-2], n, x.shape[-1])
    s = torch.zeros(x.shape[:-1], dtype=torch.float64)
    s[..., :n] = (a / TOP[fmt]).reshape(*x.shape[:-2], -1).repeat_interleave(G, -1)
    return y, s


def read_back(x, fmt, G):
    """What ott_byte_read gives: fp16(fp32(code) * scale), the scale rounded to fp32."""
    c, a = codes(x, fmt, G)
    s = (a / TOP[fmt]).float()        # a has 11 bits: rounded from 53 as from all
    y = x.clone()
    n = c.shape[-3] * G
    y[..., :n, :] = (c.float() * s).half().reshape(*x.shape[:-2], n, x.shape[-1])
    return y


def same(a, b):
    """Equal numbers (a zero's sign is lost in an int8 code, and may be in an e4m3 one)."""
    return bool((a.cpu() == b.cpu()).all())


def attend(q, K, V, fmt, G, k=None, v=None, chosen=None):
    """One sequence: q [Hq][n][d] over its tokens K, V [Hkv][T][d] and, causally, new ones k, v [Hkv][n][d]; chosen
    [n][Hkv]: lists of the complete blocks that are attended. Returns (out, tol), 64 bits.

    tol, element by element, with A = sum w |v|: a weight times its value scale is rounded to fp16 once, half a step,
    2^-11, and the result once more. A weight is held down to 2^-25, taken at least 2^7 above the largest: 2^-32 of the largest product
    of weight and scale per code (at most 448; an fp16 value counts as its own code). A logit is a sum of d products
    of exact numbers in fp32 (d/16 + 2 accumulations, each off by at most 2^-22 of the sum of magnitudes, truncation
    allowed), then scale, multiply-add, difference: six roundings of numbers up to its size and log2 of the scale (at
    most 40), and 2^x is good to 2^-21; an error e in the logits moves each weight by e and their sum by e. Sums on the
    tensor cores lose up to 6e-9 of themselves per token."""
    Hq, n, d = q.shape
    Hkv, T = K.shape[:2]
    g = Hq // Hkv
    Kh, _ = held(K, fmt, G)
    Vh, S = held(V, fmt, G)
    out = torch.zeros(Hq, n, d, dtype=torch.float64)
    tol = torch.zeros_like(out)
    m = 0 if k is None else k.shape[1]
    for h in range(Hq):
        hk = h // g
        Kx, Vx, sx = Kh[hk], Vh[hk], S[hk]
        if m:
            Kx, Vx = torch.cat([Kx, k[hk].double()]), torch.cat([Vx, v[hk].double()])
            sx = torch.cat([sx, torch.zeros(m, dtype=torch.float64)])
        see = torch.arange(T + m) <= (T + torch.arange(n)[:, None] if m else T)
        see = see.expand(n, -1).clone()
        if chosen is not None:
            for i in range(n):
                for j in range(T // G):
                    if j not in chosen[i][hk]:
                        see[i, j * G:(j + 1) * G] = False
        lg = (q[h].double() @ Kx.t()) / d ** 0.5
        mag = ((q[h].double().abs() @ Kx.abs().t()) / d ** 0.5).masked_fill(~see, 0).amax(1, keepdim=True)
        w = torch.softmax(lg.masked_fill(~see, -float("inf")), 1)
        o, A = w @ Vx, w @ Vx.abs()
        e = (d / 16 + 4) * 2.0 ** -21 * mag + 6 * 2.0 ** -23 * (mag + 40) + 2.0 ** -21
        big = (w * torch.where(sx > 0, sx * 448, Vx.abs().amax(1))).amax(1, keepdim=True)
        out[h] = o
        tol[h] = 2.0 ** -11 * (A + o.abs()) * 1.01 + 2 * e * A + 6e-9 * (T + m) * A + 2.0 ** -32 * 448 * (T + m) * big + 2.0 ** -24
    return out, tol


def bounds(q, K, G):
    """Block bounds of q [Hq][n][d] over K [Hkv][T][d]: [n][Hkv][nb], 32-bit sums in channel order."""
    Hq, n, d = q.shape
    Hkv, T = K.shape[:2]
    nb, g = T // G, Hq // Hkv
    blk = K[:, :nb * G].reshape(Hkv, nb, G, d).float()
    lo, hi = blk.amin(2), blk.amax(2)
    qf = q.float().reshape(Hkv, g, n, 1, d)
    s = torch.zeros(Hkv, g, n, nb)
    for c in range(d):
        s = s + torch.maximum(qf[..., c] * lo[:, None, None, :, c], qf[..., c] * hi[:, None, None, :, c])
    return s.amax(1).permute(1, 0, 2)


def choose(q, K, G, topk):
    """The blocks that each token and kv head selects: [n][Hkv] ascending lists."""
    b = bounds(q, K, G)
    return [[sorted(sorted(range(b.shape[2]), key=lambda j: (-float(x[j]), j))[:topk]) for x in row] for row in b]
