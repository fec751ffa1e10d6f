"""The chunk operators' plain 64-bit form, over an exported cache state, with
the error bound that their arithmetic allows.

The state's own correctness (codes, pool, tokens) is the parity tests' matter;
here the exported arrays say what the cache stands for.
"""
from __future__ import annotations

import numpy as np
import torch


def draw(seed, B, H, n, d, rate=0.05, outliers=True):
    """fp16 [B][H][n][d] with four large channels and a few tokens of small norm."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, H, n, d, generator=g)
    if outliers:
        x[..., torch.randperm(d, generator=g)[:4]] *= 15
        x[torch.rand(B, H, n, generator=g) < rate] *= 0.03
    return x.half()


def _f16(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.float16).astype(np.float64))


def unit_tokens(c, b):
    """Sequence b's tokens as the cache holds them: per kv head (keys, values, token indices, value scales), 64 bits."""
    e = c.export_state(b * c.Hkv, c.Hkv)
    out = []
    d, nf, T, nt, npool = c.d, e["nf"], e["T"], e["tail"], e["npool"]
    sh = np.arange(4) * 2
    for h in range(c.Hkv):
        K, V, idx, S = [], [], [], []
        for j in range(nf):
            cnt = int(e["bcount"][h][j]) if c.cold is not None else int(e["bcount"][j])
            if cnt == 0:
                continue
            code = lambda a: torch.from_numpy((((a[h, j, :cnt, :, None] >> sh) & 3).reshape(cnt, d)).astype(np.float64))
            ks, kz = _f16(e["ks"][h, j]), _f16(e["kz"][h, j])
            vs, vz = (_f16(e[x][h, j, :cnt]).repeat_interleave(32, 1) for x in ("vs", "vz"))
            K.append(kz + ks * code(e["kcode"]))
            V.append(vz + vs * code(e["vcode"]))
            S.append(vs)
            idx.append(torch.from_numpy(e["bidx"][h, j, :cnt].astype(np.int64)))
        K += [_f16(e["tk"][h]), _f16(e["pk"][h, :npool])]
        V += [_f16(e["tv"][h]), _f16(e["pv"][h, :npool])]
        idx += [torch.arange(T - nt, T), torch.from_numpy(e["pidx"][h, :npool].astype(np.int64))]
        if c.cold is not None:
            m = int(e["ncold"][h])
            K.append(_f16(e["ck"][h, :m]))
            V.append(_f16(e["cv"][h, :m]))
            idx.append(torch.from_numpy(e["cidx"][h, :m].astype(np.int64)))
        K, V, idx = torch.cat(K).view(-1, d), torch.cat(V).view(-1, d), torch.cat(idx)
        S = torch.cat(S + [torch.zeros(0, d, dtype=torch.float64)])
        out.append((K, V, idx, torch.cat([S, torch.zeros(len(idx) - len(S), d, dtype=torch.float64)])))
    return out, T


def attend(c, b, q, pos0, window, sinks, k=None, v=None, folded=False):
    """q [Hq][n][d] (fp16, CPU) at positions pos0.., with new tokens k, v [Hkv][n][d] behind the cache's: (out, tol).

    tol, element by element: the weights and the values carry one fp16 rounding each (half a step, 2^-11 relative), the
    result another. A weight below 2^-14 of the row's largest is held in steps of 2^-24 of it: 2^-25 per token and
    value. A logit is a sum of d products in fp32 (d/16 + 2 accumulations, each off by at most 2^-22 of the sum of
    magnitudes, truncation allowed) and three more fp32 operations (2^-23 of its size); the offsets' low part is cut
    at 2^-22 of theirs, and 2^x is good to 2^-21. An error e in the logits moves each weight by e and their sum by
    e: 2 e in all.

    folded (calls of up to four rows per kv head, as ott_decode_attn): a value is not rounded but taken as w s code +
    w z, its code an fp16 subnormal of 2^-24 per unit. Tensor cores align what they add to the operands' exponents, a
    subnormal's being 2^-14, and keep 24 bits: 2^-14 - 23 = 2^-37 per unit of w s, which is 2^-13 of a code's 2^-24.
    A product and its sum lose that much each: 2^-12 w s per token, however small z + s code itself is."""
    Hq, n, d = q.shape
    g = Hq // c.Hkv
    units, T = unit_tokens(c, b)
    out = torch.zeros(Hq, n, d, dtype=torch.float64)
    tol = torch.zeros_like(out)
    p = (pos0 + torch.arange(n))[:, None]
    for h in range(c.Hkv):
        K, V, idx, S = units[h]
        if k is not None:
            K, V = torch.cat([K, k[h].double()]), torch.cat([V, v[h].double()])
            idx = torch.cat([idx, T + torch.arange(n)])
            S = torch.cat([S, torch.zeros(n, d, dtype=torch.float64)])
        see = idx <= p
        if window:
            see = see & ((idx > p - window) | (idx < sinks))
        for hh in range(h * g, (h + 1) * g):
            qd = q[hh].double()
            lg = (qd @ K.t()) / d ** 0.5
            mag = ((qd.abs() @ K.abs().t()) / d ** 0.5).masked_fill(~see, 0).amax(1, keepdim=True)
            lg = lg.masked_fill(~see, -float("inf"))
            w = torch.softmax(lg, 1).nan_to_num(0.0)      # a row that sees nothing: zeros
            o, A = w @ V, w @ V.abs()
            e = (d / 16 + 4) * 2.0 ** -22 * 2 * mag + 3 * 2.0 ** -23 * mag + 2.0 ** -21
            out[hh] = o
            tol[hh] = 2.0 ** -11 * (2 * A + o.abs()) * 1.01 + 2 * e * A + 2.0 ** -24 * (see.double() @ V.abs()) + 2.0 ** -24
            if folded:
                tol[hh] += 2.0 ** -12 * (w @ S)
    return out, tol


def check(got, ref, tol, where=""):
    got = got.detach().double().cpu()
    assert torch.isfinite(got).all(), f"{where}: non-finite"
    over = ((got - ref).abs() - tol).max().item()
    assert over <= 0, f"{where}: {over:.3e} over the bound; max |d| {(got - ref).abs().max().item():.3e}"
