"""Plain references of the rollout step's operators for their GPU tests: numpy and
torch on the CPU, in 64 bits (in 32 where the operator's bits are defined so),
sharing nothing with the library."""
from __future__ import annotations

import numpy as np
import torch


def rope_pairs(D, R, inter):
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if inter else (i, i + R // 2)


def rope(x, pos, table, R, inter=False, inverse=False, dtype=np.float64):
    """x [T, H, D] -> rotated, in `dtype`, one rounding an operation."""
    x = x.astype(dtype)
    a, b = rope_pairs(x.shape[-1], R, inter)
    c = table[pos][:, None, :R // 2].astype(dtype)
    s = table[pos][:, None, R // 2:].astype(dtype)
    if inverse:
        s = -s
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def bf16(x):
    """Round to bf16 (fp32 numpy in, fp32 numpy out)."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def e4m3_codes(x, scale):
    """fl32(x / scale) rounded to E4M3 and saturated, as codes."""
    q = torch.from_numpy(np.ascontiguousarray(x, np.float32)) / torch.tensor([scale], dtype=torch.float32)
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def e4m3_values(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).float().numpy()


def attention(q, k, v, scale, window=0):
    """One sequence: q [Lq, Hq, D], k, v [len, Hkv, D] fp64 -> o, lse and the bound on
    |o - exact| of an implementation that multiplies bf16 or fp16 operands with fp32
    sums (below), all fp64."""
    Lq, Hq, D = q.shape
    n, Hkv, _ = k.shape
    o = np.zeros((Lq, Hq, D))
    lse = np.full((Lq, Hq), -np.inf)
    tol = np.zeros((Lq, Hq, D))
    ltol = np.zeros((Lq, Hq))
    for i in range(Lq):
        p = n - Lq + i
        if p < 0:
            continue
        lo = max(0, p - window + 1) if window else 0
        for h in range(Hq):
            kk, vv = k[lo:p + 1, h // (Hq // Hkv)], v[lo:p + 1, h // (Hq // Hkv)]
            x = scale * (kk @ q[i, h])
            m = x.max()
            w = np.exp(x - m)
            total = w.sum()
            o[i, h] = (w / total) @ vv
            lse[i, h] = np.log(total) + m
            # a score: D fp32 additions, two roundings of the scaled value, and the
            # query held to 2^-24 of its row's largest value
            dx = 2.0 ** -23 * scale * ((D + 8) * (np.abs(kk) @ np.abs(q[i, h])).max()
                                       + np.abs(q[i, h]).max() * np.abs(kk).sum(axis=1).max()) \
                + 2.0 ** -21 * np.abs(x).max()
            terms = x.size
            mean = (w / total) @ np.abs(vv)
            # probabilities rounded to 2^-8 of themselves (bf16's unit roundoff), or up
            # to 2^-24 of the row's largest where fp16 runs out; fp32 sums over the
            # tokens; bf16 result, 2^-8 of itself
            small = 2.0 ** -24 / total * np.abs(vv).sum(axis=0)
            tol[i, h] = (2.0 ** -8 + 2 * dx + terms * 2.0 ** -23 + 2.0 ** -20) * mean + small \
                + 2.0 ** -8 * 1.01 * np.abs(o[i, h]) + 1e-38
            ltol[i, h] = dx + terms * 2.0 ** -23 + 2.0 ** -20 * (1 + abs(lse[i, h]))
    return o, lse, tol, ltol


def verify(P, Q, drafts, lens, u, noise):
    """The definition, one sequence at a time; fp32 P, Q, u, noise."""
    B, K1, V = P.shape
    K = K1 - 1
    out = np.full((B, K1), -1, np.int32)
    acc = np.zeros(B, np.int32)
    for b in range(B):
        n = 0
        while n < lens[b]:
            t = drafts[b, n]
            qt = 1.0 if Q is None else np.float64(Q[b, n, t])
            if not np.float64(u[b, n]) * qt < np.float64(P[b, n, t]):
                break
            out[b, n] = t
            n += 1
        w = P[b, n].astype(np.float32)
        if n < lens[b]:
            r = w.copy()
            if Q is None:
                r[drafts[b, n]] = 0
            else:
                r = np.maximum(w - Q[b, n].astype(np.float32), np.float32(0))
            if (r > 0).any():
                w = r
        with np.errstate(divide="ignore", invalid="ignore"):
            s = np.where(w > 0, w / noise[b], np.float32(0))
        out[b, n] = int(np.argmax(s))           # the lowest of equal scores
        acc[b] = n
    return out, acc
