"""The trainer's losses and their gradients in 64 bits, from the formulas, with bounds on
what 32-bit sums and one rounding of each operand may be off."""
import math

import torch


def logits(H, W, targets, scale):
    """-> (x [M, V] with rows that do not count as zeros, which rows count, the sum of
    magnitudes behind each logit)."""
    live = (targets >= 0) & (targets < W.shape[0])
    h = torch.where(live[:, None], H.double(), 0.0)
    w = W.double()
    return h @ w.T * scale, live, h.abs() @ w.abs().T * scale, h, w


def linear_logp(H, W, targets, scale=1.0):
    """-> (logp, lse, entropy), each (value, bound)."""
    V, K = W.shape
    x, live, mag, _, _ = logits(H, W, targets, scale)
    lse = torch.logsumexp(x, dim=1)
    p = torch.exp(x - lse[:, None])
    at = targets.clamp(0, V - 1).long()[:, None]
    logp = x.gather(1, at)[:, 0] - lse
    entropy = -(p * (x - lse[:, None])).sum(1)
    # a logit: K/16 steps of 16 products, each off by at most two units of 2^-23 of the
    # sum of magnitudes, the scale and one more rounding
    d = mag.amax(1) * (max(K / 16, 1) * 2.0 ** -22 + 2.0 ** -22)
    # a sum of exponentials: their arguments' rounding (weighted: log V and a little), the
    # exponential's own 2^-22, and V additions in groups of at most 256
    r = 2.0 ** -21 + (math.log(V) + 8) * 2.0 ** -22 + (256 + V / 256 + 16) * 2.0 ** -24
    e_lse = d + r + lse.abs() * 2.0 ** -22
    e_logp = 2 * d + r + (logp.abs() + lse.abs()) * 2.0 ** -22
    span = math.log(V) + 1
    e_ent = 2 * entropy.abs() * d + r * (entropy.abs() + span) + (entropy.abs() + span) * 2.0 ** -22
    zero = torch.zeros_like(lse)
    return tuple((torch.where(live, v, zero), torch.where(live, e, zero))
                 for v, e in ((logp, e_logp), (lse, e_lse), (entropy, e_ent)))


def linear_logp_grad(H, W, targets, g, ge=None, scale=1.0):
    """-> (dH, dW), each (value, bound)."""
    V, K = W.shape
    x, live, mag, h, w = logits(H, W, targets, scale)
    lse = torch.logsumexp(x, dim=1, keepdim=True)
    logp = x - lse
    p = torch.exp(logp)
    zero = torch.zeros(len(g), dtype=torch.float64, device=g.device)
    g = torch.where(live, g.double(), zero)[:, None]
    e = torch.where(live, ge.double(), zero)[:, None] if ge is not None else zero[:, None]
    ent = -(p * logp).sum(1, keepdim=True)
    hot = torch.zeros_like(x).scatter_(1, targets.clamp(0, V - 1).long()[:, None], 1.0)
    D = g * (hot - p) - e * p * (logp + ent)
    # each D rounded once to bf16 (2^-8 of itself); p from a logit and a log-sum that are
    # off by d each; the target's 1 - p and the entropy's part by fp32 roundings
    d = (mag.amax(1) * (max(K / 16, 1) * 2.0 ** -21 + 2.0 ** -21) + (256 + V / 256 + 64) * 2.0 ** -23
         + lse[:, 0].abs() * 2.0 ** -21)[:, None] + logp.abs() * 2.0 ** -22
    off = D.abs() * 2.0 ** -8 + g.abs() * (p * d + hot * 2.0 ** -23) + e.abs() * p * (d * (2 + 2 * (logp + ent).abs())
                                                                                      + (logp.abs() + ent) * 2.0 ** -21)
    # fp32 below 2^-126 may come out as 0: a probability there, and D in units of the largest gradient
    off = off + 2.0 ** -126 * (g.abs() + e.abs() * (1 + (logp + ent).abs()) + torch.maximum(g.abs().amax(), e.abs().amax()))
    sums = 2.0 ** -20 + max(V, len(g)) / 16 * 2.0 ** -22
    out = []
    for a, b, ab in ((D, w, off), (D.T, h, off.T)):
        value = a @ b * scale
        out.append((value, (ab @ b.abs() + a.abs() @ b.abs() * sums) * scale * (1 + 2.0 ** -7) + value.abs() * 2.0 ** -8
                    + 2.0 ** -126))
    return out


def teacher(ids, T, teacher_lse, V, scale):
    """-> (q [M, k] with 0 for entries that are none, log q, which entries are)."""
    there = (ids >= 0) & (ids < V)
    t = torch.where(there, T.double() * scale, float("-inf"))
    if teacher_lse is None:
        logq = t - torch.logsumexp(t, dim=1, keepdim=True)
    else:
        logq = t - teacher_lse.double()[:, None]
    logq = torch.where(there, logq, float("-inf"))
    return torch.exp(logq), logq, there


def distill(X, ids, T, teacher_lse=None, rest=False, scale=1.0):
    """-> (loss, lse, rest_lse), each (value, bound); rest_lse None without rest."""
    V = X.shape[1]
    q, logq, there = teacher(ids, T, teacher_lse, V, scale)
    live = there.any(1)
    y = torch.where(live[:, None], X.double(), 0.0) * scale
    lse = torch.logsumexp(y, dim=1)
    at = ids.clamp(0, V - 1).long()
    logp = y.gather(1, at) - lse[:, None]
    ratio = torch.where(q > 0, logq - logp, 0.0)
    loss = (q * ratio).sum(1)
    # relative error of a sum of exponentials: arguments off by 2^-22 of themselves
    # (weighted by the exponential: below log V and a little), the exponential's 2^-21,
    # additions in runs of at most V / 256 and a tree
    r = 2.0 ** -21 + (math.log(V) + 8) * 2.0 ** -22 + (V / 256 + 32) * 2.0 ** -24
    # a teacher's probability: 2^-20 of itself
    e_loss = q.sum(1) * r + (q * ratio.abs()).sum(1) * 2.0 ** -20
    left = None
    if rest:
        inside = torch.zeros_like(y).scatter_(1, torch.where(there, at, at[:, :1]), there.double()) > 0
        for j in range(ids.shape[1]):                 # a later entry that is none may have written over one that is
            rows = there[:, j]
            inside[rows.nonzero()[:, 0], at[rows, j]] = True
        left = torch.logsumexp(y.masked_fill(inside, float("-inf")), dim=1)
        qr = torch.where(inside.all(1), 0.0, (1.0 - q.sum(1)).clamp(min=0.0))
        some = qr > 0
        part = torch.where(some, qr * (torch.log(torch.where(some, qr, 1.0)) - (left - lse)), 0.0)
        loss = loss + part
        dq = q.sum(1) * 2.0 ** -20 + 2.0 ** -24
        e_loss = e_loss + qr * 2 * r + torch.where(
            dq > 0, dq * (2 + torch.where(some, (torch.log(torch.where(some, qr, 1.0)) - (left - lse)).abs(),
                                          (torch.log(dq) - (left - lse)).abs())), 0.0)
    e_loss = e_loss + loss.abs() * 2.0 ** -23 + 1e-12
    zero = torch.zeros_like(lse)
    out = [(torch.where(live, loss, zero), torch.where(live, e_loss, zero)),
           (torch.where(live, lse, zero), torch.where(live, r + lse.abs() * 2.0 ** -23, zero)), None]
    if rest:
        out[2] = (torch.where(live, left, zero),
                  torch.where(live & torch.isfinite(left), r + left.abs() * 2.0 ** -23, zero))
    return out


def distill_grad(X, ids, T, g, teacher_lse=None, rest=False, scale=1.0):
    """-> (dX, bound), before the rounding to X's type, which the bound includes."""
    M, V = X.shape
    q, _, there = teacher(ids, T, teacher_lse, V, scale)
    live = there.any(1)
    y = torch.where(live[:, None], X.double(), 0.0) * scale
    lse = torch.logsumexp(y, dim=1, keepdim=True)
    p = torch.exp(y - lse)
    at = torch.where(there, ids, 0).long()
    inside = torch.zeros_like(p).scatter_add_(1, at, torch.where(there, q, 0.0))
    named = torch.zeros_like(p).scatter_add_(1, at, there.double()) > 0
    Q = q.sum(1, keepdim=True)
    second = torch.zeros_like(p)
    dq = Q * 2.0 ** -20 + 2.0 ** -24
    if rest:
        left = torch.logsumexp(y.masked_fill(named, float("-inf")), dim=1, keepdim=True)
        qr = torch.where(named.all(1, keepdim=True), 0.0, (1.0 - Q).clamp(min=0.0))
        share = torch.where(named | torch.isinf(left), 0.0, torch.exp(y - left))
        second = qr * share
        Q = Q + qr
    f = g.double()[:, None] * scale
    value = f * (p * Q - inside - second)
    # the log-sums arrive in fp32, the exponents are rounded once more
    # (a logit of -inf is a probability of exactly 0)
    r = 2.0 ** -20 + lse.abs() * 2.0 ** -22 + torch.where(torch.isinf(y), 0.0, y.abs()) * 2.0 ** -22
    bound = f.abs() * ((p * Q + second) * (2 * r + 2.0 ** -20) + inside * 2.0 ** -19)
    if rest:
        bound = bound + f.abs() * (p + torch.where(named, 0.0, share)) * dq
        bound = bound + f.abs() * torch.where(named, 0.0, share) * qr * torch.where(torch.isinf(left), 0.0, left.abs()) * 2.0 ** -22
    half = 2.0 ** -8 if X.dtype == torch.bfloat16 else 2.0 ** -24
    bound = bound * (1 + 2.0 ** -7) + value.abs() * half * (1 + 2.0 ** -7) + 1e-38
    zero = torch.zeros_like(value)
    return torch.where(live[:, None], value, zero), torch.where(live[:, None], bound, zero)


def check(got, want, what=""):
    """Element by element within the bound; infinities equal."""
    value, bound = want
    got = got.double()
    fine = torch.isfinite(value)
    assert torch.equal(got[~fine], value[~fine]), what
    over = (got - value).abs()[fine] - bound[fine]
    worst = over.max().item() if over.numel() else 0.0
    assert not torch.isnan(got[fine]).any() and worst <= 0.0, (
        what, worst, ((got - value).abs()[fine] / bound[fine].clamp(min=1e-300)).max().item())
