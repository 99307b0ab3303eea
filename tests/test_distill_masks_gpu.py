"""Distillation where logits are masks: rows of the type's lowest value, -inf and both, and
teachers without weight, against 64 bits taken relative to each maximum."""
import math

import pytest
import torch

import losses_ref as ref
from precision_rl_rollout_gb300 import binding as fb

pytestmark = pytest.mark.gpu


def _apart(z, where, scale):
    """-> (maximum, log of the sum of exponentials, scaled, relative to it) over the entries of each row."""
    z = z.masked_fill(~where, float("-inf"))
    top = z.amax(dim=1)
    safe = torch.where(torch.isinf(top), 0.0, top)
    return safe, torch.log(torch.exp((z - safe[:, None]) * scale).sum(1))


def _exact(X, ids, T, teacher_lse, rest, scale):
    """-> [(loss, bound), (lse, bound), (rest_lse, bound)], p [M, V], the outside's share of each token, q, q_r"""
    M, V = X.shape
    y, t = X.double(), T.double()
    everything = torch.ones_like(y, dtype=torch.bool)
    inside = torch.zeros_like(everything).scatter_(1, ids.long(), True)
    top, L = _apart(y, everything, scale)
    logp = (y - top[:, None]) * scale - L[:, None]
    if teacher_lse is None:
        t = t - t.amax(dim=1, keepdim=True)
        logq = t * scale - torch.logsumexp(t * scale, dim=1, keepdim=True)
    else:
        logq = t * scale - teacher_lse.double()[:, None]
    q = torch.exp(logq)
    ratio = torch.where(q > 0, logq - logp.gather(1, ids.long()), 0.0)
    loss = (q * ratio).sum(1)
    # as for distill in losses_ref: a sum of exponentials, a teacher's probability
    r = 2.0 ** -21 + (math.log(V) + 8) * 2.0 ** -22 + (V / 256 + 32) * 2.0 ** -24
    e = q.sum(1) * r + (q * ratio.abs()).sum(1) * 2.0 ** -20
    otop, o = _apart(y, ~inside, scale)
    R = o + (otop - top) * scale - L                      # log of the outside's share
    qr = (1.0 - q.sum(1)).clamp(min=0.0)
    share = torch.where(inside, 0.0, torch.exp((y - otop[:, None]) * scale - o[:, None]))
    if rest:
        loss = loss + qr * (torch.log(qr) - R)
        e = e + qr * 2 * r + (q.sum(1) * 2.0 ** -20 + 2.0 ** -24) * (2 + (torch.log(qr) - R).abs())
    lse, left = L + top * scale, o + otop * scale
    out = [(loss, e + loss.abs() * 2.0 ** -22 + 1e-12), (lse, r + lse.abs() * 2.0 ** -23), (left, r + left.abs() * 2.0 ** -23)]
    return out, torch.exp(logp), share, q, qr


def _rows(M, V, k, dtype, scale, seed=0):
    """Rows of each kind in turn: all lowest, lowest outside the entries, lowest inside, a teacher of
    lowest entries, both, lowest and -inf, and none of it."""
    g = torch.Generator(device="cuda").manual_seed(seed + M + V + k)
    X = (torch.randn((M, -(-V // 8) * 8), generator=g, device="cuda") * 2.5).to(dtype)[:, :V]
    T, ids = (X.float() + torch.randn((M, V), generator=g, device="cuda")).topk(k, dim=1)
    T, ids = T.contiguous(), ids.int().contiguous()
    inside = torch.zeros((M, V), dtype=torch.bool, device="cuda").scatter_(1, ids.long(), True)
    low = torch.finfo(dtype).min
    kind = torch.arange(M, device="cuda") % 7
    X[kind == 0], X[kind == 4], X[kind == 5] = low, low, low
    X[(kind == 1)[:, None] & ~inside] = low
    X[(kind == 2)[:, None] & inside] = low
    some = torch.rand((M, V), generator=g, device="cuda") < 0.5
    X[(kind == 5)[:, None] & some & ~inside] = float("-inf")
    lse = torch.logsumexp(T.double() * scale, dim=1).float() + 0.3
    T[(kind == 3) | (kind == 4)] = torch.finfo(torch.float32).min
    return X, ids, T, lse, kind, torch.randn(M, generator=g, device="cuda")


SIZES = [(1, 1000, 8), (7, 1003, 8), (14, 40000, 20), (700, 2000, 5), (7, 152064, 64)]


@pytest.mark.parametrize("M,V,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [0.5, 1.0])
def test_losses_of_masks(cuda_lib, M, V, k, dtype, scale):
    X, ids, T, lse, kind, _ = _rows(M, V, k, dtype, scale)
    got = fb.fp8rl_distill_topk(X, ids, T, scale=scale)
    want = _exact(X, ids, T, None, False, scale)[0]
    keep = (kind != 2) | (scale < 1.0)                     # q x 3.4e38 may round past fp32
    for a, b in zip(got, want):
        ref.check(a[keep], tuple(x[keep] for x in b))
    keep &= (kind != 3) & (kind != 4)                      # a teacher of masks has a log-sum that fp32 cannot tell
    got = fb.fp8rl_distill_topk(X, ids, T, teacher_lse=lse, rest=True, scale=scale)
    want = _exact(X, ids, T, lse, True, scale)[0]
    for a, b in zip(got, want):
        ref.check(a[keep], tuple(x[keep] for x in b))
    assert fb.fp8rl_check_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", [1e29, 1e31, 3e37, -1e29, -1e31])
def test_one_huge_logit(cuda_lib, dtype, value):
    """Inside the entries or outside, above the others or below: the log-sums of the others stay."""
    X, ids, T, _, _, _ = _rows(6, 2000, 10, dtype, 0.6)
    X = (torch.randn((6, 2000), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * 2.5).to(dtype)
    T = X.float().gather(1, ids.long()) + 1.0
    lse = torch.logsumexp(T.double() * 0.6, dim=1).float() + 0.3
    inside = torch.zeros((6, 2000), dtype=torch.bool, device="cuda").scatter_(1, ids.long(), True)
    X[0, ids[0, 3].long()], X[1, ids[1, 0].long()] = value, value
    X[2, (~inside[2]).nonzero()[7, 0]], X[3, (~inside[3]).nonzero()[1500, 0]] = value, value
    X[4] = torch.where(inside[4], value, X[4])
    X[5] = torch.where(inside[5], X[5], value)
    for tl in (None, lse):
        got = fb.fp8rl_distill_topk(X, ids, T, teacher_lse=tl, rest=tl is not None, scale=0.6)
        for name, a, b in zip(("loss", "lse", "rest_lse"), got, _exact(X, ids, T, tl, tl is not None, 0.6)[0]):
            ref.check(a, b, name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("student,teacher", [(300.0, 0.0), (-2e4, 0.0), (1e6, 0.0), (0.0, 3e7), (5e5, 5e5), (-4e9, 1e9)])
def test_what_logits_share_costs_nothing(cuda_lib, dtype, student, teacher):
    """A constant in the student's logits or in the teacher's is none of the loss's: it keeps its bound."""
    g = torch.Generator(device="cuda").manual_seed(3)
    X = (torch.randn((40, 3000), generator=g, device="cuda") * 2.5).to(dtype)
    T, ids = (X.float() + 0.1 * torch.randn((40, 3000), generator=g, device="cuda")).topk(30, dim=1)
    ids = ids.int().contiguous()
    X, T = (X.float() + student).to(dtype), (T + teacher).contiguous()
    lse = torch.logsumexp(T.double() * 0.8, dim=1) + 0.3
    for tl in (None, lse.float()):
        if tl is not None and teacher:
            continue                                       # a log-sum in fp32 has not the bits
        got = fb.fp8rl_distill_topk(X, ids, T, teacher_lse=tl, rest=tl is not None, scale=0.8)
        for name, a, b in zip(("loss", "lse", "rest_lse"), got, _exact(X, ids, T, tl, tl is not None, 0.8)[0]):
            ref.check(a, b, name)


def _check_grad(dX, X, ids, T, teacher_lse, g, scale, keep):
    rest = teacher_lse is not None
    out, p, share, q, qr = _exact(X, ids, T, teacher_lse, rest, scale)
    inside = torch.zeros_like(p).scatter_(1, ids.long(), q)
    Q = q.sum(1, keepdim=True)
    dq = Q * 2.0 ** -20 + 2.0 ** -24
    second = qr[:, None] * share if rest else torch.zeros_like(p)
    Q = Q + qr[:, None] if rest else Q
    f = g.double()[:, None] * scale
    value = f * (p * Q - inside - second)
    # by log-sums in fp32 up to 65536, past it by sums anew
    sums = [x[0].abs()[:, None] for x in (out[1:] if rest else out[1:2])]
    r = 2.0 ** -18 + sum(torch.where(s > 65536, 0.0, s) for s in sums) * 2.0 ** -21
    bound = f.abs() * ((p * Q + second) * 2 * r + inside * 2.0 ** -19 + (p + share if rest else p) * dq)
    half = 2.0 ** -8 if X.dtype == torch.bfloat16 else 2.0 ** -24
    bound = bound * (1 + 2.0 ** -7) + value.abs() * half * (1 + 2.0 ** -7) + 1e-38
    ref.check(dX[keep], (value[keep], bound[keep]), "dX")


@pytest.mark.parametrize("M,V,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [0.5, 0.7, 1.0])
def test_gradients_of_masks(cuda_lib, M, V, k, dtype, scale):
    """Rows whose log-sums are a mask's value: softmax and its gradient are those of equal logits; in place too."""
    X, ids, T, lse, kind, g = _rows(M, V, k, dtype, scale)
    s = fb.fp8rl_distill_topk(X, ids, T, scale=scale)[1]
    dX = fb.fp8rl_distill_topk_backward(X, ids, T, s, g, scale=scale)
    _check_grad(dX, X, ids, T, None, g, scale, kind >= 0)
    _, s, r = fb.fp8rl_distill_topk(X, ids, T, teacher_lse=lse, rest=True, scale=scale)
    dX = fb.fp8rl_distill_topk_backward(X, ids, T, s, g, teacher_lse=lse, rest_lse=r, scale=scale)
    _check_grad(dX, X, ids, T, lse, g, scale, (kind != 3) & (kind != 4))
    wide = torch.zeros((M, -(-V // 8) * 8), dtype=dtype, device="cuda")
    Y = wide[:, :V]
    Y.copy_(X)
    fb.fp8rl_distill_topk_backward(Y, ids, T, s, g, teacher_lse=lse, rest_lse=r, scale=scale, dX=Y)
    assert torch.equal(Y, dX) and (wide[:, V:] == 0).all()
    assert fb.fp8rl_check_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift", [300.0, -2e4, 7e4, -3e6, 1e9])
def test_gradients_of_shifted_logits(cuda_lib, dtype, shift):
    g = torch.Generator(device="cuda").manual_seed(3)
    X = (torch.randn((30, 3000), generator=g, device="cuda") * 2.5).to(dtype)
    T, ids = (X.float() + torch.randn((30, 3000), generator=g, device="cuda")).topk(30, dim=1)
    T, ids, gl = T.contiguous(), ids.int().contiguous(), torch.randn(30, generator=g, device="cuda")
    X = (X.float() + shift).to(dtype)
    lse = (torch.logsumexp(T.double() * 0.8, dim=1) + 0.3).float()
    _, s = fb.fp8rl_distill_topk(X, ids, T, scale=0.8)
    _check_grad(fb.fp8rl_distill_topk_backward(X, ids, T, s, gl, scale=0.8), X, ids, T, None, gl, 0.8, gl == gl)
    _, s, r = fb.fp8rl_distill_topk(X, ids, T, teacher_lse=lse, rest=True, scale=0.8)
    dX = fb.fp8rl_distill_topk_backward(X, ids, T, s, gl, teacher_lse=lse, rest_lse=r, scale=0.8)
    _check_grad(dX, X, ids, T, lse, gl, 0.8, gl == gl)


@pytest.mark.parametrize("M,V", [(4, 1003), (4, 152064), (700, 2000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("whole", [False, True])
def test_a_teacher_without_weight(cuda_lib, M, V, dtype, whole):
    """Entries of -inf alone: the loss is 0, and so is the gradient, whatever the row's logits are."""
    X, ids, T, lse, kind, g = _rows(M, V, 5, dtype, 1.0)
    T[:] = float("-inf")
    X[::4], X[1::4, 3], X[2::4] = float("-inf"), float("nan"), torch.finfo(dtype).min
    tl = lse if whole else None
    loss, s = fb.fp8rl_distill_topk(X, ids, T, teacher_lse=tl)
    dX = fb.fp8rl_distill_topk_backward(X, ids, T, s, g, teacher_lse=tl)
    assert (loss == 0).all() and (dX == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,k", [(20000, 64), (152064, 64), (300, 300)])
@pytest.mark.parametrize("rest", [False, True])
def test_a_small_divergence(cuda_lib, dtype, V, k, rest):
    """A student 0.004 from its teacher in every logit: losses of some 1e-6 to 1e-5, the differences of terms near
    1.  With both cut to the entries a relative error of the student's sum is the loss's absolute one:
    arguments (2^-24 of some 5, weighted) and exponentials (2^-22) that all err alike, 2^-20 at most.  With the
    rest, errors that all of the sums share cancel: half of that."""
    g = torch.Generator(device="cuda").manual_seed(V + k)
    M = 64
    X = (torch.randn((M, -(-V // 8) * 8), generator=g, device="cuda") * 2.5).to(dtype)[:, :V]
    teacher = X.float() + 0.004 * torch.randn((M, V), generator=g, device="cuda")
    T, ids = teacher.topk(k, dim=1)
    if not rest:
        X.masked_fill_(~torch.zeros((M, V), dtype=torch.bool, device="cuda").scatter_(1, ids, True), float("-inf"))
    T, ids = T.contiguous(), ids.int().contiguous()
    lse = torch.logsumexp(teacher.double(), dim=1).float() if rest else None
    if rest and k == V:
        # a teacher's log-sum in fp32 leaves a rest of up to 2^-22 to a class that no token is in; as in losses_ref it is none
        want = ref.distill(X, ids, T, lse, True)[0][0]
    else:
        want = _exact(X, ids, T, lse, rest, 1.0)[0][0][0]
    loss = fb.fp8rl_distill_topk(X, ids, T, teacher_lse=lse, rest=rest)[0].double()
    bound = 2.0 ** -20 if not rest else 2.0 ** -21
    if k < V or not rest:
        assert want.median() > 2 * bound                   # so that a loss of 0 would not pass
    assert ((loss - want).abs() <= bound + want.abs() * 2.0 ** -20).all(), (loss - want).abs().max().item()
