"""Distillation from a teacher's top logits and its gradient, against 64 bits."""
import pytest
import torch

import losses_ref as ref
from precision_rl_rollout_gb300 import binding as fb

pytestmark = pytest.mark.gpu

# from 153 rows (gradient) and 609 (loss) on CTAs are smaller
SIZES = [(700, 2000, 300), (1300, 4099, 7), (200, 40000, 200), (1, 1, 1), (1, 152064, 64), (2, 37, 5), (3, 1000, 20), (16, 4096, 1), (5, 4097, 300), (130, 2049, 8), (33, 50257, 100),
         (7, 1100, 1024), (40, 513, 64), (20, 30001, 33)]


def _inputs(M, V, k, dtype, seed=0, noise=1.0, masked=0.2, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + M + 7 * V + 13 * k)
    pad = -(-V // 8) * 8
    X = (torch.randn((M, pad), generator=g, device="cuda") * 2.5).to(dtype)[:, :V]
    teacher = X.float() + noise * torch.randn((M, V), generator=g, device="cuda")
    T, ids = teacher.topk(min(k, V), dim=1)
    T, ids = T.contiguous(), ids.to(torch.int32).contiguous()
    lse = torch.logsumexp(teacher.double() * scale, dim=1).float()
    if M > 1:
        out = torch.rand(M, generator=g, device="cuda") < masked
        ids[out] = -1
        X[out] = float("nan")
        ids[1, -1] = V + 3 if k > 1 else ids[1, -1]                 # fewer entries than k
    return X, ids, T, lse, torch.randn(M, generator=g, device="cuda")


def _run(X, ids, T, lse, g, rest, cut, scale):
    kw = dict(teacher_lse=None if cut else lse, scale=scale)
    out = fb.fp8rl_distill_topk(X, ids, T, rest=rest, **kw)
    dX = fb.fp8rl_distill_topk_backward(X, ids, T, out[1], g, rest_lse=out[2] if rest else None, **kw)
    return (*out, dX)


def _check(X, ids, T, lse, g, rest, cut, scale):
    got = _run(X, ids, T, lse, g, rest, cut, scale)
    teacher_lse = None if cut else lse
    want = ref.distill(X, ids, T, teacher_lse, rest, scale)
    for name, a, b in zip(("loss", "lse", "rest_lse"), got[:-1], want):
        ref.check(a, b, name)
    ref.check(got[-1], ref.distill_grad(X, ids, T, g, teacher_lse, rest, scale), "dX")
    assert got[-1].shape == X.shape and got[-1].dtype == X.dtype
    assert fb.fp8rl_check_device_error() == 0


@pytest.mark.parametrize("M,V,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mode", ["cut", "whole", "rest"])
def test_loss_and_gradient(cuda_lib, M, V, k, dtype, mode):
    scale = 0.6
    X, ids, T, lse, g = _inputs(M, V, k, dtype, scale=scale)
    _check(X, ids, T, lse, g, mode == "rest", mode == "cut", scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rest", [False, True])
def test_a_near_student_keeps_its_loss(cuda_lib, dtype, rest):
    """A divergence of some 1e-5, the difference of terms near 1."""
    X, ids, T, lse, g = _inputs(30, 20000, 64, dtype, noise=0.004, masked=0.0)
    _check(X, ids, T, lse, g, rest, not rest, 1.0)


@pytest.mark.parametrize("rest", [False, True])
def test_a_token_named_twice(cuda_lib, rest):
    X, ids, T, lse, g = _inputs(12, 3000, 40, torch.float32, masked=0.0)
    T = T - 2.0                                                     # so that doubled entries leave a rest
    ids[:, 7] = ids[:, 3]
    ids[::2, 39] = ids[::2, 3]
    lse = lse + 0.5
    _check(X, ids, T, lse, g, rest, not rest, 1.0)


def test_every_token_named(cuda_lib):
    X, ids, T, lse, g = _inputs(6, 96, 96, torch.float32, masked=0.0)
    ids[1, -1] = ids[1, 0]                                          # but one, in one row
    _check(X, ids, T, lse, g, True, False, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_infinite_and_extreme_logits(cuda_lib, dtype):
    X, ids, T, lse, g = _inputs(9, 2000, 16, dtype, masked=0.0)
    inside = torch.zeros((9, 2000), dtype=torch.bool, device="cuda").scatter_(1, ids.clamp(0, 1999).long(), True)
    X[(torch.arange(2000, device="cuda") % 3 == 0)[None, :] & ~inside] = float("-inf")   # a vocabulary mask
    X[4] = torch.where(torch.isinf(X[4]), X[4], X[4] * 3e4)
    T[5, 8:] = float("-inf")                                        # entries without weight
    for rest in (False, True):
        _check(X, ids, T, lse, g, rest, not rest, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [0.3, 0.7, 1.0, 1.3])
def test_a_lowest_logit_under_a_huge_one(cuda_lib, dtype, scale):
    """Their difference is -inf in 32 bits, the second's share still 0; a row of masks alone costs nothing
    where the teacher has no weight either."""
    X, ids, T, lse, g = _inputs(9, 1000, 20, dtype, masked=0.0)
    X, ids, T = X.clone(), ids.clone(), T.clone()
    last = X.argsort(dim=1)
    X[0, last[0, 500]], X[3, last[3, 999]] = 1e37, 3e37
    X[0, last[0, :100]], X[3, last[3, 0]] = torch.finfo(dtype).min, torch.finfo(dtype).min
    X[5] = float("-inf")
    T[5] = float("-inf")
    got = fb.fp8rl_distill_topk(X, ids, T, scale=scale)
    want = ref.distill(X, ids, torch.where(torch.isinf(T), 0.0, T), None, False, scale)
    keep = torch.arange(9, device="cuda") != 5
    for a, b in zip(got, want):
        ref.check(a[keep], tuple(x[keep] for x in b))
    assert got[0][5].item() == 0.0


@pytest.mark.parametrize("M", [1, 9, 700])
def test_the_largest_vocabulary(cuda_lib, M):
    """As many parts a row as there are, with the bits of 2^20 tokens in each one's shared memory."""
    X, ids, T, lse, g = _inputs(M, 1 << 20, 1024 if M < 10 else 20, torch.bfloat16)
    out = fb.fp8rl_distill_topk(X, ids, T, teacher_lse=lse, rest=True)
    dX = fb.fp8rl_distill_topk_backward(X, ids, T, out[1], g, teacher_lse=lse, rest_lse=out[2])
    few = slice(max(0, M - 9), M)
    want = ref.distill(X[few], ids[few], T[few], lse[few], True)
    for a, b in zip(out, want):
        ref.check(a[few], b)
    ref.check(dX[few], ref.distill_grad(X[few], ids[few], T[few], g[few], lse[few], True))


def test_masked_token_of_the_teacher_costs_everything(cuda_lib):
    X, ids, T, lse, g = _inputs(1, 500, 4, torch.float32)
    X[0, ids[0, 0].long()] = float("-inf")
    loss, _ = fb.fp8rl_distill_topk(X, ids, T)
    assert loss.item() == float("inf")


def test_gradient_against_differences(cuda_lib):
    X, ids, T, lse, g = _inputs(6, 300, 10, torch.float32, masked=0.0)
    *_, dX = _run(X, ids, T, lse, g, True, False, 0.8)
    gen = torch.Generator(device="cuda").manual_seed(2)
    for _ in range(3):
        u = torch.randn(X.shape, generator=gen, device="cuda", dtype=torch.float64)
        up, down = ((ref.distill(X.double() + s * 1e-5 * u, ids, T, lse, True, 0.8)[0][0] * g.double()).sum() for s in (1, -1))
        slope = ((up - down) / 2e-5).item()
        assert abs((dX.double() * u).sum().item() - slope) <= 1e-6 * (dX.double() * u).abs().sum().item() + 1e-8


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V", [(1, 152064), (50, 3001), (700, 4096)])
def test_in_place_and_guards(cuda_lib, dtype, M, V):
    X, ids, T, lse, g = _inputs(M, V, 24, dtype)
    _, s, r, dX = _run(X, ids, T, lse, g, True, False, 1.0)
    ld = -(-V // 8) * 8 + 16
    wide = torch.full((M, ld), 9.0, dtype=dtype, device="cuda")
    wide[:, :V] = X
    Y = wide[:, :V]
    out = fb.fp8rl_distill_topk_backward(Y, ids, T, s, g, teacher_lse=lse, rest_lse=r, dX=Y)
    assert out.data_ptr() == Y.data_ptr() and torch.equal(Y, dX)
    assert (wide[:, V:] == 9).all()


def test_no_rows(cuda_lib):
    X, ids, T, lse, g = _inputs(4, 100, 4, torch.float32)
    out = _run(X[:0], ids[:0], T[:0], lse[:0], g[:0], True, False, 1.0)
    assert [tuple(x.shape) for x in out] == [(0,), (0,), (0,), (0, 100)]


@pytest.mark.parametrize("M", [1, 3, 400])
def test_determinism_streams_and_graphs(cuda_lib, M):
    X, ids, T, lse, g = _inputs(M, 20000, 50, torch.bfloat16)

    def step(**kw):
        out = fb.fp8rl_distill_topk(X, ids, T, teacher_lse=lse, rest=True, **kw)
        return (*out, fb.fp8rl_distill_topk_backward(X, ids, T, out[1], g, teacher_lse=lse, rest_lse=out[2], **kw))

    want = [x.clone() for x in step()]
    assert all(torch.equal(a, b) for a, b in zip(want, step()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    other = _inputs(M, 20000, 50, torch.bfloat16, seed=4)
    for a, b in zip((X, ids, T, lse, g), other):
        a.copy_(b)
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    want = step()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_offsets_past_32_bits(cuda_lib):
    """Logits of more than 2^32 bytes: the last rows against 64 bits."""
    M, V = 16400, 152064
    X = torch.zeros((M, V), dtype=torch.bfloat16, device="cuda")
    small = _inputs(3, V, 16, torch.bfloat16, masked=0.0)
    X[-3:] = small[0]
    ids = small[1].repeat(M // 3 + 1, 1)[-M:].contiguous()
    T = small[2].repeat(M // 3 + 1, 1)[-M:].contiguous()
    lse, g = small[3].repeat(M // 3 + 1)[-M:].contiguous(), small[4].repeat(M // 3 + 1)[-M:].contiguous()
    # (how a row is cut goes by the number of rows, so the bits do not compare: the bounds do)
    out = fb.fp8rl_distill_topk(X, ids, T, teacher_lse=lse, rest=True)
    for a, b in zip(out, ref.distill(*small[:4], True, 1.0)):
        ref.check(a[-3:], b)
    dX = fb.fp8rl_distill_topk_backward(X, ids, T, out[1], g, teacher_lse=lse, rest_lse=out[2], dX=X)
    ref.check(dX[-3:], ref.distill_grad(small[0], small[1], small[2], small[4], small[3], True, 1.0))
