"""CPU checks of the trainer's losses: invalid arguments are refused synchronously, before
any CUDA call, and the binding refuses what only it can see."""
import pytest
import torch

from precision_rl_rollout_gb300 import binding, build

A = 0x10000  # a 16-byte-aligned fake device address: validation never dereferences it


@pytest.fixture(scope="module")
def lib():
    try:
        build.build()
    except RuntimeError as e:  # no nvcc on this machine
        pytest.skip(str(e))
    return binding.load()


def test_linear_logp_validation(lib):
    def f(H=A, ldh=64, W=A, ldw=64, t=A, M=4, V=100, K=64, scale=1.0, logp=A, lse=A, ent=None, ws=A, wb=None):
        need = lib.fp8rl_linear_logp_workspace_bytes(M, V, K)
        return lib.fp8rl_linear_logp(H, ldh, W, ldw, t, M, V, K, scale, logp, lse, ent, ws, need if wb is None else wb, None)
    assert f(M=0) == 0 and f(M=0, H=None, t=None, logp=None, lse=None, ws=None) == 0
    for name in ("H", "W", "t", "logp", "lse"):
        assert f(**{name: None}) == 1, name
    assert f(M=-1) == 2 and f(V=0) == 2 and f(K=0) == 2 and f(K=60) == 2 and f(ldh=56) == 2 and f(ldw=56) == 2
    assert f(H=A + 8) == 3 and f(W=A + 2) == 3 and f(ldh=68) == 3 and f(ldw=68) == 3 and f(t=A + 1) == 3
    assert f(logp=A + 2) == 3 and f(lse=A + 1) == 3 and f(ent=A + 2) == 3 and f(ws=A + 8) == 3
    need = lib.fp8rl_linear_logp_workspace_bytes(4, 100, 64)
    assert need > 0 and f(wb=need - 1) == 4 and f(ws=None) == 4
    assert f(M=(1 << 21) + 1) == 6 and f(V=(1 << 21) + 1) == 6 and f(K=65544, ldh=65544, ldw=65544) == 6
    for scale in (0.0, -1.0, float("nan"), float("inf"), 2.1e38):
        assert f(scale=scale) == 6
    for bad in ((0, 5, 8), (5, 0, 8), (5, 5, 0), (-1, 5, 8), ((1 << 21) + 1, 5, 8), (1 << 55, 5, 8), (1 << 62, 5, 8),
                (5, 1 << 62, 8), (5, 5, 65544)):
        assert lib.fp8rl_linear_logp_workspace_bytes(*bad) == 0
        assert lib.fp8rl_linear_logp_backward_workspace_bytes(*bad) == 0


def test_linear_logp_backward_validation(lib):
    def f(H=A, ldh=64, W=A, ldw=64, t=A, lse=A, ent=None, g=A, ge=None, M=4, V=100, K=64, scale=1.0, dH=A, dW=A, ws=A,
          wb=None):
        need = lib.fp8rl_linear_logp_backward_workspace_bytes(M, V, K)
        return lib.fp8rl_linear_logp_backward(H, ldh, W, ldw, t, lse, ent, g, ge, M, V, K, scale, dH, dW, ws,
                                              need if wb is None else wb, None)
    for name in ("H", "W", "t", "lse", "g"):
        assert f(**{name: None}) == 1, name
    assert f(dH=None, dW=None) == 1 and f(ge=A) == 1
    assert f(M=0, dW=None) == 0                                     # nothing to write
    assert f(M=-1) == 2 and f(V=0) == 2 and f(K=12) == 2 and f(ldh=56) == 2 and f(ldw=8) == 2
    for name in ("H", "W", "dH", "dW", "ws"):
        assert f(**{name: A + 8}) == 3, name
    assert f(ldw=66) == 3 and f(lse=A + 2) == 3 and f(g=A + 1) == 3 and f(ent=A, ge=A + 2) == 3 and f(ent=A + 2) == 3
    need = lib.fp8rl_linear_logp_backward_workspace_bytes(4, 100, 64)
    assert need > 0 and f(wb=need - 1) == 4 and f(ws=None) == 4
    assert f(scale=0.0) == 6 and f(V=1 << 22) == 6


def test_distill_validation(lib):
    def f(X=A, ld=104, dtype=1, ids=A, T=A, tl=A, M=4, V=100, k=8, scale=1.0, loss=A, lse=A, rest=None):
        return lib.fp8rl_distill_topk(X, ld, dtype, ids, T, tl, M, V, k, scale, loss, lse, rest, None)

    def b(X=A, ld=104, dtype=1, ids=A, T=A, tl=A, lse=A, rest=None, g=A, M=4, V=100, k=8, scale=1.0, dX=A + 4096, ldd=104):
        return lib.fp8rl_distill_topk_backward(X, ld, dtype, ids, T, tl, lse, rest, g, M, V, k, scale, dX, ldd, None)
    assert f(M=0) == 0 and b(M=0) == 0
    for name in ("X", "ids", "T", "lse"):
        assert f(**{name: None}) == 1 and b(**{name: None}) == 1, name
    assert f(loss=None) == 1 and b(g=None) == 1 and b(dX=None) == 1
    assert f(rest=A, tl=None) == 1 and b(rest=A, tl=None) == 1      # the rest needs the teacher's log-sum
    for h in (f, b):
        assert h(M=-1) == 2 and h(V=0) == 2 and h(k=0) == 2 and h(ld=96) == 2
        assert h(X=A + 8) == 3 and h(ld=108) == 3 and h(ids=A + 1) == 3 and h(T=A + 2) == 3 and h(tl=A + 1) == 3
        assert h(ld=102, dtype=0) == 3 and h(rest=A + 1) == 3 and h(lse=A + 3) == 3
        assert h(dtype=2) == 6 and h(k=1025) == 6 and h(V=(1 << 20) + 1, ld=1 << 21) in (2, 6)
        assert h(scale=0.0) == 6 and h(scale=float("nan")) == 6 and h(M=1 << 31) == 6
    assert b(ldd=96) == 2 and b(ldd=108) == 3 and b(dX=A + 8) == 3
    assert b(dX=A, ldd=112) == 2                                    # in place with another pitch


def test_binding_refusals():
    h, w = torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros((9, 64), dtype=torch.bfloat16)
    t, v = torch.zeros(2, dtype=torch.int32), torch.zeros(2)
    try:
        binding.load()
    except RuntimeError as e:
        pytest.skip(str(e))
    with pytest.raises(ValueError):
        binding.fp8rl_linear_logp(h, w, t)                          # not on a GPU
    with pytest.raises(ValueError):
        binding.fp8rl_linear_logp_backward(h, w, t, v, v)
    with pytest.raises(ValueError):
        binding.fp8rl_distill_topk(h, t[:, None], v[:, None])
    with pytest.raises(ValueError):
        binding.fp8rl_distill_topk_backward(h, t[:, None], v[:, None], v, v)


@pytest.mark.gpu
def test_binding_refusals_on_the_device(cuda_lib):
    fb, dev = binding, dict(device="cuda")
    h, w = torch.zeros((2, 64), dtype=torch.bfloat16, **dev), torch.zeros((9, 64), dtype=torch.bfloat16, **dev)
    t, v = torch.zeros(2, dtype=torch.int32, **dev), torch.zeros(2, **dev)
    x, ids, T = torch.zeros((2, 16), **dev), torch.zeros((2, 3), dtype=torch.int32, **dev), torch.zeros((2, 3), **dev)
    bad = [lambda: fb.fp8rl_linear_logp(h.float(), w, t), lambda: fb.fp8rl_linear_logp(h, w.half(), t),
           lambda: fb.fp8rl_linear_logp(h, w[:, :32], t), lambda: fb.fp8rl_linear_logp(h, w, t.long()),
           lambda: fb.fp8rl_linear_logp(h, w, t[:1]), lambda: fb.fp8rl_linear_logp(h, w, t.cpu()),
           lambda: fb.fp8rl_linear_logp(h, w.cpu(), t), lambda: fb.fp8rl_linear_logp(h, w, t, logp=v[:1]),
           lambda: fb.fp8rl_linear_logp(h, w.T.contiguous().T, t), lambda: fb.fp8rl_linear_logp(h, w, t, scale="1"),
           lambda: fb.fp8rl_linear_logp(h, w, t, workspace=torch.zeros(64)),
           lambda: fb.fp8rl_linear_logp_backward(h, w, t, v, v[:1]),
           lambda: fb.fp8rl_linear_logp_backward(h, w, t, v, v, g_entropy=v),
           lambda: fb.fp8rl_linear_logp_backward(h, w, t, v, v, want_dH=False, want_dW=False),
           lambda: fb.fp8rl_linear_logp_backward(h, w, t, v, v, dH=h[:1]),
           lambda: fb.fp8rl_linear_logp_backward(h, w, t, v, v, dW=w.float()),
           lambda: fb.fp8rl_distill_topk(x.half(), ids, T), lambda: fb.fp8rl_distill_topk(x, ids.long(), T),
           lambda: fb.fp8rl_distill_topk(x, ids, T[:, :2]), lambda: fb.fp8rl_distill_topk(x, ids, T, rest=True),
           lambda: fb.fp8rl_distill_topk(x.T, ids, T), lambda: fb.fp8rl_distill_topk(x, ids, T.double()),
           lambda: fb.fp8rl_distill_topk_backward(x, ids, T, v, v, rest_lse=v),
           lambda: fb.fp8rl_distill_topk_backward(x, ids, T, v, v, dX=x[:1]),
           lambda: fb.fp8rl_distill_topk_backward(x, ids, T, v, v, dX=x.bfloat16())]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(str(i))
    for call, status in ((lambda: fb.fp8rl_linear_logp(h[:, :60], w[:, :60], t), 2),
                         (lambda: fb.fp8rl_linear_logp(h, w, t, scale=-1.0), 6),
                         (lambda: fb.fp8rl_linear_logp(h[:, 1:9], w[:, 1:9], t), 3),
                         (lambda: fb.fp8rl_linear_logp(h[:1].expand(2, 64), w, t), 2),
                         (lambda: fb.fp8rl_linear_logp(h, w, t, workspace=torch.zeros(16, dtype=torch.uint8, **dev)), 4),
                         (lambda: fb.fp8rl_distill_topk(x[:, :0], ids, T), 2),
                         (lambda: fb.fp8rl_distill_topk(torch.zeros((2, 15), **dev), ids, T), 3),
                         (lambda: fb.fp8rl_distill_topk(x, ids[:, :0], T[:, :0]), 2)):
        with pytest.raises(fb.Fp8rlError) as e:
            call()
        assert e.value.status == status
    assert fb.fp8rl_check_device_error() == 0
