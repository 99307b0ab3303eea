"""The trainer's losses on a stream that is given: what they allocate, workspaces among it,
is that stream's memory, and results are the same."""
import pytest
import torch

from precision_rl_rollout_gb300 import binding as fb
from test_streams_gpu import _outputs, _stream_of, _unused_stream

pytestmark = pytest.mark.gpu


def _calls():
    g = torch.Generator(device="cuda").manual_seed(4)
    H = torch.randn((200, 128), generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn((3001, 128), generator=g, device="cuda").to(torch.bfloat16)
    t = torch.randint(-200, 3001, (200,), generator=g, device="cuda", dtype=torch.int32)
    v = torch.randn(200, generator=g, device="cuda")
    lse = fb.fp8rl_linear_logp(H, W, t)[1]
    X = torch.randn((200, 3008), generator=g, device="cuda")[:, :3001]
    T, ids = X.topk(16, dim=1)
    T, ids, tl = T.contiguous(), ids.int().contiguous(), torch.logsumexp(X, 1) + 0.1
    _, s, r = fb.fp8rl_distill_topk(X, ids, T, teacher_lse=tl, rest=True)
    return {"logp": lambda **kw: fb.fp8rl_linear_logp(H, W, t, want_entropy=True, **kw),
            "logp_few": lambda **kw: fb.fp8rl_linear_logp(H[:50], W, t[:50], **kw),
            "logp_backward": lambda **kw: fb.fp8rl_linear_logp_backward(H, W, t, lse, v, **kw),
            "distill": lambda **kw: fb.fp8rl_distill_topk(X, ids, T, teacher_lse=tl, rest=True, **kw),
            "distill_backward": lambda **kw: fb.fp8rl_distill_topk_backward(X, ids, T, s, v, teacher_lse=tl, rest_lse=r, **kw)}


@pytest.mark.parametrize("raw", [False, True])
def test_allocations_on_the_given_stream(cuda_lib, raw):
    for name, call in _calls().items():
        want = [t.clone() for t in _outputs(call())]
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = _outputs(call(stream=s.cuda_stream if raw else s))
        assert all(_stream_of(t) == s.cuda_stream for t in got), name
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), name
        assert all(_stream_of(t) != s.cuda_stream for t in _outputs(call())), name
    assert fb.fp8rl_check_device_error() == 0


@pytest.mark.parametrize("name,keys", [("logp", ("logp", "lse", "entropy")), ("logp_few", ("logp", "lse")),
                                       ("logp_backward", ("dH", "dW"))])
def test_workspaces_on_the_given_stream(cuda_lib, name, keys):
    call = _calls()[name]
    given = dict(zip(keys, _outputs(call())))
    s = _unused_stream()
    call(stream=s, **given)
    s.synchronize()
    assert any(seg["stream"] == s.cuda_stream for seg in torch.cuda.memory_snapshot())
