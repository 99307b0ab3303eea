"""Calls on a stream that is given: what they allocate is that stream's memory.  A block
of the caller's own stream could have work queued there that still reads it."""
import pytest
import torch

from precision_rl_rollout_gb300 import binding as fb

pytestmark = pytest.mark.gpu


def _stream_of(t):
    """The raw stream whose memory a tensor's is."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the caching allocator's")


def _unused_stream():
    """A stream that has no memory yet (they come from a pool, in turn)."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    used = {seg["stream"] for seg in torch.cuda.memory_snapshot()}
    return next(t for t in (torch.cuda.Stream() for _ in range(64)) if t.cuda_stream not in used)


def _rollout_calls():
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((64, 8, 128), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    table = torch.rand((64, 128), generator=g, device="cuda")
    K, V = (torch.randn((700, 16, 2, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    kv = x[:, :2]
    slots = torch.arange(64, device="cuda") + 690 * 16
    pages = torch.arange(680, dtype=torch.int32, device="cuda").view(2, 340)
    lens = torch.tensor([5440, 333], dtype=torch.int32, device="cuda")
    P = torch.softmax(torch.randn((3, 4, 1000), generator=g, device="cuda"), -1)
    drafts = torch.randint(0, 1000, (3, 3), generator=g, device="cuda", dtype=torch.int32)
    u, noise = torch.rand((3, 3), generator=g, device="cuda"), torch.rand((3, 1000), generator=g, device="cuda") + 0.1
    return {
        "rope": lambda **kw: fb.fp8rl_rope(x, pos, table, **kw),
        "append": lambda **kw: fb.fp8rl_rope_append_paged(x, kv, kv, pos, table, K, V, slots, **kw),
        "attn": lambda **kw: fb.fp8rl_attn_paged(x[:2].view(2, 1, 8, 128), K, V, pages, lens, 5440, want_lse=True, **kw),
        "verify": lambda **kw: fb.fp8rl_spec_verify(P, drafts, u, noise, **kw)}


def _outputs(r):
    return r if isinstance(r, tuple) else (r,)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["rope", "append", "attn", "verify"])
def test_rollout_calls_allocate_on_the_given_stream(cuda_lib, name, raw):
    call = _rollout_calls()[name]
    want = [t.clone() for t in _outputs(call())]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = _outputs(call(stream=s.cuda_stream if raw else s))
    assert all(_stream_of(t) == s.cuda_stream for t in got)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(_stream_of(t) != s.cuda_stream for t in _outputs(call()))
    assert fb.fp8rl_check_device_error() == 0


def test_attention_takes_its_workspace_from_the_given_stream(cuda_lib):
    call = _rollout_calls()["attn"]
    o, lse = call()
    assert fb.fp8rl_attn_paged_workspace_bytes(2, 1, 8, 2, 128, 5440) > 0
    s = _unused_stream()
    call(o=o, lse=lse, stream=s)
    s.synchronize()
    assert any(seg["stream"] == s.cuda_stream for seg in torch.cuda.memory_snapshot())


def test_a_freed_tensor_that_is_still_read_is_not_overwritten(cuda_lib):
    # a slow stream reads a tensor that has been freed already; calls of its size on
    # another stream are through long before
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((4096, 8, 128), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.zeros(4096, dtype=torch.int32, device="cuda")
    table = torch.ones((1, 128), device="cuda")
    kept = torch.empty_like(x)
    s = torch.cuda.Stream()
    for _ in range(3):
        held = x + 1
        want = held.cpu()
        torch.cuda.synchronize()
        torch.cuda._sleep(40_000_000)                          # some 20 ms
        kept.copy_(held)
        del held
        outs = [fb.fp8rl_rope(x, pos, table, stream=s) for _ in range(4)]
        s.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(kept.cpu(), want)
        del outs


def _layer_calls():
    g = torch.Generator(device="cuda").manual_seed(3)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    W, X, kv, P, Q = rand(512, 1024), rand(32, 1024), rand(8192, 1024), rand(4, 9000), rand(4, 9000)
    (Wq, Ws), (Xq, Xs) = fb.fp8rl_quant_weight_block(W), fb.fp8rl_quant_act_group(X)
    (W8, Ws8), (X8, Xs8) = fb.int8rl_quant_weight_channel(W), fb.int8rl_quant_act_token(X)
    scale = fb.fp8rl_quant_kv_tensor(kv)[1]
    lt, lr = (torch.randn(5000, generator=g, device="cuda") for _ in range(2))
    E, offs = Wq.view(4, 128, 1024), torch.tensor([0, 9, 9, 20, 32], dtype=torch.int32, device="cuda")
    freq = torch.rand(32, generator=g, device="cuda", dtype=torch.float64)
    return {
        "quant_weight": lambda **kw: fb.fp8rl_quant_weight_block(W, **kw),
        "quant_act": lambda **kw: fb.fp8rl_quant_act_group(X, **kw),
        "gemm": lambda **kw: fb.fp8rl_gemm_w8a8_block(Xq, Xs, Wq, Ws, **kw),
        "gemm_grouped": lambda **kw: fb.fp8rl_gemm_w8a8_block_grouped(Xq, Xs, E, Ws.view(4, 1, 8), offs, **kw),
        "linear": lambda **kw: fb.fp8rl_linear_w8a8_block(X, Wq, Ws, want_codes=True, **kw),
        "int8_quant_weight": lambda **kw: fb.int8rl_quant_weight_channel(W, **kw),
        "int8_quant_act": lambda **kw: fb.int8rl_quant_act_token(X, **kw),
        "int8_gemm": lambda **kw: fb.int8rl_gemm_w8a8(X8, Xs8, W8, Ws8, want_acc=True, **kw),
        "kv": lambda **kw: fb.fp8rl_quant_kv_tensor(kv, **kw),
        "kv_with_scale": lambda **kw: fb.fp8rl_quant_kv_with_scale(kv, scale, **kw),
        "importance": lambda **kw: fb.fp8rl_rollout_is_weights(lt, lr, **kw),
        "kl": lambda **kw: fb.fp8rl_logits_kl(P, Q, **kw),
        "table": lambda **kw: fb.fp8rl_rope_table(freq, 1000, **kw)}


@pytest.mark.parametrize("raw", [False, True])
def test_layer_calls_allocate_on_the_given_stream(cuda_lib, raw):
    for name, call in _layer_calls().items():
        want = [t.clone() for t in _outputs(call())]
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = _outputs(call(stream=s.cuda_stream if raw else s))
        assert all(_stream_of(t) == s.cuda_stream for t in got), name
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), name
    assert fb.fp8rl_check_device_error() == 0


@pytest.mark.parametrize("name", ["kv", "importance", "kl"])
def test_layer_calls_take_workspaces_from_the_given_stream(cuda_lib, name):
    call = _layer_calls()[name]
    keys = {"kv": ("KVq", "scale"), "importance": ("weights", "stats"), "kl": ("kl",)}[name]
    given = dict(zip(keys, _outputs(call())))
    s = _unused_stream()
    call(stream=s, **given)
    s.synchronize()
    assert any(seg["stream"] == s.cuda_stream for seg in torch.cuda.memory_snapshot())
    assert fb.fp8rl_check_device_error() == 0
