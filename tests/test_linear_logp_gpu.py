"""Log-probabilities from hidden states and their gradient, against 64 bits."""
import pytest
import torch

import losses_ref as ref
from precision_rl_rollout_gb300 import binding as fb

pytestmark = pytest.mark.gpu

# (M, V, K): one row, one word, tiles and their edges, few rows and more (from 65 and 129 on other
# kernels), odd vocabularies, short and long products, a vocabulary in several pieces
SIZES = [(65, 300, 128), (128, 1000, 192), (129, 600, 64), (3, 300, 65536), (150, 520, 16392), (70001, 3000, 64),
         (1, 1, 8), (1, 1000, 64), (2, 130, 72), (31, 513, 136), (32, 40000, 64), (33, 257, 200), (64, 128, 8), (130, 515, 264),
         (255, 2049, 512), (256, 256, 256), (257, 4100, 1024), (700, 1537, 328), (1025, 300, 96), (5, 7, 4104)]


def _inputs(M, V, K, masked=0.3, seed=0, spread=2.5, h_pad=0, w_pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed + M + 7 * V + 13 * K)
    H = torch.randn((M, K + h_pad), generator=g, device="cuda").to(torch.bfloat16)[:, :K]
    W = (torch.randn((V, K + w_pad), generator=g, device="cuda") * spread / K ** 0.5).to(torch.bfloat16)[:, :K]
    t = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    out = torch.rand(M, generator=g, device="cuda") < masked
    t[out] = torch.where(torch.arange(M, device="cuda")[out] % 2 == 0, -1, V).to(torch.int32)
    H[out] = float("nan")
    grads = [torch.randn(M, generator=g, device="cuda"), torch.randn(M, generator=g, device="cuda") * 0.1]
    return H, W, t, grads


@pytest.mark.parametrize("M,V,K", SIZES)
@pytest.mark.parametrize("masked", [0.0, 0.3])
def test_forward(cuda_lib, M, V, K, masked):
    H, W, t, _ = _inputs(M, V, K, masked)
    want = ref.linear_logp(H, W, t, 1.3)
    got = fb.fp8rl_linear_logp(H, W, t, scale=1.3, want_entropy=True)
    for name, a, b in zip(("logp", "lse", "entropy"), got, want):
        ref.check(a, b, name)
    two = fb.fp8rl_linear_logp(H, W, t, scale=1.3)
    assert len(two) == 2 and torch.equal(two[0], got[0]) and torch.equal(two[1], got[1])
    assert fb.fp8rl_check_device_error() == 0


@pytest.mark.parametrize("M,V,K", SIZES)
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient(cuda_lib, M, V, K, entropy):
    H, W, t, (g, ge) = _inputs(M, V, K, 0.3 if M > 1 else 0.0)
    (want_h, want_w) = ref.linear_logp_grad(H, W, t, g, ge if entropy else None, 0.7)
    _, lse, ent = fb.fp8rl_linear_logp(H, W, t, scale=0.7, want_entropy=True)
    kw = dict(entropy=ent, g_entropy=ge) if entropy else {}
    dH, dW = fb.fp8rl_linear_logp_backward(H, W, t, lse, g, scale=0.7, **kw)
    ref.check(dH, want_h, "dH")
    ref.check(dW, want_w, "dW")
    one, none = fb.fp8rl_linear_logp_backward(H, W, t, lse, g, scale=0.7, want_dW=False, **kw)
    assert none is None and torch.equal(one, dH)
    none, one = fb.fp8rl_linear_logp_backward(H, W, t, lse, g, scale=0.7, want_dH=False, **kw)
    assert none is None and torch.equal(one, dW)
    assert fb.fp8rl_check_device_error() == 0


def test_gradient_against_differences(cuda_lib):
    H, W, t, (g, ge) = _inputs(90, 700, 128, 0.2, seed=3)
    _, lse, ent = fb.fp8rl_linear_logp(H, W, t, want_entropy=True)
    dH, dW = fb.fp8rl_linear_logp_backward(H, W, t, lse, g, entropy=ent, g_entropy=ge)
    live = t.ge(0) & t.lt(700)
    gen = torch.Generator(device="cuda").manual_seed(9)

    def loss(h, w):
        full = torch.log_softmax(h @ w.T, dim=1)
        logp = full.gather(1, t.clamp(0, 699).long()[:, None])[:, 0]
        entropy = -(full.exp() * full).sum(1)
        return (torch.where(live, g, 0.0).double() * logp + torch.where(live, ge, 0.0).double() * entropy).sum()

    h, w = torch.where(live[:, None], H, 0).double(), W.double()
    for x, d, at in ((h, dH, 0), (w, dW, 1)):
        for _ in range(3):
            u = torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)
            eps = 1e-5
            up, down = (loss(*((x + s * eps * u, w) if at == 0 else (h, x + s * eps * u))) for s in (1, -1))
            slope = ((up - down) / (2 * eps)).item()
            # the gradient's entries are off by at most some 2^-7 of terms that add up at random
            noise = 2.0 ** -7 * (d.double() * u).norm().item() * 3 + 1e-6 * abs(slope)
            assert abs((d.double() * u).sum().item() - slope) <= noise


def test_constant_gradient_keeps_its_precision(cuda_lib):
    """The mean's gradient, one over a count that is no power of two, over a nearly uniform
    distribution: D is relative to the largest gradient, so its rounding does not show."""
    M, V, K = 300, 4099, 256
    H, W, t, _ = _inputs(M, V, K, 0.0, spread=0.1)
    g = torch.full((M,), -1.0 / 303, device="cuda")
    _, lse = fb.fp8rl_linear_logp(H, W, t)
    dH, _ = fb.fp8rl_linear_logp_backward(H, W, t, lse, g, want_dW=False)
    value = ref.linear_logp_grad(H, W, t, g)[0][0]
    # one rounding to bf16 is 2^-8 / sqrt 3 of a value's binade, between 0.5 and 1 of that of the value:
    # below 2^-8.5 of the norm with the small probabilities' own roundings, where 1/303 rounded to bf16 alone is off by 2^-8.6
    assert ((dH.double() - value).norm() / value.norm()).item() <= 2.0 ** -9


@pytest.mark.parametrize("M", [3, 300])
def test_nobody_counts(cuda_lib, M):
    H, W, _, (g, _) = _inputs(M, 500, 64, 0.0)
    H.fill_(float("inf"))
    t = torch.full((M,), -100, dtype=torch.int32, device="cuda")
    out = fb.fp8rl_linear_logp(H, W, t, want_entropy=True)
    assert all((x == 0).all() for x in out)
    grads = fb.fp8rl_linear_logp_backward(H, W, t, out[1], g, entropy=out[2], g_entropy=g)
    assert all((x == 0).all() for x in grads)


def test_no_rows(cuda_lib):
    H, W, t, (g, _) = _inputs(4, 300, 64)
    out = fb.fp8rl_linear_logp(H[:0], W, t[:0], want_entropy=True)
    assert [tuple(x.shape) for x in out] == [(0,)] * 3
    dW = torch.full((300, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    dH, _ = fb.fp8rl_linear_logp_backward(H[:0], W, t[:0], out[1], g[:0], dW=dW)
    assert dH.shape == (0, 64) and (dW == 0).all()


@pytest.mark.parametrize("M", [20, 333])
def test_pitches_and_given_outputs(cuda_lib, M):
    H, W, t, (g, _) = _inputs(M, 777, 200, 0.2, h_pad=24, w_pad=8)
    W = W[5:700]                                            # an odd part of the matrix, rows 208 values apart
    t = torch.where(t >= 695, -1, t)
    logp, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    out = fb.fp8rl_linear_logp(H, W, t, logp=logp, lse=lse)
    assert out[0] is logp or out[0].data_ptr() == logp.data_ptr()
    want = ref.linear_logp(H, W, t)
    ref.check(logp, want[0], "logp")
    ref.check(lse, want[1], "lse")
    guard = torch.full((M + 2, 200), 3.0, dtype=torch.bfloat16, device="cuda")
    wide = torch.full((697, 200), 3.0, dtype=torch.bfloat16, device="cuda")
    fb.fp8rl_linear_logp_backward(H, W, t, lse, g, dH=guard[1:-1], dW=wide[1:-1])
    wants = ref.linear_logp_grad(H, W, t, g)
    ref.check(guard[1:-1], wants[0], "dH")
    ref.check(wide[1:-1], wants[1], "dW")
    assert (guard[[0, -1]] == 3).all() and (wide[[0, -1]] == 3).all()


@pytest.mark.parametrize("M", [7, 200])
def test_extreme_logits(cuda_lib, M):
    """A row that is sure of its token, and logits of both signs in the thousands."""
    H, W, t, (g, ge) = _inputs(M, 900, 128, 0.0)
    H = (H.float() * 40).to(torch.bfloat16)
    out = fb.fp8rl_linear_logp(H, W, t, scale=8.0, want_entropy=True)
    for a, b in zip(out, ref.linear_logp(H, W, t, 8.0)):
        ref.check(a, b)
    grads = fb.fp8rl_linear_logp_backward(H, W, t, out[1], g, entropy=out[2], g_entropy=ge, scale=8.0)
    for a, b in zip(grads, ref.linear_logp_grad(H, W, t, g, ge, 8.0)):
        ref.check(a, b)


@pytest.mark.parametrize("M", [9, 300])
def test_same_token_and_zero_gradients(cuda_lib, M):
    H, W, t, (g, _) = _inputs(M, 300, 64, 0.0)
    t = torch.full_like(t, 299)
    _, lse = fb.fp8rl_linear_logp(H, W, t)
    dH, dW = fb.fp8rl_linear_logp_backward(H, W, t, lse, torch.zeros_like(g))
    assert (dH == 0).all() and (dW == 0).all()
    g[::2] = 0.0
    g = g * 1e-30
    for a, b in zip(fb.fp8rl_linear_logp_backward(H, W, t, lse, g), ref.linear_logp_grad(H, W, t, g)):
        ref.check(a, b)


@pytest.mark.parametrize("M", [20, 128, 300])
def test_words_of_minus_infinity(cuda_lib, M):
    """Logits of -inf for every word of a tile and some of the next are probabilities of 0; no
    row's gradient reaches their words."""
    H, W, t, (g, _) = _inputs(M, 700, 64, 0.0)
    H, t = (H.abs() + 0.125).to(torch.bfloat16), t.clamp(min=300)
    W[:300] = float("-inf")
    for scale in (0.5, 3.0):
        out = fb.fp8rl_linear_logp(H, W, t, scale=scale, want_entropy=True)
        finite = [ref.linear_logp(H, W[300:], t - 300, scale), ref.linear_logp_grad(H, W[300:], t - 300, g, None, scale)]
        for a, b in zip(out, finite[0]):
            ref.check(a, b)
        _, dW = fb.fp8rl_linear_logp_backward(H, W, t, out[1], g, scale=scale, want_dH=False)
        assert (dW[:300] == 0).all()
        ref.check(dW[300:], finite[1][1])


@pytest.mark.parametrize("what", [float("inf"), float("nan")])
def test_a_broken_gradient_stays_in_its_row(cuda_lib, what):
    H, W, t, (g, ge) = _inputs(300, 700, 64, 0.2)
    broken, zero = g.clone(), g.clone()
    t[5], broken[5], zero[5] = 3, what, 0.0
    H[5] = 1.0
    _, lse, ent = fb.fp8rl_linear_logp(H, W, t, want_entropy=True)
    a, _ = fb.fp8rl_linear_logp_backward(H, W, t, lse, broken, entropy=ent, g_entropy=ge)
    b, _ = fb.fp8rl_linear_logp_backward(H, W, t, lse, zero, entropy=ent, g_entropy=ge)
    others = torch.arange(300, device="cuda") != 5
    assert torch.equal(a[others], b[others]) and not torch.isfinite(a[5]).any()


@pytest.mark.parametrize("M,V,K", [(1 << 21, 9, 8), (2, 1 << 21, 64), (140, 1 << 21, 64)])
def test_most_rows_and_words(cuda_lib, M, V, K):
    H, W, t, (g, ge) = _inputs(M, V, K)
    t[-1], H[-1] = V - 1, 1.0
    out = fb.fp8rl_linear_logp(H, W, t, want_entropy=True)
    for a, b in zip(out, ref.linear_logp(H, W, t)):
        ref.check(a, b)
    grads = fb.fp8rl_linear_logp_backward(H, W, t, out[1], g, entropy=out[2], g_entropy=ge)
    for a, b in zip(grads, ref.linear_logp_grad(H, W, t, g, ge)):
        ref.check(a, b)


def test_offsets_past_32_bits(cuda_lib):
    """A matrix of more than 2^32 bytes and 2^31 values, the target in its last row."""
    V, K, M = 152064, 16384, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    W = torch.zeros((V, K), dtype=torch.bfloat16, device="cuda")
    W[V - 300:] = (torch.randn((300, K), generator=g, device="cuda") / 128).to(torch.bfloat16)
    H = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    t = torch.tensor([V - 1, 5, V - 300], dtype=torch.int32, device="cuda")
    logp, lse, entropy = fb.fp8rl_linear_logp(H, W, t, want_entropy=True)
    x = torch.cat([H.double() @ W[V - 300:].double().T, torch.zeros((M, V - 300), dtype=torch.float64, device="cuda")], 1)
    want = torch.logsumexp(x, 1)
    picked = torch.stack([x[0, 299], x[1, 300], x[2, 0]])
    assert (lse.double() - want).abs().max() <= 1e-3 and (logp.double() - (picked - want)).abs().max() <= 2e-3
    gl = torch.tensor([1.0, -1.0, 0.5], device="cuda")
    dH, dW = fb.fp8rl_linear_logp_backward(H, W, t, lse, gl)
    p = torch.exp(x - want[:, None])[:, :300]
    D = -p * gl.double()[:, None]
    D[0, 299] += 1.0
    D[2, 0] += 0.5
    for got, value in ((dH, D @ W[V - 300:].double()), (dW[V - 300:], D.T @ H.double())):
        assert ((got.double() - value).norm() / value.norm()).item() <= 2.0 ** -7
    base = -(torch.exp(-want)[:, None] * gl.double()[:, None] * H.double()).sum(0)
    base5 = base - H[1].double()                           # row 5 is the target of g = -1
    assert ((dW[5].double() - base5).norm() / base5.norm()).item() <= 2.0 ** -7
    assert ((dW[77000].double() - base).norm() / base.norm()).item() <= 2.0 ** -7


@pytest.mark.parametrize("M,V,K", [(20, 3000, 128), (400, 3000, 128)])
def test_determinism_streams_and_graphs(cuda_lib, M, V, K):
    H, W, t, (g, ge) = _inputs(M, V, K)

    def step(**kw):
        out = fb.fp8rl_linear_logp(H, W, t, want_entropy=True, **kw)
        return (*out, *fb.fp8rl_linear_logp_backward(H, W, t, out[1], g, entropy=out[2], g_entropy=ge, **kw))

    want = [x.clone() for x in step()]
    assert all(torch.equal(a, b) for a, b in zip(want, step()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # an odd number of bytes of dirt in the workspace changes nothing
    need = fb.fp8rl_linear_logp_backward_workspace_bytes(M, V, K)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    again = fb.fp8rl_linear_logp_backward(H, W, t, want[1], g, entropy=want[2], g_entropy=ge, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(want[3:], again))
    # captured, replayed on other inputs, and two graphs in turn
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    other = _inputs(M, V, K, seed=5)
    H.copy_(other[0]), W.copy_(other[1]), t.copy_(other[2])
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    want = step()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(want, out))
    assert fb.fp8rl_check_device_error() == 0


def test_two_calls_at_once(cuda_lib):
    H, W, t, (g, _) = _inputs(300, 5000, 256)
    want = fb.fp8rl_linear_logp(H, W, t)
    grads = fb.fp8rl_linear_logp_backward(H, W, t, want[1], g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [(fb.fp8rl_linear_logp(H, W, t, stream=s), fb.fp8rl_linear_logp_backward(H, W, t, want[1], g, stream=s))
           for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    for out, back in got:
        assert all(torch.equal(a, b) for a, b in zip((*want, *grads), (*out, *back)))
