"""The trainer's losses where logits, weights or sums are at their ends: words of -inf under
an entropy's gradient, rows of lowest logits, targets that the policy is sure of, long sums."""
import pytest
import torch

import losses_ref as ref
from precision_rl_rollout_gb300 import binding as fb

pytestmark = pytest.mark.gpu


def _head(M, V, K, seed=0, spread=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed + M + 7 * V + 13 * K)
    H = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn((V, K), generator=g, device="cuda") * spread / K ** 0.5).to(torch.bfloat16)
    t = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    return H, W, t, torch.randn(M, generator=g, device="cuda"), torch.randn(M, generator=g, device="cuda") * 0.1


@pytest.mark.parametrize("M", [1, 20, 128, 300])
@pytest.mark.parametrize("scale", [0.5, 3.0])
def test_entropys_gradient_at_words_of_minus_infinity(cuda_lib, M, scale):
    """Words whose logit is -inf in every row have a gradient of 0, in rows without an
    entropy's gradient and with one; the other words' is as if those were not there."""
    H, W, t, g, ge = _head(M, 700, 64)
    H, t = (H.abs() + 0.125).to(torch.bfloat16), t.clamp(min=300)
    W[:300] = float("-inf")
    ge[::3] = 0.0
    _, lse, ent = fb.fp8rl_linear_logp(H, W, t, scale=scale, want_entropy=True)
    _, dW = fb.fp8rl_linear_logp_backward(H, W, t, lse, g, entropy=ent, g_entropy=ge, scale=scale, want_dH=False)
    assert (dW[:300] == 0).all()
    ref.check(dW[300:], ref.linear_logp_grad(H, W[300:], t - 300, g, ge, scale)[1], "dW")


def test_a_row_with_one_word_of_minus_infinity(cuda_lib):
    """One row's logit is -inf, the others' at that word are finite: its own part is 0."""
    H, W, t, g, ge = _head(150, 300, 64)
    W[7, 0], W[:, 1:8], H[:, 0] = -3.0e38, 0.0, 0.0       # only row 5 meets the word's lowest entry
    H[5, 0] = 4.0                                          # -1.2e39 is -inf in 32 bits
    t[5] = 3
    _, lse, ent = fb.fp8rl_linear_logp(H, W, t, want_entropy=True)
    _, dW = fb.fp8rl_linear_logp_backward(H, W, t, lse, g, entropy=ent, g_entropy=ge, want_dH=False)
    W2 = W.clone()
    W2[7, 0] = -1.0e4                                      # exp(-4e4) is 0 in 64 bits too
    ref.check(dW, ref.linear_logp_grad(H, W2, t, g, ge)[1], "dW")


@pytest.mark.parametrize("M", [20, 300])
def test_nan_passes_the_entropys_gradient(cuda_lib, M):
    """A word of NaN stays NaN in the gradient of every row that counts."""
    H, W, t, g, ge = _head(M, 300, 64)
    W[40] = float("nan")
    ones = torch.ones(M, device="cuda")
    dH, _ = fb.fp8rl_linear_logp_backward(H, W, t, ones, g, entropy=ones, g_entropy=ge, want_dW=False)
    assert dH.isnan().all()


def _sure(M, V, K, seed=0):
    """Rows whose targets have from a thousandth to all but 1e-6 of the probability and less."""
    H, W, t, g, ge = _head(M, V, K, seed)
    w = W[t.long()].float()
    lean = torch.linspace(4, 26, M, device="cuda")[:, None]
    return (H.float() + lean * w / (w ** 2).sum(1, keepdim=True)).to(torch.bfloat16), W, t, g, ge


@pytest.mark.parametrize("M", [100, 256])
@pytest.mark.parametrize("K", [64, 1024, 3584, 16384])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient_of_targets_that_are_all_but_sure(cuda_lib, M, K, entropy):
    """A target's D is g (1 - p): what its logit and the log-sum are off by differently is not
    relative to 1 - p.  In 32 bits that is the roundings of the log-sum and its product with
    log2 e (2^-24 each), of the argument (2^-24) and the exponential (2^-22): below |lse| 2^-22 +
    2^-21; with the entropy's gradient the same twice more (its logarithm, and the entropy's
    own).  All else is relative: D's rounding and the result's (2^-8 each) and a
    logit's error against the others', below 2^-12."""
    H, W, t, g, ge = _sure(M, 2048, K)
    x = H.double() @ W.double().T
    lse = torch.logsumexp(x, dim=1)
    logp = x - lse[:, None]
    others = logp.exp().scatter_(1, t.long()[:, None], 0.0)
    left = others.sum(1)                                   # 1 - p of the target
    logp.scatter_(1, t.long()[:, None], torch.log1p(-left)[:, None])
    p = logp.exp()
    D = -g.double()[:, None] * others
    D.scatter_(1, t.long()[:, None], (g.double() * left)[:, None])
    e = ge.double()[:, None] if entropy else torch.zeros((M, 1), dtype=torch.float64, device="cuda")
    ent = -(p * logp).sum(1, keepdim=True)
    D = D - e * p * (logp + ent)
    want = D @ W.double()
    _, mine, mine_ent = fb.fp8rl_linear_logp(H, W, t, want_entropy=True)
    kw = dict(entropy=mine_ent, g_entropy=ge) if entropy else {}
    dH, _ = fb.fp8rl_linear_logp_backward(H, W, t, mine, g, want_dW=False, **kw)
    most = W.double().norm(dim=1).max()
    once = lse.abs() * 2.0 ** -22 + 2.0 ** -21
    bound = most * ((g.double().abs() + 2 * e[:, 0].abs()) * once + D.abs().sum(1) * (2.0 ** -8 + 2.0 ** -12))
    bound = bound * (1 + 2.0 ** -7) + want.norm(dim=1) * 2.0 ** -8
    over = (dH.double() - want).norm(dim=1) / bound
    assert left.min() < 1e-6 and left.max() > 0.1 and over.max() <= 1.0, over.max().item()


@pytest.mark.parametrize("M,V,K", [(1 << 20, 24, 8), (300001, 9, 72), (70000, 300, 64)])
@pytest.mark.parametrize("sign", [False, True])
def test_gradient_over_many_rows(cuda_lib, M, V, K, sign):
    """dW sums over the rows that count.  With terms of one sign (sign) what a sum's steps lose
    adds up, and D's roundings (2^-8 each) do not: what is left is the result's rounding (2^-8 of
    itself, 2^-8 / sqrt 3 of its binade at most in the norm), some 2^-12 of the longest sum held in one
    place (65536 rows), and, at one in a few hundred of the terms' size, D's roundings.  Without, D's
    roundings are some 2^-8 / sqrt 3 as well: the two together 2^-8 sqrt(2 / 3), at most."""
    H, W, t, g, _ = _head(M, V, K)
    if sign:
        H, W, g = H.abs(), W.abs(), g.abs()
    t[::5] = -1
    _, lse = fb.fp8rl_linear_logp(H, W, t)
    _, dW = fb.fp8rl_linear_logp_backward(H, W, t, lse, g, want_dH=False)
    want = torch.zeros((V, K), dtype=torch.float64, device="cuda")
    for i in range(0, M, 1 << 16):
        rows = torch.arange(i, min(M, i + (1 << 16)), device="cuda")
        rows = rows[t[rows] >= 0]
        h = H[rows].double()
        D = -torch.softmax(h @ W.double().T, dim=1)
        D.scatter_add_(1, t[rows].long()[:, None], torch.ones((len(rows), 1), dtype=torch.float64, device="cuda"))
        want += (D * g[rows].double()[:, None]).T @ h
    off = ((dW.double() - want).norm() / want.norm()).item()
    assert off <= 2.0 ** -8 * ((1 / 3) ** 0.5 + 2.0 ** -4 if sign else (2 / 3) ** 0.5 + 2.0 ** -4), off
    assert fb.fp8rl_check_device_error() == 0


@pytest.mark.parametrize("M", [40, 100, 300])
@pytest.mark.parametrize("K", [3584, 5120, 16392])
def test_log_probabilities_keep_their_precision(cuda_lib, M, K):
    """In the norm.  A sum of n products in tensor memory goes through n / 16 steps, each of which drops
    up to one unit of 2^-23 of what is summed so far, on average half of it: with sums that grow
    evenly n / 64 units of 2^-23 of the whole; n is 256 at most up to 128 rows, 896 at
    most above.  Two more units for the rest of a log-probability, twice all for an entropy, where the
    errors meet weights p log p.  (A sum of all 3584 products would be off by 56 units.)"""
    H, W, t, _, _ = _head(M, 3000, K)
    out = fb.fp8rl_linear_logp(H, W, t, want_entropy=True)
    units = (256 if M <= 128 else 896) / 64 + 2
    for name, a, (value, _), times in zip(("logp", "lse", "entropy"), out, ref.linear_logp(H, W, t), (1, 1, 2)):
        off = ((a.double() - value).norm() / value.norm()).item()
        assert off <= times * units * 2.0 ** -23, (name, off / 2.0 ** -23)
