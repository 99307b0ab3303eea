"""Verification of drafted tokens against the definition, exactly."""
import numpy as np
import pytest
import torch

import rollout_ops_ref as ref
from precision_rl_rollout_gb300 import binding as fb

pytestmark = pytest.mark.gpu


def _case(B, K, V, seed, near=0.5, dtype=torch.float32, drafter=True):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, K, V), generator=g) * 2
    p = torch.randn((B, K + 1, V), generator=g) * near
    p[:, :K] += q
    P, Q = torch.softmax(p, -1).to(dtype), torch.softmax(q, -1).to(dtype)
    drafts = torch.zeros((B, K), dtype=torch.int32)
    for b in range(B):
        for i in range(K):
            drafts[b, i] = int(torch.multinomial(Q[b, i].float(), 1, generator=g))
    lens = torch.randint(0, K + 1, (B,), generator=g, dtype=torch.int32)
    u = torch.rand((B, K), generator=g)
    noise = torch.empty((B, V)).exponential_(generator=g)
    return P, (Q if drafter else None), drafts, lens, u, noise


def _run(P, Q, drafts, lens, u, noise):
    t, a = fb.fp8rl_spec_verify(P.cuda(), drafts.cuda(), u.cuda(), noise.cuda(), Q=None if Q is None else Q.cuda(),
                                draft_lens=None if lens is None else lens.cuda())
    return t.cpu().numpy(), a.cpu().numpy()


def _want(P, Q, drafts, lens, u, noise):
    B, K = drafts.shape
    return ref.verify(P.float().numpy(), None if Q is None else Q.float().numpy(), drafts.numpy(),
                      np.full(B, K) if lens is None else lens.numpy(), u.numpy(), noise.numpy())


@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,K,V", [(1, 4, 1000), (37, 1, 257), (5, 8, 4099), (3, 32, 63), (64, 3, 1), (2, 2, 50257),
                                   (1, 5, 152064), (700, 2, 40)])
def test_against_the_definition(cuda_lib, B, K, V, dtype, drafter):
    c = _case(B, K, V, B + K + V, dtype=dtype, drafter=drafter)
    t, a = _run(*c)
    wt, wa = _want(*c)
    assert np.array_equal(a, wa) and np.array_equal(t, wt)
    t, a = _run(c[0], c[1], c[2], None, c[4], c[5])
    wt, wa = _want(c[0], c[1], c[2], None, c[4], c[5])
    assert np.array_equal(a, wa) and np.array_equal(t, wt)
    assert fb.fp8rl_check_device_error() == 0


def test_no_drafts_at_all(cuda_lib):
    P, _, _, _, _, noise = _case(6, 1, 999, 3)
    P = P[:, :1].contiguous()
    z = torch.zeros((6, 0))
    t, a = fb.fp8rl_spec_verify(P.cuda(), z.int().cuda(), z.cuda(), noise.cuda())
    assert not a.any()
    assert np.array_equal(t.cpu().numpy()[:, 0], (P[:, 0] / noise).argmax(-1).numpy())


def test_equal_scores_go_to_the_lowest_token(cuda_lib):
    V = 30000
    P = torch.zeros((3, 1, V))
    P[0, 0, [29999, 17, 4096, 20000]] = 0.25
    P[1, 0, :] = 1.0 / V
    P[2, 0, 12345] = 1.0
    noise = torch.ones((3, V))
    z = torch.zeros((3, 0))
    t, _ = fb.fp8rl_spec_verify(P.cuda(), z.int().cuda(), z.cuda(), noise.cuda())
    assert t.cpu().numpy()[:, 0].tolist() == [17, 0, 12345]


def test_certain_and_impossible_drafts_and_empty_residuals(cuda_lib):
    V = 5000
    P = torch.zeros((4, 2, V))
    Q = torch.zeros((4, 1, V))
    P[:, 1, 7] = 1.0
    P[0, 0, 3] = 1.0; Q[0, 0, 3] = 1.0                  # kept for every u below 1
    P[1, 0, 4] = 1.0; Q[1, 0, 3] = 1.0                  # p is 0 there: never kept, not even at u = 0
    P[2, 0, 3] = 0.5; P[2, 0, 9] = 0.5; Q[2, 0, 3] = 1.0
    P[3, 0, 3] = 0.5; P[3, 0, 8] = 0.25; Q[3, 0, 3] = 1.0; Q[3, 0, 8] = 0.25   # refused, residual empty: from p
    drafts = torch.full((4, 1), 3, dtype=torch.int32)
    u = torch.tensor([[1 - 2.0 ** -24], [0.0], [0.5], [0.75]])
    noise = torch.ones((4, V))
    noise[3, 3] = 4.0                                     # 0.5 / 4 < 0.25 / 1
    t, a = _run(P, Q, drafts, None, u, noise)
    assert a.tolist() == [1, 0, 0, 0]
    assert t.tolist() == [[3, 7], [4, -1], [9, -1], [8, -1]]


def test_products_that_32_bits_would_round(cuda_lib):
    # u q just below, at and above p, by less than an fp32 rounding of the product
    V = 64
    u = np.float32(1 - 2.0 ** -24)
    q = np.float32(0.3)
    exact = np.float64(u) * np.float64(q)
    p = np.float32(exact)
    up, down = np.nextafter(p, np.float32(1)), np.nextafter(p, np.float32(0))
    P, Q = torch.zeros((3, 2, V)), torch.zeros((3, 1, V))
    for b, x in enumerate((p, up, down)):
        P[b, 0, 1], P[b, 0, 2], Q[b, 0, 1] = float(x), 0.5, float(q)
    P[:, 1, 5] = 1.0
    drafts = torch.ones((3, 1), dtype=torch.int32)
    _, a = _run(P, Q, drafts, None, torch.full((3, 1), float(u)), torch.ones((3, V)))
    assert a.tolist() == [int(exact < p), int(exact < up), int(exact < down)]


def test_zero_noise_nan_and_infinities(cuda_lib):
    V = 300
    P = torch.full((3, 1, V), 1.0 / V)
    noise = torch.ones((3, V))
    noise[0, 211] = 0.0                                   # an infinite score wins
    P[1, 0, 40] = float("nan")                            # takes no part
    P[1, 0, 41] = 0.5
    P[2] = 0.0                                            # nothing has weight: token 0
    z = torch.zeros((3, 0))
    t, _ = fb.fp8rl_spec_verify(P.cuda(), z.int().cuda(), z.cuda(), noise.cuda())
    assert t.cpu().numpy()[:, 0].tolist() == [211, 41, 0]


def test_drafts_and_lengths_out_of_range_are_recorded(cuda_lib):
    P, Q, drafts, _, u, noise = _case(3, 2, 100, 8)
    u = torch.zeros_like(u)
    drafts[1, 0] = 100
    drafts[2, 1] = -1
    lens = torch.tensor([2, 2, 2], dtype=torch.int32)
    _, a = _run(P, Q, drafts, lens, u, noise)
    assert a.tolist() == [2, 0, 1]
    assert fb.fp8rl_check_device_error() != 0
    drafts = drafts.clamp(0, 99)
    _, a = _run(P, Q, drafts, torch.tensor([5, -2, 1], dtype=torch.int32), u, noise)
    assert a.tolist() == [2, 0, 1]
    assert fb.fp8rl_check_device_error() != 0
    assert fb.fp8rl_check_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,pad", [(4096, 0), (4097, 0), (4096, 5), (1003, 1)])
def test_strides_and_alignment(cuda_lib, V, pad, dtype):
    P, Q, drafts, lens, u, noise = _case(6, 3, V, V + pad, dtype=dtype)

    def wide(x, lead):
        w = torch.full((*x.shape[:-1], x.shape[-1] + pad + lead), float("nan"), dtype=x.dtype, device="cuda")
        w[..., lead:lead + V] = x.cuda()
        return w[..., lead:lead + V]

    for lead in (0, 1):
        t, a = fb.fp8rl_spec_verify(wide(P, lead), drafts.cuda(), u.cuda(), wide(noise, 0), Q=wide(Q, lead),
                                    draft_lens=lens.cuda())
        wt, wa = _want(P, Q, drafts, lens, u, noise)
        assert np.array_equal(a.cpu().numpy(), wa) and np.array_equal(t.cpu().numpy(), wt)


def test_the_race_draws_the_targets_distribution(cuda_lib):
    # 40000 sequences, one draft from q each, every random number fresh: the first
    # emitted token is distributed as p, whatever q is.  A cell of expected count
    # n is within 5 sqrt(n) (about 6 cells: chance of a failure below 1e-5)
    B, V = 40000, 6
    g = torch.Generator().manual_seed(99)
    p = torch.tensor([0.3, 0.05, 0.2, 0.0, 0.4, 0.05])
    q = torch.tensor([0.05, 0.25, 0.2, 0.3, 0.1, 0.1])
    P = p.expand(B, 2, V).contiguous()
    Q = q.expand(B, 1, V).contiguous()
    drafts = torch.multinomial(q, B, replacement=True, generator=g).int()[:, None].contiguous()
    u, noise = torch.rand((B, 1), generator=g), torch.empty((B, V)).exponential_(generator=g)
    t, _ = _run(P, Q, drafts, None, u, noise)
    n = np.bincount(t[:, 0], minlength=V)
    want = p.numpy() * B
    assert np.all(np.abs(n - want) <= 5 * np.sqrt(want)), (n, want)


def test_scores_among_subnormal_numbers(cuda_lib):
    # products and quotients below 2^-126 have no relative rounding error: nothing that
    # spares divisions may assume one.  Units of the smallest number, 2^-149: 7 / 1.2627378
    # is 6, 2 / 0.3063047 is 7, and the second wins
    tiny = 2.0 ** -149
    V = 8
    P, noise = torch.zeros((1, 1, V)), torch.ones((1, V))
    P[0, 0, 0], P[0, 0, 1] = 7 * tiny, 2 * tiny
    noise[0, 0], noise[0, 1] = 1.2627378, 0.3063047
    z = torch.zeros((1, 0))
    t, _ = fb.fp8rl_spec_verify(P.cuda(), z.int().cuda(), z.cuda(), noise.cuda())
    assert t.tolist() == [[1]]
    # rows of such numbers, 8 and 16 entries a thread and unaligned ones
    for B, V in ((600, 61), (3, 4096), (200, 16001)):
        g = torch.Generator().manual_seed(V)
        P = (torch.randint(0, 9, (B, 1, V), generator=g).double() * tiny).float()
        noise = torch.empty((B, V)).exponential_(generator=g) + 0.25
        z = torch.zeros((B, 0))
        t, _ = fb.fp8rl_spec_verify(P.cuda(), z.int().cuda(), z.cuda(), noise.cuda())
        want, _ = ref.verify(P.numpy(), None, np.zeros((B, 0), np.int32), np.zeros(B, int), np.zeros((B, 0)), noise.numpy())
        assert np.array_equal(t.cpu().numpy(), want)


@pytest.mark.parametrize("V,at", [(64, 9), (50001, 40000), (152064, 151999)])
def test_a_residual_whose_scores_underflow_is_not_empty(cuda_lib, V, at):
    # the residual's only positive entry is two units of 2^-149, its score a quarter of
    # one, which rounds to 0: it takes part and wins all the same, and the entries without
    # weight, whose scores are 0 too, do not
    tiny = 2.0 ** -149
    for drafter in (True, False):
        P, Q = torch.zeros((2, 2, V)), torch.zeros((2, 1, V))
        P[:, 0, 7] = 0.0 if not drafter else 0.5
        Q[:, 0, 7] = 0.5
        P[:, 0, at], Q[:, 0, at] = 5 * tiny, 3 * tiny
        Q[:, 0, 3] = 0.5
        drafts = torch.full((2, 1), 3, dtype=torch.int32)           # p is 0 there: refused
        noise = torch.ones((2, V))
        noise[:, at] = 32.0 if not drafter else 8.0
        t, a = _run(P, Q if drafter else None, drafts, None, torch.full((2, 1), 0.5), noise)
        assert a.tolist() == [0, 0] and t.tolist() == [[at, -1]] * 2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,K,V", [(40, 3, 50257), (200, 2, 32001), (40, 3, 50260)])
def test_many_entries_a_thread(cuda_lib, B, K, V, dtype):
    # rows off the boundary of four entries that a thread goes over several times, and
    # the same for rows on it
    c = _case(B, K, V, B + V, dtype=dtype)
    t, a = _run(*c)
    wt, wa = _want(*c)
    assert np.array_equal(a, wa) and np.array_equal(t, wt)
    assert fb.fp8rl_check_device_error() == 0
