"""Paged attention against a plain 64-bit reference, element by element within the
bound rollout_ops_ref.attention derives from the operand types."""
import numpy as np
import pytest
import torch

import rollout_ops_ref as ref
from precision_rl_rollout_gb300 import binding as fb

pytestmark = pytest.mark.gpu


class Cache:
    """Random pages in a random order; everything no sequence owns is NaN."""

    def __init__(self, lens, Hkv, D, page, e4m3, heads_first, seed, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.e4m3, self.page = e4m3, page
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g)
        self.ks, self.vs = (0.013, 0.009) if e4m3 else (1.0, 1.0)
        cols = max(1, max(need))
        self.table = torch.full((len(lens), cols), -1, dtype=torch.int32)      # unused entries: never read
        shape = (pages, page, Hkv, D)
        pools = []
        for s in (self.ks, self.vs):
            x = (torch.randn(shape, generator=g) * spread).numpy()
            if e4m3:
                pools.append(torch.from_numpy(ref.e4m3_codes(x, np.float32(s))))
            else:
                pools.append(torch.from_numpy(x).to(torch.bfloat16))
        self.seq, own, at = [], torch.zeros((pages, page), dtype=torch.bool), 0
        for b, n in enumerate(lens):
            ids = order[at:at + need[b]]
            at += need[b]
            self.table[b, :need[b]] = ids.int()
            j = torch.arange(n)
            where = (ids[j // page], j % page) if n else (j, j)
            own[where] = True
            val = [ref.e4m3_values(p[where].numpy()).astype(np.float64) * float(np.float32(s)) if e4m3 else
                   p[where].double().numpy() for p, s in zip(pools, (self.ks, self.vs))]
            self.seq.append(val)
        self.pools = []
        for p in pools:
            p = p.clone()
            p[~own] = 0x7F if e4m3 else float("nan")
            t = p.cuda()
            if heads_first:
                t = t.transpose(1, 2).contiguous().transpose(1, 2)
            self.pools.append(t)
        self.lens = torch.tensor(lens, dtype=torch.int32)

    def scales(self):
        if not self.e4m3:
            return {}
        return dict(k_scale=torch.tensor([self.ks], device="cuda"), v_scale=torch.tensor([self.vs], device="cuda"))


def _check(c, q, window=0, scale=None, max_len=None, **kw):
    o, lse = fb.fp8rl_attn_paged(q.cuda() if not q.is_cuda else q, c.pools[0], c.pools[1], c.table.cuda(),
                                 c.lens.cuda(), int(max_len or c.lens.max()), window=window, scale=scale,
                                 want_lse=True, **c.scales(), **kw)
    o, lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
    qh = q.cpu().double().numpy()
    for b in range(qh.shape[0]):
        k, v = c.seq[b]
        wo, wl, tol, ltol = ref.attention(qh[b], k, v, scale or qh.shape[-1] ** -0.5, window)
        assert np.all(np.isfinite(o[b])), f"sequence {b}: non-finite output"
        err = np.abs(o[b] - wo)
        assert np.all(err <= tol), (b, float((err / np.maximum(tol, 1e-300)).max()))
        empty = np.isneginf(wl)
        assert np.array_equal(np.isneginf(lse[b]), empty)
        assert np.all(np.abs(lse[b][~empty] - wl[~empty]) <= ltol[~empty])
    assert fb.fp8rl_check_device_error() == 0
    return o, lse


def _q(B, Lq, Hq, D, seed, size=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, Lq, Hq, D), generator=g) * size).to(torch.bfloat16)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,page,Lq,window", [
    (28, 4, 128, 16, 1, 0), (5, 1, 128, 7, 1, 0), (40, 8, 128, 32, 5, 0), (6, 6, 64, 16, 1, 0), (8, 1, 64, 1, 2, 0),
    (16, 1, 128, 64, 3, 9), (28, 4, 128, 16, 8, 0), (7, 1, 256, 24, 1, 0), (9, 3, 256, 8, 4, 33), (4, 2, 16, 16, 1, 0),
    (10, 2, 96, 12, 3, 0), (3, 1, 80, 128, 1, 100), (64, 1, 128, 16, 2, 1), (2, 2, 128, 16, 17, 0)])
def test_ragged_batch(cuda_lib, Hq, Hkv, D, page, Lq, window, e4m3):
    # lengths of zero and one, shorter than the query block, at tile and page edges
    lens = [0, 1, 2, 15, 16, 17, 31, 64, 65, 127, 128, 129, 300, 511]
    c = Cache(lens, Hkv, D, page, e4m3, (Hq + page) % 2 == 0, D + Lq)
    _check(c, _q(len(lens), Lq, Hq, D, Hq), window)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,L,Lq,Hq,Hkv,D,window", [(1, 20000, 1, 8, 2, 128, 0), (2, 9001, 4, 5, 1, 128, 0),
                                                    (1, 6000, 2, 4, 1, 64, 2500), (3, 5000, 1, 2, 1, 256, 0),
                                                    (1, 3000, 1, 1, 1, 128, 0)])
def test_long_sequences_split_and_joined(cuda_lib, B, L, Lq, Hq, Hkv, D, window, e4m3):
    lens = [max(1, L - 777 * b) for b in range(B)]
    c = Cache(lens, Hkv, D, 16, e4m3, False, L)
    _check(c, _q(B, Lq, Hq, D, L, size=3.0), window)


@pytest.mark.parametrize("Hq,Hkv,D,page,Lq,window", [
    (33, 1, 128, 16, 1, 0), (40, 8, 128, 8, 5, 0), (48, 3, 96, 32, 5, 0), (28, 4, 64, 64, 8, 0), (16, 2, 128, 24, 8, 40),
    (48, 3, 128, 128, 8, 0), (65, 1, 64, 16, 1, 7), (6, 2, 80, 8, 43, 0), (10, 5, 128, 16, 150, 0), (4, 4, 64, 256, 70, 19),
    (12, 1, 16, 16, 11, 0)])
def test_many_query_rows(cuda_lib, Hq, Hkv, D, page, Lq, window):
    # more than 32 rows a kv head, one and several chunks of them, over bf16
    lens = [0, 1, 2, 15, 16, 17, 31, 64, 65, 127, 128, 129, 300, 511]
    c = Cache(lens, Hkv, D, page, False, (Hq + page) % 2 == 0, D + Lq)
    _check(c, _q(len(lens), Lq, Hq, D, Hq), window)


@pytest.mark.parametrize("D,window", [(128, 0), (64, 30), (112, 200)])
@pytest.mark.parametrize("rows", [48, 49, 80, 81, 96, 97, 112, 129, 192, 193, 385])
def test_row_counts_at_the_edges_of_the_configurations(cuda_lib, rows, D, window):
    lens = [rows + 1, 130, 256, 257, 1000]
    c = Cache(lens, 1, D, 16, False, False, rows + D)
    _check(c, _q(len(lens), rows, 1, D, rows), window)


@pytest.mark.parametrize("B,L,Lq,Hq,Hkv,D,window", [(1, 9000, 5, 14, 2, 128, 0), (2, 4001, 9, 40, 8, 128, 0),
                                                    (3, 3000, 16, 8, 1, 64, 1111), (1, 2500, 300, 2, 1, 96, 0)])
def test_many_query_rows_of_long_sequences(cuda_lib, B, L, Lq, Hq, Hkv, D, window):
    lens = [max(1, L - 777 * b) for b in range(B)]
    c = Cache(lens, Hkv, D, 16, False, False, L)
    q = _q(B, Lq, Hq, D, L, size=3.0)
    o, lse = _check(c, q, window)
    again, lse2 = _check(c, q, window)
    assert np.array_equal(o, again) and np.array_equal(lse, lse2)


@pytest.mark.parametrize("Hq,Lq,D", [(40, 2, 128), (12, 9, 64), (3, 50, 96)])
def test_many_query_rows_do_not_see_later_values(cuda_lib, Hq, Lq, D):
    # NaN and infinities among the newest tokens, and below a window's edge
    lens, page = [200, 133, 129], 8
    for window in (0, 61):
        c = Cache(lens, 1, D, page, False, False, 11)
        q = _q(3, Lq, Hq, D, 12)
        want, _ = _check(c, q, window)
        for bad_keys in (False, True):
            hit = []
            for b, n in enumerate(lens):
                for i, t in enumerate([n - 1, n - 2] if not window else [n - Lq - window + 1, n - Lq - window + 2]):
                    value = float("nan") if i else float("inf")
                    at = (int(c.table[b, t // page]), t % page)
                    c.pools[1][at] = value
                    if bad_keys:
                        c.pools[0][at] = value
                    hit.append((b, t))
            o, _ = fb.fp8rl_attn_paged(q.cuda(), *c.pools, c.table.cuda(), c.lens.cuda(), max(lens), window=window,
                                       want_lse=True)
            o = o.cpu().double().numpy()
            for b, n in enumerate(lens):
                for i in range(Lq):
                    p = n - Lq + i
                    if any(x == b and t <= p and (not window or t > p - window) for x, t in hit):
                        assert not np.any(np.isfinite(o[b, i])), (window, b, i)
                    else:
                        assert np.array_equal(o[b, i], want[b, i]), (window, b, i)
        assert fb.fp8rl_check_device_error() == 0


def test_many_short_sequences(cuda_lib):
    lens = [(37 * i) % 90 for i in range(300)]
    c = Cache(lens, 2, 64, 16, False, True, 3)
    _check(c, _q(300, 1, 6, 64, 3))


@pytest.mark.parametrize("e4m3", [False, True])
def test_values_only_later_queries_see_do_not_leak(cuda_lib, e4m3):
    # the newest cached tokens hold NaN and infinities: queries before them must
    # not notice, with and without a window whose lower edge does the same
    lens, Lq, Hq, Hkv, D, page = [40, 133], 4, 6, 2, 128, 16
    for window in (0, 21):
        c = Cache(lens, Hkv, D, page, e4m3, False, 11)
        q = _q(2, Lq, Hq, D, 12)
        want, _ = _check(c, q, window)
        bad = [torch.tensor(0x7F, dtype=torch.uint8)] * 2 if e4m3 else [torch.tensor(float("nan")), torch.tensor(float("inf"))]
        hit = []
        for b, n in enumerate(lens):
            j = [n - 1, n - 2] if not window else [n - Lq - window + 1, n - Lq - window + 2]
            for i, t in enumerate(j):                      # seen by the newest queries, or by the oldest only
                at = (int(c.table[b, t // page]), t % page)
                for pool in c.pools:
                    pool[at] = bad[i].to(pool.dtype).cuda()
                hit.append((b, t))
        o, _ = fb.fp8rl_attn_paged(q.cuda(), *c.pools, c.table.cuda(), c.lens.cuda(), max(lens), window=window,
                                   want_lse=True, **c.scales())
        o = o.cpu().double().numpy()
        for b, n in enumerate(lens):
            for i in range(Lq):
                p = n - Lq + i
                sees = any(x == b and t <= p and (not window or t > p - window) for x, t in hit)
                if sees:
                    assert not np.all(np.isfinite(o[b, i])), (window, b, i)
                else:
                    assert np.array_equal(o[b, i], want[b, i]), (window, b, i)


def test_masked_by_the_types_lowest_value_and_infinite_scores(cuda_lib):
    # keys of bf16's lowest value drive scores to the bottom of fp32 and to -inf:
    # such tokens weigh nothing, and a row of only such scores of -inf is empty
    lens = [3, 50]
    c = Cache(lens, 1, 64, 16, False, False, 5)
    low = torch.finfo(torch.bfloat16).min
    K = c.pools[0]
    q = torch.ones((2, 1, 2, 64), dtype=torch.bfloat16)
    for t in range(3):
        K[int(c.table[0, 0]), t] = low                     # sums to -inf in fp32
    for t in (0, 17, 49):
        K[int(c.table[1, t // 16]), t % 16] = low
        c.seq[1][0][t] = -1e30                              # weighs nothing
    o, lse = fb.fp8rl_attn_paged(q.cuda(), *c.pools, c.table.cuda(), c.lens.cuda(), 50, want_lse=True)
    assert not o[0].any() and torch.isneginf(lse[0]).all()
    wo, wl, tol, ltol = ref.attention(q[1].double().numpy(), c.seq[1][0], c.seq[1][1], 0.125)
    keep = [t for t in range(50) if t not in (0, 17, 49)]
    _, _, tol, _ = ref.attention(q[1].double().numpy(), c.seq[1][0][keep], c.seq[1][1][keep], 0.125)
    assert np.all(np.abs(o[1].cpu().double().numpy() - wo) <= tol)


def test_sharp_and_flat_rows(cuda_lib):
    # one token far above the rest, late and early; and equal scores everywhere
    lens = [2000, 2000, 2000]
    for e4m3 in (False, True):
        c = Cache(lens, 1, 128, 16, e4m3, False, 21)
        q = torch.zeros((3, 1, 4, 128), dtype=torch.bfloat16)
        for b, t in ((0, 1990), (1, 3)):
            k = torch.from_numpy(c.seq[b][0][t, 0]).to(torch.bfloat16)
            q[b, 0, :] = k * 6
        _check(c, q)


def test_lengths_and_pages_out_of_range_are_recorded(cuda_lib):
    c = Cache([20, 20], 1, 64, 16, False, False, 2)
    q = _q(2, 1, 2, 64, 2).cuda()
    good = fb.fp8rl_attn_paged(q, *c.pools, c.table.cuda(), c.lens.cuda(), 20)
    for lens in ([20, 21], [20, -3]):
        o = fb.fp8rl_attn_paged(q, *c.pools, c.table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 20)
        assert fb.fp8rl_check_device_error() != 0
        assert torch.equal(o[0], good[0])
        assert torch.equal(o[1], good[1] if lens[1] > 0 else torch.zeros_like(o[1]))
    table = c.table.clone()
    table[1, 0] = 1000
    o = fb.fp8rl_attn_paged(q, *c.pools, table.cuda(), c.lens.cuda(), 20)
    assert fb.fp8rl_check_device_error() != 0
    assert torch.equal(o[0], good[0])
    assert fb.fp8rl_check_device_error() == 0


def test_strided_queries_shared_pool_and_bound_above_the_lengths(cuda_lib):
    # K and V as halves of one pool, queries inside a fused projection, a length
    # bound far above the lengths, and a caller's workspace full of garbage
    c = Cache([5, 200, 77], 2, 64, 16, False, False, 9)
    both = torch.stack([c.pools[0], c.pools[1]], dim=2).contiguous()        # [pages, page, 2, heads, D]
    c.pools = [both[:, :, 0], both[:, :, 1]]
    fused = torch.zeros((3, 1, 12, 64), dtype=torch.bfloat16, device="cuda")
    q = _q(3, 1, 6, 64, 9)
    fused[:, :, 2:8] = q.cuda()
    c.table = torch.nn.functional.pad(c.table, (0, 700), value=-1)
    n = fb.fp8rl_attn_paged_workspace_bytes(3, 1, 6, 2, 64, 10000)
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    _check(c, fused[:, :, 2:8], max_len=10000, workspace=ws)


@pytest.mark.parametrize("e4m3", [False, True])
def test_offsets_beyond_32_bits(cuda_lib, e4m3):
    # pages whose byte and element offsets pass 2^32
    page, D = 16, 128
    stride = (1 << 30) + 64
    buf = [torch.empty(5 * stride + page * D, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")
           for _ in range(2)]
    pools = [b.as_strided((6, page, 1, D), (stride, D, D, 1)) for b in buf]
    c = Cache([page + 9], 1, D, page, e4m3, False, 4)
    for big, small in zip(pools, c.pools):
        big[5], big[4] = small[int(c.table[0, 0])], small[int(c.table[0, 1])]
    c.pools, c.table = pools, torch.tensor([[5, 4]], dtype=torch.int32)
    _check(c, _q(1, 1, 4, D, 4))


def test_determinism_streams_and_graph(cuda_lib):
    c = Cache([3000, 10, 700], 4, 128, 16, True, False, 6)
    q = _q(3, 2, 28, 128, 6).cuda()
    table, lens = c.table.cuda(), c.lens.cuda()
    kw = c.scales()
    first = fb.fp8rl_attn_paged(q, *c.pools, table, lens, 3000, **kw)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        again = fb.fp8rl_attn_paged(q, *c.pools, table, lens, 3000, stream=s, **kw)
    s.synchronize()
    assert torch.equal(first, again)
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(first)
    n = fb.fp8rl_attn_paged_workspace_bytes(3, 2, 28, 4, 128, 3000)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    with torch.cuda.graph(g):
        fb.fp8rl_attn_paged(q, *c.pools, table, lens, 3000, o=out, workspace=ws, **kw)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out)
    # new lengths through the same graph
    lens.copy_(torch.tensor([2999, 0, 650], dtype=torch.int32))
    g.replay()
    assert torch.equal(out, fb.fp8rl_attn_paged(q, *c.pools, table, lens, 3000, **kw))
    assert fb.fp8rl_check_device_error() == 0


def test_empty_batch_and_zero_bound(cuda_lib):
    c = Cache([4], 1, 64, 16, False, False, 1)
    q = _q(1, 2, 2, 64, 1).cuda()
    o, lse = fb.fp8rl_attn_paged(q, *c.pools, c.table.cuda(), torch.zeros(1, dtype=torch.int32).cuda(), 0,
                                 want_lse=True)
    assert not o.any() and torch.isneginf(lse).all()
    o = fb.fp8rl_attn_paged(q[:0], *c.pools, c.table[:0].cuda(), torch.zeros(0, dtype=torch.int32).cuda(), 16)
    assert o.shape == (0, 2, 2, 64)


@pytest.mark.parametrize("n", [1, 7])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Hq,D,page,Lq", [(8, 128, 16, 1), (8, 128, 7, 1), (5, 64, 16, 3), (16, 64, 16, 1), (7, 256, 16, 1),
                                          (4, 256, 16, 4), (8, 96, 32, 2), (25, 128, 16, 1), (40, 128, 16, 1), (9, 256, 16, 5)])
def test_probabilities_are_as_exact_as_promised(cuda_lib, Hq, D, page, Lq, e4m3, n):
    """Tokens of value 1 and weight 1 against tokens of value -1 and a weight that bf16
    and fp16 hold badly, so many of each that they nearly cancel: what the rounding of the
    weights leaves stands in the result.  Promised: 2^-16 of a weight over bf16 for up to
    16 query rows a kv head, 2^-8 above; 2^-11 over E4M3."""
    # 0.70117 + 0.45 of bf16's spacing there (2^-8), and off fp16's grid by 0.4 of its spacing
    w = 0.69921875 + 0.45 * 2.0 ** -8
    w = np.floor(w * 2048) / 2048 + 0.4 / 2048
    na, nb = 70 * n, 100 * n
    length = na + nb + Lq - 1                                  # the newest Lq - 1 tokens weigh nothing to the last bit
    pages = -(-length // page)
    k, v = torch.zeros((pages * page, 1, D)), torch.zeros((pages * page, 1, D))
    k[na:na + nb, 0, 0] = 1.0
    k[na + nb:, 0, 0] = 448.0
    v[:na], v[na:na + nb] = 1.0, -1.0
    one = torch.ones(1, device="cuda")
    pools = [x.to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else x.to(torch.bfloat16) for x in (k, v)]
    pools = [x.view(pages, page, 1, D).cuda() for x in pools]
    q = torch.zeros((1, Lq, Hq, D), dtype=torch.bfloat16)
    q[..., 0] = -1.0
    scale = float(np.float32(-np.log(w)))
    o = fb.fp8rl_attn_paged(q.cuda(), *pools, torch.arange(pages, dtype=torch.int32).view(1, -1).cuda(),
                            torch.tensor([length], dtype=torch.int32).cuda(), length, scale=scale,
                            **(dict(k_scale=one, v_scale=one) if e4m3 else {}))
    w = np.exp(-scale)
    total = na + nb * w
    want = (na - nb * w) / total
    rows = Hq * Lq
    each = 2.0 ** -11 if e4m3 else 2.0 ** -16 if rows <= 16 else 2.0 ** -8
    # the weights' rounding; a score of at most 0.36 in D fp32 sums and three roundings,
    # and the exponential's 2^-22; fp32 sums; the result's bf16 rounding
    tol = each + 2 * (2.0 ** -23 * (D + 8) * 0.36 + 2.0 ** -21) + (na + nb) * 2.0 ** -23 + 2.0 ** -8 * 1.01 * abs(want)
    err = np.abs(o.cpu().double().numpy() - want).max()
    assert err <= tol, (err, tol)
    assert fb.fp8rl_check_device_error() == 0
