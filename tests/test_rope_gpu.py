"""Rotary positions and the rotating append against plain references: bit for bit
against the 32-bit definition, and within a derived bound of the 64-bit one."""
import numpy as np
import pytest
import torch

import rollout_ops_ref as ref
from precision_rl_rollout_gb300 import binding as fb

pytestmark = pytest.mark.gpu


def _table(max_pos, R, seed=0, magnitude=1.0):
    freq = 1.0 / (10000.0 ** (np.arange(R // 2) * 2.0 / R))
    angle = np.arange(max_pos)[:, None] * freq[None, :]
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32) * np.float32(magnitude), freq


def _x(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def _no_error():
    assert fb.fp8rl_check_device_error() == 0


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,D,R", [(1, 1, 2, 2), (1, 32, 128, 128), (5, 3, 64, 32), (7, 5, 80, 20), (3, 7, 96, 24),
                                     (33, 2, 256, 256), (257, 8, 128, 64), (2, 40, 128, 120), (4, 3, 18, 6),
                                     (1000, 1, 16, 16), (9, 2, 64, 0)])
def test_rope_bits_and_bound(cuda_lib, T, H, D, R, inter, inverse):
    if R == 0:
        table = np.zeros((11, 0), np.float32)
    else:
        table, _ = _table(501, R, magnitude=1.1)
    x = _x((T, H, D), T + D)
    pos = np.random.default_rng(T).integers(0, table.shape[0], T).astype(np.int32)
    y = fb.fp8rl_rope(x.cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda(), interleaved=inter,
                      inverse=inverse).cpu().float().numpy()
    xf = x.float().numpy()
    assert np.array_equal(y, ref.bf16(ref.rope(xf, pos, table, R, inter, inverse, np.float32)))
    want = ref.rope(xf, pos, table, R, inter, inverse)
    a, b = ref.rope_pairs(D, R, inter)
    size = np.abs(xf).astype(np.float64)
    size[..., a] = size[..., b] = 1.2 * (np.abs(xf[..., a]) + np.abs(xf[..., b]))
    # three fp32 roundings of at most the pair's size, then one to bf16 (unit
    # roundoff 2^-8)
    assert np.all(np.abs(y - want) <= 2.0 ** -8 * 1.01 * np.abs(want) + 2.0 ** -22 * size)
    _no_error()


@pytest.mark.parametrize("inter", [False, True])
def test_rope_strided_heads_in_place_and_output_strides(cuda_lib, inter):
    # q heads of a fused [T, heads, D] projection, rotated in place, with the
    # other heads untouched; then the same into a wider output
    T, H, D, R = 19, 4, 64, 48
    table, _ = _table(64, R)
    base = _x((T, H + 3, D), 5)
    pos = np.arange(T, dtype=np.int32)[::-1].copy()
    want = ref.bf16(ref.rope(base[:, 1:1 + H].float().numpy(), pos, table, R, inter, False, np.float32))
    d = base.cuda()
    tp, tt = torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda()
    wide = torch.zeros((T, H, D + 8), dtype=torch.bfloat16, device="cuda")
    fb.fp8rl_rope(d[:, 1:1 + H], tp, tt, interleaved=inter, Y=wide[:, :, :D])
    assert np.array_equal(wide[:, :, :D].cpu().float().numpy(), want) and not wide[:, :, D:].any()
    fb.fp8rl_rope(d[:, 1:1 + H], tp, tt, interleaved=inter, Y=d[:, 1:1 + H])
    got = d.cpu().float().numpy()
    assert np.array_equal(got[:, 1:1 + H], want)
    assert np.array_equal(got[:, :1], base[:, :1].float().numpy())
    assert np.array_equal(got[:, 1 + H:], base[:, 1 + H:].float().numpy())
    # odd strides and a misaligned start take the narrow form
    odd = torch.zeros((T, H, D + 1), dtype=torch.bfloat16, device="cuda")
    odd[:, :, 1:] = base[:, 1:1 + H].cuda()
    y = fb.fp8rl_rope(odd[:, :, 1:], tp, tt, interleaved=inter)
    assert np.array_equal(y.cpu().float().numpy(), want)
    _no_error()


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient_against_differences(cuda_lib, inter):
    # the map is linear: column j is the difference y(e_j) - y(0), one token per
    # unit vector; the gradient of <dy, y> is the columns' products with dy
    D, R, pos0 = 32, 24, 37
    table, _ = _table(64, R, magnitude=1.05)
    tt = torch.from_numpy(table).cuda()
    pos = torch.full((D,), pos0, dtype=torch.int32, device="cuda")
    eye = torch.eye(D).to(torch.bfloat16)[:, None, :].cuda()
    cols = fb.fp8rl_rope(eye, pos, tt, interleaved=inter) - fb.fp8rl_rope(torch.zeros_like(eye), pos, tt,
                                                                          interleaved=inter)
    cols = cols[:, 0].cpu().double().numpy()
    dy = _x((1, 1, D), 3)
    dx = fb.fp8rl_rope(dy.cuda(), pos[:1], tt, interleaved=inter, inverse=True)[0, 0].cpu().double().numpy()
    g = dy[0, 0].double().numpy()
    # two column entries of at most 1.05, each to 2^-8, and dx itself to 2^-8
    assert np.all(np.abs(dx - cols @ g) <= 2.0 ** -8 * 1.02 * (np.abs(cols) @ np.abs(g) + np.abs(dx)) + 1e-6)


def test_rope_positions_out_of_range_are_recorded(cuda_lib):
    table, _ = _table(16, 32)
    x = _x((3, 2, 32), 1)
    pos = torch.tensor([-5, 3, 16], dtype=torch.int32, device="cuda")
    y = fb.fp8rl_rope(x.cuda(), pos, torch.from_numpy(table).cuda())
    assert fb.fp8rl_check_device_error() != 0
    want = ref.bf16(ref.rope(x.float().numpy(), np.array([0, 3, 15]), table, 32, False, False, np.float32))
    assert np.array_equal(y.cpu().float().numpy(), want)
    _no_error()


def test_rope_beyond_32_bit_offsets(cuda_lib):
    # the second token lies more than 2^32 bytes behind the first
    step = (1 << 31) + 64
    buf = torch.empty(step + 256, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, 2, 128), (step, 128, 1))
    x.copy_(_x((2, 2, 128), 4))
    table, _ = _table(9, 128)
    pos = np.array([8, 5], np.int32)
    y = fb.fp8rl_rope(x, torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda())
    want = ref.bf16(ref.rope(x.cpu().float().numpy(), pos, table, 128, False, False, np.float32))
    assert np.array_equal(y.cpu().float().numpy(), want)


def test_rope_table_in_64_bits(cuda_lib):
    _, freq = _table(1, 64)
    table = fb.fp8rl_rope_table(torch.from_numpy(freq).cuda(), 70001, magnitude=1.25).cpu().numpy()
    angle = np.arange(70001)[:, None] * freq[None, :]
    want = 1.25 * np.concatenate([np.cos(angle), np.sin(angle)], axis=1)
    assert np.all(np.abs(table - want) <= 2.0 ** -24 * 1.25 + 1e-9)     # fp32 rounding, fp64 angle


# ---------------------------------------------------------------- append

def _pools(n, page, heads, D, e4m3, heads_first, fill=0):
    shape = (n, heads, page, D) if heads_first else (n, page, heads, D)
    t = torch.full(shape, fill, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")
    return t.transpose(1, 2) if heads_first else t


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,page,inter", [(1, 28, 4, 128, 128, 16, False), (61, 8, 2, 64, 64, 16, True),
                                                     (17, 3, 3, 96, 48, 7, False), (5, 0, 1, 256, 256, 1, False),
                                                     (130, 7, 1, 16, 6, 5, False), (9, 4, 2, 80, 20, 3, True),
                                                     (12, 2, 2, 64, 0, 8, False)])
def test_append_bits(cuda_lib, T, Hq, Hkv, D, R, page, inter, e4m3, heads_first):
    rng = np.random.default_rng(T + D)
    table = _table(300, R)[0] if R else None
    qkv = _x((T, Hq + 2 * Hkv, D), T * 3 + D)
    pos = rng.integers(0, 300, T).astype(np.int32)
    pages = -(-T // page) + 3
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if T > 4:
        slots[2] = -1                                          # a padding token
    ks, vs = 0.011, 0.007
    K, V = _pools(pages, page, Hkv, D, e4m3, heads_first, 3), _pools(pages, page, Hkv, D, e4m3, heads_first, 5)
    d = qkv.cuda()
    args = dict(k_scale=torch.tensor([ks], device="cuda"), v_scale=torch.tensor([vs], device="cuda")) if e4m3 else {}
    q = fb.fp8rl_rope_append_paged(d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], torch.from_numpy(pos).cuda(),
                                   None if table is None else torch.from_numpy(table).cuda(), K, V,
                                   torch.from_numpy(slots).cuda(), interleaved=inter, **args)
    f = qkv.float().numpy()
    rot = f if R == 0 else ref.rope(f, pos, table, R, inter, False, np.float32)
    assert np.array_equal(q.cpu().float().numpy(), ref.bf16(rot[:, :Hq]))
    for pool, x, s, fill in ((K, rot[:, Hq:Hq + Hkv], ks, 3), (V, f[:, Hq + Hkv:], vs, 5)):
        got = pool.cpu()
        got = got.numpy() if e4m3 else got.float().numpy()
        want = np.full(got.shape, fill, got.dtype)
        for t in range(T):
            if slots[t] >= 0:
                want[slots[t] // page, slots[t] % page] = ref.e4m3_codes(x[t], np.float32(s)) if e4m3 else ref.bf16(x[t])
        assert np.array_equal(got, want)
    _no_error()


@pytest.mark.parametrize("kind", ["boundary", "power of two", "tiny", "huge"])
def test_append_codes_at_the_boundaries_between_codes(cuda_lib, kind):
    """Scales that put a value's quotient on a boundary between two codes or a unit or
    two beside it; and scales whose reciprocal is exact, or out of range."""
    rng = np.random.default_rng(5)
    x = _x((1, 4, 64), 9)
    f = x.float().numpy()[0]
    normal = [m * 2.0 ** e for e in range(-6, 9) for m in (17 / 16, 19 / 16, 21 / 16, 23 / 16, 25 / 16, 27 / 16, 29 / 16, 31 / 16)]
    ties = np.array([i * 2.0 ** -10 for i in range(1, 16, 2)] + [t for t in normal if t < 448])
    zero = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    for i in range(48):
        if kind == "boundary":
            s = np.float32(abs(float(f.flat[i])) / ties[rng.integers(len(ties))])
            s = np.float32(s * (1 + (i % 5 - 2) * 2.0 ** -24))
        else:
            s = np.float32({"power of two": 2.0 ** (i % 12 - 8), "tiny": 2.0 ** -(100 + i % 49), "huge": 1.3 * 2.0 ** (90 + i % 37)}[kind])
        K, V = (torch.zeros((1, 1, 4, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
        scale = torch.tensor([s], device="cuda")
        fb.fp8rl_rope_append_paged(zero, x.cuda(), x.cuda(), None, None, K, V, torch.zeros(1, dtype=torch.int64, device="cuda"),
                                   k_scale=scale, v_scale=scale)
        want = ref.e4m3_codes(f, s)
        assert np.array_equal(K.cpu().numpy()[0, 0], want) and np.array_equal(V.cpu().numpy()[0, 0], want), s
    _no_error()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,R,shift", [(80, 56, 0), (80, 40, 0), (96, 24, 0), (64, 64, 4), (128, 72, 4), (48, 8, 0), (16, 16, 4)])
def test_append_in_8_byte_chunks(cuda_lib, D, R, shift, e4m3, inter):
    """Halves of R that are no multiple of 8, and heads that begin 8 bytes past a
    16-byte boundary; an odd number of chunks past R."""
    T, Hq, Hkv = 37, 5, 2
    table = _table(300, R)[0]
    big = _x((T, (Hq + 2 * Hkv) * D + 2 * shift), D + R).cuda()
    qkv = big[:, shift:shift + (Hq + 2 * Hkv) * D].unflatten(1, (Hq + 2 * Hkv, D))
    pos = np.random.default_rng(R).integers(0, 300, T).astype(np.int32)
    slots = np.arange(T, dtype=np.int64)[::-1].copy()
    K, V = _pools(5, 8, Hkv, D, e4m3, False), _pools(5, 8, Hkv, D, e4m3, False)
    ks, vs = 0.013, 0.006
    args = dict(k_scale=torch.tensor([ks], device="cuda"), v_scale=torch.tensor([vs], device="cuda")) if e4m3 else {}
    q = fb.fp8rl_rope_append_paged(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], torch.from_numpy(pos).cuda(),
                                   torch.from_numpy(table).cuda(), K, V, torch.from_numpy(slots).cuda(),
                                   interleaved=inter, **args)
    f = qkv.cpu().float().numpy()
    rot = ref.rope(f, pos, table, R, inter, False, np.float32)
    assert np.array_equal(q.cpu().float().numpy(), ref.bf16(rot[:, :Hq]))
    for pool, x, s in ((K, rot[:, Hq:Hq + Hkv], ks), (V, f[:, Hq + Hkv:], vs)):
        got = pool.cpu().reshape(40, Hkv, D)
        got = got.numpy() if e4m3 else got.float().numpy()
        for t in range(T):
            assert np.array_equal(got[slots[t]], ref.e4m3_codes(x[t], np.float32(s)) if e4m3 else ref.bf16(x[t]))
    _no_error()


def test_append_saturates_and_keeps_specials(cuda_lib):
    v = torch.zeros((1, 1, 16), dtype=torch.bfloat16)
    v[0, 0, :6] = torch.tensor([3e38, -3e38, float("inf"), float("-inf"), float("nan"), 1e-30])
    K, V = (torch.zeros((1, 1, 1, 16), dtype=torch.uint8, device="cuda") for _ in range(2))
    one = torch.tensor([1e-6], device="cuda")
    z = torch.zeros((1, 1, 16), dtype=torch.bfloat16, device="cuda")
    fb.fp8rl_rope_append_paged(z, z, v.cuda(), None, None, K, V, torch.zeros(1, dtype=torch.int64, device="cuda"),
                               k_scale=one, v_scale=one)
    got = V.cpu().view(-1)[:6].tolist()
    assert got[:4] == [0x7E, 0xFE, 0x7E, 0xFE] and (got[4] & 0x7F) == 0x7F and got[5] == 0


def test_append_slots_out_of_range_are_recorded(cuda_lib):
    K, V = (torch.full((2, 4, 1, 32), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x = _x((3, 1, 32), 2).cuda()
    slots = torch.tensor([8, 1, 1 << 40], dtype=torch.int64, device="cuda")
    fb.fp8rl_rope_append_paged(x, x, x, None, None, K, V, slots)
    assert fb.fp8rl_check_device_error() != 0
    want = torch.full((2, 4, 1, 32), 7.0, dtype=torch.bfloat16)
    want[0, 1] = x[1].cpu()
    assert torch.equal(K.cpu(), want) and torch.equal(V.cpu(), want)
    _no_error()


def test_append_on_a_side_stream_and_empty_batch(cuda_lib):
    s = torch.cuda.Stream()
    K, V = (torch.zeros((3, 4, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x = _x((6, 2, 64), 8).cuda()
    slots = torch.arange(6, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    q = fb.fp8rl_rope_append_paged(x, x, x, None, None, K, V, slots, stream=s)
    s.synchronize()
    assert torch.equal(q, x) and torch.equal(K.view(12, 2, 64)[:6], x)
    e = x[:0]
    assert fb.fp8rl_rope_append_paged(e, e, e, None, None, K, V, slots[:0]).shape == (0, 2, 64)
    assert fb.fp8rl_rope(e, slots[:0].int(), torch.zeros((1, 64), device="cuda")).shape == (0, 2, 64)
    _no_error()


# ---------------------------------------------------------------- prompt-sized calls
# Large enough that a thread goes over several batches of heads and a CTA over several
# tokens, the last of them with tokens that are not there (T is prime).

@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,D,R", [(1747, 48, 128, 128), (2999, 32, 128, 64), (3001, 36, 80, 56), (1201, 21, 256, 256),
                                     (2003, 41, 96, 0)])
def test_rope_of_many_tokens(cuda_lib, T, H, D, R, inter, in_place):
    table = _table(4099, R, magnitude=1.1)[0] if R else np.zeros((4099, 0), np.float32)
    x = _x((T, H + 2, D), T + R)
    pos = np.random.default_rng(T).integers(0, 4099, T).astype(np.int32)
    d = x.cuda()
    heads = d[:, 1:1 + H]
    for inverse in (False, True):
        if inverse and in_place:
            heads.copy_(x[:, 1:1 + H])
        y = fb.fp8rl_rope(heads, torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda(), interleaved=inter,
                          inverse=inverse, Y=heads if in_place else None)
        want = ref.bf16(ref.rope(x[:, 1:1 + H].float().numpy(), pos, table, R, inter, inverse, np.float32))
        assert np.array_equal(y.cpu().float().numpy(), want)
    assert torch.equal(d[:, 0].cpu(), x[:, 0]) and torch.equal(d[:, -1].cpu(), x[:, -1])
    _no_error()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,in_place", [(2003, 28, 4, 128, 128, False), (1733, 40, 8, 96, 48, True),
                                                   (3001, 28, 4, 80, 56, True), (1511, 8, 8, 256, 256, False),
                                                   (2999, 40, 8, 64, 0, False)])
def test_append_of_many_tokens(cuda_lib, T, Hq, Hkv, D, R, in_place, e4m3, inter):
    rng = np.random.default_rng(T)
    table = _table(4099, R)[0] if R else None
    page, pages = 16, -(-T // 16) + 3
    x = _x((T, Hq + 2 * Hkv, D), T)
    pos = rng.integers(0, 4099, T).astype(np.int32)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[rng.permutation(T)[:T // 7]] = -1                   # padding
    ks, vs = np.float32(0.011), np.float32(0.007)
    K, V = _pools(pages, page, Hkv, D, e4m3, inter, 3), _pools(pages, page, Hkv, D, e4m3, inter, 5)
    args = dict(k_scale=torch.tensor([ks], device="cuda"), v_scale=torch.tensor([vs], device="cuda")) if e4m3 else {}
    d = x.cuda()
    q = fb.fp8rl_rope_append_paged(d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], torch.from_numpy(pos).cuda(),
                                   None if table is None else torch.from_numpy(table).cuda(), K, V,
                                   torch.from_numpy(slots).cuda(), interleaved=inter,
                                   q_out=d[:, :Hq] if in_place else None, **args)
    f = x.float().numpy()
    rot = f if R == 0 else ref.rope(f, pos, table, R, inter, False, np.float32)
    assert np.array_equal(q.cpu().float().numpy(), ref.bf16(rot[:, :Hq]))
    assert torch.equal(d[:, Hq:].cpu(), x[:, Hq:])
    keep = slots >= 0
    for pool, y, s, fill in ((K, rot[:, Hq:Hq + Hkv], ks, 3), (V, f[:, Hq + Hkv:], vs, 5)):
        got = pool.cpu()
        got = got.numpy() if e4m3 else got.float().numpy()
        want = np.full(got.shape, fill, got.dtype)
        want[slots[keep] // page, slots[keep] % page] = ref.e4m3_codes(y[keep], s) if e4m3 else ref.bf16(y[keep])
        assert np.array_equal(got, want)
    _no_error()
