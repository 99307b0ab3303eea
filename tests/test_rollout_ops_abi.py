"""CPU checks of the rotary, paged-cache and verification calls: invalid arguments are
refused synchronously, before any CUDA call, and the binding refuses what only it
can see."""
import ctypes

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


def _kv(**kw):
    d = dict(K=A, V=A, k_scale=None, v_scale=None, num_pages=4, page_size=16, kv_heads=2, head_dim=64,
             page_stride=16 * 128, token_stride=128, head_stride=64, dtype=0)
    d.update(kw)
    return binding.FP8RL_PAGED_KV(*[d[n] for n, _ in binding.FP8RL_PAGED_KV._fields_])


def test_rope_validation(lib):
    def f(X=A, T=4, H=2, D=64, xt=128, xh=64, pos=A, table=A, max_pos=16, R=64, flags=0, Y=A, yt=128, yh=64):
        return lib.fp8rl_rope(X, T, H, D, xt, xh, pos, table, max_pos, R, flags, Y, yt, yh, None)
    assert f(T=0) == 0
    assert f(X=None) == 1 and f(Y=None) == 1 and f(pos=None) == 1 and f(table=None) == 1
    assert f(T=-1) == 2 and f(H=0) == 2 and f(D=0) == 2
    assert f(R=63) == 2 and f(R=66) == 2 and f(R=-2) == 2
    assert f(max_pos=0) == 2 and f(xt=-1) == 2 and f(yh=-64) == 2
    assert f(X=A + 1) == 3 and f(table=A + 2) == 3 and f(pos=A + 1) == 3
    assert f(flags=4) == 6 and f(H=1 << 20, D=64) == 6 and f(T=1 << 31) == 6


def test_rope_table_validation(lib):
    f = lib.fp8rl_rope_table
    assert f(A, 0, 64, 1.0, A, None) == 0
    assert f(None, 8, 64, 1.0, A, None) == 1 and f(A, 8, 64, 1.0, None, None) == 1
    assert f(A, 8, 63, 1.0, A, None) == 2 and f(A, 8, 0, 1.0, A, None) == 2 and f(A, -1, 64, 1.0, A, None) == 2
    assert f(A + 4, 8, 64, 1.0, A, None) == 3
    assert f(A, 1 << 40, 64, 1.0, A, None) == 6


def test_append_validation(lib):
    def f(kv=None, q=A, Hq=4, k=A, v=A, T=4, pos=A, table=A, max_pos=16, R=64, flags=0, qo=A, slots=A, qt=512):
        return lib.fp8rl_rope_append_paged(q, Hq, qt, 64, k, 512, 64, v, 512, 64, T, pos, table, max_pos, R, flags,
                                           qo, 256, 64, kv if kv is not None else _kv(), slots, None)
    assert f(T=0) == 0
    for name in ("q", "k", "v", "qo", "slots", "pos", "table"):
        assert f(**{name: None}) == 1, name
    assert lib.fp8rl_rope_append_paged(A, 4, 512, 64, A, 512, 64, A, 512, 64, 4, A, A, 16, 64, 0, A, 256, 64, None,
                                       A, None) == 1
    assert f(kv=_kv(K=None)) == 1 and f(kv=_kv(dtype=1)) == 1                      # E4M3 without scales
    assert f(kv=_kv(dtype=1, k_scale=A, v_scale=None)) == 1
    assert f(kv=_kv(num_pages=0)) == 2 and f(kv=_kv(page_size=0)) == 2 and f(kv=_kv(head_dim=40)) == 2
    assert f(kv=_kv(token_stride=-128)) == 2 and f(Hq=-1) == 2 and f(R=128) == 2
    assert f(kv=_kv(K=A + 8)) == 3 and f(kv=_kv(token_stride=132)) == 3 and f(slots=A + 4) == 3
    assert f(kv=_kv(dtype=1, k_scale=A, v_scale=A, head_stride=72)) == 3            # 72 bytes
    assert f(kv=_kv(dtype=2)) == 6 and f(kv=_kv(head_dim=512)) == 6 and f(flags=2) == 6
    assert f(kv=_kv(kv_heads=1 << 17)) == 6


def test_attn_validation(lib):
    def f(kv=None, q=A, B=2, Lq=1, Hq=4, qs=256, table=A, ts=8, lens=A, max_len=100, window=0, o=A, lse=None, ws=A,
          wb=None):
        need = lib.fp8rl_attn_paged_workspace_bytes(B, Lq, Hq, 2, 64, max_len)
        return lib.fp8rl_attn_paged(q, B, Lq, Hq, qs, 256, 64, kv if kv is not None else _kv(), table, ts, lens,
                                    max_len, window, 0.125, o, lse, ws, need if wb is None else wb, None)
    assert f(B=0) == 0
    for name in ("q", "table", "lens", "o"):
        assert f(**{name: None}) == 1, name
    assert f(Hq=3) == 2 and f(Lq=0) == 2 and f(B=-1) == 2 and f(max_len=-1) == 2 and f(window=-1) == 2
    assert f(ts=6) == 2                                                            # too few columns for max_len
    assert f(kv=_kv(page_size=-1)) == 2
    assert f(q=A + 8) == 3 and f(qs=252) == 3 and f(lse=A + 2) == 3 and f(table=A + 1) == 3 and f(ws=A + 8) == 3
    assert f(max_len=(1 << 30) + 1, ts=1 << 30) == 6 and f(B=1 << 30, Hq=4, ws=A, wb=0) in (4, 6)
    for B, L in ((1, 100000), (64, 8192)):
        need = lib.fp8rl_attn_paged_workspace_bytes(B, 1, 4, 2, 64, L)
        if need:
            assert f(B=B, max_len=L, ts=10000, wb=need - 1) == 4 and f(B=B, max_len=L, ts=10000, ws=None) == 4
    c = lib.fp8rl_attn_paged_kernel_count
    assert c(0, 1, 4, 2, 64, 100, 0) == 0 and c(2, 1, 3, 2, 64, 100, 0) == -2 and c(2, 1, 4, 2, 64, 100, 2) == -6
    for dtype in (0, 1):
        assert c(2, 1, 4, 2, 64, 16, dtype) == 1 and c(2, 1, 4, 2, 64, 100000, dtype) == 2


def test_verify_validation(lib):
    def f(P=A, Q=A, dtype=0, drafts=A, lens=None, u=A, noise=A, B=2, K=3, V=100, tokens=A, acc=A, ps=400):
        return lib.fp8rl_spec_verify(P, ps, 100, Q, 300, 100, dtype, drafts, lens, u, noise, 100, B, K, V, tokens,
                                     acc, None)
    assert f(B=0) == 0
    for name in ("P", "drafts", "u", "noise", "tokens", "acc"):
        assert f(**{name: None}) == 1, name
    assert f(B=-1) == 2 and f(K=-1) == 2 and f(V=0) == 2 and f(ps=-1) == 2
    assert f(P=A + 2) == 3 and f(P=A + 1, dtype=1) == 3 and f(noise=A + 2) == 3 and f(tokens=A + 1) == 3
    assert f(dtype=2) == 6 and f(K=33) == 6 and f(B=65536) == 6 and f(V=(1 << 30) + 1) == 6


def test_binding_refusals():
    cpu = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    try:
        binding.load()
    except RuntimeError as e:
        pytest.skip(str(e))
    pos, table = torch.zeros(2, dtype=torch.int32), torch.zeros((4, 64))
    with pytest.raises(ValueError):
        binding.fp8rl_rope(cpu, pos, table)                                # not on a GPU
    with pytest.raises(ValueError):
        binding.fp8rl_attn_paged(cpu[None], cpu[None], cpu[None], pos[None], pos, 4)
    with pytest.raises(ValueError):
        binding.fp8rl_spec_verify(torch.zeros((1, 2, 8)), pos[None, :1], table[:1, :1], table[:1, :8])
    with pytest.raises(ValueError):
        binding.fp8rl_rope_append_paged(cpu, cpu, cpu, pos, table, cpu[None], cpu[None], pos.long())
    with pytest.raises(ValueError):
        binding.fp8rl_rope_table(torch.zeros(4, dtype=torch.float64), 8)


@pytest.mark.gpu
def test_binding_refusals_on_the_device(cuda_lib):
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = torch.zeros((4, 64), device="cuda")
    pool = torch.zeros((2, 4, 2, 64), dtype=torch.bfloat16, device="cuda")
    bt = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    fb = binding
    bad = [lambda: fb.fp8rl_rope(x.float(), pos, table), lambda: fb.fp8rl_rope(x, pos.long(), table),
           lambda: fb.fp8rl_rope(x, pos[:1], table), lambda: fb.fp8rl_rope(x, pos.cpu(), table),
           lambda: fb.fp8rl_rope(x, pos, table, Y=x[:1]), lambda: fb.fp8rl_rope(x.transpose(1, 2), pos, table),
           lambda: fb.fp8rl_rope_append_paged(x, x, x, pos, table, pool, pool[:1], pos.long()),
           lambda: fb.fp8rl_rope_append_paged(x, x, x, pos, table, pool, pool.transpose(1, 2), pos.long()),
           lambda: fb.fp8rl_rope_append_paged(x, x[:, :1], x, pos, table, pool, pool, pos.long()),
           lambda: fb.fp8rl_rope_append_paged(x, x, x, pos, table, pool.byte(), pool.byte(), pos.long()),
           lambda: fb.fp8rl_attn_paged(x[None], pool, pool, bt, pos[:1], 9),          # table too narrow
           lambda: fb.fp8rl_attn_paged(x[None], pool, pool, bt.long(), pos[:1], 8),
           lambda: fb.fp8rl_attn_paged(x[None][..., :32], pool, pool, bt, pos[:1], 8),
           lambda: fb.fp8rl_spec_verify(table[None].double(), pos[None, :1], table[:1, :1], table[:1]),
           lambda: fb.fp8rl_spec_verify(table[None], pos[None, :1], table[:1, :3], table[:1])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fb.Fp8rlError) as e:
        fb.fp8rl_rope(x, pos, torch.zeros((4, 66), device="cuda"))                     # R above the head
    assert e.value.status == 2
    with pytest.raises(fb.Fp8rlError):
        fb.fp8rl_attn_paged(x[None, :, :1].repeat(1, 1, 3, 1), pool, pool, bt, pos[:1], 8)   # 3 heads over 2
    assert fb.fp8rl_check_device_error() == 0


@pytest.mark.gpu
def test_other_threads_run_during_a_launch(cuda_lib, tmp_path):
    """A launch can wait (for room in the driver's queue, for a module to load): other
    Python threads must run meanwhile.  The calls are bound to libc's poll here, given no
    descriptors and 300 ms by the arguments that come second and third."""
    import importlib.machinery
    import importlib.util
    import shutil
    import threading
    import time
    dev = dict(device="cuda")
    x = torch.zeros((0, 300, 64), dtype=torch.bfloat16, **dev)
    pos, table = torch.zeros(0, dtype=torch.int32, **dev), torch.zeros((4, 64), **dev)
    binding.fp8rl_rope(x, pos, table)                          # loads the module
    copy = str(tmp_path / "_calls.so")                         # a module of its own, with its own functions
    shutil.copy(binding._calls.__spec__.origin, copy)
    calls = importlib.util.module_from_spec(importlib.util.spec_from_loader(
        "_calls", importlib.machinery.ExtensionFileLoader("_calls", copy)))
    calls.__spec__.loader.exec_module(calls)
    poll = ctypes.cast(ctypes.CDLL(None).poll, ctypes.c_void_p).value
    calls.bind(poll, poll, poll, poll, poll, binding.Fp8rlError)
    pool = torch.zeros((2, 4, 2, 64), dtype=torch.bfloat16, **dev)
    kv = torch.zeros((2, 2, 64), dtype=torch.bfloat16, **dev)
    buf = torch.zeros(1000, **dev)
    q = torch.zeros(1000, dtype=torch.bfloat16, **dev).as_strided((2, 0, 64), (300, 64, 1))
    ws = torch.zeros(16, dtype=torch.uint8, **dev)
    made = {"rope": lambda: calls.rope(x, pos, table, False, False, None, None),
            "append": lambda: calls.rope_append_paged(q, kv, kv, None, None, pool, pool, torch.zeros(2, dtype=torch.int64, **dev),
                                                      None, None, False, None, None),
            "attn": lambda: calls.attn_paged(x.view(0, 300, 1, 64).expand(0, 300, 2, 64), pool, pool,
                                             torch.zeros((0, 2), dtype=torch.int32, **dev), pos, 8, None, 0, None, None,
                                             None, None, False, ws, None),
            "verify": lambda: calls.spec_verify(buf.as_strided((1, 2, 8), (0, 300, 1)), torch.zeros((1, 1), dtype=torch.int32, **dev),
                                                buf[:1].view(1, 1), buf[:8].view(1, 8), None, None, None, None, None)}
    for name, call in made.items():
        ticks, stop = [0], threading.Event()

        def tick():
            while not stop.wait(0.002):
                ticks[0] += 1
        t = threading.Thread(target=tick)
        t.start()
        while not ticks[0]:
            time.sleep(0.001)
        before, t0 = ticks[0], time.perf_counter()
        call()
        took, ran = time.perf_counter() - t0, ticks[0] - before
        stop.set()
        t.join()
        assert took > 0.25, (name, took)                       # the function did wait
        assert ran > 20, (name, ran)                           # of some 140
