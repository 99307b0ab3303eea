"""Cases of the rollout step's cache operators: rotary positions, the rotating
append to a paged key-value cache, attention over that cache, and verification
of drafted tokens.  ``run`` computes them in elementary torch operations where
``own`` is false, and through the framework's entry points where it is true.

Head counts, widths and the vocabulary are those of the 7B- and 32B-shaped
layers the benchmark runs (28/4 and 40/8 heads of 128, 152064 logits); the other
head layouts are generic."""
import math
import random

import torch

own = False

BF16 = torch.bfloat16
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of one sequence: q and k heads of a 7B-shaped layer, as in a
        # rollout's last running sequence; latency is all that counts
        dict(name="rope_one_token", op="rope", T=1, Hq=28, Hkv=4, D=128, R=128, inter=False, back=False,
             max_pos=32768, scaled=False),
        # a prefill batch of a 32B-shaped layer, positions scaled to a long context
        dict(name="rope_prefill", op="rope", T=8192, Hq=40, Hkv=8, D=128, R=128, inter=False, back=False,
             max_pos=131072, scaled=True),
        # the trainer's side: gradient for a packed batch with an odd token count,
        # interleaved pairs over half of each head
        dict(name="rope_gradient", op="rope", T=16411, Hq=28, Hkv=4, D=128, R=64, inter=True, back=True,
             max_pos=32768, scaled=False),
        # one decode step of 61 sequences into 8-bit pages of 16 tokens
        dict(name="append_decode_e4m3", op="append", T=61, Hq=28, Hkv=4, D=128, R=128, inter=False, page=16,
             cache="e4m3", heads_first=False, prefill=False, pad=0, max_pos=32768),
        # a prefill chunk of a 32B-shaped layer into bf16 pages of 64 tokens
        dict(name="append_prefill_bf16", op="append", T=8192, Hq=40, Hkv=8, D=128, R=128, inter=False, page=64,
             cache="bf16", heads_first=True, prefill=True, pad=0, max_pos=32768),
        # the last sequence of a rollout early in its life: latency
        dict(name="attn_one_short", op="attn", B=1, L=777, Lq=1, Hq=28, Hkv=4, D=128, page=16, cache="bf16",
             heads_first=False, window=0, spread=0.0),
        # the long tail: one sequence, a long bf16 cache, split over its length
        dict(name="attn_one_long", op="attn", B=1, L=131072, Lq=1, Hq=40, Hkv=8, D=128, page=64, cache="bf16",
             heads_first=True, window=0, spread=0.0),
        # the usual decode step: 64 ragged sequences over an 8-bit cache
        dict(name="attn_decode_e4m3", op="attn", B=64, L=8191, Lq=1, Hq=28, Hkv=4, D=128, page=16, cache="e4m3",
             heads_first=False, window=0, spread=1.0),
        # verification of four drafted tokens: five query rows per sequence
        dict(name="attn_verify_e4m3", op="attn", B=32, L=16384, Lq=5, Hq=40, Hkv=8, D=128, page=32, cache="e4m3",
             heads_first=False, window=0, spread=1.0),
        # a full batch late in a rollout, bf16 cache: the largest read
        dict(name="attn_full_batch", op="attn", B=128, L=16384, Lq=1, Hq=40, Hkv=8, D=128, page=16, cache="bf16",
             heads_first=False, window=0, spread=1.0),
        # verification of four drafted tokens of one sequence
        dict(name="verify_one", op="verify", B=1, K=4, V=152064, probs="fp32", draft_probs=True, near=0.5),
        # a full batch's verification, eight drafted tokens each
        dict(name="verify_batch", op="verify", B=256, K=8, V=152064, probs="fp32", draft_probs=True, near=0.5),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(n, lo), hi)


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "verify"])
    Hq, Hkv = rng.choice([(28, 4), (40, 8), (16, 16), (8, 1), (10, 5), (7, 1), (48, 3)])
    if op == "rope":
        D = rng.choice([64, 80, 128, 256])
        R = rng.choice([D, D, D // 2, D // 4 * 3 // 8 * 8])
        T = _log(rng, 1, 16384)
        return dict(op=op, T=T, Hq=Hq, Hkv=Hkv, D=D, R=R, inter=rng.random() < 0.4, back=rng.random() < 0.5,
                    max_pos=rng.choice([4096, 32768, 131072]), scaled=rng.random() < 0.5)
    if op == "append":
        D = rng.choice([64, 96, 128, 256])
        return dict(op=op, T=_log(rng, 1, 8192), Hq=Hq, Hkv=Hkv, D=D, R=rng.choice([D, D, D // 2]),
                    inter=rng.random() < 0.4, page=rng.choice([8, 16, 24, 32, 64]),
                    cache=rng.choice(["bf16", "e4m3"]), heads_first=rng.random() < 0.5,
                    prefill=rng.random() < 0.5, pad=rng.choice([0, 0, 3]), max_pos=32768)
    if op == "attn":
        D = rng.choice([64, 96, 128, 128, 256])
        Lq = rng.choice([1, 1, 1, 2, 3, 5, 8])
        B = _log(rng, 1, 128)
        # no more cached values than the largest listed case
        most = min(131072, 128 * 16384 * 8 * 128 // (B * Hkv * D * 2))
        L = _log(rng, 1, most)
        # many query rows against many tokens are bounded by their products
        if Lq * Hq * L * B > 128 * 16384 * 40:
            Lq = 1
        return dict(op=op, B=B, L=L, Lq=Lq, Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([8, 16, 24, 32, 64, 128]),
                    cache=rng.choice(["bf16", "e4m3"]), heads_first=rng.random() < 0.5,
                    window=rng.choice([0, 0, 0, 1 + L // 3]), spread=rng.choice([0.0, 1.0, 1.0]))
    V = rng.choice([152064, 151936, 32000, 50257, _log(rng, 1000, 150000)])
    return dict(op=op, B=_log(rng, 1, 200), K=rng.randint(1, 8), V=V, probs=rng.choice(["fp32", "fp32", "bf16"]),
                draft_probs=rng.random() < 0.75, near=round(rng.uniform(0.1, 2.0), 3))


def _lengths(c):
    """Cached tokens of each sequence: the first is the longest; with spread 1 the
    others fall off towards short ones, as in a batch of rollouts."""
    golden = 0.6180339887498949
    out = []
    for i in range(c["B"]):
        f = 1.0 - (i * golden) % 1.0
        out.append(max(1, int(round(c["L"] * (1.0 - c["spread"] * (1.0 - f))))))
    return out


def work(c):
    if c["op"] == "rope":
        H = c["Hq"] + c["Hkv"]
        return dict(bytes=4 * c["T"] * H * c["D"] + c["T"] * (4 + 4 * c["R"]), flops=3 * c["T"] * H * c["R"])
    if c["op"] == "append":
        n = 1 if c["cache"] == "e4m3" else 2
        T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
        return dict(bytes=T * ((Hq + 2 * Hkv) * D * 2 + Hq * D * 2 + 2 * Hkv * D * n + 12 + 4 * c["R"]),
                    flops=3 * T * (Hq + Hkv) * c["R"])
    if c["op"] == "attn":
        n = 1 if c["cache"] == "e4m3" else 2
        seen = pairs = pages = 0
        for length in _lengths(c):
            first = max(0, length - c["Lq"] - c["window"] + 1) if c["window"] else 0
            seen += length - first
            pages += -(-length // c["page"]) - first // c["page"]
            for i in range(c["Lq"]):
                p = length - c["Lq"] + i
                if p >= 0:
                    pairs += min(p + 1, c["window"]) if c["window"] else p + 1
        rows = c["B"] * c["Lq"] * c["Hq"]
        return dict(bytes=2 * seen * c["Hkv"] * c["D"] * n + rows * (4 * c["D"] + 4) + 4 * pages + 4 * c["B"],
                    flops=4 * c["D"] * c["Hq"] * pairs)
    # one row of the target's probabilities and of the race's numbers for every
    # sequence; the drafter's row too for the half or so that refuse a token
    n = 4 if c["probs"] == "fp32" else 2
    rows = n + 4 + (n / 2 if c["draft_probs"] else 0)
    return dict(bytes=c["B"] * (c["V"] * rows + c["K"] * 12 + 4 * c["K"] + 8), flops=2 * c["B"] * c["V"])


# ---------------------------------------------------------------- inputs

def _table(c, dev):
    """cos | sin of every position, fp32 [max_pos, R], computed in 64 bits.  A
    scaled table stretches the slow frequencies to four times the context and
    blends towards the fast ones, with the usual magnitude correction."""
    half = c["R"] // 2
    inv = 1.0 / (1e6 ** (torch.arange(half, dtype=torch.float64, device=dev) * 2.0 / c["R"]))
    mag = 1.0
    if c.get("scaled"):
        turns = 32768.0 * inv / (2.0 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        inv = inv * (keep + (1.0 - keep) / 4.0)
        mag = 0.1 * math.log(4.0) + 1.0
    angle = torch.arange(c["max_pos"], dtype=torch.float64, device=dev)[:, None] * inv[None, :]
    return torch.cat([torch.cos(angle) * mag, torch.sin(angle) * mag], dim=1).float()


def _pools(c, pages, g, dev, fill):
    """Key and value pools [pages, page, Hkv, D]; heads_first lays each page out
    head by head.  E4M3 pools hold codes, with one scale each."""
    shape = (pages, c["Hkv"], c["page"], c["D"]) if c["heads_first"] else (pages, c["page"], c["Hkv"], c["D"])
    out = []
    for spread in (1.0, 0.5):
        if not fill:
            x = torch.zeros(shape, dtype=BF16, device=dev)
            scale = 5.5 / 448.0
        else:
            x = torch.randn(shape, generator=g, device=dev, dtype=BF16)
            x.mul_(spread)
            scale = 5.5 * spread / 448.0
        s = torch.full((1,), scale, dtype=torch.float32, device=dev)
        if c["cache"] == "e4m3":
            if fill:
                x.mul_(1.0 / scale).clamp_(-448.0, 448.0)
            x = x.to(E4M3).view(torch.uint8)
        out.append((x.transpose(1, 2) if c["heads_first"] else x, s))
    return out


def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    if c["op"] == "rope":
        T, H, D = c["T"], c["Hq"] + c["Hkv"], c["D"]
        if c["back"]:
            x = torch.randn((T, H, D), generator=g, device=dev, dtype=BF16)
        else:  # the q and k heads of a fused projection's output
            x = torch.randn((T, H + c["Hkv"], D), generator=g, device=dev, dtype=BF16)[:, :H]
        pos = torch.randint(0, c["max_pos"], (T,), generator=g, device=dev, dtype=torch.int32)
        return dict(c=c, x=x, pos=pos, table=_table(c, dev))
    if c["op"] == "append":
        T, Hq, Hkv, D, page = c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
        qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=dev, dtype=BF16)
        if c["prefill"]:  # consecutive tokens of one sequence, pages anywhere in the pool
            pages = -(-T // page) + 5
            t = torch.arange(T, device=dev)
            start = int(torch.randint(0, c["max_pos"] - T, (1,), generator=g, device=dev)) if T < c["max_pos"] else 0
            where = torch.randperm(pages, generator=g, device=dev)
            slots = where[t // page] * page + t % page
            pos = (t + start).to(torch.int32)
        else:  # one token for each of T sequences
            pages = 2 * T + 1
            where = torch.randperm(pages, generator=g, device=dev)[:T]
            pos = torch.randint(0, c["max_pos"], (T,), generator=g, device=dev, dtype=torch.int32)
            slots = where * page + pos % page
        if c["pad"]:  # a step padded to a fixed batch: those tokens go nowhere
            slots[::c["pad"]] = -1
        (K, ks), (V, vs) = _pools(c, pages, g, dev, False)
        return dict(c=c, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], pos=pos,
                    slots=slots.to(torch.int64), table=_table(c, dev), K=K, V=V, ks=ks, vs=vs)
    if c["op"] == "attn":
        lens = _lengths(c)
        need = [-(-n // c["page"]) for n in lens]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        table = torch.zeros((c["B"], max(need)), dtype=torch.int32, device=dev)
        used = torch.arange(max(need), device=dev)[None, :] < torch.tensor(need, device=dev)[:, None]
        table[used] = order[:sum(need)]
        (K, ks), (V, vs) = _pools(c, pages, g, dev, True)
        q = torch.randn((c["B"], c["Lq"], c["Hq"], c["D"]), generator=g, device=dev, dtype=BF16) * 2.0
        return dict(c=c, q=q, K=K, V=V, ks=ks, vs=vs, table=table, L=max(lens),
                    lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    B, K, V = c["B"], c["K"], c["V"]
    dt = torch.float32 if c["probs"] == "fp32" else BF16
    q = torch.randn((B, K, V), generator=g, device=dev)
    q.mul_(2.5)
    p = torch.randn((B, K + 1, V), generator=g, device=dev)
    p.mul_(c["near"])
    p[:, :K].add_(q)
    p[:, K].add_(torch.randn((B, V), generator=g, device=dev), alpha=2.5)
    p, q = torch.softmax(p, dim=-1).to(dt), torch.softmax(q, dim=-1).to(dt)
    tokens = torch.empty((B, K), dtype=torch.int32, device=dev)
    for i in range(K):  # drafted tokens are drawn from the drafter's own row
        e = torch.empty((B, V), device=dev).exponential_(generator=g)
        tokens[:, i] = (q[:, i].float() / e).argmax(dim=-1).to(torch.int32)
    if not c["draft_probs"]:  # a drafter that only proposes tokens: half of them the target's best
        best = p[:, :K].float().argmax(dim=-1).to(torch.int32)
        tokens = torch.where(torch.rand((B, K), generator=g, device=dev) < 0.5, best, tokens)
        q = None
    return dict(c=c, p=p, q=q, tokens=tokens, u=torch.rand((B, K), generator=g, device=dev),
                lens=torch.randint(0 if B > 1 else K, K + 1, (B,), generator=g, device=dev, dtype=torch.int32),
                noise=torch.empty((B, V), device=dev).exponential_(generator=g))


# ---------------------------------------------------------------- plain forms

def _rotate(x, pos, table, R, inter, back):
    """The rotated first R values of each head, in 32 bits, before rounding."""
    x = x.float()
    rows = table[pos.long()]
    cos, sin = rows[:, None, :R // 2], rows[:, None, R // 2:]
    if back:
        sin = -sin
    if inter:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([y, x[..., R:]], dim=-1)


def _store(pool, slots, x, scale, page):
    keep = slots >= 0
    at, x = slots[keep], x[keep]
    if pool.dtype == torch.uint8:
        x = (x / scale).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
    else:
        x = x.to(BF16)
    pool[at // page, at % page] = x


def _values(pool):
    """What a pool holds, as numbers (of an E4M3 pool: in units of its scale)."""
    return pool.view(E4M3) if pool.dtype == torch.uint8 else pool


def _plain_attn(s):
    c, q = s["c"], s["q"].float()
    B, Lq, Hq, D = q.shape
    Hkv, page = c["Hkv"], c["page"]
    n = s["table"].shape[1] * page
    at = torch.arange(n, device=q.device)
    seen = torch.arange(Lq, device=q.device)[None, :] + (s["lens"][:, None] - Lq)      # [B, Lq]: position
    mask = at[None, None, :] <= seen[:, :, None]
    if c["window"]:
        mask = mask & (at[None, None, :] > seen[:, :, None] - c["window"])

    def side(pool, scale):
        x = pool[s["table"].long()].reshape(B, n, Hkv, D)
        if x.dtype == torch.uint8:
            return x.view(E4M3).float() * scale
        return x.float()

    rows = q.reshape(B, Lq, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    x = rows @ side(s["K"], s["ks"]).permute(0, 2, 3, 1)
    x = x.view(B, Hkv, Lq, -1, n) * (1.0 / math.sqrt(D))
    x = torch.where(mask[:, None, :, None, :], x, float("-inf"))
    top = x.amax(dim=-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    x = torch.exp(x - top)
    total = x.sum(dim=-1, keepdim=True)
    o = x.view(B, Hkv, -1, n) @ side(s["V"], s["vs"]).permute(0, 2, 1, 3)
    o = o.view(B, Hkv, Lq, -1, D) / torch.where(total == 0, 1.0, total)
    lse = (torch.log(total) + top)[..., 0]
    return (o.permute(0, 2, 1, 3, 4).reshape(B, Lq, Hq, D).to(BF16),
            lse.permute(0, 2, 1, 3).reshape(B, Lq, Hq))


def _plain_verify(s):
    c, p, q, tokens = s["c"], s["p"], s["q"], s["tokens"].long()
    B, K = tokens.shape
    V = p.shape[-1]
    pt = p[:, :K].gather(2, tokens[:, :, None])[:, :, 0].double()
    qt = q.gather(2, tokens[:, :, None])[:, :, 0].double() if q is not None else torch.ones_like(pt)
    step = torch.arange(K, device=p.device)[None, :]
    good = (s["u"].double() * qt < pt) & (step < s["lens"][:, None])
    n = good.long().cumprod(dim=1).sum(dim=1)                       # accepted drafts
    at = torch.arange(B, device=p.device)
    w = p[at, n].float()
    short = n < s["lens"]                                            # a draft was refused
    last = n.clamp(max=K - 1)
    if q is not None:
        less = (w - q[at, last].float()).clamp(min=0.0)
    else:
        less = w.clone()
        less[at, tokens[at, last]] = 0.0
    some = (less > 0).any(dim=1)
    w = torch.where((short & some)[:, None], less, w)
    score = torch.where(w > 0, w / s["noise"], 0.0)
    best = score.amax(dim=1, keepdim=True)
    ids = torch.arange(V, device=p.device)
    token = torch.where(score == best, ids[None, :], V).amin(dim=1)
    out = torch.where(step < n[:, None], tokens, -1)
    out = torch.cat([out, torch.full((B, 1), -1, device=p.device)], dim=1)
    out[at, n] = token
    return out.to(torch.int32), n.to(torch.int32)


def run(s):
    c = s["c"]
    if own:
        from precision_rl_rollout_gb300 import binding as fb
    if c["op"] == "rope":
        if own:
            return fb.fp8rl_rope(s["x"], s["pos"], s["table"], interleaved=c["inter"], inverse=c["back"])
        return _rotate(s["x"], s["pos"], s["table"], c["R"], c["inter"], c["back"]).to(BF16)
    if c["op"] == "append":
        if own:
            q = fb.fp8rl_rope_append_paged(s["q"], s["k"], s["v"], s["pos"], s["table"], s["K"], s["V"], s["slots"],
                                           k_scale=s["ks"], v_scale=s["vs"], interleaved=c["inter"])
        else:
            q = _rotate(s["q"], s["pos"], s["table"], c["R"], c["inter"], False).to(BF16)
            k = _rotate(s["k"], s["pos"], s["table"], c["R"], c["inter"], False)
            _store(s["K"], s["slots"], k, s["ks"], c["page"])
            _store(s["V"], s["slots"], s["v"].float(), s["vs"], c["page"])
        return q, _values(s["K"]), _values(s["V"])
    if c["op"] == "attn":
        if own:
            return fb.fp8rl_attn_paged(s["q"], s["K"], s["V"], s["table"], s["lens"], s["L"], window=c["window"],
                                       k_scale=s["ks"], v_scale=s["vs"], want_lse=True)
        return _plain_attn(s)
    if own:
        return fb.fp8rl_spec_verify(s["p"], s["tokens"], s["u"], s["noise"], Q=s["q"], draft_lens=s["lens"])
    return _plain_verify(s)


# ---------------------------------------------------------------- 64 bits

def _turn(x, pos, table, R, inter, back):
    """Rotation as a product of complex numbers."""
    x = x.double()
    rows = table[pos.long()].double()
    turn = torch.complex(rows[:, :R // 2], -rows[:, R // 2:] if back else rows[:, R // 2:])[:, None, :]
    y = x.clone()
    if inter:
        z = torch.complex(x[..., 0:R:2].contiguous(), x[..., 1:R:2].contiguous()) * turn
        y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * turn
        y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
    return y


def exact(c, seed):
    if c["op"] == "verify":  # whole numbers only
        return None
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _turn(s["x"], s["pos"], s["table"], c["R"], c["inter"], c["back"])
    if c["op"] == "append":
        q = _turn(s["q"], s["pos"], s["table"], c["R"], c["inter"], False)
        pools = []
        for pool, scale, x in ((s["K"], s["ks"], _turn(s["k"], s["pos"], s["table"], c["R"], c["inter"], False)),
                               (s["V"], s["vs"], s["v"].double())):
            out = _values(pool).to(torch.float64)
            keep = s["slots"] >= 0
            at = s["slots"][keep]
            out[at // c["page"], at % c["page"]] = ((x[keep] / scale.double()).clamp(-448.0, 448.0)
                                                      if c["cache"] == "e4m3" else x[keep])
            pools.append(out)
        return (q, *pools)
    B, Lq, Hq, D = s["q"].shape
    o = torch.zeros((B, Lq, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Lq, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    group = Hq // c["Hkv"]
    for b, length in enumerate(_lengths(c)):
        ids = s["table"][b, :-(-length // c["page"])].long()
        for h in range(c["Hkv"]):
            k, v = (_values(pool[ids, :, h]).double().reshape(-1, D)[:length]
                    * (scale.double() if c["cache"] == "e4m3" else 1.0)
                    for pool, scale in ((s["K"], s["ks"]), (s["V"], s["vs"])))
            for i in range(Lq):
                last = length - Lq + i + 1
                if last <= 0:
                    continue
                first = max(0, last - c["window"]) if c["window"] else 0
                heads = slice(h * group, (h + 1) * group)
                x = s["q"][b, i, heads].double() @ k[first:last].T / math.sqrt(D)
                lse[b, i, heads] = torch.logsumexp(x, dim=-1)
                o[b, i, heads] = torch.softmax(x, dim=-1) @ v[first:last]
    return o, lse
