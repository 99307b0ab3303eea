"""Cases of the trainer's side of an 8-bit rollout: log-probabilities of sampled
tokens straight from the hidden states and the output matrix, whose logits are not
kept, with their gradient; and distillation from a teacher's top logits, with its
gradient.  ``run`` computes them in elementary torch operations where ``own`` is
false, and through the framework's entry points where it is true.

The vocabulary of 152064 and the hidden sizes 3584 and 5120 are those of the 7B-
and 32B-shaped layers that the benchmark runs; the others are generic."""
import math
import random

import torch

own = False

BF16 = torch.bfloat16


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the log-probability of one sampled token: a single sequence scored as it
        # is generated; one pass over the matrix
        dict(name="logp_one_token", op="logp", M=1, V=152064, K=3584, masked=0.0, entropy=False, scale=1.0),
        # one decode step of 48 sequences, at the sampling temperature of 0.7
        dict(name="logp_decode", op="logp", M=48, V=152064, K=5120, masked=0.0, entropy=False, scale=1.0 / 0.7),
        # a small draft model over an odd vocabulary, a ragged batch with entropies
        dict(name="logp_small", op="logp", M=333, V=50257, K=1024, masked=0.2, entropy=True, scale=1.0),
        # the trainer's scoring of a packed batch: prompts and padding (0.3 of the rows) do not count
        dict(name="logp_batch", op="logp", M=8192, V=152064, K=3584, masked=0.3, entropy=True, scale=1.0),
        # the gradient of a small model's step, entropy bonus included
        dict(name="grad_small", op="grad", M=500, V=32000, K=1024, masked=0.2, entropy=True, scale=1.0, dh=True, dw=True),
        # the output matrix frozen, as with low-rank adapters: only the hidden states' gradient
        dict(name="grad_frozen_head", op="grad", M=1531, V=151936, K=5120, masked=0.0, entropy=False,
             scale=1.0 / 0.7, dh=True, dw=False),
        # the trainer's step on a packed batch: both gradients, a third of the rows not counted
        dict(name="grad_batch", op="grad", M=4096, V=152064, K=3584, masked=1.0 / 3.0, entropy=False, scale=1.0,
             dh=True, dw=True),
        # distillation loss of one token: latency
        dict(name="distill_one", op="distill", M=1, V=152064, k=64, dtype="bf16", rest=True, masked=0.0, scale=1.0),
        # a batch, the teacher's 64 best tokens and what they leave as one more class
        dict(name="distill_batch", op="distill", M=4096, V=152064, k=64, dtype="bf16", rest=True, masked=0.1,
             scale=0.5),
        # fp32 logits over an odd vocabulary (rows padded to their alignment), distributions cut to the teacher's 20 best
        dict(name="distill_fp32", op="distill", M=777, V=50257, k=20, dtype="fp32", rest=False, masked=0.1, scale=1.0),
        # its gradient
        dict(name="distill_grad_fp32", op="distill_grad", M=777, V=50257, k=20, dtype="fp32", rest=False, masked=0.1,
             scale=1.0),
        # the batch's gradient: the largest read and write
        dict(name="distill_grad_batch", op="distill_grad", M=4096, V=152064, k=64, dtype="bf16", rest=True,
             masked=0.1, scale=0.5),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(n, lo), hi)


def draw(rng):
    op = rng.choice(["logp", "logp", "grad", "grad", "distill", "distill_grad"])
    V = rng.choice([152064, 151936, 32000, 50257, _log(rng, 1000, 150000)])
    masked = rng.choice([0.0, 0.0, round(rng.uniform(0.05, 0.8), 3)])
    scale = rng.choice([1.0, 1.0, 1.0 / 0.7, 0.5])
    if op in ("logp", "grad"):
        K = rng.choice([512, 896, 1024, 2048, 3584, 4096, 5120, 8 * _log(rng, 32, 800)])
        most = (8192 if op == "logp" else 4096) * 152064 * 3584
        M = _log(rng, 1, min(8192, most // (V * K)))
        c = dict(op=op, M=M, V=V, K=K, masked=masked, entropy=rng.random() < 0.5, scale=scale)
        if op == "grad":
            c["dh"], c["dw"] = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        return c
    return dict(op=op, M=_log(rng, 1, min(8192, 4096 * 152064 // V)), V=V, k=rng.choice([1, 8, 20, 64, 100, 128, 256]),
                dtype=rng.choice(["bf16", "bf16", "fp32"]), rest=rng.random() < 0.5, masked=masked, scale=scale)


def _live(c):
    """Rows that count: the share left out, but never all of them."""
    return max(1, c["M"] - int(round(c["M"] * c["masked"])))


def work(c):
    M, V, n = c["M"], c["V"], _live(c)
    if c["op"] in ("logp", "grad"):
        K = c["K"]
        read = 2 * K * (n + V) + 4 * M
        if c["op"] == "logp":
            return dict(bytes=read + 4 * M * (3 if c["entropy"] else 2), flops=2 * n * V * K)
        # the logits again, then a product for each gradient
        back = (2 * M * K if c["dh"] else 0) + (2 * V * K if c["dw"] else 0)
        return dict(bytes=read + back + 4 * M * (4 if c["entropy"] else 2), flops=2 * n * V * K * (1 + c["dh"] + c["dw"]))
    size = 2 if c["dtype"] == "bf16" else 4
    teacher = 8 * M * c["k"] + (4 * M if c["rest"] else 0)
    sums = 8 * M if c["rest"] else 4 * M
    if c["op"] == "distill":
        return dict(bytes=n * V * size + teacher + 4 * M + sums, flops=4 * n * V)
    return dict(bytes=(n + M) * V * size + teacher + 4 * M + sums, flops=4 * n * V)


# ---------------------------------------------------------------- inputs

def _rows_left_out(c, g, dev):
    out = torch.zeros(c["M"], dtype=torch.bool, device=dev)
    out[torch.randperm(c["M"], generator=g, device=dev)[:c["M"] - _live(c)]] = True
    return out


def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    M, V = c["M"], c["V"]
    out = _rows_left_out(c, g, dev)
    if c["op"] in ("logp", "grad"):
        K = c["K"]
        h = torch.randn((M, K), generator=g, device=dev, dtype=BF16)
        w = torch.randn((V, K), generator=g, device=dev, dtype=BF16)
        w.mul_(2.5 / math.sqrt(K))
        t = torch.randint(0, V, (M,), generator=g, device=dev, dtype=torch.int32)
        # sampled tokens are likely ones: the hidden states lean towards their rows of the matrix
        lean = torch.rand((M, 1), generator=g, device=dev) * 2.0
        h = (h.float() + lean * w[t.long()].float()).to(BF16)
        t[out] = -1
        h[out] = float("nan")                               # what a row of padding holds is nobody's
        s = dict(c=c, h=h, w=w, t=t)
        if c["op"] == "grad":
            # the forward pass has left each row's log-sum and entropy; the loss its gradient:
            # advantages times importance weights over the count, and an entropy bonus
            s["lse"], s["entropy"] = _plain_logp(s)[1:]
            s["g"] = torch.randn(M, generator=g, device=dev) / M
            s["ge"] = torch.rand(M, generator=g, device=dev) * (-0.01 / M) if c["entropy"] else None
        return s
    dt = BF16 if c["dtype"] == "bf16" else torch.float32
    pad = -(-V // 8) * 8
    x = torch.randn((M, pad), generator=g, device=dev)
    x.mul_(2.5)
    teacher = torch.randn((M, V), generator=g, device=dev)
    teacher.add_(x[:, :V])                                  # a student on the way to its teacher
    best, ids = teacher.topk(min(c["k"], V), dim=1)
    s = dict(c=c, x=x.to(dt)[:, :V], t=best.contiguous(), ids=ids.to(torch.int32).contiguous())
    s["ids"][out] = -1
    s["x"][out] = float("nan")
    top = best[:, :1]
    s["teacher_lse"] = ((((teacher - top) * c["scale"]).exp_().sum(1).log() + top[:, 0] * c["scale"])
                        if c["rest"] else None)
    if c["op"] == "distill_grad":
        _, s["lse"], s["rest_lse"] = _plain_distill(s)
        s["g"] = torch.rand(M, generator=g, device=dev) * (2.0 / M)
    return s


# ---------------------------------------------------------------- plain forms

def _logits(s):
    """Scaled logits in 32 bits, rows left out as zeros; and which rows count."""
    live = s["t"] >= 0
    h = torch.where(live[:, None], s["h"].float(), 0.0)
    w = s["w"].float()
    return (h @ w.T).mul_(s["c"]["scale"]), h, w, live


def _plain_logp(s):
    x, _, _, live = _logits(s)
    top = x.amax(dim=1)
    picked = x.gather(1, s["t"].clamp(min=0).long()[:, None])[:, 0]
    x.sub_(top[:, None])
    e = torch.exp(x)
    total = e.sum(dim=1)
    lse = torch.log(total) + top
    entropy = torch.log(total) - x.mul_(e).sum(dim=1) / total
    zero = torch.zeros_like(lse)
    return tuple(torch.where(live, v, zero) for v in (picked - lse, lse, entropy))


def _plain_grad(s):
    c = s["c"]
    x, h, w, live = _logits(s)
    g = torch.where(live, s["g"], 0.0)
    logp = x.sub_(s["lse"][:, None])
    p = torch.exp(logp)
    if c["entropy"]:
        ge = torch.where(live, s["ge"], 0.0)
        d = -p * (g[:, None] + ge[:, None] * (logp + s["entropy"][:, None]))
    else:
        d = p.mul_(-g[:, None])
    at = torch.arange(c["M"], device=d.device)
    d[at, s["t"].clamp(min=0).long()] += g
    d.mul_(c["scale"])
    return (d @ w).to(BF16) if c["dh"] else None, (d.T @ h).to(BF16) if c["dw"] else None


def _teacher(s):
    """The teacher's probabilities of its entries and of the rest, in 64 bits."""
    c = s["c"]
    t = s["t"].double() * c["scale"]
    there = s["ids"] >= 0
    if s["teacher_lse"] is not None:
        q = torch.where(there, torch.exp(t - s["teacher_lse"].double()[:, None]), 0.0)
        return q, (1.0 - q.sum(dim=1)).clamp(min=0.0)
    e = torch.where(there, torch.exp(t - t.amax(dim=1, keepdim=True)), 0.0)
    return e / e.sum(dim=1, keepdim=True).clamp(min=1e-300), None


def _plain_distill(s):
    c, ids = s["c"], s["ids"].clamp(min=0).long()
    x = s["x"].float() * c["scale"]
    there = s["ids"] >= 0
    live = there.any(dim=1)
    top = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - top)
    lse = (torch.log(e.sum(dim=1, dtype=torch.float64)) + top[:, 0].double())
    q, qr = _teacher(s)
    logq = torch.log(torch.where(q > 0, q, 1.0))
    loss = (q * (logq - (x.gather(1, ids).double() - lse[:, None]))).sum(dim=1)
    rest = None
    if c["rest"]:
        e.scatter_(1, ids, 0.0)
        rest = torch.log(e.sum(dim=1, dtype=torch.float64)) + top[:, 0].double()
        loss = loss + torch.where(qr > 0, qr * (torch.log(torch.where(qr > 0, qr, 1.0)) - (rest - lse)), 0.0)
    zero = torch.zeros_like(lse)
    loss, lse = torch.where(live, loss, zero).float(), torch.where(live, lse, zero).float()
    return loss, lse, torch.where(live, rest, zero).float() if rest is not None else None


def _plain_distill_grad(s):
    c, ids = s["c"], s["ids"].clamp(min=0).long()
    live = (s["ids"] >= 0).any(dim=1)
    x = s["x"].float() * c["scale"]
    q, qr = _teacher(s)
    p = torch.exp(x - s["lse"][:, None])
    total = q.sum(dim=1) + (qr if qr is not None else 0.0)
    d = p * total.float()[:, None]
    inside = d.gather(1, ids).double() - q
    if c["rest"]:
        d.sub_(torch.exp(x - s["rest_lse"][:, None]).mul_(qr.float()[:, None]))
    d.scatter_(1, ids, inside.float())
    d.mul_((s["g"] * c["scale"])[:, None])
    return torch.where(live[:, None], d, 0.0).to(s["x"].dtype)


def run(s):
    c = s["c"]
    if own:
        from precision_rl_rollout_gb300 import binding as fb
        if c["op"] == "logp":
            return fb.fp8rl_linear_logp(s["h"], s["w"], s["t"], scale=c["scale"], want_entropy=c["entropy"])
        if c["op"] == "grad":
            return fb.fp8rl_linear_logp_backward(
                s["h"], s["w"], s["t"], s["lse"], s["g"], entropy=s["entropy"] if c["entropy"] else None,
                g_entropy=s["ge"], scale=c["scale"], want_dH=c["dh"], want_dW=c["dw"])
        if c["op"] == "distill":
            return fb.fp8rl_distill_topk(s["x"], s["ids"], s["t"], teacher_lse=s["teacher_lse"], rest=c["rest"],
                                         scale=c["scale"])
        return fb.fp8rl_distill_topk_backward(s["x"], s["ids"], s["t"], s["lse"], s["g"],
                                              teacher_lse=s["teacher_lse"], rest_lse=s["rest_lse"], scale=c["scale"])
    if c["op"] == "logp":
        out = _plain_logp(s)
        return out if c["entropy"] else out[:2]
    if c["op"] == "grad":
        return _plain_grad(s)
    if c["op"] == "distill":
        out = _plain_distill(s)
        return out if c["rest"] else out[:2]
    return _plain_distill_grad(s)


# ---------------------------------------------------------------- 64 bits

def exact(c, seed):
    """The definitions in 64 bits over the rows that count alone; the gradients by
    differentiating them."""
    s = prepare(c, seed)
    if c["op"] in ("logp", "grad"):
        rows = torch.nonzero(s["t"] >= 0)[:, 0]
        back = c["op"] == "grad"
        w = s["w"].double().requires_grad_(back and c["dw"])
        h = s["h"][rows].double().requires_grad_(back and c["dh"])
        t = s["t"][rows].long()
        with torch.set_grad_enabled(back):
            full = torch.log_softmax(torch.nn.functional.linear(h, w) * c["scale"], dim=1)
            logp = full.gather(1, t[:, None])[:, 0]
            if not back or c["entropy"]:
                entropy = -(full.exp() * full).sum(dim=1)
        if not back:
            picked = (h * w[t]).sum(dim=1) * c["scale"]
            outs = []
            for v in (logp, picked - logp, entropy)[:3 if c["entropy"] else 2]:
                outs.append(torch.zeros(c["M"], dtype=torch.float64, device="cuda").index_copy_(0, rows, v))
            return tuple(outs)
        loss = (logp * s["g"][rows].double()).sum()
        if c["entropy"]:
            loss = loss + (entropy * s["ge"][rows].double()).sum()
        loss.backward()
        dh = torch.zeros((c["M"], c["K"]), dtype=torch.float64, device="cuda").index_copy_(0, rows, h.grad) if c["dh"] else None
        return dh, w.grad
    M, V = c["M"], c["V"]
    back = c["op"] == "distill_grad"
    loss, lse, rest = (torch.zeros(M, dtype=torch.float64, device="cuda") for _ in range(3))
    dx = torch.zeros((M, V), dtype=torch.float64, device="cuda") if back else None
    for first in range(0, M, 512):                           # a few rows at a time
        rows = torch.arange(first, min(M, first + 512), device="cuda")
        rows = rows[(s["ids"][rows] >= 0).any(dim=1)]
        if not rows.numel():
            continue
        ids, t = s["ids"][rows].long(), s["t"][rows].double() * c["scale"]
        x = s["x"][rows].double().requires_grad_(back)
        with torch.set_grad_enabled(back):
            y = x * c["scale"]
            total = torch.logsumexp(y, dim=1)
            inside = torch.zeros_like(y, dtype=torch.bool).scatter_(1, ids, True)
            if c["rest"]:
                logq = t - s["teacher_lse"][rows].double()[:, None]
                left = torch.logsumexp(y.masked_fill(inside, float("-inf")), dim=1)
                qr = (1.0 - logq.exp().sum(dim=1)).clamp(min=0.0)
                part = torch.special.xlogy(qr, qr) - qr * (left - total)
            else:
                logq, left, part = torch.log_softmax(t, dim=1), total, 0.0
            value = torch.nn.functional.kl_div(y.gather(1, ids) - total[:, None], logq, reduction="none",
                                               log_target=True).sum(dim=1) + part
        if back:
            (value * s["g"][rows].double()).sum().backward()
            dx[rows] = x.grad
        else:
            loss[rows], lse[rows], rest[rows] = value, total, left
    if back:
        return dx
    return (loss, lse, rest) if c["rest"] else (loss, lse)
