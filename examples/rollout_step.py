"""One speculative rollout step of a small 8-bit layer, end to end on the GPU:

    python examples/rollout_step.py [--sequences 8] [--drafts 3] [--bf16-cache]

A batch of sequences with prompts in a paged cache gets its drafted tokens: the
qkv projection runs in 8 bits, queries and keys are rotated and keys and values
stored in the cache's pages, the new tokens attend over the cache, the output
projection and the LM head run in 8 bits, and the drafts are verified against the
target's probabilities.  The prompts are written with the same append; E4M3 caches
take their scales from the prompts' keys and values.  Weights and inputs are
random; what is printed is how many drafts were kept, and the difference of the
attention output from one computed in plain 64-bit torch over the same cache.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from precision_rl_rollout_gb300 import binding as fb
from precision_rl_rollout_gb300.positions import rope_frequencies

HIDDEN, HQ, HKV, D, VOCAB, PAGE = 1024, 8, 2, 128, 4096, 16


def weights(n, k, g):
    return fb.fp8rl_quant_weight_block(torch.randn((n, k), generator=g, device="cuda").mul_(k ** -0.5).to(torch.bfloat16))


def project(x, w):
    return fb.fp8rl_linear_w8a8_block(x, *w)


def heads_of(qkv):
    q, k, v = qkv.view(-1, HQ + 2 * HKV, D).split([HQ, HKV, HKV], dim=1)
    return q, k, v


def step(sequences=8, drafts=3, e4m3=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w_qkv, w_o, w_head = weights((HQ + 2 * HKV) * D, HIDDEN, g), weights(HIDDEN, HQ * D, g), weights(VOCAB, HIDDEN, g)
    embed = torch.randn((VOCAB, HIDDEN), generator=g, device="cuda").to(torch.bfloat16)
    freq, magnitude = rope_frequencies(D, base=1e6, scaling="bands", factor=4.0, trained=1024)
    table = fb.fp8rl_rope_table(torch.tensor(freq, dtype=torch.float64, device="cuda"), 4096, magnitude)

    # ragged prompts, and pages for them and the new tokens
    new = drafts + 1
    prompt = torch.randint(1, 300, (sequences,), generator=g, device="cuda")
    lens = (prompt + new).to(torch.int32)
    columns = (int(lens.max()) + PAGE - 1) // PAGE
    pages = torch.randperm(sequences * columns, generator=g, device="cuda").view(sequences, columns)
    shape = (sequences * columns, PAGE, HKV, D)
    K, V = (torch.zeros(shape, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda") for _ in range(2))

    def slots(seq, pos):
        return pages[seq, pos // PAGE] * PAGE + pos % PAGE

    # the prompts: project, calibrate the cache's scales, rotate and store
    seq = torch.repeat_interleave(torch.arange(sequences, device="cuda"), prompt)
    pos = torch.cat([torch.arange(int(n), device="cuda") for n in prompt])
    tokens = torch.randint(0, VOCAB, (seq.numel(),), generator=g, device="cuda")
    q, k, v = heads_of(project(embed[tokens], w_qkv))
    scales = {}
    if e4m3:
        rotated = fb.fp8rl_rope(k, pos.int(), table)
        scales = dict(k_scale=fb.fp8rl_quant_kv_tensor(rotated.view(-1, HKV * D))[1],
                      v_scale=fb.fp8rl_quant_kv_tensor(v.reshape(-1, HKV * D))[1])
    fb.fp8rl_rope_append_paged(q, k, v, pos.int(), table, K, V, slots(seq, pos), **scales)

    # the step: the last accepted token and its drafts, all at once
    draft = torch.randint(0, VOCAB, (sequences, drafts), generator=g, device="cuda", dtype=torch.int32)
    last = torch.randint(0, VOCAB, (sequences, 1), generator=g, device="cuda", dtype=torch.int32)
    seq = torch.arange(sequences, device="cuda").repeat_interleave(new)
    pos = prompt.repeat_interleave(new) + torch.arange(new, device="cuda").repeat(sequences)
    q, k, v = heads_of(project(embed[torch.cat([last, draft], dim=1).flatten().long()], w_qkv))
    q = fb.fp8rl_rope_append_paged(q, k, v, pos.int(), table, K, V, slots(seq, pos), **scales)
    q = q.view(sequences, new, HQ, D)
    o, lse = fb.fp8rl_attn_paged(q, K, V, pages.to(torch.int32), lens, columns * PAGE, want_lse=True, **scales)
    logits = project(project(o.view(-1, HQ * D), w_o), w_head)
    P = torch.softmax(logits.float() * 0.2, dim=-1).view(sequences, new, VOCAB)

    # a drafter that agrees with the target up to noise, and its drafts' verdict
    Q = torch.softmax(torch.log(P[:, :drafts]) + 0.3 * torch.randn(P[:, :drafts].shape, generator=g, device="cuda"), -1)
    u = torch.rand((sequences, drafts), generator=g, device="cuda")
    noise = torch.empty((sequences, VOCAB), device="cuda").exponential_(generator=g)
    out, kept = fb.fp8rl_spec_verify(P, draft, u, noise, Q=Q)
    assert fb.fp8rl_check_device_error() == 0
    return dict(q=q, K=K, V=V, pages=pages, lens=lens, scales=scales, o=o, lse=lse, draft=draft, P=P, Q=Q, u=u,
                noise=noise, out=out, kept=kept)


def exact_attention(r):
    """The attention output of ``step`` in 64 bits, sequence by sequence."""
    outs = []
    for b, n in enumerate(r["lens"].tolist()):
        kv = []
        for pool, s in ((r["K"], "k_scale"), (r["V"], "v_scale")):
            x = pool[r["pages"][b]].flatten(0, 1)[:n]
            x = x.view(torch.float8_e4m3fn).double() * r["scales"][s].double() if r["scales"] else x.double()
            kv.append(x.repeat_interleave(HQ // HKV, dim=1))
        q = r["q"][b].double()
        x = torch.einsum("ihd,jhd->hij", q, kv[0]) * D ** -0.5
        new = q.shape[0]
        mask = torch.arange(n, device=x.device)[None, :] > torch.arange(n - new, n, device=x.device)[:, None]
        x = torch.softmax(x.masked_fill(mask, float("-inf")), dim=-1)
        outs.append(torch.einsum("hij,jhd->ihd", x, kv[1]))
    return torch.stack(outs)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--sequences", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--bf16-cache", action="store_true")
    a = ap.parse_args()
    r = step(a.sequences, a.drafts, not a.bf16_cache)
    want = exact_attention(r)
    err = ((r["o"].double() - want).norm() / want.norm()).item()
    print(f"kept {r['kept'].tolist()} of {a.drafts} drafts; attention error against 64 bits {err:.2e}")
    print("tokens of the first sequence:", r["out"][0].tolist())


if __name__ == "__main__":
    main()
