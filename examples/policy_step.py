"""A trainer's step behind an 8-bit rollout, on the calls that the framework has for it:

- tokens sampled by the 8-bit policy (its output layer runs as a W8A8 linear layer) get
  their log-probability there;
- the trainer's own log-probabilities and entropies come straight from the hidden states
  and the bf16 output matrix (``fp8rl_linear_logp``), prompts and padding left out;
- importance weights between the two (``fp8rl_rollout_is_weights``);
- the policy gradient with an entropy bonus, back to hidden states and output matrix
  (``fp8rl_linear_logp_backward``);
- distillation of a smaller student from the policy's top logits (``fp8rl_distill_topk``
  and its gradient), the tokens that the policy did not name as one more class.

    python examples/policy_step.py [--tokens 512] [--steps 5]
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
from precision_rl_rollout_gb300 import binding as fb  # noqa: E402

HIDDEN, VOCAB, TOP = 512, 2048, 32
BONUS = 0.01


def setup(tokens, seed=0):
    """Hidden states, an output matrix, sampled tokens (a third of the rows prompt or
    padding), advantages, and a student's hidden states and matrix."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    H, W = rand(tokens, HIDDEN), rand(VOCAB, HIDDEN, scale=2.0 / HIDDEN ** 0.5)
    Wq, Ws = fb.fp8rl_quant_weight_block(W)
    logits = fb.fp8rl_linear_w8a8_block(H, Wq, Ws).float()
    rollout = torch.log_softmax(logits, dim=1)
    noise = torch.empty((tokens, VOCAB), device="cuda").exponential_(generator=g)
    sampled = (rollout.exp() / noise).argmax(dim=1)
    logp_rollout = rollout.gather(1, sampled[:, None])[:, 0].contiguous()
    counted = torch.rand(tokens, generator=g, device="cuda") < 2 / 3
    counted[0] = True
    targets = torch.where(counted, sampled, -1).to(torch.int32)
    H[~counted] = float("nan")                              # whatever padding holds
    return dict(H=H, W=W, targets=targets, logp_rollout=logp_rollout, counted=counted,
                advantage=torch.randn(tokens, generator=g, device="cuda"),
                student_H=rand(tokens, HIDDEN // 2), student_W=rand(VOCAB, HIDDEN // 2, scale=0.05))


def policy_gradient(s):
    """-> what a step computes: log-probabilities, entropies, importance weights, the
    loss's gradients with respect to them, and dH and dW."""
    logp, lse, entropy = fb.fp8rl_linear_logp(s["H"], s["W"], s["targets"], want_entropy=True)
    weights, stats = fb.fp8rl_rollout_is_weights(logp, s["logp_rollout"], mask=s["counted"].to(torch.uint8))
    n = s["counted"].sum()
    # loss = -(weights * advantage * logp + BONUS * entropy).sum() / n, the weights held
    g_logp = -weights * s["advantage"] / n
    g_entropy = torch.full_like(g_logp, -BONUS) / n
    dH, dW = fb.fp8rl_linear_logp_backward(s["H"], s["W"], s["targets"], lse, g_logp, entropy=entropy,
                                           g_entropy=g_entropy)
    return dict(logp=logp, lse=lse, entropy=entropy, weights=weights, stats=stats, g_logp=g_logp, g_entropy=g_entropy,
                dH=dH, dW=dW)


def distill(s):
    """-> the student's loss a row and its gradients, from the policy's TOP best logits."""
    teacher = s["H"].nan_to_num(0.0) @ s["W"].T
    top, ids = teacher.float().topk(TOP, dim=1)
    ids = torch.where(s["counted"][:, None], ids, -1).to(torch.int32)
    teacher_lse = torch.logsumexp(teacher.float(), dim=1)
    X = s["student_H"] @ s["student_W"].T
    loss, lse, rest = fb.fp8rl_distill_topk(X, ids, top.contiguous(), teacher_lse=teacher_lse, rest=True)
    g = s["counted"].float() / s["counted"].sum()
    dX = fb.fp8rl_distill_topk_backward(X, ids, top.contiguous(), lse, g, teacher_lse=teacher_lse, rest_lse=rest)
    return dict(X=X, ids=ids, top=top, teacher_lse=teacher_lse, loss=loss, g=g, dX=dX,
                dH=dX @ s["student_W"], dW=dX.T @ s["student_H"])


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args()
    s = setup(a.tokens)
    for i in range(a.steps):
        p, d = policy_gradient(s), distill(s)
        n = s["counted"].sum().item()
        objective = (p["weights"] * s["advantage"]).sum().item() / n
        print(f"step {i}: weighted advantage {objective:+.4f}, entropy {p['entropy'].sum().item() / n:.4f}, mean weight "
              f"{p['stats'][2].item() / n:.4f}, student's divergence {(d['loss'] * d['g']).sum().item():.4f}")
        s["W"] -= 0.05 * p["dW"]
        s["student_W"] -= 0.5 * d["dW"]
    assert fb.fp8rl_check_device_error() == 0


if __name__ == "__main__":
    main()
