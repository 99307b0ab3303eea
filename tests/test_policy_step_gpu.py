"""The trainer's step of examples/policy_step.py: log-probabilities, importance weights,
policy gradient and distillation together, against 64 bits and autograd."""
import importlib.util
import os

import pytest
import torch

import losses_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("policy_step", os.path.join(ROOT, "examples", "policy_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens", [1, 100, 700])
def test_policy_gradient(cuda_lib, example, tokens):
    s = example.setup(tokens, seed=tokens)
    p = example.policy_gradient(s)
    want = ref.linear_logp(s["H"], s["W"], s["targets"])
    for name, w in zip(("logp", "lse", "entropy"), want):
        ref.check(p[name], w, name)
    # the weights from the 64-bit log-probabilities: exp of a difference off by the bound of logp
    # and a rounding; truncated at 2
    d = want[0][0] - s["logp_rollout"].double()
    weights = torch.where(s["counted"], torch.exp(d.clamp(max=0.6931472)), 0.0)
    off = weights * (want[0][1] * 1.01 + d.abs() * 2.0 ** -22 + 2.0 ** -20)
    assert ((p["weights"].double() - weights).abs() <= off).all()
    assert p["stats"][0].item() == s["counted"].sum().item()
    # the step's gradient by autograd in 64 bits, given the weights
    rows = s["counted"].nonzero()[:, 0]
    h = s["H"][rows].double().requires_grad_()
    w = s["W"].double().requires_grad_()
    full = torch.log_softmax(h @ w.T, dim=1)
    logp = full.gather(1, s["targets"][rows].long()[:, None])[:, 0]
    entropy = -(full.exp() * full).sum(1)
    n = len(rows)
    loss = -((p["weights"][rows].double() * s["advantage"][rows].double() * logp) + example.BONUS * entropy).sum() / n
    loss.backward()
    bounds = ref.linear_logp_grad(s["H"], s["W"], s["targets"], p["g_logp"], p["g_entropy"])
    whole = torch.zeros((tokens, h.shape[1]), dtype=torch.float64, device="cuda").index_copy_(0, rows, h.grad)
    for got, value, (_, bound), what in ((p["dH"], whole, bounds[0], "dH"), (p["dW"], w.grad, bounds[1], "dW")):
        # g in fp32: two roundings of each gradient that goes in
        ref.check(got, (value, bound * (1 + 2.0 ** -6) + value.abs() * 2.0 ** -20 + 1e-12), what)


@pytest.mark.parametrize("tokens", [1, 300])
def test_distillation(cuda_lib, example, tokens):
    s = example.setup(tokens, seed=tokens)
    d = example.distill(s)
    top = d["top"].contiguous()
    ref.check(d["loss"], ref.distill(d["X"], d["ids"], top, d["teacher_lse"], True)[0], "loss")
    ref.check(d["dX"], ref.distill_grad(d["X"], d["ids"], top, d["g"], d["teacher_lse"], True), "dX")
    assert (d["dX"][~s["counted"]] == 0).all()


def test_runs(cuda_lib, example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["policy_step.py", "--tokens", "200", "--steps", "2"])
    example.main()
    assert len(capsys.readouterr().out.strip().splitlines()) == 2
