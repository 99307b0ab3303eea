"""The example's rollout step: its attention within bf16 rounding of 64 bits, its
verification exactly the definition's, and the same step over a bf16 cache near the
one over an 8-bit cache."""
import importlib.util
import os

import numpy as np
import pytest

import rollout_ops_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("rollout_step", os.path.join(ROOT, "examples", "rollout_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("sequences,drafts", [(1, 1), (8, 3), (5, 7)])
def test_step(cuda_lib, example, sequences, drafts, e4m3):
    r = example.step(sequences, drafts, e4m3, seed=sequences)
    want = example.exact_attention(r)
    # the output and each probability are rounded to at most 2^-8 of themselves
    assert ((r["o"].double() - want).norm() / want.norm()).item() <= 2.0 ** -7
    out, kept = ref.verify(r["P"].cpu().numpy(), r["Q"].cpu().numpy(), r["draft"].cpu().numpy(),
                           np.full(sequences, drafts), r["u"].cpu().numpy(), r["noise"].cpu().numpy())
    assert np.array_equal(out, r["out"].cpu().numpy()) and np.array_equal(kept, r["kept"].cpu().numpy())
