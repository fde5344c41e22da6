"""The optimizer step with 8-bit moments where the second moment's root, or its quotient with the block's largest, leaves
fp32's normal range: the weight's update reads the moments before their rounding, so it holds also where a block's
codes are all 0 for want of a step that fp32 can hold, where an element is tiny beside its block's largest, and where
the root is so large that its reciprocal is not a normal number.  eps is the least that the call takes, so that it hides
nothing.  Bounds as in the tests of single steps (test_gpu_adamw): the update is 16 roundings of 2^-24 off at most."""

import numpy as np
import pytest
import torch

import test_gpu_adamw as base

pytestmark = pytest.mark.gpu
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1.2e-38, weight_decay=0.05)


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import bit_quantized_fine_qlora_amd as lib
    lib._lib.load()
    return lib


def gradients(kind, n, rng):
    g = rng.uniform(1.0, 2.0, n) * rng.choice([-1.0, 1.0], n)
    if kind == "small blocks":
        return g * 2e-35  # roots of 1e-36 .. 1e-35: no step that fp32 holds
    if kind == "small beside large":
        return np.where(np.arange(n) % 128 == 5, g * 1e8, g * 1e-27)
    if kind == "large":
        return g * 1.6e38  # to 3.2e38: roots past 2^126, fp32 ends at 3.4e38
    # the largest that there are, with zeros between
    return np.sign(g) * np.where(np.arange(n) % 3 == 0, 0.0, float(np.finfo(np.float32).max))


@pytest.mark.parametrize("kind", ["small blocks", "small beside large", "large", "largest"])
def test_updates_at_any_magnitude(Q, kind):
    base.say(f"adamw, {kind}")
    rng = np.random.default_rng(23)
    hyper = HYPER | dict(beta2=0.9999) if kind == "largest" else HYPER  # whose first root rounds past the largest
    t = base.Tensor(Q, 6, 128 * 5 + 17, (8, torch.float32, True))
    step_of = Q.AdamWStep([t.entry()])
    for step in (1, 2, 3):
        t.g.copy_(torch.from_numpy(gradients(kind, t.n, rng).astype(np.float32)))
        want = base.expect(t, step, hyper, 1.0)
        assert np.all(np.abs(want[0]) < 100.0)
        step_of.run(**hyper, step=step)
        torch.cuda.synchronize()
        base.check_step(t, want, f"{kind} step {step}")
