"""Infinite margins of the preference loss: a label whose logit is -infinity
has probability 0, so its sequence's log-probability is -infinity.  The loss
term is then infinite or 0 by its direction and the smoothing; a term with the
factor 0 counts as 0, and the coefficients are finite throughout."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def softplus(z):
    return np.maximum(z, 0.0) + np.log1p(np.exp(-np.abs(z)))


@pytest.mark.parametrize("V", [50, 9000])
@pytest.mark.parametrize("smoothing", [0.0, 0.1, 1.0])
@pytest.mark.parametrize("loser", [0, 1])
@pytest.mark.parametrize("pairs", [1, 2])
def test_infinite_margin(V, smoothing, loser, pairs):
    """The sequence `loser` of the first pair is impossible: z = -inf for the preferred one, +inf for the other."""
    import bit_quantized_fine_qlora_amd as Q
    print(f"[case] infinite margin V {V} e {smoothing} loser {loser} pairs {pairs}", flush=True)
    lens, beta = [3, 2, 4, 4][:2 * pairs], 0.5
    T = sum(lens)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(V)
    logits = torch.randn((T, V), generator=gen, device="cuda")
    labels = torch.randint(0, V, (T,), generator=gen, device="cuda")
    cut = np.concatenate([[0], np.cumsum(lens)])
    offsets = torch.from_numpy(cut.astype(np.int32)).cuda()
    t = int(cut[loser]) + 1
    logits[t, labels[t]] = float("-inf")
    r = Q.preference_fwd(logits, labels, offsets, beta=beta, label_smoothing=smoothing)
    grad = Q.preference_bwd(logits, labels, r)
    e = float(np.float32(smoothing))
    # weight of the infinite logarithm, and the limit of e sigma(z) - (1 - e) sigma(-z)
    weight, slope = (1 - e, -(1 - e)) if loser == 0 else (e, e)
    want = np.inf if weight else 0.0
    if pairs == 2:
        z = beta * (r.logps[2].double() - r.logps[3].double()).item()
        want += (1 - e) * softplus(-z) + e * softplus(z)
    assert r.logps[loser].item() == float("-inf") and bool(torch.isfinite(r.logps[1 - loser]))
    if np.isinf(want):
        assert r.loss.item() == want
    else:
        assert abs(r.loss.item() - want / pairs) <= 1e-6 * max(1.0, want)
    first = r.coef[:lens[0] + lens[1]].cpu().numpy()
    sign = np.repeat([1.0, -1.0], lens[:2])
    assert np.all(np.abs(first - sign * beta / pairs * slope) <= 2.0 ** -22)
    assert bool(torch.isfinite(grad).all())
