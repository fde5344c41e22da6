"""The experts' and the 8-bit moments' oracle against torch in float64, central differences and direct search."""

import numpy as np
import pytest
import torch

from oracle import experts_oracle as X


def random_layer(rng, E=4, M=19, n=6, m=5, r=3):
    f = rng.standard_normal
    return f((M, n)), f((M, m)), f((E, m, n)), f((E, r, n)), f((E, m, r))


@pytest.mark.parametrize("offsets", [[0, 4, 4, 11, 19], [2, 2, 7, 7, 15], [0, 0, 0, 0, 0], [-3, 5, 2, 40, 1]])
def test_experts_against_autograd(offsets):
    rng = np.random.default_rng(3)
    x, g, W, A, B = random_layer(rng)
    s = 0.7
    h, u, rows = X.experts_fwd(x, offsets, W, A, B, s)
    tx, tA, tB = (torch.tensor(t, requires_grad=True) for t in (x, A, B))
    spans = X.expert_rows(offsets, x.shape[0])
    loss = torch.zeros((), dtype=torch.float64)
    for e, (a, b) in enumerate(spans):
        out = tx[a:b] @ torch.tensor(W[e]).t() + s * (tx[a:b] @ tA[e].t()) @ tB[e].t()
        assert np.allclose(out.detach().numpy(), h[a:b], rtol=1e-12, atol=1e-12)
        loss = loss + (out * torch.tensor(g[a:b])).sum()
    assert rows.sum() == sum(b - a for a, b in spans)
    gx, gA, gB = X.experts_bwd(x, g, offsets, W, A, B, s, u)
    if rows.any():
        loss.backward()
        for t, want in ((tx, gx), (tA, gA), (tB, gB)):
            assert np.allclose(t.grad.numpy(), want, rtol=1e-11, atol=1e-12)
    else:
        assert not gx.any() and not gA.any() and not gB.any()


def test_experts_against_differences():
    rng = np.random.default_rng(5)
    x, g, W, A, B = random_layer(rng)
    offsets, s, d = [0, 7, 7, 12, 18], 1.3, 1e-6
    h, u, _ = X.experts_fwd(x, offsets, W, A, B, s)
    grads = X.experts_bwd(x, g, offsets, W, A, B, s, u)
    for which, t in enumerate((x, A, B)):
        for _ in range(12):
            at = tuple(rng.integers(0, k) for k in t.shape)
            keep, ends = t[at], []
            for sign in (1, -1):
                t[at] = keep + sign * d
                ends.append((X.experts_fwd(x, offsets, W, A, B, s)[0] * g).sum())
            t[at] = keep
            assert abs((ends[0] - ends[1]) / (2 * d) - grads[which][at]) < 1e-6


def test_expert_rows_are_disjoint_whatever_the_offsets():
    rng = np.random.default_rng(1)
    for _ in range(300):
        M = int(rng.integers(1, 50))
        spans = X.expert_rows(rng.integers(-60, 100, size=int(rng.integers(2, 20))), M)
        assert all(0 <= a <= b <= M for a, b in spans)
        assert all(p[1] == q[0] for p, q in zip(spans, spans[1:]))


@pytest.mark.parametrize("signed", [True, False])
def test_moment8(signed):
    rng = np.random.default_rng(7)
    x = rng.standard_normal(1000) * 10.0 ** rng.uniform(-6, 2, 1000)
    if not signed:
        x = x * x
    x[::17] = 0.0
    x[128:256] = 0.0
    x[256:384] *= 1e-45 if signed else 1e-90
    codes, steps = X.moment8_pack(x, signed)
    got = X.moment8_values(codes, steps, signed)
    assert np.array_equal(got == 0, codes == 0) and np.all(got[x == 0] == 0)
    assert np.all(np.sign(got) * np.sign(x) >= 0)
    assert steps[1] == 0 and steps[2] == 0 and not codes[128:384].any()
    # half the distance between neighbouring codes: (2 k + 1) / 2 steps of the value, or of its root
    most = 127 if signed else 255
    k = (codes & 127 if signed else codes).astype(np.float64)
    d = np.repeat(steps.astype(np.float64), 128)[:1000]
    off = np.abs(got - x) if signed else np.abs(np.sqrt(got) - np.sqrt(x))
    near = off <= (k + 0.5) * d * (1 + 1e-6)
    if not signed:
        near |= (codes == 1) & (x > 0)  # no value but 0 takes code 0
        assert np.all((codes > 0) == ((x > 0) & (d > 0)))
    assert np.all(near[d > 0])
    for b in (0, 3, 4, 5, 6, 7):
        assert k[128 * b:128 * (b + 1)].max() == most


def test_grad_clip():
    norm, factor = X.grad_clip([np.array([3.0]), np.array([4.0, 0.0])], 1.0)
    assert norm == 5.0 and abs(factor - 1.0 / (5.0 + 1e-6)) < 1e-15
    assert X.grad_clip([np.array([0.1])], 1.0)[1] == 1.0 and X.grad_clip([np.array([0.0])], 1.0) == (0.0, 1.0)
    assert np.isnan(X.grad_clip([np.array([np.inf])], 1.0)[1]) and np.isnan(X.grad_clip([np.array([np.nan])], 1.0)[1])


def test_adamw_against_torch():
    rng = np.random.default_rng(2)
    p = rng.standard_normal(50)
    t = torch.tensor(p, requires_grad=True)
    opt = torch.optim.AdamW([t], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    m, v = np.zeros(50), np.zeros(50)
    for step in range(1, 5):
        g = rng.standard_normal(50)
        t.grad = torch.tensor(g * 0.25)
        opt.step()
        p, m, v = X.adamw_step(p, g, m, v, step, 1e-2, 0.8, 0.95, 1e-6, 0.1, factor=0.25)
        assert np.allclose(p, t.detach().numpy(), rtol=1e-12, atol=1e-14)
