"""The optimizer step's drawn codes of 8-bit second moments (qlora_adamw_step_ex): every code is the one that the oracle
draws, for the same seed, step and place in the plan; a running average kept in them follows the exact one over
thousands of steps; and what a seed leaves alone.

Bounds as in the tests of single steps (test_gpu_adamw) and of the oracle's draws (test_oracle_moment_draws): codes are
equal (a draw would have to fall within 1e-15 of a border to differ) but next to a code: the lower code comes from an
fp32 root that is 8 roundings of 2^-24 off and its own root, two more, so within 12 2^-24 k^2 of k^2 it may be one off,
which is 6 2^-24 k, at most 1e-4, of the way from one code to the other; there v takes the code that it is next to.  An
average is off by five times the root of the summed bounds of its draws' variances, and by 1e-3.
"""

import ctypes

import numpy as np
import pytest
import torch

import test_gpu_adamw as base
from oracle import experts_oracle as X

pytestmark = pytest.mark.gpu
HYPER = base.HYPER


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import bit_quantized_fine_qlora_amd as lib
    lib._lib.load()
    return lib


def chunks(n):
    return -(-n // 2048)


def check_drawn(moment, exact, words):
    codes, steps = X.moment8_pack_drawn(exact, words)
    assert np.array_equal(moment.steps.cpu().numpy(), steps)
    got, d = moment.codes.cpu().numpy().astype(int), np.repeat(steps.astype(np.float64), 128)[:exact.size]
    off = got != codes
    for i in np.flatnonzero(off):
        a = (got[i] ** 2 * d[i]) ** 2
        way = ((got[i] + 1) ** 2 * d[i]) ** 2 - a if exact[i] > a else a - ((got[i] - 1) ** 2 * d[i]) ** 2
        assert abs(exact[i] - a) <= 1e-4 * way, (got[i], codes[i])
    assert off.sum() <= 2


@pytest.mark.parametrize("seed,step", [(0, 1), (2 ** 64 - 3, 2), (-7, 1000), (123456789012345, 2 ** 31 + 5)])
def test_codes_are_the_oracles(Q, seed, step):
    base.say(f"drawn codes, seed {seed} step {step}")
    kinds = base.KINDS
    sizes = [1, 3, 4, 7, 8, 127, 129, 2047, 2048, 2049, 5000, 70001]
    ts = [base.Tensor(Q, 10 * i, n, kinds[i % 4]) for i, n in enumerate(sizes)]
    ts += [base.Tensor(Q, 10 * i + 1, n, kinds[(i + 2) % 4]) for i, n in enumerate(sizes)]
    step_of = Q.AdamWStep([t.entry() for t in ts])
    for at in (step, step + 1):
        for i, t in enumerate(ts):
            t.gradient(100 * i + at % 97, 10.0 ** (-3 + i % 3))
        c = step_of.clip(0.5)
        torch.cuda.synchronize()
        want = [base.expect(t, at, HYPER, float(c[1].item())) for t in ts]
        step_of.run(**HYPER, step=at, clip=c, seed=seed)
        torch.cuda.synchronize()
        first = 0
        for t, w in zip(ts, want):
            if t.eight:
                base.check_moment8(t.m, w[1], "exp_avg")
                check_drawn(t.v, w[2], X.moment8_draws(seed & (2 ** 64 - 1), at, first, t.n))
            else:
                assert np.all(np.abs(base.host(t.v) - w[2]) <= w[5])
            assert np.all(np.abs(base.host(t.p) - w[0]) <= w[3])
            first += chunks(t.n)


def test_magnitudes(Q):
    """Gradients from 1e-30 to 1e10 in one block, blocks of zeros and of values that no step holds."""
    base.say("drawn codes, magnitudes")
    rng = np.random.default_rng(3)
    n = 128 * 6
    t = base.Tensor(Q, 5, n, (8, torch.float32, True))
    g = rng.standard_normal(n) * 10.0 ** rng.uniform(-30, 10, n)
    g[128:256] = 0.0
    g[256:384] *= 1e-20
    g[384:512] = np.float32(3e-45)
    step_of = Q.AdamWStep([t.entry()])
    for step in (1, 2, 3):
        t.g.copy_(torch.from_numpy(g.astype(np.float32)))
        want = base.expect(t, step, HYPER, 1.0)
        step_of.run(**HYPER, step=step, seed=11)
        torch.cuda.synchronize()
        check_drawn(t.v, want[2], X.moment8_draws(11, step, 0, n))
        assert np.all(np.abs(base.host(t.p) - want[0]) <= want[3])
        g = -g * 0.5


@pytest.mark.parametrize("change", [1.0, 0.2, 2.0])
def test_the_average_follows(Q, change):
    """Gradients of every other element change by a factor after 1500 of 5500 steps."""
    base.say(f"drawn codes over 5500 steps, change {change}")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    n, b2 = 128 * 48, 0.999
    m, v = Q.alloc_moment8(n, True), Q.alloc_moment8(n, False)
    g = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    step_of = Q.AdamWStep([(torch.zeros(n, device="cuda"), None, g, m, v)])
    odd = torch.arange(n, device="cuda") % 2 == 1
    after = torch.where(odd, change, 1.0)
    exact, var = (torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2))
    for step in range(1, 5501):
        x = torch.randn(n, generator=gen, device="cuda")
        g.copy_(x if step <= 1500 else x * after)
        step_of.run(1e-4, 0.9, b2, 1e-8, 0.0, step, seed=77)
        exact.mul_(b2).add_(g.double().square_(), alpha=1 - b2)
        if step % 10 == 0:  # of ten steps' variances the last, which changes by less than a tenth over them
            k, d = v.codes.double(), v.steps.double().repeat_interleave(128)
            apart = ((k + 1).square() * d).square() - ((k - 1).clamp_min(0).square() * d).square()
            var.mul_(b2 ** 20).add_(apart.square_(), alpha=1.1 * 10 / 4)
    kept = Q.moment8_values(v).double()
    for part in (odd, ~odd):
        off = (kept - exact)[part].sum().abs().item()
        assert off <= 5 * var[part].sum().sqrt().item() + 1e-3 * exact[part].sum().item()
        ratio = (kept / exact)[part].sqrt()
        print(f"[case] root kept / exact: median {ratio.median().item():.3f}", flush=True)


def state_after(Q, seeds, kinds=None, seed_of_gradients=1):
    ts = [base.Tensor(Q, 30 + i, n, (kinds or base.KINDS)[i % 4]) for i, n in enumerate((3000, 129, 70001, 17))]
    plan = Q.AdamWStep([t.entry() for t in ts])
    for step, seed in enumerate(seeds, 1):
        for i, t in enumerate(ts):
            t.gradient(500 * seed_of_gradients + 10 * step + i, 0.1)
        plan.run(**HYPER, step=step, seed=seed)
    torch.cuda.synchronize()
    return ts


def test_what_a_seed_changes(Q):
    base.say("drawn codes, seeds")
    a, b = state_after(Q, (3, 4)), state_after(Q, (3, 4))
    for s, t in zip(a, b):  # run to run
        assert all(torch.equal(x, y) for x, y in zip(s.raw(), t.raw()))
    c, none = state_after(Q, (3, 5)), state_after(Q, (None, None))
    assert not torch.equal(a[0].v.codes, c[0].v.codes) and not torch.equal(a[0].v.codes, none[0].v.codes)
    one, other = state_after(Q, (3,)), state_after(Q, (None,))
    for s, t in zip(one, other):  # one step: everything but the codes of the second moments
        for x, y in zip(s.raw(), t.raw()):
            same = torch.equal(x, y)
            assert same or (s.eight and x is s.v.codes)
    for s, t in zip(a, none):
        if not s.eight:
            assert all(torch.equal(x, y) for x, y in zip(s.raw(), t.raw()))


def test_a_call_without_a_seed_is_the_plain_step(Q):
    """qlora_adamw_step, and qlora_adamw_step_ex with NULL."""
    base.say("step and step_ex")
    lib = Q._lib.load()
    want = state_after(Q, (None,))
    ts = [base.Tensor(Q, 30 + i, n, base.KINDS[i % 4]) for i, n in enumerate((3000, 129, 70001, 17))]
    plan = Q.AdamWStep([t.entry() for t in ts])
    for i, t in enumerate(ts):
        t.gradient(510 + i, 0.1)
    h = HYPER
    torch.cuda.synchronize()
    assert lib.qlora_adamw_step(ctypes.byref(plan._handle), h["lr"], h["beta1"], h["beta2"], h["eps"],
                                h["weight_decay"], 1, None, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    for s, t in zip(want, ts):
        assert all(torch.equal(x, y) for x, y in zip(s.raw(), t.raw()))


def test_no_step_without_a_finite_norm(Q):
    base.say("drawn codes, gradients that are not finite")
    ts = state_after(Q, (3,))
    ts[0].g[5] = float("nan")
    plan = Q.AdamWStep([t.entry() for t in ts])
    before = [t.state() for t in ts]
    plan.run(**HYPER, step=2, clip=plan.clip(1.0), seed=4)
    torch.cuda.synchronize()
    for t, old in zip(ts, before):
        assert all(torch.equal(x, y) for x, y in zip(t.raw(), old))


def test_graph(Q):
    """A captured step replays its seed and number: each replay is the eager step with these."""
    base.say("drawn codes, graph")
    make = lambda: [base.Tensor(Q, 50 + i, n, base.KINDS[i % 4]) for i, n in enumerate((3000, 129, 70001, 17))]
    a, b = make(), make()
    plan_a, plan_b = Q.AdamWStep([t.entry() for t in a]), Q.AdamWStep([t.entry() for t in b])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan_b.run(**HYPER, step=9, seed=21)
    for replay in range(4):
        for i, (s, t) in enumerate(zip(a, b)):
            s.gradient(900 + 10 * replay + i, 0.1)
            t.g.copy_(s.g)
        torch.cuda.synchronize()
        graph.replay()
        plan_a.run(**HYPER, step=9, seed=21)
        torch.cuda.synchronize()
        for s, t in zip(a, b):
            assert all(torch.equal(x, y) for x, y in zip(s.raw(), t.raw()))
