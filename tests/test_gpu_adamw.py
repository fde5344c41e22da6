"""GPU parity of the optimizer step over many tensors (qlora_adamw_step), the gradients' norm (qlora_grad_clip) and
moments in 8 bits, against the float64 oracle, one step at a time from the kernel's own state.

Bounds.  With eps = 2^-24 (half a step of fp32): an 8-bit moment is formed in 64 bits, so a code is wrong only where
another code is nearer by more than rounding of 64-bit numbers (1e-13 here).  A weight: p (1 - lr wd) - U is off by
3 eps |p| (the constant, the product, the difference) and U = step_size m / denom by 16 eps |U|: the constants,
conversions, products and the sum in the denominator are eps each (8 of them), its root and reciprocal, which are the
card's own approximations within one unit, 2 eps each.  32-bit moments: constant, product and sum, 4 eps of their terms
(5 for the square), and what that changes in U.
"""

import numpy as np
import pytest
import torch

import qlora_inputs as QI
from oracle import experts_oracle as X
from oracle import qlora_oracle as O
from parity_utils import f64, host_bits

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import bit_quantized_fine_qlora_amd as lib
    lib._lib.load()
    return lib


def say(msg):
    print(f"[case] {msg}", flush=True)


def host(t):
    return f64(host_bits(t)) if t.dtype == torch.bfloat16 else t.cpu().numpy()


class Tensor:
    """One trained tensor; kind: (8 or 32, gradient type, bf16 copy or not)."""

    def __init__(self, Q, seed, n, kind, pinned=False):
        self.eight, gtype, copy = kind[0] == 8, kind[1], kind[2]
        kw = dict(device="cpu", pin_memory=True) if pinned else dict(device="cuda")

        def put(a):
            t = torch.empty(a.shape, dtype=torch.from_numpy(a).dtype, **kw)
            return t.copy_(torch.from_numpy(a))

        self.n = n
        self.p = put(QI.normal_f32(seed, (n,), 0.05))
        self.p16 = torch.empty(n, dtype=torch.bfloat16, device="cuda") if copy else None
        self.g = torch.empty(n, dtype=gtype, device="cuda")
        if self.eight:
            self.m, self.v = (Q.alloc_moment8(n, signed, **kw) for signed in (True, False))
        else:
            self.m, self.v = put(np.zeros(n, np.float32)), put(np.zeros(n, np.float32))

    def gradient(self, seed, scale):
        g = QI.normal_f32(seed, (self.n,), scale) * np.exp(QI.normal_f32(seed + 7, (self.n,), 1.0))
        g[::13] = 0.0
        self.g.copy_(torch.from_numpy(g))

    def entry(self):
        return self.p, self.p16, self.g, self.m, self.v

    def moments(self):
        """Both moments as float64 values."""
        if not self.eight:
            return [host(t).astype(np.float64) for t in (self.m, self.v)]
        return [X.moment8_values(host(t.codes), host(t.steps), t.signed) for t in (self.m, self.v)]

    def raw(self):
        out = [self.p] + ([self.p16] if self.p16 is not None else [])
        return out + ([self.m.codes, self.m.steps, self.v.codes, self.v.steps] if self.eight else [self.m, self.v])

    def state(self):
        return [t.clone() for t in self.raw()]


def check_moment8(moment, exact, what):
    """Steps are the roundings of the exact largest, codes the nearest."""
    n = exact.size
    codes, steps = host(moment.codes).astype(np.int64), host(moment.steps).astype(np.float64)
    most = 127 if moment.signed else 255
    x = np.abs(exact) if moment.signed else np.sqrt(exact)
    pad = np.concatenate([x, np.zeros(-n % 128)]).reshape(-1, 128)
    top = pad.max(axis=1) / most ** 2
    lo, hi = (np.float32(top * (1 + d)).astype(np.float64) for d in (-1e-13, 1e-13))
    tiny = 2.0 ** -126
    assert np.all(((steps >= lo) & (steps <= hi)) | ((steps == 0) & (lo < tiny))), f"{what}: steps"
    d = np.repeat(steps, 128)[:n]
    k = (codes & 127 if moment.signed else codes).astype(np.float64)
    off = np.abs(k * k * d - x)
    slack = 1e-13 * x
    up = np.where(k < most, np.abs((k + 1) ** 2 * d - x), np.inf)
    down = np.where(k > 0, np.abs((k - 1) ** 2 * d - x), np.inf)
    held = np.zeros(n, bool) if moment.signed else (k == 1) & (x > 0)  # not below 1
    ok = (off <= up + slack) & ((off < down + slack) | held)
    assert np.all(ok | (d == 0)), f"{what}: {int((~ok & (d > 0)).sum())} codes are not the nearest"
    assert not codes[d == 0].any(), f"{what}: codes of an empty block"
    if moment.signed:
        assert np.all((codes >> 7).astype(bool) == ((exact < 0) & (k > 0))), f"{what}: signs"
    else:
        assert np.all((codes > 0) == ((x > 0) & (d > 0))), f"{what}: zeros"


HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.05)


def expect(t, step, hp, factor):
    """The exact step from the tensor's present state: (p, m, v, tolerances of p, m, v)."""
    p, g = host(t.p).astype(np.float64), host(t.g).astype(np.float64)
    m0, v0 = t.moments()
    p1, m1, v1 = X.adamw_step(p, g, m0, v0, step, hp["lr"], hp["beta1"], hp["beta2"], hp["eps"], hp["weight_decay"],
                              factor)
    size = hp["lr"] / (1 - hp["beta1"] ** step)
    denom = np.sqrt(v1 / (1 - hp["beta2"] ** step)) + hp["eps"]
    U = size * np.abs(m1) / denom
    tol_p = 3 * EPS * np.abs(p) + 16 * EPS * U + EPS * np.abs(p1)
    tol_m = tol_v = None
    if not t.eight:
        tol_m = 4 * EPS * (hp["beta1"] * np.abs(m0) + (1 - hp["beta1"]) * np.abs(g * factor)) + 1e-44
        tol_v = 5 * EPS * v1 + 1e-44
        tol_p = tol_p + size * tol_m / denom
    return p1, m1, v1, tol_p, tol_m, tol_v


def check_step(t, want, what):
    p1, m1, v1, tol_p, tol_m, tol_v = want
    if t.eight:
        check_moment8(t.m, m1, what + " exp_avg")
        check_moment8(t.v, v1, what + " exp_avg_sq")
    else:
        assert np.all(np.abs(host(t.m) - m1) <= tol_m), what + " exp_avg"
        assert np.all(np.abs(host(t.v) - v1) <= tol_v), what + " exp_avg_sq"
    assert np.all(np.abs(host(t.p) - p1) <= tol_p), what + " param"
    if t.p16 is not None:
        assert np.array_equal(host_bits(t.p16), O.bf16_bits_rne(t.p.cpu().numpy())), what + " bf16 copy"


def train(Q, tensors, steps, clip=None, hp=HYPER, seed=1):
    step_of = Q.AdamWStep([t.entry() for t in tensors])
    for step in range(1, steps + 1):
        for i, t in enumerate(tensors):
            t.gradient(1000 * seed + 37 * i + step, 10.0 ** (-3 + i % 3))
        factor, c = 1.0, None
        if clip is not None:
            c = step_of.clip(clip)
            norm, f = X.grad_clip([host(t.g) for t in tensors], clip)
            torch.cuda.synchronize()
            assert abs(c[0].item() - norm) <= 2.0 ** -23 * norm
            assert abs(c[1].item() - f) <= 2.0 ** -23 * f
            factor = float(c[1].item())
        want = [expect(t, step, hp, factor) for t in tensors]
        step_of.run(**hp, step=step, clip=c)
        torch.cuda.synchronize()
        for i, (t, w) in enumerate(zip(tensors, want)):
            check_step(t, w, f"step {step} tensor {i} ({t.n})")


KINDS = [(8, torch.bfloat16, True), (8, torch.float32, False), (32, torch.bfloat16, False), (32, torch.float32, True)]


@pytest.mark.parametrize("kind", range(4))
@pytest.mark.parametrize("clip", [None, 0.5])
def test_sizes(Q, kind, clip):
    """One element, less than a piece, a piece, blocks and chunks and one off them."""
    say(f"adamw sizes, kind {kind}, clip {clip}")
    sizes = [1, 7, 8, 9, 127, 128, 129, 130, 2047, 2048, 2049, 4096, 5000, 70001]
    train(Q, [Tensor(Q, 10 * i + kind, n, KINDS[kind]) for i, n in enumerate(sizes)], 3, clip)


def test_mixed_kinds_in_one_launch(Q):
    say("adamw, 130 tensors of all kinds")
    train(Q, [Tensor(Q, i, 64 * (i % 9) + i, KINDS[i % 4]) for i in range(1, 131)], 2, 1.0)


def test_many_chunks(Q):
    """More chunks than the norm's workgroups."""
    say("adamw, 5 million elements")
    train(Q, [Tensor(Q, 3, 4_500_003, KINDS[0]), Tensor(Q, 4, 500_001, KINDS[3])], 1, 0.3)


def test_moments_over_many_orders(Q):
    """Gradients from 1e-30 to 1e10 in one block, zeros, and blocks that are all zero or below what a step can hold."""
    say("adamw, magnitudes")
    n = 128 * 12
    t = Tensor(Q, 5, n, (8, torch.float32, True))
    rng = np.random.default_rng(3)
    g = rng.standard_normal(n) * 10.0 ** rng.uniform(-30, 10, n)
    g[128:256] = 0.0
    g[256:384] *= 1e-20
    g[384:512] = np.float32(3e-45)
    g[512:640] = 1.0
    g[640:768] = np.where(np.arange(128) == 5, 1e18, 1e-18)
    step_of = Q.AdamWStep([t.entry()])
    for step in (1, 2, 3):
        t.g.copy_(torch.from_numpy(g.astype(np.float32)))
        want = expect(t, step, HYPER, 1.0)
        step_of.run(**HYPER, step=step)
        torch.cuda.synchronize()
        check_step(t, want, f"magnitudes step {step}")
        g = -g * 0.5


def test_values(Q):
    say("moment8_values")
    for n in (1, 7, 8, 127, 128, 129, 2048, 5001):
        rng = np.random.default_rng(n)
        codes = rng.integers(0, 256, n).astype(np.uint8)
        steps = (10.0 ** rng.uniform(-30, 3, -(-n // 128))).astype(np.float32)
        for signed in (True, False):
            m = Q.Moment8(torch.from_numpy(codes).cuda(), torch.from_numpy(steps).cuda(), signed)
            got = Q.moment8_values(m).cpu().numpy()
            assert np.array_equal(got, X.moment8_values(codes, steps, signed).astype(np.float32))


def test_no_step_without_a_finite_norm(Q):
    say("adamw, gradients that are not finite")
    for bad in (float("inf"), float("-inf"), float("nan")):
        for gtype in (torch.bfloat16, torch.float32):
            ts = [Tensor(Q, i, 300 + i, (kind[0], gtype, True)) for i, kind in enumerate(KINDS)]
            step_of = Q.AdamWStep([t.entry() for t in ts])
            for t in ts:
                t.gradient(t.n, 0.1)
            step_of.run(**HYPER, step=1)
            ts[2].g[299] = bad
            before = [t.state() for t in ts]
            c = step_of.clip(1.0)
            step_of.run(**HYPER, step=2, clip=c)
            torch.cuda.synchronize()
            assert np.isnan(c[1].item()) and not np.isfinite(c[0].item())
            for t, old in zip(ts, before):
                for a, b in zip(t.raw(), old):
                    assert torch.equal(a, b)
    t = Tensor(Q, 1, 100, KINDS[0])
    t.g.zero_()
    c = Q.AdamWStep([t.entry()]).clip(float("inf"))
    assert c.tolist() == [0.0, 1.0]


def test_norm_of_large_and_small_gradients(Q):
    """Squares beyond fp32's range."""
    say("gradient norm, range")
    for scale in (1e30, 1e-30):
        t = Tensor(Q, 1, 1000, (32, torch.float32, False))
        t.g.copy_(torch.from_numpy(QI.normal_f32(2, (1000,), 1.0)) * scale)
        c = Q.AdamWStep([t.entry()]).clip(scale)
        norm, f = X.grad_clip([host(t.g)], scale)
        assert abs(c[0].item() - norm) <= 2.0 ** -23 * norm and abs(c[1].item() - f) <= 2.0 ** -23 * f


def test_same_bits_and_pinned_state(Q):
    """The same bits run to run, in any grouping of the tensors, and with the state in pinned host memory."""
    say("adamw, same bits")
    sizes = [5000, 129, 40000]

    def steps(pinned, together):
        ts = [Tensor(Q, 70 + i, n, KINDS[i % 2], pinned) for i, n in enumerate(sizes)]
        plans = [Q.AdamWStep([t.entry() for t in ts])] if together else [Q.AdamWStep([t.entry()]) for t in ts]
        for step in (1, 2):
            for i, t in enumerate(ts):
                t.gradient(90 + 10 * step + i, 0.01)
            for plan in plans:
                plan.run(**HYPER, step=step)
            torch.cuda.synchronize()
        return [a.cpu() for t in ts for a in t.raw()]

    first = steps(False, True)
    for other in (steps(False, True), steps(False, False), steps(True, True)):
        for a, b in zip(first, other):
            assert torch.equal(a, b)


def test_neighbours_are_left_alone(Q):
    """Tensors that are slices of one storage: nothing between them is written."""
    say("adamw, slices")
    sizes, room = [130, 1, 2047, 9], 17 * 128  # steps from 4-byte aligned places on
    for eight in (True, False):
        flat = {k: torch.full((4 * room,), 3.0, device="cuda") for k in ("p", "m", "v")}
        p16 = torch.full((4 * room,), 3.0, device="cuda", dtype=torch.bfloat16)
        codes = [torch.full((4 * room,), 77, dtype=torch.uint8, device="cuda") for _ in range(2)]
        step8 = [torch.full((4 * room // 128,), 1e-9, device="cuda") for _ in range(2)]
        g = torch.full((4 * room,), float("nan"), device="cuda")
        entries, inside = [], torch.zeros(4 * room, dtype=torch.bool, device="cuda")
        blocks = torch.zeros(4 * room // 128, dtype=torch.bool, device="cuda")
        for i, n in enumerate(sizes):
            at = slice(i * room, i * room + n)
            inside[at] = True
            g[at] = 0.5
            b = slice(i * room // 128, i * room // 128 + -(-n // 128))
            blocks[b] = True
            mv = [Q.Moment8(c[at], s[b], signed) for c, s, signed in zip(codes, step8, (True, False))] if eight else \
                [flat["m"][at], flat["v"][at]]
            entries.append((flat["p"][at], p16[at], g[at], *mv))
        Q.AdamWStep(entries).run(**HYPER, step=1)
        torch.cuda.synchronize()
        assert (flat["p"][~inside] == 3.0).all() and (p16[~inside] == 3.0).all() and (flat["p"][inside] != 3.0).all()
        if eight:
            assert all((c[~inside] == 77).all() for c in codes) and all((s[~blocks] == step8[0].new_tensor(1e-9)).all() for s in step8)
            assert all((s[blocks] != step8[0].new_tensor(1e-9)).all() for s in step8)
        else:
            assert (flat["m"][~inside] == 3.0).all() and (flat["v"][~inside] == 3.0).all()


def test_side_stream_and_graph(Q):
    """A captured clip and step: each replay reads the gradients as they are then."""
    say("adamw, graph")

    def make():
        return [Tensor(Q, 50 + i, n, KINDS[i % 4]) for i, n in enumerate((3000, 129, 70001, 17))]

    a, b = make(), make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan_a, plan_b = Q.AdamWStep([t.entry() for t in a]), Q.AdamWStep([t.entry() for t in b])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    out_b = torch.empty(2, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan_b.clip(0.5, out=out_b)
        plan_b.run(**HYPER, step=3, clip=out_b)
    for replay in range(4):
        for i, (s, t) in enumerate(zip(a, b)):
            s.gradient(500 + 10 * replay + i, 0.1)
            t.g.copy_(s.g)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            out_a = plan_a.clip(0.5)
            plan_a.run(**HYPER, step=3, clip=out_a)
        torch.cuda.synchronize()
        assert torch.equal(out_a, out_b)
        for s, t in zip(a, b):
            for x, y in zip(s.raw(), t.raw()):
                assert torch.equal(x, y)


def test_given_tensors_are_checked(Q):
    say("adamw, given tensors")
    f = torch.zeros(256, device="cuda")
    m8, v8 = Q.alloc_moment8(256, True), Q.alloc_moment8(256, False)
    Q.AdamWStep([(f, None, f.clone(), m8, v8)])
    with pytest.raises(ValueError, match="GPU or in pinned"):
        Q.AdamWStep([(f, None, f.clone(), m8, Q.alloc_moment8(256, False, device="cpu"))])
    with pytest.raises(ValueError, match="GPU or in pinned"):
        Q.AdamWStep([(f, None, f.cpu(), m8, v8)])
    with pytest.raises(Q.QloraError):  # not 16-byte aligned
        Q.AdamWStep([(f[1:129], None, f[:128].clone(), f[:128].clone(), f[:128].clone())])
    with pytest.raises(Q.QloraError):
        Q.AdamWStep([(f[:0], None, f[:0], f[:0], f[:0])])
    g, h = f.clone(), torch.zeros(256, device="cuda")
    new = lambda: [Q.alloc_moment8(256, True), Q.alloc_moment8(256, False)]
    Q.AdamWStep([(f, None, g, *new()), (h, None, g, *new())])  # a gradient that two tensors read
    for other in ((f, None, g.clone(), *new()), (h, None, g.clone(), m8, new()[1]), (h, None, f, *new()),
                  (h, g[128:].view(torch.bfloat16), h.clone(), *new()), (h, None, h, *new())):
        for pair in ([(f, None, g, m8, v8), other], [other, (f, None, g, m8, v8)]):
            with pytest.raises(ValueError, match="share"):
                Q.AdamWStep(pair)
    step_of = Q.AdamWStep([(f, None, f.clone(), m8, v8)])
    with pytest.raises(ValueError):
        step_of.run(1e-3, clip=torch.ones(2))
    with pytest.raises(ValueError):
        step_of.run(1e-3, clip=torch.ones(3, device="cuda"))
    with pytest.raises(ValueError):
        step_of.clip(1.0, out=torch.ones(2))
    with pytest.raises(Q.QloraError):
        step_of.clip(0.0)
    with pytest.raises(Q.QloraError):
        step_of.run(1e-3, eps=0.0)
    with pytest.raises(ValueError):
        Q.moment8_values(Q.Moment8(m8.codes.cpu(), m8.steps.cpu(), True))
