"""GPU parity of the experts' layer (qlora_experts_fwd, qlora_experts_bwd) against the float64 oracle.

Tolerances are bounds of the arithmetic.  With eps = 2^-24 (half a step of
fp32), a product of K terms summed in fp32 in any order is off by at most
K eps sum |terms|; operands that enter as two bf16 parts (u, v, s u, s v) keep
all but 2^-18 of themselves (2^-9 of a 2^-9 part), taken as 2^-17 with the
rounding of the product by s.  The bf16 outputs are compared with the roundings
of both ends of the allowed interval (assert_rounds_into).  Every call runs on
a workspace of NaN bytes, so that nothing unwritten is read, and on outputs of
a pattern that rows of no expert must keep.
"""

import numpy as np
import pytest
import torch

import qlora_inputs as QI
from oracle import experts_oracle as X
from oracle import qlora_oracle as O
from parity_utils import dev_bf16, f64, host_bits
from rounding_utils import assert_rounds_into

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
PAIR = 2.0 ** -17
PATTERN = 0x4A4A  # bf16 bits, and twice that as fp32


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import bit_quantized_fine_qlora_amd as lib
    lib._lib.load()
    return lib


def say(msg):
    print(f"[case] {msg}", flush=True)


class Layer:
    """E experts of one shape with M rows: device tensors and their float64 values."""

    def __init__(self, Q, seed, E, M, n, m, r):
        self.E, self.M, self.n, self.m, self.r = E, M, n, m, r
        W = QI.normal_f32(seed * 10 + 1, (E * m, n), 0.02)
        qw = O.quantize_nf4_dq(W)
        self.W = f64(O.dequant_nf4_dq(qw["codes"], qw["absmax8"], qw["c2"], E * m * n)).reshape(E, m, n)
        self.q = Q.QuantizedWeight(*(torch.from_numpy(qw[k]).to("cuda") for k in ("codes", "absmax8", "c2")), E * m, n)
        bits = {k: QI.to_bf16_bits(QI.normal_f32(seed * 10 + i, shape, sigma)) for i, (k, shape, sigma) in enumerate(
            [("x", (M, n), 1.0), ("g", (M, m), 1.0), ("A", (E, r, n), QI.A_SIGMA), ("B", (E, m, r), QI.B_SIGMA)], 2)}
        self.dev = {k: dev_bf16(v) for k, v in bits.items()}
        self.val = {k: f64(v) for k, v in bits.items()}


def offsets_dev(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


def poison(nbytes):
    return torch.full((max(nbytes, 256),), 0xFF, dtype=torch.uint8, device="cuda")


def patterned(shape, dtype=torch.bfloat16):
    bits = torch.full(shape, PATTERN, dtype=torch.int16, device="cuda") if dtype == torch.bfloat16 else \
        torch.full(shape, (PATTERN << 16) | PATTERN, dtype=torch.int32, device="cuda")
    return bits.view(dtype)


def val(t):
    return f64(host_bits(t)) if t.dtype == torch.bfloat16 else t.cpu().numpy().astype(np.float64)


def run(Q, L, offsets, s, need_grad_x=True, give_u=True):
    """(h, u, gx, gA, gB) of one forward and backward, on poisoned workspaces and patterned outputs."""
    off, d = offsets_dev(offsets), L.dev
    size = (L.M, L.E, L.n, L.m, L.r)
    h, u = patterned((L.M, L.m)), patterned((L.M, L.r), torch.float32)
    Q.experts_fwd(d["x"], off, L.q, d["A"], d["B"], s, h=h, u=u, workspace=poison(Q.experts_workspace_bytes(0, *size)))
    gx = patterned((L.M, L.n)) if need_grad_x else None
    out = (gx, patterned((L.E, L.r, L.n)), patterned((L.E, L.m, L.r)))
    got = Q.experts_bwd(d["x"], d["g"], off, L.q, d["A"], d["B"], s, u=u if give_u else None, out=out,
                        workspace=poison(Q.experts_workspace_bytes(1, *size)))
    assert got[0] is gx
    torch.cuda.synchronize()
    return h, u, *out


def check(L, offsets, s, h, u, gx, gA, gB, given_u=True):
    x, g, A, B = (L.val[k] for k in "xgAB")
    h_ref, u_ref, rows = X.experts_fwd(x, offsets, L.W, A, B, s)
    n, m, r, a = L.n, L.m, L.r, abs(s)
    for t in (h, u) + ((gx,) if gx is not None else ()):
        raw = t.view(torch.int16).cpu().numpy()
        assert np.all(raw[~rows] == PATTERN), "a row of no expert was written"
    # u: n terms.  h: n terms, r terms of s u B with u's own error
    abs_u, abs_h = np.zeros_like(u_ref), np.zeros_like(h_ref)
    abs_v, abs_gx = np.zeros_like(u_ref), np.zeros_like(x)
    tA, tB = np.zeros_like(A), np.zeros_like(B)
    got_u = val(u)
    u_bwd = np.where(rows[:, None], got_u if given_u else u_ref, 0.0)
    gx_ref, gA_ref, gB_ref = X.experts_bwd(x, g, offsets, L.W, A, B, s, u_bwd)
    for e, (i, j) in enumerate(X.expert_rows(offsets, L.M)):
        if j == i:
            continue
        ax, ag, aA, aB, aW = np.abs(x[i:j]), np.abs(g[i:j]), np.abs(A[e]), np.abs(B[e]), np.abs(L.W[e])
        abs_u[i:j] = ax @ aA.T
        lora = a * (abs_u[i:j] @ aB.T)
        abs_h[i:j] = (n + 2 * r) * EPS * (ax @ aW.T + lora) + (PAIR + n * EPS) * lora
        abs_v[i:j] = ag @ aB
        lora = a * (abs_v[i:j] @ aA)
        abs_gx[i:j] = (m + 2 * r) * EPS * (ag @ aW + lora) + (PAIR + m * EPS) * lora
        c = 2 * (j - i)  # both parts of each row
        tA[e] = a * (c * EPS + PAIR + m * EPS) * (abs_v[i:j].T @ ax)
        tB[e] = a * (c * EPS + PAIR + (0 if given_u else n * EPS)) * (
            ag.T @ (np.abs(u_bwd[i:j]) if given_u else abs_u[i:j]))
    assert np.all(np.abs(got_u - u_ref)[rows] <= (n * EPS * abs_u)[rows] + 1e-30), "u"
    assert_rounds_into(val(h)[rows], h_ref[rows], abs_h[rows], "h")
    if gx is not None:
        assert_rounds_into(val(gx)[rows], gx_ref[rows], abs_gx[rows], "grad_x")
    assert_rounds_into(val(gA), gA_ref, tA, "grad_A")
    assert_rounds_into(val(gB), gB_ref, tB, "grad_B")


def cuts(E, M, seed, idle=0.3, lead=0, tail=0):
    """Ascending offsets with some experts empty; `lead` and `tail` rows belong to none."""
    rng = np.random.default_rng(seed)
    w = rng.uniform(0.2, 3.0, E) * (rng.random(E) >= idle)
    if not w.any():
        w[-1] = 1.0
    c = np.floor(np.concatenate([[0.0], np.cumsum(w) / w.sum()]) * (M - lead - tail)).astype(int)
    return [int(v) + lead for v in c]


CASES = [  # E, M, n, m, r, offsets (None: drawn)
    (1, 1, 64, 8, 1, [0, 1]),
    (1, 40, 128, 64, 8, [0, 40]),
    (3, 7, 64, 7, 3, [0, 0, 7, 7]),                  # one expert has every row; m odd
    (4, 33, 192, 100, 12, [2, 9, 9, 30, 31]),        # rows before and behind every expert
    (5, 90, 320, 259, 16, None),                     # the weight begins inside a block group
    (6, 203, 320, 259, 20, None),
    (2, 600, 256, 128, 8, [0, 577, 600]),            # three row tiles, chunks that are summed
    (3, 1100, 128, 192, 33, [0, 700, 700, 1090]),
    (4, 300, 1088, 136, 64, None),                   # K pieces
    (3, 130, 192, 1100, 100, [0, 1, 65, 130]),       # K pieces of the backward
    (2, 520, 64, 72, 128, [0, 257, 520]),
    (70, 500, 64, 24, 4, None),                      # more experts than lanes
    (130, 90, 128, 16, 8, None),                     # more experts than rows
    (4, 64, 64, 64, 8, [0, 0, 0, 0, 0]),             # no row at all
    (4, 64, 64, 64, 8, [64, 64, 64, 64, 64]),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_parity(Q, case):
    E, M, n, m, r, offsets = CASES[case]
    say(f"experts E {E} M {M} n {n} m {m} r {r}")
    L = Layer(Q, 300 + case, E, M, n, m, r)
    offsets = cuts(E, M, case, lead=case % 2, tail=case % 3) if offsets is None else offsets
    s = (0.25, -1.5, 2.0)[case % 3]
    check(L, offsets, s, *run(Q, L, offsets, s))


@pytest.mark.parametrize("offsets", [[-7, 20, 45, 60], [0, 50, 20, 60], [10, 5, 1000, 30], [0, -1, -1, 60],
                                     [2 ** 31 - 1, 0, 5, 9], [-2 ** 31, 2 ** 31 - 1, 0, 60]])
def test_offsets_out_of_order_or_range(Q, offsets):
    say(f"experts offsets {offsets}")
    L = Layer(Q, 331, 3, 60, 128, 72, 8)
    check(L, offsets, 0.5, *run(Q, L, offsets, 0.5))


def test_u_recomputed_and_grad_x_skipped(Q):
    say("experts, u recomputed, no grad_x")
    for case, r in enumerate((8, 12, 64)):
        L = Layer(Q, 340 + case, 4, 150, 256, 120, r)
        offsets = cuts(4, 150, 40 + case)
        check(L, offsets, 0.5, *run(Q, L, offsets, 0.5, need_grad_x=case != 1, give_u=False), given_u=False)


def test_same_bits_twice_and_with_other_rows_beside(Q):
    """Results do not depend on the run, nor on the rows of other experts or of none."""
    say("experts, same bits")
    L = Layer(Q, 350, 4, 700, 192, 136, 16)
    offsets = [0, 300, 300, 420, 690]
    first, second = run(Q, L, offsets, 0.5), run(Q, L, offsets, 0.5)
    for a, b in zip(first, second):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    keep = L.dev["x"].clone(), L.dev["g"].clone()
    for t in (L.dev["x"], L.dev["g"]):
        t[:300] = 7.0
        t[690:] = float("nan")  # never read
    other = run(Q, L, offsets, 0.5)
    L.dev["x"], L.dev["g"] = keep
    for a, b in zip(first[:3], other[:3]):
        assert torch.equal(a[300:690], b[300:690])
    for a, b in zip(first[3:], other[3:]):
        assert torch.equal(a[1:], b[1:])


def test_one_expert_is_the_dense_layer(Q):
    say("one expert and linear_fwd, linear_bwd")
    L = Layer(Q, 360, 1, 300, 512, 264, 16)
    d = L.dev
    h, u, gx, gA, gB = run(Q, L, [0, 300], 0.5)
    dh, du = Q.linear_fwd(d["x"], L.q, d["A"][0], d["B"][0], 0.5)
    dgx, dgA, dgB = Q.linear_bwd(d["x"], d["g"], L.q, d["A"][0], d["B"][0], 0.5, u=du)
    for a, b in ((h, dh), (u, du), (gx, dgx), (gA[0], dgA), (gB[0], dgB)):
        a, b = a.double(), b.double()
        assert ((a - b).norm() / b.norm()).item() < 2e-3  # 2^-9, half a step of bf16, at most


def test_many_rows(Q):
    """Tiles on every XCD, feature tiles past 256, no K pieces, rows that are not whole tiles."""
    say("experts, 3000 rows")
    E, M, n, m, r = 5, 3000, 512, 1544, 16
    L = Layer(Q, 370, E, M, n, m, r)
    offsets = [3, 900, 900, 901, 2300, 2999]
    check(L, offsets, 0.25, *run(Q, L, offsets, 0.25))


def test_side_stream_and_graph(Q):
    """On another stream than the default, and captured: the offsets are read at each replay."""
    say("experts, side stream and graph")
    E, M, n, m, r = 4, 400, 256, 264, 16
    L = Layer(Q, 380, E, M, n, m, r)
    off = offsets_dev([0, 100, 200, 300, 400])
    d = L.dev
    h, u = patterned((M, m)), patterned((M, r), torch.float32)
    out = (patterned((M, n)), patterned((E, r, n)), patterned((E, m, r)))
    ws = [poison(Q.experts_workspace_bytes(op, M, E, n, m, r)) for op in (0, 1)]

    def chain():
        Q.experts_fwd(d["x"], off, L.q, d["A"], d["B"], 0.5, h=h, u=u, workspace=ws[0])
        Q.experts_bwd(d["x"], d["g"], off, L.q, d["A"], d["B"], 0.5, u=u, out=out, workspace=ws[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    check(L, off.tolist(), 0.5, h, u, *out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for offsets in ([0, 400, 400, 400, 400], [0, 0, 17, 390, 400], [5, 100, 101, 101, 350], [0, 100, 200, 300, 400]):
        off.copy_(offsets_dev(offsets))
        for t in (h, u, *out):
            t.view(torch.int16).fill_(PATTERN)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(L, offsets, 0.5, h, u, *out)
        replayed = [t.clone() for t in (h, u, *out)]
        chain()
        torch.cuda.synchronize()
        for a, b in zip(replayed, (h, u, *out)):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_two_calls_at_once(Q):
    """Two streams, a workspace each."""
    say("experts, two streams")
    layers = [Layer(Q, 390 + i, 3, 500, 256, 200, 16) for i in range(2)]
    offsets = [[0, 200, 350, 500], [0, 10, 490, 495]]
    offs = [offsets_dev(o) for o in offsets]
    alone = [run(Q, L, o, 0.5) for L, o in zip(layers, offsets)]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for L, off, stream in zip(layers, offs, streams):
            with torch.cuda.stream(stream):
                d = L.dev
                h, u = Q.experts_fwd(d["x"], off, L.q, d["A"], d["B"], 0.5)
                got.append((h, u, *Q.experts_bwd(d["x"], d["g"], off, L.q, d["A"], d["B"], 0.5, u=u)))
        torch.cuda.synchronize()
        for L, o, a, b in zip(layers, offsets, alone, got):
            live = slice(o[0], o[-1])
            for p, q in zip(a[:3], b[:3]):
                assert torch.equal(p[live], q[live])
            for p, q in zip(a[3:], b[3:]):
                assert torch.equal(p, q)


def test_gradients_are_the_forwards_slopes(Q):
    """The directional derivative of sum(h * g) along a direction of A or B: h is linear in s u B^T, so the exact
    forward's difference quotient has no truncation error in B and in A; the kernels' gradients against it."""
    say("experts, differences")
    L = Layer(Q, 410, 3, 48, 128, 72, 8)
    offsets, s = [0, 20, 20, 47], 0.5
    _, _, _, gA, gB = run(Q, L, offsets, s)
    rng = np.random.default_rng(4)
    x, g, A, B = (L.val[k] for k in "xgAB")
    base = (X.experts_fwd(x, offsets, L.W, A, B, s)[0] * g).sum()
    for name, grad in (("A", gA), ("B", gB)):
        d = rng.standard_normal(L.val[name].shape)
        args = dict(A=A, B=B)
        args[name] = args[name] + d
        slope = (X.experts_fwd(x, offsets, L.W, args["A"], args["B"], s)[0] * g).sum() - base
        got = val(grad)
        assert abs(slope - (got * d).sum()) <= 2.0 ** -8 * np.abs(got * d).sum()  # each gradient value's rounding


def test_given_buffers_are_checked(Q):
    say("experts, given buffers")
    L = Layer(Q, 400, 2, 20, 64, 16, 8)
    d, off = L.dev, offsets_dev([0, 8, 20])
    args = (d["x"], off, L.q, d["A"], d["B"], 1.0)
    for kw in (dict(h=patterned((20, 8))), dict(u=patterned((19, 8), torch.float32)), dict(h=torch.zeros(20, 16).bfloat16()),
               dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            Q.experts_fwd(*args, **kw)
    with pytest.raises(TypeError):
        Q.experts_fwd(d["x"], off.long(), *args[2:])
    with pytest.raises(ValueError):
        Q.experts_fwd(d["x"], off.cpu(), *args[2:])
    bwd = (d["x"], d["g"]) + args[1:]
    for out in ((None, d["A"][0], d["B"]), (None, torch.empty_like(d["A"]), d["B"].cpu()),
                (d["g"], torch.empty_like(d["A"]), torch.empty_like(d["B"]))):
        with pytest.raises(ValueError):
            Q.experts_bwd(*bwd, out=out)
    with pytest.raises(TypeError):
        Q.experts_bwd(*bwd, u=d["g"][:, :8].contiguous())
    small = torch.zeros(16, dtype=torch.uint8, device="cuda")  # too small: replaced
    h, _ = Q.experts_fwd(*args, workspace=small)
    assert torch.equal(h, Q.experts_fwd(*args)[0])
