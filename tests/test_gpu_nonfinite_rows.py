"""A row of the upstream gradient that holds infinities or NaN changes no other row of grad_x, whatever the layer's
number of features: the GEMM's last step of 64 features must not read on into the next row where 64 does not divide
them.  grad_x is compared bit for bit with that of the same call on finite rows; no rounding enters."""

import pytest
import torch

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import bit_quantized_fine_qlora_amd as lib
    lib._lib.load()
    return lib


def say(msg):
    print(f"[case] {msg}", flush=True)


def operands(Q, seed, E, M, n, m, r):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    f = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
    q = Q.quantize_nf4_dq(0.05 * f(E * m, n))
    bf = torch.bfloat16
    return q, f(M, n).to(bf), f(M, m).to(bf), f(E, r, n).to(bf), f(E, m, r).to(bf)


def spoilt(g, rows):
    """g with the rows holding an infinity in their first columns or all NaN, by turns."""
    g = g.clone()
    for i, t in enumerate(rows):
        if i % 3 == 2:
            g[t] = NAN
        else:
            g[t, : 8 if i % 3 else 1] = (INF, -INF)[i % 2]
    return g


def compare(run, g, rows, live=None):
    want, got = run(g), run(spoilt(g, rows))
    torch.cuda.synchronize()
    keep = torch.ones(g.shape[0], dtype=torch.bool, device="cuda") if live is None else live.clone()
    keep[rows] = False
    assert torch.isfinite(want[keep].float()).all()
    assert torch.equal(got[keep].view(torch.int16), want[keep].view(torch.int16))
    assert not torch.isfinite(got[rows].float()).all(1).any()


# m: one, two and many K steps, of which the last is short by 8 to 56 columns (136: 120 = 64 + 56 of 192), K pieces
# (1608), K halves that meet (1032 by 16384), and multiples of 64 and odd numbers, where nothing is cut
DENSE = [(40, 128, 8), (300, 128, 56), (256, 64, 72), (77, 192, 136), (300, 256, 200), (512, 128, 264), (300, 64, 520),
         (100, 256, 1608), (256, 256, 1608), (256, 16384, 1032), (200, 16384, 1032), (4160, 4096, 200), (300, 128, 192),
         (300, 128, 259), (90, 128, 9)]


@pytest.mark.parametrize("M,n,m", DENSE)
@pytest.mark.parametrize("dropout", [None, (0.25, 11, 0)])
def test_dense(Q, M, n, m, dropout):
    say(f"rows that are not finite, dense M {M} n {n} m {m} dropout {dropout}")
    r = 8
    q, x, g, A, B = operands(Q, m + M, 1, M, n, m, r)
    run = lambda g: Q.linear_bwd(x, g, q, A[0], B[0], 0.5, dropout=dropout)[0]
    compare(run, g, [1, 5, 18, M // 2, M - 2])


EXPERTS = [(3, 90, 128, 8), (3, 600, 128, 56), (2, 520, 64, 72), (4, 300, 192, 136), (5, 700, 320, 200),
           (2, 1100, 256, 264), (3, 130, 192, 1032), (3, 130, 192, 1608), (4, 2100, 4096, 72), (70, 900, 64, 24),
           (3, 300, 128, 192), (3, 300, 128, 259)]


@pytest.mark.parametrize("E,M,n,m", EXPERTS)
def test_experts(Q, E, M, n, m):
    say(f"rows that are not finite, E {E} M {M} n {n} m {m}")
    r = 8
    q, x, g, A, B = operands(Q, m + M, E, M, n, m, r)
    cut = [2] + [M * (e + 1) // E - (7 * e) % 5 for e in range(E - 1)] + [M - 3]  # ragged; rows of no expert at both ends
    off = torch.tensor(cut, dtype=torch.int32, device="cuda")
    live = torch.zeros(M, dtype=torch.bool, device="cuda")
    live[2:M - 3] = True
    run = lambda g: Q.experts_bwd(x, g, off, q, A, B, 0.5)[0]
    compare(run, g, sorted({3, 6, 19, M // 2, M - 5, cut[1] - 1, cut[1]}), live)
