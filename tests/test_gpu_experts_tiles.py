"""The experts' layer over the paths that its kernels choose between: streamed tiles of 16 and 32 rows with and without K
splits, GEMM tiles of every height, K pieces and whole tiles (both kernels launched, one of them at work), more experts
than a wave has lanes, chunks that are summed.

The reference is torch in float64 on the same card, from the weight's dequantized values (which are compared bit for
bit elsewhere); the tolerances are those of the parity tests: K 2^-24 of the sum of magnitudes for a product of K
terms in fp32, 2^-17 for operands that enter as two bf16 parts.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

EPS, PAIR = 2.0 ** -24, 2.0 ** -17


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import bit_quantized_fine_qlora_amd as lib
    lib._lib.load()
    return lib


def rounds_into(got, ref, tol, what):
    """got is the rounding of a value within tol of ref (rounding is monotone)."""
    lo, hi = ((ref + d).float().to(torch.bfloat16) for d in (-tol, tol))
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside"


def even(E, M):
    return [M * e // E for e in range(E + 1)]


def one_takes_all(E, M, e=1):
    return [0] * (e + 1) + [M] * (E - e)


HEIGHTS = [1, 64, 65, 0, 128, 129, 192, 193, 255, 256, 257, 321]


def of_rows(rows):
    out = [0]
    for r in rows:
        out.append(out[-1] + r)
    return out


CASES = [  # name, n, m, r, offsets
    ("16 rows a tile, K splits", 2048, 520, 16, one_takes_all(3, 48)),
    ("16 rows a tile, one row each", 832, 264, 8, even(40, 40)),
    ("32 rows a tile", 1024, 392, 20, [0, 3, 3, 70, 100]),
    ("32 rows a tile, K splits, odd features", 2112, 131, 64, even(4, 120)),
    ("every tile height", 256, 300, 16, of_rows(HEIGHTS)),
    ("every tile height, K pieces both ways", 1152, 1080, 8, of_rows(HEIGHTS)),
    ("forward pieces where whole tiles were possible", 1024, 4096, 16, one_takes_all(8, 1000)),
    ("forward whole tiles where pieces were possible", 1024, 4096, 16, of_rows([300, 1, 257, 130, 600, 258, 300, 154])),
    ("backward pieces where whole tiles were possible", 4096, 1024, 16, one_takes_all(8, 1000, 6)),
    ("backward whole tiles where pieces were possible", 4096, 1024, 32, of_rows([300, 1, 257, 130, 600, 258, 300, 154])),
    ("200 experts", 128, 256, 8, even(200, 8000)),
    ("1024 experts", 64, 64, 8, even(1024, 2000)),
    ("1024 experts, the last two have rows", 64, 72, 4, [0] * 1023 + [1, 700]),
    ("summed chunks at 64 ranks", 512, 448, 64, of_rows([700, 1400, 0, 90])),
    ("summed chunks at 128 ranks", 256, 320, 128, of_rows([0, 1100, 513])),
    ("summed chunks at 24 ranks, odd features", 192, 333, 24, of_rows([1025, 256])),
]


@pytest.mark.parametrize("case", range(len(CASES)), ids=[c[0].replace(" ", "_") for c in CASES])
def test_paths(Q, case):
    name, n, m, r, offsets = CASES[case]
    E, M, s = len(offsets) - 1, max(offsets), 0.5
    print(f"[case] {name}: E {E} M {M} n {n} m {m} r {r}", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(100 + case)

    def normal(*shape, sigma=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * sigma).to(dtype)

    q = Q.quantize_nf4_dq(normal(E * m, n, sigma=0.02, dtype=torch.float32))
    W = Q.dequant_nf4_dq(q).view(E, m, n)
    x, g, A, B = normal(M, n), normal(M, m), normal(E, r, n, sigma=1 / 16), normal(E, m, r, sigma=0.01)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")

    def poison(op):
        return torch.full((Q.experts_workspace_bytes(op, M, E, n, m, r),), 0xFF, dtype=torch.uint8, device="cuda")

    nan = float("nan")
    h = torch.full((M, m), nan, dtype=torch.bfloat16, device="cuda")
    u = torch.full((M, r), nan, device="cuda")
    Q.experts_fwd(x, off, q, A, B, s, h=h, u=u, workspace=poison(0))
    out = [torch.full(shape, nan, dtype=torch.bfloat16, device="cuda") for shape in ((M, n), (E, r, n), (E, m, r))]
    Q.experts_bwd(x, g, off, q, A, B, s, u=u, out=out, workspace=poison(1))
    torch.cuda.synchronize()
    gx, gA, gB = out
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        if a == b:
            assert not gA[e].any() and not gB[e].any(), f"gradients of expert {e}, which has no row"
            continue
        xe, ge, We, Ae, Be, ue = (t.double() for t in (x[a:b], g[a:b], W[e], A[e], B[e], u[a:b]))
        mag = [t.abs() for t in (xe, ge, We, Ae, Be, ue)]
        u_ref, u_mag = xe @ Ae.t(), mag[0] @ mag[3].t()
        assert ((ue - u_ref).abs() <= n * EPS * u_mag + 1e-30).all(), f"u of expert {e}"
        lora = s * (u_mag @ mag[4].t())
        rounds_into(h[a:b], xe @ We.t() + s * (u_ref @ Be.t()),
                    (n + 2 * r) * EPS * (mag[0] @ mag[2].t() + lora) + (PAIR + n * EPS) * lora, f"h of expert {e}")
        v_ref, v_mag = ge @ Be, mag[1] @ mag[4]
        lora = s * (v_mag @ mag[3])
        rounds_into(gx[a:b], ge @ We + s * (v_ref @ Ae),
                    (m + 2 * r) * EPS * (mag[1] @ mag[2] + lora) + (PAIR + m * EPS) * lora, f"grad_x of expert {e}")
        rows = 2 * (b - a) * EPS + PAIR
        rounds_into(gA[e], s * (v_ref.t() @ xe), s * (rows + m * EPS) * (v_mag.t() @ mag[0]), f"grad_A of expert {e}")
        rounds_into(gB[e], s * (ge.t() @ ue), s * rows * (mag[1].t() @ mag[5]), f"grad_B of expert {e}")


def test_rows_of_no_expert_may_hold_anything(Q):
    """NaN and infinities before the first and behind the last row that counts, in both operands, next to a tile's end."""
    print("[case] rows of no expert", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    for lead, rows, tail, n, m in ((1, [5, 9], 1, 320, 200), (70, [200, 0, 31], 33, 256, 137), (3, [300, 290], 9, 128, 72)):
        E, M, r = len(rows), lead + sum(rows) + tail, 12
        x, g = (torch.randn(M, k, generator=gen, device="cuda").bfloat16() for k in (n, m))
        A, B = (torch.randn(E, *k, generator=gen, device="cuda").bfloat16() for k in ((r, n), (m, r)))
        q = Q.quantize_nf4_dq(torch.randn(E * m, n, generator=gen, device="cuda"))
        off = torch.tensor(of_rows(rows), dtype=torch.int32, device="cuda") + lead
        live = slice(lead, lead + sum(rows))

        def both():
            h, u = Q.experts_fwd(x, off, q, A, B, 0.5)
            return [t[live].clone() for t in (h, u)] + [
                t[live].clone() if i == 0 else t for i, t in enumerate(Q.experts_bwd(x, g, off, q, A, B, 0.5, u=u))]

        first = both()
        for t, v in ((x, float("nan")), (g, float("inf"))):
            t[:lead] = v
            t[lead + sum(rows):] = -v
        for p, k in zip(first, both()):
            assert torch.equal(p, k) and p.isfinite().all()
