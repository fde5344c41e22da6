"""The experts' layer and the optimizer step where offsets pass 32 bits, where operands and workspaces end, and at the
largest numbers of experts."""

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


def normal(gen, *shape, sigma=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * sigma).bfloat16()


def generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


@pytest.mark.parametrize("rows", [3, 70])
def test_weights_past_four_gigabytes(Q, rows):
    """The last expert's codes begin past 2^32 bytes (and its blocks past 2^26): rows streamed, and the GEMM."""
    E, n, m, r, s = 150, 4096, 14336, 8, 0.5
    print(f"[case] {E} experts of {m} x {n}, {rows} rows in the last", flush=True)
    gen = generator(rows)
    cells = m * n
    q = Q.QuantizedWeight(torch.zeros(E * cells // 2, dtype=torch.uint8, device="cuda"),
                          torch.zeros(E * cells // 64, dtype=torch.uint8, device="cuda"),
                          torch.zeros(E * cells // 16384, device="cuda"), E * m, n)
    one = Q.quantize_nf4_dq(torch.randn(m, n, generator=gen, device="cuda") * 0.02)
    q.codes[-cells // 2:] = one.codes
    q.absmax8[-cells // 64:] = one.absmax8
    q.c2[-(cells // 16384):] = one.c2
    A, B = torch.zeros(E, r, n, dtype=torch.bfloat16, device="cuda"), torch.zeros(E, m, r, dtype=torch.bfloat16, device="cuda")
    A[-1], B[-1] = normal(gen, r, n, sigma=1 / 16), normal(gen, m, r, sigma=0.01)
    x, g = normal(gen, rows, n), normal(gen, rows, m)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = rows
    h, u = Q.experts_fwd(x, off, q, A, B, s)
    gx, gA, gB = Q.experts_bwd(x, g, off, q, A, B, s, u=u)
    torch.cuda.synchronize()
    W = Q.dequant_nf4_dq(one).double()
    xd, gd, Ad, Bd = (t.double() for t in (x, g, A[-1], B[-1]))
    u_ref, v_ref = xd @ Ad.t(), gd @ Bd

    def near(got, ref, mag, terms):
        tol = (terms + 2 * r) * EPS * mag + PAIR * mag
        lo, hi = ((ref + d).float().bfloat16() for d in (-tol, tol))
        assert ((got >= lo) & (got <= hi)).all()

    near(h, xd @ W.t() + s * (u_ref @ Bd.t()), xd.abs() @ W.abs().t() + s * (xd.abs() @ Ad.abs().t() @ Bd.abs().t()), 2 * n)
    near(gx, gd @ W + s * (v_ref @ Ad), gd.abs() @ W.abs() + s * (gd.abs() @ Bd.abs() @ Ad.abs()), 2 * m)
    near(gA[-1], s * (v_ref.t() @ xd), s * (gd.abs() @ Bd.abs()).t() @ xd.abs(), m + 2 * rows)
    near(gB[-1], s * (gd.t() @ u_ref), s * gd.abs().t() @ (xd.abs() @ Ad.abs().t()), n + 2 * rows)
    assert not gA[:-1].any() and not gB[:-1].any()


@pytest.mark.parametrize("case", [(2, 60, 512, 200, 12), (3, 40, 1024, 520, 8), (3, 700, 2048, 131, 16), (5, 900, 320, 259, 64),
                                  (1024, 1, 128, 64, 4), (1024, 1023, 64, 64, 8), (1, 2000, 4096, 256, 32)])
def test_nothing_is_written_behind_operands(Q, case):
    """Outputs and a workspace of the least size end where guard bytes begin."""
    E, M, n, m, r = case
    print(f"[case] guards: E {E} M {M} n {n} m {m} r {r}", flush=True)
    gen = generator(1)
    q = Q.quantize_nf4_dq(torch.randn(E * m, n, generator=gen, device="cuda"))
    x, g, A, B = normal(gen, M, n), normal(gen, M, m), normal(gen, E, r, n), normal(gen, E, m, r)
    off = torch.tensor([M * e // E for e in range(E + 1)], dtype=torch.int32, device="cuda")
    held = []

    def guarded(shape, dtype):
        size = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
        room = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        held.append((room, size))
        return room[:size].view(dtype).view(shape)

    def ws(op):
        return guarded((Q.experts_workspace_bytes(op, M, E, n, m, r),), torch.uint8)

    h, u = Q.experts_fwd(x, off, q, A, B, 0.5, h=guarded((M, m), torch.bfloat16), u=guarded((M, r), torch.float32),
                         workspace=ws(Q.QLORA_OP_FWD))
    shapes = ((M, n), (E, r, n), (E, m, r))
    out = Q.experts_bwd(x, g, off, q, A, B, 0.5, u=u, out=tuple(guarded(k, torch.bfloat16) for k in shapes),
                        workspace=ws(Q.QLORA_OP_BWD))
    torch.cuda.synchronize()
    for room, size in held:
        assert (room[size:] == 0xA5).all()
    again = (Q.experts_fwd(x, off, q, A, B, 0.5)[0], *Q.experts_bwd(x, g, off, q, A, B, 0.5))
    for p, k in zip((h, *out), again):
        assert torch.equal(p, k) and p.isfinite().all()


@pytest.mark.parametrize("eight", [True, False])
def test_elements_past_two_to_the_31(Q, eight):
    """The last elements of a tensor of more than 2^31 step as a tensor of their own does."""
    n, tail = 2 ** 31 + 6149, 2 ** 12 + 5  # the tail begins at a block's border
    print(f"[case] {n} elements, {8 if eight else 32} bits", flush=True)
    gen = generator(5)

    def state(count):
        moments = [Q.alloc_moment8(count, True), Q.alloc_moment8(count, False)] if eight else [
            torch.zeros(count, device="cuda") for _ in range(2)]
        return [torch.zeros(count, device="cuda"), torch.zeros(count, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(count, dtype=torch.bfloat16, device="cuda"), *moments]

    assert (n - tail) % 128 == 0
    large, small = state(n), state(tail)
    small[0].copy_(torch.randn(tail, generator=gen, device="cuda"))
    small[2].copy_(torch.randn(tail, generator=gen, device="cuda"))
    for i in (0, 2):
        large[i][-tail:] = small[i]
    plans = Q.AdamWStep([tuple(large)]), Q.AdamWStep([tuple(small)])
    clips = [p.clip(1.0) for p in plans]
    for p in plans:
        p.run(1e-3, weight_decay=0.1, step=1, clip=clips[1])
    torch.cuda.synchronize()
    assert abs(clips[0][0].item() / clips[1][0].item() - 1) <= 2.0 ** -23 and clips[1][0].item() > 1
    for i in (0, 1):
        assert torch.equal(large[i][-tail:], small[i])
        assert not large[i][:n - tail:4097].any()
    for a, b in zip(large[3:], small[3:]):
        if eight:
            assert torch.equal(a.codes[-tail:], b.codes) and torch.equal(a.steps[-b.steps.numel():], b.steps)
            assert torch.equal(Q.moment8_values(a)[-tail:], Q.moment8_values(b))
        else:
            assert torch.equal(a[-tail:], b)
