"""GPU parity of the 8-bit activation checkpoint and of the linear backward
that reads it.

Packing and restoring are exact integer and power-of-two arithmetic: codes,
scale bytes and restored values are compared bit for bit with the oracle.  The
linear backward from a checkpoint is compared with the oracle at the common
tolerance of the float outputs (parity_utils), its grad_x and grad_B bit for
bit with the plain call's (x does not enter them); grad_A, and the plain call's
on the restored input, are the bf16 rounding of a value within the fp32 error
bound of the oracle's.
"""

import numpy as np
import pytest
import torch

import qlora_inputs as QI
from oracle import qlora_oracle as O
from oracle import training_oracle as TO
from parity_utils import assert_close, dev_bf16, f64, host_bits
from rounding_utils import assert_rounds_into

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import bit_quantized_fine_qlora_amd as lib
    lib._lib.load()
    return lib


def say(msg):
    print(f"[case] {msg}", flush=True)


def activations(seed, M, n):
    """Channels of unequal size, a few far larger than the rest."""
    x = QI.normal_f32(seed, (M, n), 1.0)
    width = np.exp(QI.normal_f32(seed + 1, (n,), 1.0))
    width[::37] *= 30.0
    return QI.to_bf16_bits((x * width).astype(np.float32))


def check_pack(Q, bits):
    M, n = bits.shape
    c = Q.checkpoint_pack(dev_bf16(bits))
    x = Q.checkpoint_unpack(c)
    torch.cuda.synchronize()
    codes, scales = TO.checkpoint_pack(bits)
    assert np.array_equal(c.codes.cpu().numpy(), codes)
    assert np.array_equal(c.scales.cpu().numpy(), scales)
    want = TO.checkpoint_unpack(codes, scales)
    got = f64(host_bits(x))
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.array_equal(got[ok], want[ok])


@pytest.mark.parametrize("M,n", [(1, 1), (1, 7), (3, 8), (2, 31), (5, 33), (33, 100), (4, 127), (4, 129), (17, 1000),
                                 (129, 257), (64, 4096), (7, 28672), (1000, 40)])
def test_pack_and_restore(Q, M, n):
    say(f"pack {M}x{n}")
    check_pack(Q, activations(M * 31 + n, M, n))


def test_every_bf16_pattern(Q):
    """All 65536 patterns, one to a row and shuffled into blocks, non-finite ones and subnormals included."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    say("pack every pattern")
    with np.errstate(invalid="ignore"):
        check_pack(Q, bits[:, None].copy())
        check_pack(Q, np.random.default_rng(3).permutation(bits).reshape(256, 256))
        small = np.random.default_rng(4).permutation(bits[(bits & 0x7FFF) < 0x0500])
        check_pack(Q, small[: small.size // 64 * 64].reshape(-1, 64))


def test_more_than_32_bits_of_elements(Q):
    M, n = 140000, 16384  # 2.3e9 elements
    say(f"pack {M}x{n}")
    x = torch.empty((M, n), dtype=torch.bfloat16, device="cuda")
    x.fill_(0.5)
    rows = [0, 65535, 131072, M - 1]
    bits = activations(5, len(rows), n)
    for i, r in enumerate(rows):
        x[r] = dev_bf16(bits[i])
    c = Q.checkpoint_pack(x)
    y = Q.checkpoint_unpack(c)
    codes, scales = TO.checkpoint_pack(bits)
    for i, r in enumerate(rows):
        assert np.array_equal(c.codes[r].cpu().numpy(), codes[i]) and np.array_equal(c.scales[r].cpu().numpy(), scales[i])
        assert np.array_equal(f64(host_bits(y[r])), TO.checkpoint_unpack(codes[i:i + 1], scales[i:i + 1])[0])
    assert bool((y[M - 2] == 0.5).all())


def test_other_stream_and_given_outputs(Q):
    say("side stream")
    bits = activations(8, 300, 640)
    x = dev_bf16(bits)
    c = Q.alloc_checkpoint(300, 640)
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert Q.checkpoint_pack(x, out=c) is c
        assert Q.checkpoint_unpack(c, out=out) is out
    torch.cuda.current_stream().wait_stream(side)
    want = TO.checkpoint_unpack(*TO.checkpoint_pack(bits))
    assert np.array_equal(f64(host_bits(out)), want)
    assert c.nbytes() == 300 * 640 + 300 * 20


def layer(M, n, m, r, seed):
    W = QI.normal_f32(seed, (m, n), 0.02)
    g = QI.to_bf16_bits(QI.normal_f32(seed + 1, (M, m), 1.0))
    A = QI.to_bf16_bits(QI.normal_f32(seed + 2, (r, n), 1 / 16))
    B = QI.to_bf16_bits(QI.normal_f32(seed + 3, (m, r), 0.01))
    return W, activations(seed + 4, M, n), g, A, B


CASES = [(1, 64, 64, 1), (32, 256, 256, 8), (33, 128, 200, 16), (65, 320, 96, 5), (129, 576, 131, 64), (200, 1024, 512, 32),
         (300, 448, 320, 128), (700, 192, 256, 33), (1030, 2048, 256, 64), (257, 4160, 1024, 16)]


@pytest.mark.parametrize("M,n,m,r", CASES)
@pytest.mark.parametrize("dropout", [None, (0.1, 99, 7)])
def test_linear_backward(Q, M, n, m, r, dropout):
    say(f"linear_bwd M {M} n {n} m {m} r {r} dropout {dropout}")
    W, x_bits, g_bits, A_bits, B_bits = layer(M, n, m, r, 1000 + M + r)
    s = 0.5
    q = Q.quantize_nf4_dq(torch.from_numpy(W).cuda())
    x, g, A, B = (dev_bf16(v) for v in (x_bits, g_bits, A_bits, B_bits))
    _, u = Q.linear_fwd(x, q, A, B, s, dropout=dropout)
    c = Q.checkpoint_pack(x)
    restored = Q.checkpoint_unpack(c)
    gx, gA, gB = Q.linear_bwd(c, g, q, A, B, s, u=u, dropout=dropout)
    px, pA, pB = Q.linear_bwd(restored, g, q, A, B, s, u=u, dropout=dropout)
    again = Q.linear_bwd(c, g, q, A, B, s, u=u, dropout=dropout)
    none, gA2, gB2 = Q.linear_bwd(c, g, q, A, B, s, u=u, dropout=dropout, need_grad_x=False)
    torch.cuda.synchronize()
    assert none is None
    for a, b in ((gx, px), (gB, pB), (gB2, gB), (gA2, gA), (again[0], gx), (again[1], gA), (again[2], gB)):
        assert torch.equal(a, b)
    v = f64(g_bits) @ f64(B_bits)
    xd = TO.checkpoint_unpack(*TO.checkpoint_pack(x_bits))
    if dropout is not None:
        xd = xd * O.dropout_mask_np(M, n, *dropout) / (1.0 - float(np.float32(dropout[0])))
    ref = s * v.T @ xd
    assert_close(f64(host_bits(gA)), ref, "grad_A")
    # v is a sum of m products, kept as two bf16 parts (2^-15 of it), grad_A a sum of M products, all in fp32
    x_abs = np.abs(xd)
    tol = s * (m + 64) * 2.0 ** -24 * (np.abs(f64(g_bits)) @ np.abs(f64(B_bits))).T @ x_abs
    tol = tol + s * ((M + 64) * 2.0 ** -23 + 2.0 ** -15) * np.abs(v).T @ x_abs
    for name, t in (("grad_A", gA), ("grad_A of the restored input", pA)):
        assert_rounds_into(f64(host_bits(t)), ref, tol, name)


def test_not_finite_block_marks_its_columns(Q):
    M, n, m, r = 70, 256, 128, 16
    say("linear_bwd with a NaN in the input")
    W, x_bits, g_bits, A_bits, B_bits = layer(M, n, m, r, 77)
    x_bits[41, 70] = 0x7FC0
    q = Q.quantize_nf4_dq(torch.from_numpy(W).cuda())
    x, g, A, B = (dev_bf16(v) for v in (x_bits, g_bits, A_bits, B_bits))
    u = torch.zeros((M, r), dtype=torch.float32, device="cuda")
    gx, gA, gB = Q.linear_bwd(Q.checkpoint_pack(x), g, q, A, B, 1.0, u=u)
    bad = torch.isnan(gA)
    assert bool(bad[:, 64:96].all()) and int(bad.sum()) == 32 * r
    assert bool(torch.isfinite(gx.float()).all()) and bool(torch.isfinite(gB.float()).all())


def test_refusals(Q):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        Q.checkpoint_pack(x.float())
    with pytest.raises(ValueError):
        Q.checkpoint_pack(x.t())
    with pytest.raises(ValueError):
        Q.checkpoint_pack(x.cpu())
    c = Q.checkpoint_pack(x)
    with pytest.raises(ValueError):
        Q.checkpoint_unpack(Q.Checkpoint8(c.codes, c.scales[:, :2].contiguous()))
    q = Q.quantize_nf4_dq(torch.zeros((64, 64), device="cuda"))
    A = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    B = torch.zeros((64, 8), dtype=torch.bfloat16, device="cuda")
    g = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    u = torch.zeros((4, 8), dtype=torch.float32, device="cuda")
    with pytest.raises(ValueError):
        Q.linear_bwd(c, g, q, A, B, 1.0)  # u is required
    with pytest.raises(ValueError):
        Q.linear_bwd(Q.checkpoint_pack(torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")), g, q, A, B, 1.0, u=u)
