"""GPU parity of the layer norm and RMS norm against the float64 oracle.

Tolerances come from fp32 arithmetic: a row's sums pass through at most 16
additions in a thread and 6 + 8 across lanes and waves, so a sum is within
40 2^-24 of its terms' magnitudes; with the products and the reciprocal root
64 2^-24 of the sizes below bounds every step.  An output is then the rounding
to its type of a value within that of the oracle's.  The weights' gradients add up M rows, at most
M / 256 + 64 additions deep.
"""

import numpy as np
import pytest
import torch

import qlora_inputs as QI
from oracle import training_oracle as TO
from parity_utils import dev_bf16, f64, host_bits
from rounding_utils import assert_rounds_into

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import bit_quantized_fine_qlora_amd as lib
    lib._lib.load()
    return lib


def say(msg):
    print(f"[case] {msg}", flush=True)


def tensor(a, dtype):
    """(device tensor, its float64 values) of a float array in bf16 or fp32."""
    if dtype == "bf16":
        bits = QI.to_bf16_bits(a.astype(np.float32))
        return dev_bf16(bits), f64(bits)
    a = a.astype(np.float32)
    return torch.from_numpy(a).cuda(), a.astype(np.float64)


def values(t):
    return f64(host_bits(t)) if t.dtype == torch.bfloat16 else t.cpu().numpy().astype(np.float64)


def close(t, ref, tol, what):
    assert_rounds_into(values(t), ref, tol, what, bf16=t.dtype == torch.bfloat16)


def make(seed, M, n, dtype, wdtype, bias, shift=0.5):
    x = QI.normal_f32(seed, (M, n), 1.0) * np.exp(QI.normal_f32(seed + 1, (n,), 0.7)) + shift
    out = [tensor(x, dtype), tensor(1.0 + QI.normal_f32(seed + 2, (n,), 0.3), wdtype),
           tensor(QI.normal_f32(seed + 3, (M, n), 0.5), dtype)]
    out.append(tensor(QI.normal_f32(seed + 4, (n,), 0.3), wdtype) if bias else (None, None))
    return out


SHAPES = [(1, 1), (3, 5), (2, 8), (4, 9), (5, 511), (9, 512), (6, 513), (70, 1000), (5, 1025), (3, 2047), (33, 2048),
          (7, 3001), (40, 4096), (5, 4104), (600, 5001), (3, 8192), (2, 8200), (5, 16383), (300, 16384), (1500, 640)]


@pytest.mark.parametrize("M,n", SHAPES)
@pytest.mark.parametrize("kind,dtype,wdtype,bias", [("layer", "bf16", "bf16", True), ("rms", "bf16", "bf16", False),
                                                    ("layer", "fp32", "fp32", True), ("rms", "fp32", "fp32", False),
                                                    ("rms", "bf16", "fp32", True), ("layer", "bf16", "fp32", False)])
def test_norm(Q, M, n, kind, dtype, wdtype, bias):
    say(f"norm {kind} {M}x{n} {dtype} {wdtype} bias {bias}")
    layer = kind == "layer"
    (x, xv), (w, wv), (g, gv), (b, bv) = make(17 * M + n, M, n, dtype, wdtype, bias)
    eps = 1e-5
    y, mean, rstd = Q.norm_fwd(x, w, b, kind=Q.NORM_LAYER if layer else Q.NORM_RMS, eps=eps)
    gx, gw, gb = Q.norm_bwd(x, g, w, rstd, mean, bias=bias)
    gx2, no_w, no_b = Q.norm_bwd(x, g, w, rstd, mean, bias=bias, need_grad_w=False)
    again = Q.norm_bwd(x, g, w, rstd, mean, bias=bias)
    torch.cuda.synchronize()
    assert no_w is None and no_b is None and torch.equal(gx2, gx)
    assert torch.equal(again[0], gx) and torch.equal(again[1], gw) and (not bias or torch.equal(again[2], gb))
    ry, rmean, rrstd = TO.norm_fwd(xv, wv, bv, np.float64(np.float32(eps)), layer)
    C = 64 * EPS32
    size = np.abs(xv).mean(axis=1)
    spread = (np.abs(xv - rmean[:, None]) * rrstd[:, None])
    if layer:
        assert np.all(np.abs(values(mean) - rmean) <= C * size)
    else:
        assert mean is None
    # an error of the mean moves every difference: d var / var <= 2 rstd dmean
    drstd = rrstd * C * (1.0 + (rrstd * size if layer else 0.0))
    assert np.all(np.abs(values(rstd) - rrstd) <= drstd)
    move = np.abs(wv) * (spread * (drstd / rrstd)[:, None] + C * ((size * rrstd)[:, None] * layer + spread))
    close(y, ry, move + C * (0.0 if bv is None else np.abs(bv)), "y")

    # the backward takes the mean and rstd that it was given
    mv = values(mean) if layer else np.zeros(M)
    rv = values(rstd)
    rgx, rgw, rgb = TO.norm_bwd(xv, gv, wv, mv, rv, layer)
    xh = np.abs(xv - mv[:, None]) * rv[:, None]
    d = np.abs(gv * wv)
    tol = C * rv[:, None] * (d + d.mean(axis=1, keepdims=True) * layer + xh * (d * xh).mean(axis=1, keepdims=True))
    close(gx, rgx, tol, "grad_x")
    deep = (M / 256 + 64) * EPS32
    close(gw, rgw, deep * (np.abs(gv) * xh).sum(axis=0), "grad_w")
    if bias:
        close(gb, rgb, deep * np.abs(gv).sum(axis=0), "grad_b")
    else:
        assert gb is None


@pytest.mark.parametrize("M,n", [(1, 1), (3, 40), (5, 100), (33, 1000), (65, 4096), (9, 8192), (200, 5000)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_checkpoint_out_and_in(Q, M, n, kind):
    """y's checkpoint is the packing of y, and the backward from x's checkpoint is the backward of the restored x."""
    say(f"norm checkpoint {kind} {M}x{n}")
    layer = kind == "layer"
    (x, _), (w, wv), (g, gv), (b, _) = make(M + n, M, n, "bf16", "bf16", layer)
    y, mean, rstd, y8 = Q.norm_fwd(x, w, b, kind=Q.NORM_LAYER if layer else Q.NORM_RMS, checkpoint=True)
    plain = Q.norm_fwd(x, w, b, kind=Q.NORM_LAYER if layer else Q.NORM_RMS)[0]
    packed = Q.checkpoint_pack(y)
    assert torch.equal(y, plain)
    assert torch.equal(y8.codes, packed.codes) and torch.equal(y8.scales, packed.scales)
    x8 = Q.checkpoint_pack(x)
    for a, c in zip(Q.norm_bwd(x8, g, w, rstd, mean, bias=layer),
                    Q.norm_bwd(Q.checkpoint_unpack(x8), g, w, rstd, mean, bias=layer)):
        assert (a is None and c is None) or torch.equal(a, c)


def test_large_mean(Q):
    """The variance is not a difference of large numbers."""
    say("norm large mean")
    M, n = 8, 4096
    (x, xv), (w, wv), (g, _), _ = make(3, M, n, "fp32", "fp32", False, shift=1000.0)
    _, mean, rstd = Q.norm_fwd(x, w, kind=Q.NORM_LAYER, eps=0.0)
    _, rmean, rrstd = TO.norm_fwd(xv, wv, None, 0.0, True)
    # dmean <= 40 2^-24 1000 = 2.4e-3 changes the variance by its square
    assert np.all(np.abs(values(rstd) / rrstd - 1) <= 1e-5)


def test_special_rows(Q):
    """A row's infinities and NaNs stay in that row; a zero row is finite by its eps; others are untouched."""
    say("norm special rows")
    M, n = 9, 700
    (x, xv), (w, _), (g, _), (b, _) = make(4, M, n, "bf16", "bf16", True)
    clean, _, _ = Q.norm_fwd(x, w, b, kind=Q.NORM_LAYER)
    x[1, 699], x[3, 0], x[5] = float("nan"), float("inf"), 0.0
    for kind in (Q.NORM_LAYER, Q.NORM_RMS):
        y, mean, rstd, y8 = Q.norm_fwd(x, w, b, kind=kind, checkpoint=True)
        gx, gw, gb = Q.norm_bwd(x, g, w, rstd, mean, bias=True)
        finite = torch.isfinite(y.float()).all(dim=1)
        assert finite.tolist() == [True, False, True, False, True, True, True, True, True]
        assert torch.isfinite(gx.float()).all(dim=1).tolist() == finite.tolist()
        assert torch.equal(y[5], b) and bool(torch.isfinite(gb.float()).all())
        assert bool(torch.isnan(Q.checkpoint_unpack(y8)[1]).any())
        packed = Q.checkpoint_pack(y)
        assert torch.equal(y8.codes, packed.codes) and torch.equal(y8.scales, packed.scales)
        if kind == Q.NORM_LAYER:
            for i in (0, 2, 4, 6, 7, 8):
                assert torch.equal(y[i], clean[i])


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradient_against_differences(Q, kind):
    """A step along a direction changes sum(g y) by the gradient's product with it.  With y in fp32 within 1e-6
    of values of order 1, n M = 4000 of them, sum(g y) is within about 1e-4, over 2 h = 0.02: 5e-3; the third
    derivative adds h^2 times values of order 10: 1e-3 of a product of order 50."""
    say(f"norm differences {kind}")
    M, n, h = 4, 1000, 0.01
    k = Q.NORM_LAYER if kind == "layer" else Q.NORM_RMS
    (x, _), (w, _), (g, gv), (b, _) = make(6, M, n, "fp32", "fp32", True)
    _, mean, rstd = Q.norm_fwd(x, w, b, kind=k)
    gx, gw, gb = Q.norm_bwd(x, g, w, rstd, mean, bias=True)

    def total(x, w, b):
        return (values(Q.norm_fwd(x, w, b, kind=k)[0]) * gv).sum()

    for seed in range(3):
        dx = torch.from_numpy(QI.normal_f32(50 + seed, (M, n), 1.0)).cuda()
        dw = torch.from_numpy(QI.normal_f32(60 + seed, (n,), 1.0)).cuda()
        want = [(values(gx) * values(dx)).sum(), (values(gw) * values(dw)).sum(), (values(gb) * values(dw)).sum()]
        got = [(total(x + h * dx, w, b) - total(x - h * dx, w, b)) / (2 * h),
               (total(x, w + h * dw, b) - total(x, w - h * dw, b)) / (2 * h),
               (total(x, w, b + h * dw) - total(x, w, b - h * dw)) / (2 * h)]
        for a, c in zip(got, want):
            assert abs(a - c) <= 5e-3 + 1e-3 * max(50.0, abs(c))


def test_more_than_32_bits_of_elements(Q):
    M, n = 140000, 16384
    say(f"norm {M}x{n}")
    rows = [0, 70000, 131072, M - 1]
    (xr, xv), (w, wv), (gr, gv), _ = make(9, len(rows), n, "bf16", "bf16", False)
    x = torch.ones((M, n), dtype=torch.bfloat16, device="cuda")
    g = torch.zeros((M, n), dtype=torch.bfloat16, device="cuda")
    for i, r in enumerate(rows):
        x[r], g[r] = xr[i], gr[i]
    y, _, rstd = Q.norm_fwd(x, w, kind=Q.NORM_RMS)
    gx, gw, _ = Q.norm_bwd(x, g, w, rstd)
    ys, _, rs = Q.norm_fwd(xr, w, kind=Q.NORM_RMS)
    gxs, _, _ = Q.norm_bwd(xr, gr, w, rs)
    for i, r in enumerate(rows):
        assert torch.equal(y[r], ys[i]) and torch.equal(gx[r], gxs[i])
    assert not bool(gx[M - 2].any())
    rgw = TO.norm_bwd(xv, gv, wv, np.zeros(len(rows)), values(rs), False)[1]
    assert np.all(np.abs(values(gw) - rgw) <= 2.0 ** -8 * np.abs(rgw) + 1e-4)


def test_in_place_and_other_stream(Q):
    say("norm in place, side stream")
    (x, _), (w, _), (g, _), _ = make(12, 50, 3000, "bf16", "bf16", False)
    y, _, rstd = Q.norm_fwd(x, w)
    gx, gw, _ = Q.norm_bwd(x, g, w, rstd)
    x2, g2 = x.clone(), g.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gx2, gw2, _ = Q.norm_bwd(x, g2, w, rstd, out=g2)
        y2, _, rstd2 = Q.norm_fwd(x2, w, out=x2)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(gx2, gx) and torch.equal(gw2, gw) and torch.equal(y2, y) and torch.equal(rstd2, rstd)


def test_refusals(Q):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        Q.norm_fwd(x.half(), w)
    with pytest.raises(TypeError):
        Q.norm_fwd(x, w, b=w.float())
    with pytest.raises(ValueError):
        Q.norm_fwd(x, w[:32].contiguous())
    with pytest.raises(ValueError):
        Q.norm_fwd(x.t(), w[:4].contiguous())
    with pytest.raises(Q.QloraError):
        Q.norm_fwd(x.float(), w)  # fp32 rows take fp32 weights
    with pytest.raises(Q.QloraError):
        Q.norm_fwd(x.float(), w.float(), checkpoint=True)
    with pytest.raises(Q.QloraError):
        Q.norm_fwd(x, w, kind=7)
    with pytest.raises(Q.QloraError):
        Q.norm_fwd(x, w, eps=float("nan"))
    wide = torch.zeros((2, 16385), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(Q.QloraError):
        Q.norm_fwd(wide, wide[0].contiguous())
    rstd = torch.ones(4, device="cuda")
    with pytest.raises(TypeError):
        Q.norm_bwd(x, x.float(), w, rstd)
    with pytest.raises(ValueError):
        Q.norm_bwd(x, x, w, rstd[:2].contiguous())
