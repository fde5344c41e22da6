"""The norm where a workgroup (or a wave) walks several rows: three at least
and a remainder, every shape that the kernels hold a row in, both directions
and all types, all rows different, against the float64 oracle at the
tolerances of the few-row cases; then what the few-row cases leave out of
checkpoints (wide rows, fp32 weights, the RMS norm with a bias) and of calls
in place."""

import numpy as np
import pytest
import torch

from oracle import training_oracle as TO
from rounding_utils import assert_rounds_into

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24
C = 64 * EPS32
# widths of one wave a row (two shapes), 4 waves, 8 waves, and 16 / 8 / 8 waves past 4096 values; the rows make three
# iterations and a remainder on 256 compute units (the forward takes up to 16 workgroups of four rows on each)
SHAPES = [(50001, 100), (50003, 700), (6500, 1500), (3300, 3001), (3301, 4500), (3200, 8200), (4700, 2600)]


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import bit_quantized_fine_qlora_amd as lib
    lib._lib.load()
    return lib


def f64(t):
    return t.cpu().double().numpy()


def inputs(seed, M, n, dtype, wdtype, bias):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, scale, to):
        return (scale * torch.randn(*shape, generator=gen, device="cuda")).to(to)

    width = torch.exp(normal(n, scale=0.7, to=torch.float32))
    size = 1.0 + torch.rand(M, 1, generator=gen, device="cuda")  # rows of different sizes: one taken for another shows
    x = (torch.randn(M, n, generator=gen, device="cuda") * width * size + 0.5).to(dtype)
    w = (1.0 + normal(n, scale=0.3, to=torch.float32)).to(wdtype)
    return x, w, normal(M, n, scale=0.5, to=dtype), normal(n, scale=0.3, to=wdtype) if bias else None


def close(t, ref, tol, what):
    assert_rounds_into(f64(t), ref, tol, what, bf16=t.dtype == torch.bfloat16)


def check_fwd(out, x, w, b, layer, eps=1e-5):
    y, mean, rstd = out
    xv, wv, bv = f64(x), f64(w), None if b is None else f64(b)
    ry, rmean, rrstd = TO.norm_fwd(xv, wv, bv, np.float64(np.float32(eps)), layer)
    size = np.abs(xv).mean(axis=1)
    spread = np.abs(xv - rmean[:, None]) * rrstd[:, None]
    if layer:
        assert np.all(np.abs(f64(mean) - rmean) <= C * size)
    drstd = rrstd * C * (1.0 + (rrstd * size if layer else 0.0))
    assert np.all(np.abs(f64(rstd) - rrstd) <= drstd)
    move = np.abs(wv) * (spread * (drstd / rrstd)[:, None] + C * ((size * rrstd)[:, None] * layer + spread))
    close(y, ry, move + C * (0.0 if bv is None else np.abs(bv)), "y")


def check_bwd(grads, x, g, w, mean, rstd, layer):
    gx, gw, gb = grads
    M = g.shape[0]
    xv, gv, wv, rv = f64(x), f64(g), f64(w), f64(rstd)
    mv = f64(mean) if layer else np.zeros(M)
    rgx, rgw, rgb = TO.norm_bwd(xv, gv, wv, mv, rv, layer)
    xh = np.abs(xv - mv[:, None]) * rv[:, None]
    d = np.abs(gv * wv)
    tol = C * rv[:, None] * (d + d.mean(axis=1, keepdims=True) * layer + xh * (d * xh).mean(axis=1, keepdims=True))
    close(gx, rgx, tol, "grad_x")
    deep = (M / 256 + 64) * EPS32
    close(gw, rgw, deep * (np.abs(gv) * xh).sum(axis=0), "grad_w")
    if gb is not None:
        close(gb, rgb, deep * np.abs(gv).sum(axis=0), "grad_b")


@pytest.mark.parametrize("M,n", SHAPES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_rows(Q, M, n, kind, dtype):
    print(f"[case] norm rows {M}x{n} {kind} {dtype}", flush=True)
    layer = kind == "layer"
    k = Q.NORM_LAYER if layer else Q.NORM_RMS
    x, w, g, b = inputs(M + n, M, n, dtype, dtype, layer)
    y, mean, rstd = Q.norm_fwd(x, w, b, kind=k)
    check_fwd((y, mean, rstd), x, w, b, layer)
    grads = Q.norm_bwd(x, g, w, rstd, mean, bias=layer, kind=k)
    check_bwd(grads, x, g, w, mean, rstd, layer)
    for a, c in zip(grads, Q.norm_bwd(x, g, w, rstd, mean, bias=layer, kind=k)):
        assert (a is None and c is None) or torch.equal(a, c)
    # in place, all rows
    assert torch.equal(Q.norm_bwd(x, g, w, rstd, mean, bias=layer, kind=k, out=g)[0], grads[0])
    assert torch.equal(Q.norm_fwd(x, w, b, kind=k, out=x)[0], y)


@pytest.mark.parametrize("M,n", SHAPES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_many_rows_from_a_checkpoint(Q, M, n, kind):
    print(f"[case] norm rows from a checkpoint {M}x{n} {kind}", flush=True)
    layer = kind == "layer"
    k = Q.NORM_LAYER if layer else Q.NORM_RMS
    x, w, g, b = inputs(M + 2 * n, M, n, torch.bfloat16, torch.bfloat16, layer)
    y, mean, rstd, y8 = Q.norm_fwd(x, w, b, kind=k, checkpoint=True)
    packed = Q.checkpoint_pack(y)
    assert torch.equal(y8.codes, packed.codes) and torch.equal(y8.scales, packed.scales)
    x8 = Q.checkpoint_pack(x)
    restored = Q.checkpoint_unpack(x8)
    grads = Q.norm_bwd(x8, g, w, rstd, mean, bias=layer, kind=k)
    check_bwd(grads, restored, g, w, mean, rstd, layer)
    for a, c in zip(grads, Q.norm_bwd(restored, g, w, rstd, mean, bias=layer, kind=k)):
        assert (a is None and c is None) or torch.equal(a, c)
    assert torch.equal(Q.norm_bwd(x8, g, w, rstd, mean, bias=layer, kind=k, out=g)[0], grads[0])


@pytest.mark.parametrize("M,n", [(1, 8193), (5, 9001), (300, 12000), (40, 16383), (33, 16384), (7, 6), (90, 500),
                                 (40, 1000), (30, 2000), (20, 4000), (20, 8000)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("wdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bias", [False, True])
def test_checkpoints_of_every_kind(Q, M, n, kind, wdtype, bias):
    """Written and read by the norm: wide rows, fp32 weights, either norm with a bias or without."""
    print(f"[case] norm checkpoint {M}x{n} {kind} {wdtype} bias {bias}", flush=True)
    layer = kind == "layer"
    k = Q.NORM_LAYER if layer else Q.NORM_RMS
    x, w, g, b = inputs(3 * M + n, M, n, torch.bfloat16, wdtype, bias)
    y, mean, rstd, y8 = Q.norm_fwd(x, w, b, kind=k, checkpoint=True)
    check_fwd((y, mean, rstd), x, w, b, layer)
    packed = Q.checkpoint_pack(y)
    assert torch.equal(y8.codes, packed.codes) and torch.equal(y8.scales, packed.scales)
    x8 = Q.checkpoint_pack(x)
    restored = Q.checkpoint_unpack(x8)
    grads = Q.norm_bwd(x8, g, w, rstd, mean, bias=bias, kind=k)
    check_bwd(grads, restored, g, w, mean, rstd, layer)
    for a, c in zip(grads, Q.norm_bwd(restored, g, w, rstd, mean, bias=bias, kind=k)):
        assert (a is None and c is None) or torch.equal(a, c)
    only_x = Q.norm_bwd(x8, g, w, rstd, mean, kind=k, need_grad_w=False)
    assert torch.equal(only_x[0], grads[0]) and only_x[1] is None


@pytest.mark.parametrize("M,n", [(40, 7), (40, 300), (40, 900), (9, 1999), (9, 4001), (9, 8191), (9, 16381)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place(Q, M, n, kind, dtype):
    """Rows whose last values share a piece with a neighbour's, written over their own input."""
    print(f"[case] norm in place {M}x{n} {kind} {dtype}", flush=True)
    layer = kind == "layer"
    k = Q.NORM_LAYER if layer else Q.NORM_RMS
    x, w, g, b = inputs(5 * M + n, M, n, dtype, dtype, True)
    y, mean, rstd = Q.norm_fwd(x, w, b, kind=k)
    grads = Q.norm_bwd(x, g, w, rstd, mean, bias=True, kind=k)
    over_g = Q.norm_bwd(x, g, w, rstd, mean, bias=True, kind=k, out=g)
    for a, c in zip(over_g, grads):
        assert torch.equal(a, c)
    over_x = Q.norm_fwd(x, w, b, kind=k, out=x)
    assert over_x[0].data_ptr() == x.data_ptr() and torch.equal(over_x[0], y) and torch.equal(over_x[2], rstd)
