"""CPU checks of the C ABI of the norm, the 8-bit checkpoint and the preference
loss: bad arguments are rejected before anything is launched."""

import ctypes
import os

import pytest

P = ctypes.c_void_p(1 << 20)   # non-NULL and aligned; never dereferenced on error paths
MIS = ctypes.c_void_p((1 << 20) + 4)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_fine_qlora_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libqlora.so is not built (run __graft_entry__.build())")
    return _lib.load()


@pytest.mark.parametrize("name", ["qlora_checkpoint_pack", "qlora_checkpoint_unpack"])
def test_checkpoint(lib, name):
    f = getattr(lib, name)
    for M, n in ((0, 8), (-1, 8), (4, 0), (4, -8), (1 << 31, 8), (4, 1 << 30)):
        assert f(M, n, P, P, P, None) == -2, (M, n)
    for i in range(3):
        assert f(4, 8, *[None if j == i else P for j in range(3)], None) == -1
        assert f(4, 8, *[MIS if j == i else P for j in range(3)], None) == -4


def test_linear_bwd_ckpt(lib):
    from bit_quantized_fine_qlora_amd import _lib

    def f(M=32, n=256, m=256, r=8, s=1.0, x=P, xs=P, u=P, gx=P, gA=P, d=None, ws=P, wsb=1 << 30):
        return lib.qlora_linear_bwd_ckpt(M, n, m, r, s, x, xs, P, P, P, P, P, P, u, gx, gA, P, d, ws, wsb, None)

    assert f(n=100) == -2 and f(M=0) == -2 and f(r=129) == -3 and f(s=NAN) == -7
    assert f(x=None) == -1 and f(xs=None) == -1 and f(u=None) == -1 and f(gA=None) == -1
    assert f(x=MIS) == -4 and f(xs=MIS) == -4 and f(u=MIS) == -4 and f(gx=MIS) == -4
    assert f(d=ctypes.pointer(_lib.Dropout(1.0, 1, 0))) == -7
    need = lib.qlora_workspace_bytes(1, 32, 256, 256, 8)
    assert f(wsb=need - 1) == -5 and f(ws=None) == -5
    more = lib.qlora_workspace_bytes(2, 32, 256, 256, 8)
    assert f(d=ctypes.pointer(_lib.Dropout(0.1, 1, 0)), wsb=more - 1) == -5


def test_norm_fwd(lib):
    def f(kind=0, xt=0, wt=0, M=4, n=64, eps=1e-5, x=P, w=P, b=P, y=P, mean=P, rstd=P, c=None, cs=None):
        return lib.qlora_norm_fwd(kind, xt, wt, M, n, eps, x, w, b, y, mean, rstd, c, cs, None)

    assert f(kind=2) == -7 and f(kind=-1) == -7 and f(xt=2) == -7 and f(xt=3) == -7 and f(wt=2) == -7
    assert f(xt=1, wt=0) == -7 and f(eps=NAN) == -7 and f(eps=-1.0) == -7 and f(eps=INF) == -7
    assert f(M=0) == -2 and f(n=0) == -2 and f(n=16385) == -2
    assert f(x=None) == -1 and f(w=None) == -1 and f(y=None) == -1 and f(rstd=None) == -1 and f(mean=None) == -1
    assert f(c=P) == -1 and f(cs=P) == -1                 # both or neither
    assert f(xt=1, wt=1, c=P, cs=P) == -7                 # a checkpoint holds bf16
    for name in ("x", "w", "b", "y", "mean", "rstd"):
        assert f(**{name: MIS}) == -4, name
    assert f(c=MIS, cs=P) == -4 and f(c=P, cs=MIS) == -4


def test_norm_bwd(lib):
    def f(kind=0, xt=0, wt=0, M=4, n=64, x=P, xs=None, g=P, w=P, mean=P, rstd=P, gx=P, gw=P, gb=P, ws=P, wsb=1 << 30):
        return lib.qlora_norm_bwd(kind, xt, wt, M, n, x, xs, g, w, mean, rstd, gx, gw, gb, ws, wsb, None)

    assert f(kind=5) == -7 and f(xt=3) == -7 and f(xt=1) == -7 and f(n=16385) == -2 and f(M=0) == -2
    for name in ("x", "g", "w", "mean", "rstd", "gx", "gw"):
        assert f(**{name: None}) == -1, name                # gw: grad_b without grad_w
    assert f(xt=2) == -1                                    # a checkpoint needs its scales
    for name in ("x", "g", "w", "mean", "rstd", "gx", "gw", "gb", "xs", "ws"):
        assert f(**{name: MIS}) == -4, name
    size = lib.qlora_norm_workspace_bytes
    assert size(0, 4, 64, 0) == 0 and size(0, 4, 16385, 1) == 0 and size(2, 4, 64, 1) == 0 and size(0, 4, 64, 3) == 0
    assert f(wsb=size(0, 4, 64, 2) - 1) == -5 and f(ws=None) == -5
    assert f(gb=None, wsb=size(0, 4, 64, 1) - 1) == -5
    assert f(kind=1, gb=None, wsb=size(1, 4, 64, 1) - 1) == -5
    assert size(1, 4, 64, 1) < size(1, 4, 64, 2)


def test_preference(lib):
    def fwd(ty=0, T=4, V=64, pairs=1, x=P, lab=P, off=P, ref=P, beta=0.1, e=0.0, loss=P, lps=P, lse=P, coef=P, ws=P,
            wsb=1 << 30):
        return lib.qlora_preference_fwd(ty, T, V, pairs, x, lab, off, ref, beta, e, loss, lps, lse, coef, ws, wsb, None)

    assert fwd(ty=2) == -7 and fwd(beta=NAN) == -7 and fwd(e=-0.1) == -7 and fwd(e=1.1) == -7 and fwd(e=NAN) == -7
    assert fwd(T=0) == -2 and fwd(V=0) == -2 and fwd(pairs=0) == -2 and fwd(V=1 << 30) == -2
    for name in ("x", "lab", "off", "loss", "lps", "lse", "coef"):
        assert fwd(**{name: None}) == -1, name
    for name in ("x", "lab", "off", "ref", "loss", "lps", "lse", "coef", "ws"):
        assert fwd(**{name: MIS}) == -4, name
    size = lib.qlora_preference_workspace_bytes
    assert size(0, 64, 1) == 0 and size(4, 64, -1) == 0
    assert fwd(wsb=size(4, 64, 1) - 1) == -5 and fwd(ws=None) == -5

    def lps(ty=0, T=4, V=64, S=2, x=P, lab=P, off=P, out=P, lse=P, ws=P, wsb=1 << 30):
        return lib.qlora_sequence_logps(ty, T, V, S, x, lab, off, out, lse, ws, wsb, None)

    assert lps(ty=5) == -7 and lps(S=0) == -2 and lps(T=-1) == -2 and lps(off=None) == -1 and lps(out=MIS) == -4
    assert lps(wsb=size(4, 64, 0) - 1) == -5

    def bwd(ty=0, T=4, V=64, x=P, lab=P, lse=P, coef=P, scale=1.0, out=P):
        return lib.qlora_preference_bwd(ty, T, V, x, lab, lse, coef, scale, out, None)

    assert bwd(ty=2) == -7 and bwd(scale=INF) == -7 and bwd(V=0) == -2
    for name in ("x", "lab", "lse", "coef", "out"):
        assert bwd(**{name: None}) == -1 and bwd(**{name: MIS}) == -4, name
