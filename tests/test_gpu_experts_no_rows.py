"""The experts' layer for a batch without any row: empty outputs, and gradients of zero as every expert without rows has
them, on the current stream and in a captured graph.  Nothing is rounded."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import bit_quantized_fine_qlora_amd as lib
    lib._lib.load()
    return lib


@pytest.mark.parametrize("E,n,m,r", [(1, 64, 8, 1), (3, 128, 72, 12), (70, 64, 7, 128)])
def test_no_rows(Q, E, n, m, r):
    print(f"[case] experts without rows, E {E} n {n} m {m} r {r}", flush=True)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    q = Q.quantize_nf4_dq(torch.randn(E * m, n, device="cuda"))
    A, B = torch.randn(E, r, n, **bf), torch.randn(E, m, r, **bf)
    x, g, off = torch.empty(0, n, **bf), torch.empty(0, m, **bf), torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    h, u = Q.experts_fwd(x, off, q, A, B, 0.5)
    assert h.shape == (0, m) and u.shape == (0, r) and Q.experts_fwd(x, off, q, A, B, 0.5, want_u=False)[1] is None
    for kw in (dict(), dict(u=u), dict(need_grad_x=False)):
        gx, gA, gB = Q.experts_bwd(x, g, off, q, A, B, 0.5, **kw)
        assert (gx is None) == ("need_grad_x" in kw) and (gx is None or gx.shape == (0, n))
        assert gA.shape == A.shape and gB.shape == B.shape and not gA.any() and not gB.any()
    out = (None, torch.full_like(A, float("nan")), torch.full_like(B, float("nan")))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.experts_bwd(x, g, off, q, A, B, 0.5, u=u, out=out)
    for _ in range(3):
        for t in out[1:]:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert not out[1].any() and not out[2].any()


def test_what_is_refused_without_rows(Q):
    print("[case] experts without rows, wrong arguments", flush=True)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    q = Q.quantize_nf4_dq(torch.randn(16, 64, device="cuda"))
    A, B, x = torch.randn(2, 4, 64, **bf), torch.randn(2, 8, 4, **bf), torch.empty(0, 64, **bf)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    for args in ((x, off[:2], q, A, B), (x, off, q, A[:1], B), (torch.empty(0, 128, **bf), off, q, A, B)):
        with pytest.raises(ValueError):
            Q.experts_fwd(*args, 0.5)
    with pytest.raises(ValueError):
        Q.experts_bwd(x, torch.empty(0, 7, **bf), off, q, A, B, 0.5)
    with pytest.raises(ValueError):
        Q.experts_bwd(x, torch.empty(1, 8, **bf), off, q, A, B, 0.5)
