"""Workspaces and outputs that the caller gives: a host tensor, a strided one
or one of another shape is refused before anything is launched (its address
would go to a kernel), and a workspace that is too small is replaced."""

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


def calls(Q):
    """(name, call that takes a workspace) of every operator with one."""
    M, n, m, r = 40, 128, 64, 8
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    q = Q.quantize_nf4_dq(normal(m, n, dtype=torch.float32))
    x, g, A, B = normal(M, n), normal(M, m), normal(r, n), normal(m, r)
    _, u = Q.linear_fwd(x, q, A, B, 1.0)
    c = Q.checkpoint_pack(x)
    w, gn = normal(n), normal(M, n)
    _, mean, rstd = Q.norm_fwd(x, w, kind=Q.NORM_LAYER)
    labels = torch.randint(0, m, (M,), generator=gen, device="cuda")
    offsets = torch.tensor([0, 20, M], dtype=torch.int32, device="cuda")
    return [("linear_fwd", lambda ws: Q.linear_fwd(x, q, A, B, 1.0, workspace=ws)),
            ("linear_bwd", lambda ws: Q.linear_bwd(x, g, q, A, B, 1.0, u=u, workspace=ws)),
            ("linear_bwd of a checkpoint", lambda ws: Q.linear_bwd(c, g, q, A, B, 1.0, u=u, workspace=ws)),
            ("norm_bwd", lambda ws: Q.norm_bwd(x, gn, w, rstd, mean, bias=True, workspace=ws)),
            ("sequence_logps", lambda ws: (Q.sequence_logps(g, labels, offsets, workspace=ws),)),
            ("preference_fwd", lambda ws: tuple(vars(Q.preference_fwd(g, labels, offsets, workspace=ws)).values()))]


def test_workspaces(Q):
    for name, call in calls(Q):
        print(f"[case] workspace of {name}", flush=True)
        with pytest.raises(ValueError):
            call(torch.empty(1 << 20, dtype=torch.uint8))
        with pytest.raises(ValueError):
            call(torch.empty(1 << 21, dtype=torch.uint8, device="cuda")[::2])
        want = call(None)
        for size in (0, 1 << 22):
            for a, b in zip(call(torch.empty(size, dtype=torch.uint8, device="cuda")), want):
                assert torch.equal(a, b), name


def test_norm_without_weight_gradients_needs_none(Q):
    x = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    _, _, rstd = Q.norm_fwd(x, w)
    gx, gw, gb = Q.norm_bwd(x, x, w, rstd, need_grad_w=False)
    assert gw is None and gb is None and gx.shape == x.shape


def test_outputs_of_the_linear_backward(Q):
    M, n, m, r = 4, 64, 128, 8
    q = Q.quantize_nf4_dq(torch.ones((m, n), device="cuda"))

    def zeros(*shape, device="cuda"):
        return torch.zeros(shape, dtype=torch.bfloat16, device=device)

    x, g, A, B = zeros(M, n), zeros(M, m), zeros(r, n), zeros(m, r)
    u = torch.zeros((M, r), device="cuda")
    good = (zeros(M, n), zeros(r, n), zeros(m, r))
    bad = [(zeros(M, n, device="cpu"), *good[1:]), (good[0], zeros(r, n, device="cpu"), good[2]), (*good[:2], zeros(r, m)),
           (good[0].float(), *good[1:]), (good[0], zeros(n, r).t(), good[2])]
    for given in (x, Q.checkpoint_pack(x)):
        for out in bad:
            with pytest.raises((TypeError, ValueError)):
                Q.linear_bwd(given, g, q, A, B, 1.0, u=u, out=out)
        assert Q.linear_bwd(given, g, q, A, B, 1.0, u=u, out=good)[1] is good[1]
        assert Q.linear_bwd(given, g, q, A, B, 1.0, u=u, out=(None, *good[1:]))[0] is None
