"""grad_A from a checkpointed input where a workgroup's ring of stages wraps:
a wide layer leaves few splits of the tokens, so that a split has 7 to 18
stages of 64 tokens (three buffers up to 32 ranks and past 64, four between),
the last one ragged, the last columns a part of a tile.  Against float64 on
the device, at the bound of the few-stage cases.
"""

import pytest
import torch

from rounding_utils import assert_rounds_into

pytestmark = pytest.mark.gpu


# on 256 compute units: 130 tiles of 256 columns, 2 splits of 9 stages (1 of 18 past 64 ranks), 3 of 8 or 7 up to 32
@pytest.mark.parametrize("M,n,m,r", [(1150, 33088, 64, 64), (1139, 33088, 136, 33), (1150, 33088, 64, 128), (1100, 33088, 72, 96),
                                     (1350, 33088, 64, 16), (1350, 33088, 128, 8), (1339, 33088, 64, 32), (600, 65600, 64, 64)])
@pytest.mark.parametrize("dropout", [None, (0.2, 11, 5)])
def test_grad_A(M, n, m, r, dropout):
    import bit_quantized_fine_qlora_amd as Q
    print(f"[case] grad_A from a checkpoint M {M} n {n} m {m} r {r} dropout {dropout}", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M + n + r)

    def normal(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=gen, device="cuda")).to(torch.bfloat16)

    s = 0.5
    size = 1.0 + 3.0 * torch.rand(M, 1, generator=gen, device="cuda")  # a token taken for another shows
    x = (normal(M, n).float() * size).to(torch.bfloat16)
    g, A, B = normal(M, m), normal(r, n, scale=1 / 16), normal(m, r, scale=0.05)
    q = Q.quantize_nf4_dq(normal(m, n, scale=0.02).float())
    u = torch.randn(M, r, generator=gen, device="cuda")
    c = Q.checkpoint_pack(x)
    restored = Q.checkpoint_unpack(c)
    _, gA, gB = Q.linear_bwd(c, g, q, A, B, s, u=u, dropout=dropout, need_grad_x=False)
    again = Q.linear_bwd(c, g, q, A, B, s, u=u, dropout=dropout, need_grad_x=False)[1]
    _, pA, pB = Q.linear_bwd(restored, g, q, A, B, s, u=u, dropout=dropout, need_grad_x=False)
    assert torch.equal(again, gA) and torch.equal(gB, pB)
    if dropout is not None:
        assert torch.equal(gA, pA)  # the same splits, masks and products
        return
    xd, gd, Bd = restored.double(), g.double(), B.double()
    v = gd @ Bd
    # v is a sum of m products, kept as two bf16 parts (2^-15 of it), grad_A a sum of M products, all in fp32
    tol = s * (m + 64) * 2.0 ** -24 * (gd.abs() @ Bd.abs()).t() @ xd.abs()
    tol = tol + s * ((M + 64) * 2.0 ** -23 + 2.0 ** -15) * v.abs().t() @ xd.abs()
    ref = s * v.t() @ xd
    for name, t in (("grad_A", gA), ("grad_A of the restored input", pA)):
        assert_rounds_into(t.double().cpu().numpy(), ref.cpu().numpy(), tol.cpu().numpy(), name)
