"""The backward from a checkpoint stays inside a workspace of exactly the size
that the library asks for, and its gradients are right in it.

The shapes give the checkpointed product more split sums than the plain one
has room for (they go over memory of earlier stages), with and without the
single pass over g, and one where the splits are what fits.
"""

import numpy as np
import pytest
import torch

import qlora_inputs as QI
from oracle import training_oracle as TO
from parity_utils import dev_bf16, f64, host_bits
from rounding_utils import assert_rounds_into

pytestmark = pytest.mark.gpu

GUARD = 4096


@pytest.mark.parametrize("M,n,m,r", [(1030, 2048, 256, 64), (2048, 1024, 512, 32), (600, 2048, 131, 33), (1100, 512, 264, 128),
                                     (308, 7808, 8, 5)])
@pytest.mark.parametrize("dropout", [None, (0.1, 5, 3)])
def test_exact_workspace(M, n, m, r, dropout):
    import bit_quantized_fine_qlora_amd as Q
    print(f"[case] exact workspace M {M} n {n} m {m} r {r} dropout {dropout}", flush=True)
    x_bits = QI.to_bf16_bits(QI.normal_f32(1 + M, (M, n), 1.0))
    g_bits = QI.to_bf16_bits(QI.normal_f32(2 + M, (M, m), 1.0))
    A_bits = QI.to_bf16_bits(QI.normal_f32(3 + M, (r, n), 1 / 16))
    B_bits = QI.to_bf16_bits(QI.normal_f32(4 + M, (m, r), 0.01))
    q = Q.quantize_nf4_dq(torch.from_numpy(QI.normal_f32(5 + M, (m, n), 0.02)).cuda())
    x, g, A, B = (dev_bf16(v) for v in (x_bits, g_bits, A_bits, B_bits))
    c = Q.checkpoint_pack(x)
    _, u = Q.linear_fwd(x, q, A, B, 0.5, dropout=dropout)
    need = Q.workspace_bytes(Q.QLORA_OP_BWD if dropout is None else Q.QLORA_OP_BWD_DROPOUT, M, n, m, r)
    room = torch.full((need + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    inside = room[GUARD:GUARD + need]
    gx, gA, gB = Q.linear_bwd(c, g, q, A, B, 0.5, u=u, workspace=inside, dropout=dropout)
    px, pA, pB = Q.linear_bwd(Q.checkpoint_unpack(c), g, q, A, B, 0.5, u=u, dropout=dropout)
    torch.cuda.synchronize()
    assert bool((room[:GUARD] == 0xA5).all()) and bool((room[GUARD + need:] == 0xA5).all())
    assert torch.equal(gx, px) and torch.equal(gB, pB)
    if dropout is not None:
        assert torch.equal(gA, pA)  # the same splits, the same masks
        return
    v = f64(g_bits) @ f64(B_bits)
    xd = TO.checkpoint_unpack(*TO.checkpoint_pack(x_bits))
    # v is a sum of m products, kept as two bf16 parts (2^-15 of it), grad_A a sum of M products, all in fp32
    tol = 0.5 * (m + 64) * 2.0 ** -24 * (np.abs(f64(g_bits)) @ np.abs(f64(B_bits))).T @ np.abs(xd)
    tol = tol + 0.5 * ((M + 64) * 2.0 ** -23 + 2.0 ** -15) * np.abs(v).T @ np.abs(xd)
    assert_rounds_into(f64(host_bits(gA)), 0.5 * v.T @ xd, tol, "grad_A")
