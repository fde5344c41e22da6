"""The norm's backward told its kind: a mean that does not go with it is an
error instead of the other norm's gradients, and with the right one the
gradients are those of the call without a kind, bit for bit."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("checkpoint", [False, True])
def test_kind(checkpoint):
    import bit_quantized_fine_qlora_amd as Q
    print(f"[case] norm_bwd kind, checkpoint {checkpoint}", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    x, g = (torch.randn((9, 200), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.randn(200, generator=gen, device="cuda").to(torch.bfloat16)
    saved = Q.checkpoint_pack(x) if checkpoint else x
    for kind, other in ((Q.NORM_LAYER, Q.NORM_RMS), (Q.NORM_RMS, Q.NORM_LAYER)):
        _, mean, rstd = Q.norm_fwd(x, w, kind=kind)
        told = Q.norm_bwd(saved, g, w, rstd, mean, bias=True, kind=kind)
        for a, b in zip(told, Q.norm_bwd(saved, g, w, rstd, mean, bias=True)):
            assert torch.equal(a, b)
        with pytest.raises(ValueError):
            Q.norm_bwd(saved, g, w, rstd, mean, kind=other)
    with pytest.raises(ValueError):
        Q.norm_bwd(saved, g, w, rstd, kind=Q.NORM_LAYER)  # the mean forgotten
    with pytest.raises(Q.QloraError):
        Q.norm_bwd(saved, g, w, rstd, kind=7)
