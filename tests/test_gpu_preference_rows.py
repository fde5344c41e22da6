"""Rows that are no sequence's: whatever they hold, with a label or without,
they change no output of the sequences, and their own outputs are zeros."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,V", [(24, 1000), (30, 20011), (1500, 300)])  # rows in one chunk, in many, and whole rows
@pytest.mark.parametrize("spoil", ["nan", "inf", "-inf", "label"])
def test_rows_outside_every_sequence(dtype, tokens, V, spoil):
    import bit_quantized_fine_qlora_amd as Q
    print(f"[case] rows outside {dtype} {tokens}x{V} {spoil}", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(tokens + V)
    logits = (2.0 * torch.randn((tokens, V), generator=gen, device="cuda")).to(dtype)
    labels = torch.randint(0, V, (tokens,), generator=gen, device="cuda")
    labels[::5] = -100
    # tokens before the first sequence and after the last are no sequence's
    a, b = tokens // 8, tokens - tokens // 8
    cut = np.array([a, a + (b - a) // 4, a + (b - a) // 2, a + (b - a) // 2, b], dtype=np.int32)
    offsets = torch.from_numpy(cut).cuda()
    outside = torch.ones(tokens, dtype=torch.bool, device="cuda")
    outside[a:b] = False

    def run(x, lab):
        r = Q.preference_fwd(x, lab, offsets, beta=0.3, label_smoothing=0.1)
        return r, Q.preference_bwd(x, lab, r), Q.sequence_logps(x, lab, offsets)

    clean, grad, lps = run(logits, labels)
    x, lab = logits.clone(), labels.clone()
    lab[outside] = 7 if spoil != "label" else 2 * V  # all with a label now
    if spoil != "label":
        x[outside] = float(spoil)
    r, g, s = run(x, lab)
    assert bool(torch.isfinite(r.loss))
    for p, q in ((r.loss, clean.loss), (r.logps, clean.logps), (r.coef, clean.coef), (g, grad), (s, lps),
                 (r.lse[a:b], clean.lse[a:b])):
        assert torch.equal(p, q)
    assert not bool(r.coef[outside].any()) and not bool(g[outside].any())
