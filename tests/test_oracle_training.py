"""Pins for the oracle of the norm, the 8-bit checkpoint and the preference loss.

Pinned by: torch's own norms, log-softmax and autograd in float64, central
differences of the forward formulas, and for the checkpoint its definition
value by value (an exhaustive walk over bf16) and its error bound.
"""

import numpy as np
import pytest
import torch

import qlora_inputs as QI
from oracle import training_oracle as TO


def bf16_values(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def test_checkpoint_every_bf16_value():
    """One value a row: every finite bf16 number within half a step of its restored value."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)[:, None]
    codes, scales = TO.checkpoint_pack(bits)
    assert scales.shape == (65536, 4) and not scales[:, 1:].any()
    v, r = bf16_values(bits)[:, 0], TO.checkpoint_unpack(codes, scales)[:, 0]
    finite = np.isfinite(v)
    assert np.array_equal(np.isnan(r), ~finite)
    step = np.exp2(scales[finite, 0].astype(np.float64) - 127)
    assert np.all(np.abs(r[finite] - v[finite]) <= step / 2)
    big = finite & (np.abs(v) >= 2.0 ** -120)
    k = np.abs(codes[big, 0].astype(int))
    assert k.min() >= 64 and k.max() == 127
    # a restored value is a bf16 number
    back = torch.from_numpy(r[finite]).to(torch.bfloat16).double().numpy()
    assert np.array_equal(back, r[finite])


@pytest.mark.parametrize("n", [1, 31, 32, 33, 100, 128, 160])
def test_checkpoint_blocks(n):
    bits = QI.to_bf16_bits(QI.normal_f32(7 + n, (9, n), 3.0))
    codes, scales = TO.checkpoint_pack(bits)
    assert scales.shape == (9, TO.checkpoint_pitch(n)) and not scales[:, -(-n // 32):].any()
    v, r = bf16_values(bits), TO.checkpoint_unpack(codes, scales)
    for b in range(-(-n // 32)):
        sl = slice(32 * b, min(n, 32 * b + 32))
        top = np.abs(v[:, sl]).max(axis=1)
        assert np.all(np.abs(r[:, sl] - v[:, sl]).max(axis=1) <= top / 128)
        assert np.array_equal(np.floor(np.log2(top)) + 127 - 6, scales[:, b])


def test_checkpoint_special_blocks():
    bits = QI.to_bf16_bits(QI.normal_f32(3, (4, 96), 1.0))
    bits[0, 5], bits[1, 40], bits[2, :32] = 0x7F80, 0xFFC1, 0
    bits[3, :32] = 0x0001  # the smallest subnormal: restored as zero
    r = TO.checkpoint_unpack(*TO.checkpoint_pack(bits))
    assert np.isnan(r[0, :32]).all() and np.isfinite(r[0, 32:]).all()
    assert np.isnan(r[1, 32:64]).all() and np.isfinite(r[1, :32]).all() and np.isfinite(r[1, 64:]).all()
    assert not r[2, :32].any() and not r[3, :32].any()


@pytest.mark.parametrize("layer", [True, False])
def test_norm_against_torch_and_differences(layer):
    rng = np.random.default_rng(5)
    x, g, w, b = rng.standard_normal((6, 37)) + 0.3, rng.standard_normal((6, 37)), rng.standard_normal(37), rng.standard_normal(37)
    eps = 1e-3
    y, mean, rstd = TO.norm_fwd(x, w, b, eps, layer)
    tx, tw, tb = (torch.tensor(v, requires_grad=True) for v in (x, w, b))
    if layer:
        ty = torch.nn.functional.layer_norm(tx, (37,), tw, tb, eps)
    else:
        ty = tx * torch.rsqrt(tx.square().mean(1, keepdim=True) + eps) * tw + tb
    assert np.allclose(y, ty.detach().numpy(), rtol=1e-12, atol=1e-12)
    ty.backward(torch.tensor(g))
    grads = TO.norm_bwd(x, g, w, mean, rstd, layer)
    for got, want in zip(grads, (tx.grad, tw.grad, tb.grad)):
        assert np.allclose(got, want.numpy(), rtol=1e-10, atol=1e-11)
    # central differences: error h^2 / 6 of a third derivative of order 10, plus rounding 1e-16 / h
    h = 1e-5
    for at in [(0, 0), (3, 17), (5, 36)]:
        e = np.zeros_like(x)
        e[at] = h
        d = ((TO.norm_fwd(x + e, w, b, eps, layer)[0] - TO.norm_fwd(x - e, w, b, eps, layer)[0]) * g).sum() / (2 * h)
        assert abs(d - grads[0][at]) <= 1e-8
    for col in (0, 36):
        e = np.zeros(37)
        e[col] = h
        d = ((TO.norm_fwd(x, w + e, b, eps, layer)[0] - TO.norm_fwd(x, w - e, b, eps, layer)[0]) * g).sum() / (2 * h)
        assert abs(d - grads[1][col]) <= 1e-8


def packed_case(seed, lens, V, masked=0.3):
    rng = np.random.default_rng(seed)
    T = sum(lens)
    logits = 2.0 * rng.standard_normal((T, V))
    labels = rng.integers(0, V, T)
    labels[rng.random(T) < masked] = -100
    offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return logits, labels, offsets


@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_preference_against_torch_and_differences(smoothing):
    lens, V, beta = [5, 1, 7, 4], 11, 0.7
    logits, labels, offsets = packed_case(11, lens, V)
    ref = np.random.default_rng(1).standard_normal(4) - 8.0
    out = TO.preference(logits, labels, offsets, ref, beta, smoothing)
    tl = torch.tensor(logits, requires_grad=True)
    lp = torch.log_softmax(tl, 1)
    lp = torch.stack([lp[t, labels[t]] if labels[t] >= 0 else lp[t, 0] * 0 for t in range(len(labels))])
    seq = torch.stack([lp[a:b].sum() for a, b in zip(offsets, offsets[1:])])
    z = beta * ((seq[0::2] - torch.tensor(ref[0::2])) - (seq[1::2] - torch.tensor(ref[1::2])))
    ls = torch.nn.functional.logsigmoid
    loss = (-(1 - smoothing) * ls(z) - smoothing * ls(-z)).mean()
    loss.backward()
    assert np.allclose(out["loss"], loss.item(), rtol=1e-13)
    assert np.allclose(out["logps"], seq.detach().numpy(), rtol=1e-13)
    assert np.allclose(out["grad"], tl.grad.numpy(), rtol=1e-11, atol=1e-14)
    h = 1e-5
    for t in np.flatnonzero(labels >= 0)[:3]:
        for v in (0, labels[t]):
            e = np.zeros_like(logits)
            e[t, v] = h
            d = (TO.preference(logits + e, labels, offsets, ref, beta, smoothing)["loss"]
                 - TO.preference(logits - e, labels, offsets, ref, beta, smoothing)["loss"]) / (2 * h)
            assert abs(d - out["grad"][t, v]) <= 1e-9


def test_preference_empty_and_masked_sequences():
    logits, labels, offsets = packed_case(3, [3, 0, 4, 2], 7, masked=0.0)
    labels[3:7] = -1  # a sequence with nothing scored
    out = TO.preference(logits, labels, offsets, None, 0.5)
    assert out["logps"][1] == 0.0 and out["logps"][2] == 0.0
    assert not out["grad"][3:7].any() and np.isfinite(out["loss"])


def test_masked_logits_have_probability_zero():
    logits, labels, offsets = packed_case(4, [3, 3], 9, masked=0.0)
    logits[:, 8] = -np.inf
    labels = labels % 8
    out = TO.preference(logits, labels, offsets, None, 0.5)
    assert np.isfinite(out["loss"]) and not out["grad"][:, 8].any()
    less = TO.preference(logits[:, :8], labels, offsets, None, 0.5)
    assert np.allclose(out["grad"][:, :8], less["grad"], rtol=1e-14)
