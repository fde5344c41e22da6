"""GPU parity of the packed sequences' log-probabilities, the preference loss
and its gradient against the float64 oracle.

Tolerances from fp32 arithmetic.  A row's sum of exponentials: the largest
term is 1, a thread adds V / 256 terms one after another and the joins add 16
more steps, each term's exponential within 2^-22 (4 + |x - m|) of itself, of
which only terms near the maximum weigh: lse is within
(V / 256 + 128) 2^-24 + 2^-22 |lse|.  A log-probability adds two roundings of
its operands, a sequence adds its scored tokens' errors, z adds its two
sequences', times beta; the loss moves by at most z's error, the coefficient
by beta / pairs times a quarter of it.  A gradient is the rounding to its type
of a value within that of the oracle's.
"""

import numpy as np
import pytest
import torch

import qlora_inputs as QI
from oracle import training_oracle as TO
from parity_utils import dev_bf16, f64, host_bits
from rounding_utils import assert_rounds_into

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import bit_quantized_fine_qlora_amd as lib
    lib._lib.load()
    return lib


def say(msg):
    print(f"[case] {msg}", flush=True)


def values(t):
    return f64(host_bits(t)) if t.dtype == torch.bfloat16 else t.cpu().numpy().astype(np.float64)


def packed(seed, lens, V, dtype, masked=0.4, spread=3.0, likely=True):
    """(logits on the device, their float64 values, labels, offsets)."""
    rng = np.random.default_rng(seed)
    T = sum(lens)
    x = (spread * rng.standard_normal((T, V))).astype(np.float32)
    labels = rng.integers(0, V, T)
    if likely:
        x[np.arange(T), labels] = np.log(V) + spread ** 2 / 2 + rng.standard_normal(T)
    labels[rng.random(T) < masked] = -100
    offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    if dtype == "bf16":
        bits = QI.to_bf16_bits(x)
        return dev_bf16(bits), f64(bits), labels, offsets
    return torch.from_numpy(x).cuda(), x.astype(np.float64), labels, offsets


def on_device(a):
    return torch.from_numpy(a).cuda()


def check(Q, logits, v, labels, offsets, ref, beta, smoothing, scale=1.0):
    T, V = v.shape
    dl, do = on_device(labels), on_device(offsets)
    dr = None if ref is None else on_device(ref.astype(np.float32))
    r = Q.preference_fwd(logits, dl, do, dr, beta=beta, label_smoothing=smoothing)
    grad = Q.preference_bwd(logits, dl, r, grad_scale=scale)
    again = Q.preference_fwd(logits, dl, do, dr, beta=beta, label_smoothing=smoothing)
    lps = Q.sequence_logps(logits, dl, do)
    torch.cuda.synchronize()
    for a, b in ((again.loss, r.loss), (again.logps, r.logps), (again.lse, r.lse), (again.coef, r.coef), (lps, r.logps)):
        assert torch.equal(a, b)
    want = TO.preference(v, labels, offsets, None if ref is None else ref.astype(np.float32), np.float64(np.float32(beta)),
                         np.float64(np.float32(smoothing)))
    live = labels >= 0
    tol = np.where(live, (V / 256 + 128) * 2.0 ** -24 + 2.0 ** -22 * np.abs(want["lse"]), 0.0)
    assert np.all(np.abs(values(r.lse) - want["lse"]) <= tol)
    at = np.abs(v[np.arange(T), np.maximum(labels, 0)])
    token = np.where(live, tol + 2.0 ** -23 * (at + np.abs(want["lse"])), 0.0)
    seq = np.array([token[a:b].sum() for a, b in zip(offsets, offsets[1:])])
    assert np.all(np.abs(values(r.logps) - want["logps"]) <= seq + 2.0 ** -23 * np.abs(want["logps"]))
    pairs = len(seq) // 2
    dz = abs(beta) * (seq[0::2] + seq[1::2])
    assert abs(r.loss.item() - want["loss"]) <= dz.mean() + 2.0 ** -22 * abs(want["loss"])
    dc = np.zeros(T)
    for s in range(2 * pairs):
        dc[offsets[s]:offsets[s + 1]] = abs(beta) / pairs * dz[s // 2] / 4
    dc = np.where(live, dc + 2.0 ** -22 * np.abs(want["coef"]), 0.0)
    assert np.all(np.abs(values(r.coef) - want["coef"]) <= dc)
    ref_grad = scale * want["grad"]
    p = np.zeros_like(v)
    p[live] = np.exp(v[live] - want["lse"][live, None])
    hit = np.zeros_like(v)
    hit[np.arange(T)[live], labels[live]] = 1.0
    far = np.where(p > 0, np.abs(np.where(p > 0, v, 0.0) - want["lse"][:, None]), 0.0)
    gtol = abs(scale) * (np.abs(want["coef"])[:, None] * p * (tol[:, None] + (8 + 4 * far) * 2.0 ** -23)
                         + dc[:, None] * (p + hit) + 2.0 ** -22 * np.abs(want["coef"])[:, None] * (p + hit))
    got = values(grad)
    assert_rounds_into(got, ref_grad, gtol + 2.0 ** -126, "grad", bf16=logits.dtype == torch.bfloat16)
    assert not got[~live].any()
    return r, grad


CASES = [([1, 1], 1), ([2, 3], 5), ([3, 1], 8), ([4, 0], 9), ([5, 7, 1, 2], 100), ([20, 13], 2048), ([3, 2], 8191),
         ([6, 9, 2, 4, 3, 3], 32000), ([40, 25], 50021), ([3, 4], 131072), ([300, 200, 1, 150, 2, 260], 777),
         ([1200, 900], 1000)]


@pytest.mark.parametrize("lens,V", CASES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_parity(Q, lens, V, dtype):
    say(f"preference {lens} V {V} {dtype}")
    logits, v, labels, offsets = packed(sum(lens) + V, lens, V, dtype)
    ref = np.random.default_rng(V).standard_normal(len(lens)) * 4 + TO.sequence_logps(v, labels, offsets)[0]
    check(Q, logits, v, labels, offsets, ref, 0.1, 0.05)


@pytest.mark.parametrize("beta,smoothing,scale,with_ref", [(0.1, 0.0, 1.0, True), (0.5, 0.2, -2.5, True), (2.0, 1.0, 1.0, False),
                                                           (0.0, 0.0, 1.0, True), (-0.3, 0.5, 0.0, False)])
def test_parameters(Q, beta, smoothing, scale, with_ref):
    say(f"preference beta {beta} e {smoothing} scale {scale} ref {with_ref}")
    lens = [7, 4, 9, 11]
    logits, v, labels, offsets = packed(5, lens, 3001, "fp32")
    ref = TO.sequence_logps(v, labels, offsets)[0] + np.array([1.0, -2.0, 0.5, 3.0]) if with_ref else None
    check(Q, logits, v, labels, offsets, ref, beta, smoothing, scale)


def test_nothing_scored(Q):
    say("preference nothing scored")
    logits, v, labels, offsets = packed(6, [5, 3, 0, 0], 640, "bf16", masked=1.0)
    r, grad = check(Q, logits, v, labels, offsets, None, 0.1, 0.0)
    assert abs(r.loss.item() - np.log(2.0)) < 1e-6 and not bool(grad.any())


def test_unscored_rows_are_not_read(Q):
    """A masked token's row may hold anything, and so may rows outside every sequence."""
    say("preference unscored rows")
    logits, v, labels, offsets = packed(7, [6, 5, 4, 5], 1000, "bf16")
    offsets = np.array([0, 6, 11, 15, 18], dtype=np.int32)  # the last two rows belong to none
    clean = Q.preference_fwd(logits, on_device(labels), on_device(offsets))
    grad = Q.preference_bwd(logits, on_device(labels), clean)
    labels2 = labels.copy()
    spoiled = logits.clone()
    spoiled[on_device(labels) < 0] = float("nan")
    r = Q.preference_fwd(spoiled, on_device(labels2), on_device(offsets))
    g = Q.preference_bwd(spoiled, on_device(labels2), r)
    assert torch.equal(r.loss, clean.loss) and torch.equal(g, grad)
    assert not bool(grad[18:].any()) and not bool(clean.coef[18:].any())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [37, 5000, 70000])
def test_masked_vocabulary(Q, dtype, V):
    """Logits of minus infinity, and of the type's lowest value, have probability 0."""
    say(f"preference masked vocabulary {V} {dtype}")
    logits, v, labels, offsets = packed(8, [3, 4], V, dtype, masked=0.0)
    labels = labels // 2  # the upper half is masked, all of a row's last chunk with it
    low = float(torch.finfo(logits.dtype).min)
    logits[:, V // 2 + 1:] = float("-inf")
    logits[2, V // 2 + 1:] = low
    v = values(logits)
    r, grad = check(Q, logits, v, labels, offsets, None, 0.1, 0.0)
    assert not bool(grad[:, V // 2 + 1:].any())


def test_not_finite_rows(Q):
    """A scored row with NaN, +inf or nothing finite, or a label past the vocabulary, makes its pair's loss NaN."""
    say("preference not finite")
    for spoil in ("nan", "inf", "none", "label"):
        logits, v, labels, offsets = packed(9, [3, 2, 4, 4], 500, "fp32", masked=0.0)
        if spoil == "nan":
            logits[1, 77] = float("nan")
        elif spoil == "inf":
            logits[1, 499] = float("inf")
        elif spoil == "none":
            logits[1] = float("-inf")
        else:
            labels[1] = 500
        r = Q.preference_fwd(logits, on_device(labels), on_device(offsets))
        g = Q.preference_bwd(logits, on_device(labels), r)
        assert bool(torch.isnan(r.loss)), spoil
        assert torch.isnan(r.logps).tolist() == [True, False, False, False], spoil
        assert bool(torch.isfinite(g[5:]).all()), spoil  # the other pair


def test_saturated_pairs(Q):
    """Margins far beyond what exp can hold: loss and gradient stay finite and right."""
    say("preference saturated")
    lens = [4, 4, 4, 4]
    logits, v, labels, offsets = packed(10, lens, 300, "fp32", masked=0.0)
    ref = np.array([-5000.0, 5000.0, 5000.0, -5000.0])
    r, g = check(Q, logits, v, labels, offsets, ref, 1.0, 0.1)
    assert bool(torch.isfinite(g).all())


def test_gradient_against_differences(Q):
    """Loss differences along random directions.  The loss is within 1e-5 (its log-probabilities of order 30 are
    within 1e-5 in fp32), over 2 h = 0.04: 5e-4; h^2 times a third derivative of order 1: 4e-4."""
    say("preference differences")
    lens, V, h = [5, 4, 6, 5], 400, 0.02
    logits, v, labels, offsets = packed(12, lens, V, "fp32")
    dl, do = on_device(labels), on_device(offsets)
    r = Q.preference_fwd(logits, dl, do, beta=0.5)
    g = values(Q.preference_bwd(logits, dl, r))
    for seed in range(3):
        d = torch.from_numpy(QI.normal_f32(90 + seed, v.shape, 1.0)).cuda()
        up = Q.preference_fwd(logits + h * d, dl, do, beta=0.5).loss.item()
        down = Q.preference_fwd(logits - h * d, dl, do, beta=0.5).loss.item()
        assert abs((up - down) / (2 * h) - (g * values(d)).sum()) <= 1e-3


def test_more_than_32_bits_of_logits(Q):
    say("preference 20000 x 131072")
    T, V = 20000, 131072  # 2.6e9 elements, 5.2e9 bytes
    rows = np.array([0, 9999, 16385, T - 1])
    small, v, labels, _ = packed(13, [2, 2], V, "bf16", masked=0.0)
    logits = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    all_labels = np.full(T, -1)
    for i, t in enumerate(rows):
        logits[t] = small[i]
        all_labels[t] = labels[i]
    offsets = np.array([0, 10000, T], dtype=np.int32)
    r = Q.preference_fwd(logits, on_device(all_labels), on_device(offsets))
    g = Q.preference_bwd(logits, on_device(all_labels), r, out=logits)  # in place
    want = TO.preference(v, labels, np.array([0, 2, 4]))
    assert abs(r.loss.item() - want["loss"]) <= 1e-4
    got = values(g[on_device(rows)])
    assert np.all(np.abs(got - want["grad"]) <= 2.0 ** -8 * np.abs(want["grad"]) + 1e-7)
    assert not bool(g[T - 2].any()) and not bool(g[9998].any())


def test_offsets_are_held_within_the_tokens(Q):
    """Offsets come from the device: values outside 0 .. T read nothing outside the tokens."""
    say("preference offsets")
    logits, v, labels, _ = packed(14, [6, 6], 100, "fp32", masked=0.0)
    odd = np.array([-5, 6, 400], dtype=np.int32)
    r = Q.preference_fwd(logits, on_device(labels), on_device(odd))
    s = Q.preference_fwd(logits, on_device(labels), on_device(np.array([0, 6, 12], dtype=np.int32)))
    assert torch.equal(r.loss, s.loss) and torch.equal(r.coef, s.coef)
    back = Q.sequence_logps(logits, on_device(labels), on_device(np.array([8, 3, 12], dtype=np.int32)))
    assert back[0].item() == 0.0


def test_other_stream_and_in_place(Q):
    say("preference side stream")
    logits, v, labels, offsets = packed(15, [30, 20, 25, 28], 4001, "bf16")
    dl, do = on_device(labels), on_device(offsets)
    r = Q.preference_fwd(logits, dl, do)
    g = Q.preference_bwd(logits, dl, r)
    side = torch.cuda.Stream()
    copy = logits.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r2 = Q.preference_fwd(copy, dl, do)
        g2 = Q.preference_bwd(copy, dl, r2, out=copy)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(r2.loss, r.loss) and torch.equal(g2, g) and g2.data_ptr() == copy.data_ptr()


def test_refusals(Q):
    logits = torch.zeros((6, 50), device="cuda")
    labels = torch.zeros(6, dtype=torch.int64, device="cuda")
    offsets = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        Q.preference_fwd(logits.half(), labels, offsets)
    with pytest.raises(TypeError):
        Q.preference_fwd(logits, labels.int(), offsets)
    with pytest.raises(TypeError):
        Q.preference_fwd(logits, labels, offsets.long())
    with pytest.raises(ValueError):
        Q.preference_fwd(logits, labels[:5].contiguous(), offsets)
    with pytest.raises(ValueError):
        Q.preference_fwd(logits, labels, offsets[:2].contiguous())  # one sequence is no pair
    with pytest.raises(ValueError):
        Q.preference_fwd(logits, labels, offsets, ref_logps=torch.zeros(3, device="cuda"))
    with pytest.raises(Q.QloraError):
        Q.preference_fwd(logits, labels, offsets, beta=float("inf"))
    with pytest.raises(Q.QloraError):
        Q.preference_fwd(logits, labels, offsets, label_smoothing=1.5)
    with pytest.raises(ValueError):
        Q.sequence_logps(logits, labels, offsets[:1].contiguous())
    r = Q.preference_fwd(logits, labels, offsets)
    with pytest.raises(Q.QloraError):
        Q.preference_bwd(logits, labels, r, grad_scale=float("nan"))
