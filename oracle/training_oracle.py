"""Plain numpy oracle of the operators next to the adapted linear layer.

float64 throughout (the 8-bit checkpoint is exact integer and power-of-two
arithmetic); shares no code with the library.

  checkpoint_pack / checkpoint_unpack   the 8-bit activation checkpoint
  norm_fwd / norm_bwd                   layer norm and RMS norm
  sequence_logps / preference           packed sequences' log-probabilities,
                                        the paired log-ratio loss, its gradient
"""

from __future__ import annotations

import numpy as np

CKPT_BLOCK = 32


def checkpoint_pitch(n: int) -> int:
    return 4 * (-(-n // 128))


def checkpoint_pack(bits: np.ndarray):
    """(codes int8 [M, n], scales uint8 [M, pitch]) of bf16 bits [M, n], block by block."""
    M, n = bits.shape
    codes = np.zeros((M, n), dtype=np.int8)
    scales = np.zeros((M, checkpoint_pitch(n)), dtype=np.uint8)
    values = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    for b in range(-(-n // CKPT_BLOCK)):
        sl = slice(CKPT_BLOCK * b, min(n, CKPT_BLOCK * (b + 1)))
        field = ((bits[:, sl] >> 7) & 0xFF).max(axis=1).astype(np.int64)
        bad = field == 255
        c = np.where(bad, 255, np.maximum(field, 7) - 6)
        scales[:, b] = c
        with np.errstate(invalid="ignore", over="ignore"):
            k = np.rint(values[:, sl] * np.exp2(127.0 - c)[:, None])  # numpy rounds half to even
            k = np.clip(k, -127, 127)
        codes[:, sl] = np.where(bad[:, None], 0, k).astype(np.int8)
    return codes, scales


def checkpoint_unpack(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values of a checkpoint (NaN where a block was not finite)."""
    n = codes.shape[1]
    c = np.repeat(scales.astype(np.float64), CKPT_BLOCK, axis=1)[:, :n]
    return np.where(c == 255, np.nan, codes.astype(np.float64) * np.exp2(c - 127.0))


def norm_fwd(x, w, b=None, eps=1e-5, layer=True):
    """(y, mean, rstd); mean is zeros for the RMS norm."""
    x = np.asarray(x, dtype=np.float64)
    n = x.shape[1]
    mean = x.sum(axis=1) / n if layer else np.zeros(x.shape[0])
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).sum(axis=1) / n + eps)
    y = d * rstd[:, None] * w
    return (y if b is None else y + b), mean, rstd


def norm_bwd(x, g, w, mean, rstd, layer=True):
    """(grad_x, grad_w, grad_b) with the forward's mean and rstd as given."""
    x, g = np.asarray(x, dtype=np.float64), np.asarray(g, dtype=np.float64)
    n = x.shape[1]
    xh = (x - mean[:, None]) * rstd[:, None]
    d = g * w
    p = (d * xh).sum(axis=1, keepdims=True) / n
    q = d.sum(axis=1, keepdims=True) / n if layer else 0.0
    return rstd[:, None] * (d - q - xh * p), (g * xh).sum(axis=0), g.sum(axis=0)


def log_sum_exp(rows):
    rows = np.asarray(rows, dtype=np.float64)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        m = rows.max(axis=1, keepdims=True)
        base = np.where(np.isfinite(m), m, 0.0)
        return (base + np.log(np.exp(rows - base).sum(axis=1, keepdims=True)))[:, 0]


def sequence_logps(logits, labels, offsets):
    """(logps [sequences], lse [T], lp [T]); unscored tokens have lp 0."""
    logits = np.asarray(logits, dtype=np.float64)
    T = logits.shape[0]
    lse, lp = np.zeros(T), np.zeros(T)
    live = np.flatnonzero(labels >= 0)
    lse[live] = log_sum_exp(logits[live]) if live.size else 0.0
    lp[live] = logits[live, labels[live]] - lse[live]
    logps = np.array([lp[a:b].sum() for a, b in zip(offsets, offsets[1:])])
    return logps, lse, lp


def _log_sigmoid(z):
    return -(np.maximum(-z, 0.0) + np.log1p(np.exp(-np.abs(z))))


def preference(logits, labels, offsets, ref=None, beta=0.1, smoothing=0.0):
    """dict(loss, logps, lse, coef, grad) of the paired log-ratio loss."""
    logits = np.asarray(logits, dtype=np.float64)
    logps, lse, _ = sequence_logps(logits, labels, offsets)
    pairs = (len(offsets) - 1) // 2
    ratio = logps - (0.0 if ref is None else np.asarray(ref, dtype=np.float64))
    z = beta * (ratio[0::2] - ratio[1::2])
    e = smoothing
    loss = np.mean(-(1 - e) * _log_sigmoid(z) - e * _log_sigmoid(-z))
    slope = beta / pairs * (e * np.exp(_log_sigmoid(z)) - (1 - e) * np.exp(_log_sigmoid(-z)))
    coef = np.zeros(len(labels))
    for s in range(2 * pairs):
        sl = slice(offsets[s], offsets[s + 1])
        coef[sl] = np.where(labels[sl] >= 0, slope[s // 2] * (1 if s % 2 == 0 else -1), 0.0)
    grad = np.zeros_like(logits)
    for t in np.flatnonzero(coef != 0):
        grad[t] = -coef[t] * np.exp(logits[t] - lse[t])
        grad[t, labels[t]] += coef[t]
    return dict(loss=loss, logps=logps, lse=lse, coef=coef, grad=grad)
