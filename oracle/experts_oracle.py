"""Plain numpy oracle of the experts' layer and of the optimizer step over many tensors.

float64 throughout; shares no code with the library.

  experts_fwd / experts_bwd   the adapted layer over the rows of many experts
  moment8_values / moment8_pack   moments in 8 bits
  moment8_draws / moment8_pack_drawn   second moments in 8 bits with drawn codes
  grad_clip                   norm of all gradients and the factor that holds it to a maximum
  adamw_step                  the step of one tensor, moments given and returned in float64
"""

from __future__ import annotations

import numpy as np

from . import qlora_oracle as O

MOMENT_BLOCK = 128


def expert_rows(offsets, M: int):
    """(begin, end) of each expert's rows: offsets held within 0 .. M and below none before them."""
    end = min(max(int(offsets[0]), 0), M)
    out = []
    for o in offsets[1:]:
        begin, end = end, max(end, min(max(int(o), 0), M))
        out.append((begin, end))
    return out


def experts_fwd(x, offsets, W, A, B, s: float):
    """(h, u, rows): rows is True where a row belongs to an expert (the others are 0 in h and u).  W: E x m x n."""
    M = x.shape[0]
    h, u = np.zeros((M, W.shape[1])), np.zeros((M, A.shape[1]))
    rows = np.zeros(M, dtype=bool)
    for e, (a, b) in enumerate(expert_rows(offsets, M)):
        if b > a:
            h[a:b], u[a:b] = O.linear_fwd(x[a:b], W[e], A[e], B[e], s)
            rows[a:b] = True
    return h, u, rows


def experts_bwd(x, g, offsets, W, A, B, s: float, u):
    """grad_x (0 for rows of no expert), grad_A, grad_B (0 for experts without rows)."""
    gx, gA, gB = np.zeros_like(x), np.zeros_like(A), np.zeros_like(B)
    for e, (a, b) in enumerate(expert_rows(offsets, x.shape[0])):
        if b > a:
            out = O.linear_bwd(x[a:b], g[a:b], W[e], A[e], B[e], s, u=u[a:b])
            gx[a:b], gA[e], gB[e] = out["grad_x"], out["grad_A"], out["grad_B"]
    return gx, gA, gB


def moment8_values(codes, steps, signed: bool):
    """The values that an 8-bit moment stands for."""
    c = np.asarray(codes, dtype=np.int64)
    d = np.repeat(np.asarray(steps, dtype=np.float64), MOMENT_BLOCK)[:c.size]
    if signed:
        k = (c & 127).astype(np.float64)
        return np.where(c & 128, -1.0, 1.0) * k * k * d
    return (c.astype(np.float64) ** 2 * d) ** 2


def moment8_pack(values, signed: bool):
    """(codes, steps) of a moment, by trying every code of each block."""
    values = np.asarray(values, dtype=np.float64)
    most = 127 if signed else 255
    codes = np.zeros(values.size, dtype=np.uint8)
    steps = np.zeros(-(-values.size // MOMENT_BLOCK), dtype=np.float32)
    squares = np.arange(most + 1, dtype=np.float64) ** 2
    for b in range(steps.size):
        sl = slice(MOMENT_BLOCK * b, min(values.size, MOMENT_BLOCK * (b + 1)))
        x = np.abs(values[sl]) if signed else np.sqrt(values[sl])
        d = np.float32(x.max() / most ** 2)
        if d < np.float32(2.0 ** -126):
            continue
        steps[b] = d
        k = np.argmin(np.abs(x[:, None] - squares[None, :] * float(d)), axis=1)  # the first of two as near
        if signed:
            k = np.where((values[sl] < 0) & (k > 0), k + 128, k)
        else:
            k = np.where((values[sl] > 0) & (k == 0), 1, k)
        codes[sl] = k
    return codes, steps


def moment8_draws(seed: int, step: int, chunk: int, count: int):
    """The random words of a tensor of `count` elements that begins at chunk `chunk` of its plan."""
    group = (step * 2 ** 33 + 512 * chunk + np.arange(-(-count // 4)).astype(object)) % 2 ** 64
    group = group.astype(np.uint64)
    words = O.philox4x32_10_np(group & np.uint64(0xFFFFFFFF), group >> np.uint64(32),
                               (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    return np.stack(words, axis=1).reshape(-1)[:count]


def moment8_pack_drawn(values, words):
    """(codes, steps) of a second moment: of the two codes about a value the one that its word picks."""
    values = np.asarray(values, dtype=np.float64)
    codes = np.zeros(values.size, dtype=np.uint8)
    steps = np.zeros(-(-values.size // MOMENT_BLOCK), dtype=np.float32)
    for b in range(steps.size):
        sl = slice(MOMENT_BLOCK * b, min(values.size, MOMENT_BLOCK * (b + 1)))
        v = values[sl]
        d = np.float32(np.sqrt(v.max()) / 255 ** 2)
        if d < np.float32(2.0 ** -126):
            continue
        steps[b] = d
        table = (np.arange(258, dtype=np.float64) ** 2 * float(d)) ** 2
        k = np.searchsorted(table, v, side="right") - 1
        a, up = table[k], table[k + 1]
        k = k + (v - a > (up - a) * ((words[sl].astype(np.float64) + 0.5) / 2.0 ** 32))
        codes[sl] = np.where((v > 0) & (k == 0), 1, np.minimum(k, 255))
    return codes, steps


def grad_clip(grads, max_norm: float):
    """(norm, factor): the factor is NaN where the norm is not finite."""
    with np.errstate(over="ignore", invalid="ignore"):
        norm = np.sqrt(sum(float(np.sum(np.asarray(g, dtype=np.float64) ** 2)) for g in grads))
    return norm, min(1.0, max_norm / (norm + 1e-6)) if np.isfinite(norm) else float("nan")


def adamw_step(p, g, m, v, t: int, lr: float, beta1: float, beta2: float, eps: float, weight_decay: float,
               factor: float = 1.0):
    """(p, m, v) after step t, before any rounding."""
    g = np.asarray(g, dtype=np.float64) * factor
    return O.adam_step(p, g, m, v, t, lr, beta1, beta2, eps, weight_decay)
