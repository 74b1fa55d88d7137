"""Oracle of the training operators: the definitions in float64 NumPy, written for reading
and not for speed.  Shares no code with the GPU path.

* the 8-bit checkpoint: blocks of 32 rows of one column, scale the smallest power of two
  2^k >= 2^-126 with max |x| <= 127 * 2^k, codes x / 2^k rounded to nearest even;
* activations: silu(x) = x sigmoid(x); gelu in its tanh form;
* the weight gradient dY^T X, the embedding and its gradient;
* the clipped policy loss with the KL estimate exp(d) - d - 1, d = ref - logp.
"""

from __future__ import annotations

import numpy as np

BLOCK, PITCH = 32, 16
K_GELU = np.sqrt(2.0 / np.pi)


def act8_scale_exponent(amax: float) -> int:
    """k of the block's scale 2^k, by search."""
    if amax == 0.0:
        return -126
    k = int(np.floor(np.log2(amax))) - 9
    while amax > 127.0 * 2.0 ** k:
        k += 1
    return max(k, -126)


def act8_store(x):
    """(codes int8 [R, P], exponents uint8 [R / 32, P]) of a float matrix."""
    x = np.asarray(x, np.float64)
    t, c = x.shape
    rows, pitch = -(-t // BLOCK) * BLOCK, -(-c // PITCH) * PITCH
    codes = np.zeros((rows, pitch), np.int8)
    scales = np.ones((rows // BLOCK, pitch), np.uint8)
    for b in range(rows // BLOCK):
        blk = x[b * BLOCK:(b + 1) * BLOCK]
        for j in range(c):
            col = blk[:, j]
            if not np.all(np.isfinite(col)):
                scales[b, j] = 255
                continue
            k = act8_scale_exponent(float(np.max(np.abs(col))))
            top = 63 if 64.0 * 2.0 ** k >= 2.0 ** 128 else 127
            scales[b, j] = k + 127
            codes[b * BLOCK:b * BLOCK + len(col), j] = np.clip(np.rint(col / 2.0 ** k), -top, top)
    return codes, scales


def act8_load(codes, scales, t, c):
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127.0))
    return (codes.astype(np.float64).reshape(len(scales), BLOCK, -1) * s[:, None]).reshape(codes.shape)[:t, :c]


def act_argument(x, kind):
    """z with a(x) = x / (1 + exp(-z)), and dz/dx."""
    if kind == "silu":
        return x, np.ones_like(x)
    return 2 * K_GELU * (x + 0.044715 * x ** 3), 2 * K_GELU * (1 + 3 * 0.044715 * x ** 2)


def activation(x, kind):
    z, _ = act_argument(np.asarray(x, np.float64), kind)
    with np.errstate(over="ignore"):
        return x / (1 + np.exp(-z))


def activation_derivative(x, kind):
    x = np.asarray(x, np.float64)
    z, dz = act_argument(x, kind)
    with np.errstate(over="ignore"):
        sg = 1 / (1 + np.exp(-z))
    return sg + x * sg * (1 - sg) * dz


def embedding(table, ids, scale):
    out = np.zeros((len(ids), table.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < table.shape[0]:
            out[t] = scale * np.asarray(table[v], np.float64)
    return out


def embedding_grad(dout, ids, vocab, scale):
    g = np.zeros((vocab, dout.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < vocab:
            g[v] += scale * np.asarray(dout[t], np.float64)
    return g


def log_softmax(z):
    z = np.asarray(z, np.float64)
    m = np.max(z, axis=1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        return z - m - np.log(np.sum(np.exp(z - m), axis=1, keepdims=True))


def policy(z, y, old, adv, w, ref=None, clip_low=0.2, clip_high=0.2, kl=0.0):
    """Loss, log-probabilities, gradient, and per row the size of the terms the gradient's
    coefficient is made of (for error bounds).  Rows with w = 0 or a target outside the
    vocabulary count for nothing."""
    z = np.asarray(z, np.float64)
    rows, vocab = z.shape
    loss, logp, dz, size = 0.0, np.zeros(rows), np.zeros((rows, vocab)), np.zeros(rows)
    for t in range(rows):
        if w[t] == 0 or not 0 <= y[t] < vocab:
            continue
        lp = log_softmax(z[t:t + 1])[0]
        logp[t] = lp[y[t]]
        r = np.exp(lp[y[t]] - float(old[t]))
        a = float(adv[t])
        plain, clipped = r * a, float(np.clip(r, 1 - clip_low, 1 + clip_high)) * a
        l = -min(plain, clipped)
        g = -plain if plain <= clipped else 0.0
        size[t] = abs(plain)
        if kl > 0:
            d = float(ref[t]) - lp[y[t]]
            l += kl * (np.exp(d) - d - 1)
            g += kl * (1 - np.exp(d))
            size[t] += kl * (1 + np.exp(d) + abs(d))
        size[t] *= abs(float(w[t]))
        loss += float(w[t]) * l
        p = np.exp(lp)
        dz[t] = -float(w[t]) * g * p
        dz[t, y[t]] += float(w[t]) * g
    return loss, logp, dz, size
