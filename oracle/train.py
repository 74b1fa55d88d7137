"""Oracle of the training operators: the definitions in float64 NumPy, written for reading
and not for speed.  Shares no code with the GPU path.

* the 8-bit checkpoint: blocks of 32 rows of one column, scale the smallest power of two
  2^k >= 2^-126 with max |x| <= 127 * 2^k, codes x / 2^k rounded to nearest even;
* activations: silu(x) = x sigmoid(x); gelu in its tanh form;
* the weight gradient dY^T X, the embedding and its gradient;
* the clipped policy loss with the KL estimate exp(d) - d - 1, d = ref - logp;
* e4m3 with a scale for each block of 128 columns, scale the smallest power of two 2^k >= 2^-126
  with max |x| <= 448 * 2^k, codes the nearest of the e4m3 numbers, ties to the even code;
* dropout by the Philox 4 x 32 generator of ten rounds;
* the norms, gate, residual sum and dropout at the ends of a block, and their gradients.
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


def e4m3_numbers():
    """The 127 numbers of codes 0 .. 126, in order (code 127 is NaN)."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.astype(np.float64) - 7))


def e4m3_code(v):
    """The nearest number's code, by search among all of them; ties to the even code."""
    numbers = e4m3_numbers()
    a = np.abs(v)
    hi = np.minimum(np.searchsorted(numbers, a), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - numbers[lo], numbers[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.signbit(v), code + 128, code).astype(np.uint8)


def e4m3_value(codes):
    numbers = np.concatenate([e4m3_numbers(), [np.nan]])
    return np.where(codes >= 128, -1.0, 1.0) * numbers[codes & 127]


def fp8_scale_exponent(amax: float) -> int:
    if amax == 0.0:
        return -126
    k = int(np.floor(np.log2(amax))) - 11
    while amax > 448.0 * 2.0 ** k:
        k += 1
    return max(k, -126)


def fp8_store(x, block_rows=1):
    """(codes uint8 [rows, P], exponents uint8 [rows / block_rows, S]) of a float matrix."""
    x = np.asarray(x, np.float64)
    t, c = x.shape
    pitch, sp = -(-c // 128) * 128, -(-c // 512) * 4
    codes = np.zeros((t, pitch), np.uint8)
    scales = np.ones((-(-t // block_rows), sp), np.uint8)
    for b in range(len(scales)):
        for j in range(pitch // 128):
            rows, cols = slice(b * block_rows, (b + 1) * block_rows), slice(j * 128, min(c, (j + 1) * 128))
            blk = x[rows, cols]
            if not np.all(np.isfinite(blk)):
                scales[b, j] = 255
                continue
            k = fp8_scale_exponent(float(np.max(np.abs(blk))))
            scales[b, j] = k + 127
            top = 240 if 256.0 * 2.0 ** k >= 2.0 ** 128 else 448
            codes[rows, cols] = e4m3_code(np.clip(blk / 2.0 ** k, -top, top))
    return codes, scales


def fp8_load(codes, scales, c, block_rows=1):
    t, pitch = codes.shape
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127.0))[:, :pitch // 128]
    s = np.repeat(np.repeat(s, block_rows, 0)[:t], 128, 1)
    return (e4m3_value(codes) * s)[:, :c]


def philox(counter, key):
    """Ten rounds of Philox 4 x 32 on one counter (four words) with one key (two words), in Python's
    integers."""
    x, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * x[0], 0xCD9E8D57 * x[2]
        x = [(b >> 32) ^ x[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ x[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return x


def dropout_keep(rows, cols, p, seed, call, row0=0, col0=0):
    """[rows, cols] booleans, of the elements from (row0, col0) on (col0 a multiple of 8)."""
    seed, call = seed % 2 ** 64, call % 2 ** 64
    keep = np.zeros((rows, -(-cols // 8) * 8), bool)
    for t in range(rows):
        for q in range(keep.shape[1] // 8):
            w = philox([col0 // 8 + q, row0 + t, call % 2 ** 32, call >> 32], [seed % 2 ** 32, seed >> 32])
            bits = [(w[j // 2] >> (16 * (j % 2))) & 0xFFFF for j in range(8)]
            keep[t, 8 * q:8 * q + 8] = np.array(bits) >= np.rint(p * 65536)
    return keep[:, :cols]


def dropout_scale(p):
    return 65536.0 / (65536.0 - np.rint(p * 65536))


def rstd(v, eps):
    """1 / sqrt(mean v^2 + eps) per row."""
    return 1 / np.sqrt(np.mean(np.square(np.asarray(v, np.float64)), axis=1, keepdims=True) + eps)


def block_end(x, h, post, gate, drop, rho, eps):
    """x' in float64.  post, gate, drop: arrays that broadcast, or None (drop: keep times its scale)."""
    z = np.asarray(h, np.float64)
    if post is not None:
        z = z * rstd(z, eps) * post
    if drop is not None:
        z = np.where(drop > 0, z, 0.0) * drop
    return rho * np.asarray(x, np.float64) + (1.0 if gate is None else gate) * z


def block_backward(dy, dres, x, weight, h, post, gate, drop, rho, eps):
    """Gradients by the formulas, and the sizes of the terms that each is made of (for error bounds):
    dictionaries of dx, dh, dweight, dpost, dgate (dgate by element; a vector gate's is its sum over
    rows)."""
    x = np.asarray(x, np.float64)
    out, size = {}, {}
    g = np.zeros_like(x) if dres is None else np.asarray(dres, np.float64)
    sg = np.abs(g)
    if weight is not None:
        r = rstd(x, eps)
        xh, t = x * r, dy * weight
        g = g + r * (t - xh * np.mean(t * xh, 1, keepdims=True))
        sg = sg + r * (np.abs(t) + np.abs(xh) * np.mean(np.abs(t * xh), 1, keepdims=True))
        out["dweight"], size["dweight"] = np.sum(dy * xh, 0), np.sum(np.abs(dy * xh), 0)
    out["dx"], size["dx"] = rho * g, abs(rho) * sg
    if h is None:
        return out, size
    h = np.asarray(h, np.float64)
    hr = rstd(h, eps) if post is not None else 1.0
    hh, p = h * hr, 1.0 if post is None else post
    d = np.ones_like(x) if drop is None else drop
    z = np.where(d > 0, hh * p, 0.0) * d
    out["dgate"], size["dgate"] = g * z, sg * np.abs(z)
    gt = 1.0 if gate is None else gate
    dn, sn = d * g * gt, d * sg * np.abs(gt)
    out["dpost"], size["dpost"] = np.sum(dn * hh, 0), np.sum(sn * np.abs(hh), 0)
    if post is None:
        out["dh"], size["dh"] = dn, sn
    else:
        u, su = dn * p, sn * np.abs(p)
        out["dh"] = hr * (u - hh * np.mean(u * hh, 1, keepdims=True))
        size["dh"] = hr * (su + np.abs(hh) * np.mean(su * np.abs(hh), 1, keepdims=True))
    return out, size
