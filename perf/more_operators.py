"""The products and the ends of a residual block in training, as cases to time and compare.

Operators: the linear layer in 8-bit floating point with a scale for each block of 128 ("linear": forward,
or the gradient of its input; "weights": the weight quantised in both orientations), the norms before and
after a block fused with its gate, its residual scale and its dropout ("block"), and dropout from a
counter-based generator ("dropout").

`run` computes a case in plain torch, or (own = True) through bit_quantized_shampoo_amd.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


# -- cases -----------------------------------------------------------------------------

def listed():
    return [
        # one new token through a 4096-wide layer: the weight's bytes and the launch count
        {"name": "linear_token", "op": "linear", "dtype": "bf16", "T": 1, "N": 4096, "K": 4096, "back": False},
        # a decoding step of 64 sequences through a layer that widens 1024 channels
        {"name": "linear_few", "op": "linear", "dtype": "bf16", "T": 64, "N": 4096, "K": 1024, "back": False},
        # the forward product of a [4096, 4096] layer over a 16384-token batch, the largest product
        {"name": "linear_large", "op": "linear", "dtype": "bf16", "T": 16384, "N": 4096, "K": 4096, "back": False},
        # the gradient of the input of a [4096, 1024] layer, added to that of its twin (a gated feed-forward)
        {"name": "linear_back", "op": "linear", "dtype": "bf16", "T": 8192, "N": 4096, "K": 1024, "back": True},
        # a small layer of odd sizes in float32 over a ragged batch
        {"name": "linear_ragged", "op": "linear", "dtype": "f32", "T": 777, "N": 577, "K": 1153, "back": False},
        # the master weight of a [4096, 4096] layer after an optimizer step, for both directions
        {"name": "weights_large", "op": "weights", "dtype": "f32", "N": 4096, "K": 4096},
        # a small float16 weight of odd sizes
        {"name": "weights_odd", "op": "weights", "dtype": "f16", "N": 577, "K": 1153},
        # between two blocks of a decoding step of eight sequences, the next product's operand kept
        {"name": "block_token", "op": "block", "dtype": "bf16", "T": 8, "C": 1024, "post": True, "gate": "channel",
         "p": 0.0, "rho": 1.0, "train": False, "keep8": True},
        # between two blocks of a 16384-token batch, forward and backward, with dropout
        {"name": "block_large", "op": "block", "dtype": "bf16", "T": 16384, "C": 4096, "post": True, "gate": "channel",
         "p": 0.1, "rho": 1.0, "train": True, "keep8": False},
        # float32, an odd width, a gate for every token and a scaled residual, without a norm behind the block
        {"name": "block_ragged", "op": "block", "dtype": "f32", "T": 1000, "C": 2309, "post": False, "gate": "token",
         "p": 0.0, "rho": 0.7071, "train": True, "keep8": False},
        # dropout behind the embedding of a 16-token micro-batch: only the launches count
        {"name": "dropout_small", "op": "dropout", "dtype": "bf16", "T": 16, "C": 1024, "p": 0.1},
        # a 16384-token batch of a 4096-wide layer, forward and backward
        {"name": "dropout_large", "op": "dropout", "dtype": "bf16", "T": 16384, "C": 4096, "p": 0.1},
    ]


def _size(rng, lo, hi):
    """A size in [lo, hi], spread over its logarithm; one in three a multiple of 64 where that fits."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    v = min(max(v, lo), hi)
    if rng.random() < 1 / 3 and v >= max(lo, 64):
        v = v // 64 * 64
    return v


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "weights", "block", "block", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    b = BYTES[dtype] // 2
    c = {"op": op, "dtype": dtype}
    if op == "linear":
        c["T"] = _size(rng, 1, 16384 // b)
        c["N"] = _size(rng, 16, 4096)
        c["K"] = _size(rng, 16, 4096)
        c["back"] = rng.random() < 0.4
    elif op == "weights":
        c["N"] = _size(rng, 16, 4096)
        c["K"] = _size(rng, 16, 4096)
    elif op == "block":
        c["T"] = _size(rng, 1, 16384 // b)
        c["C"] = _size(rng, 16, 4096)
        c["train"] = rng.random() < 0.7
        c.update(post=rng.random() < 0.6, gate=rng.choice(["none", "channel", "token"]),
                 p=rng.choice([0.0, 0.05, 0.3]) if c["train"] else 0.0, rho=rng.choice([1.0, 1.0, 0.7071]),
                 keep8=rng.random() < 0.3)
    else:
        c["T"] = _size(rng, 1, 16384 // b)
        c["C"] = _size(rng, 16, 4096)
        c["p"] = rng.choice([0.02, 0.1, 0.5])
    return c


def work(case):
    """Bytes and operations that a pass cannot do without: inputs read once, outputs written once."""
    op, b = case["op"], BYTES[case["dtype"]]
    if op == "linear":
        t, n, k = case["T"], case["N"], case["K"]
        ends = t * (2 * k + n) if case["back"] else t * (n + k)      # the added gradient is read and written
        return {"bytes": ends * b + n * k, "flops": 2 * t * n * k}
    if op == "weights":
        n = case["N"] * case["K"]
        return {"bytes": n * (b + 2) + 2 * n * (1 + 2), "flops": 4 * n}      # quantised twice, both read back
    n = case["T"] * case["C"]
    if op == "dropout":
        return {"bytes": 4 * n * b, "flops": 4 * n}
    token = 1 if case["gate"] == "token" else 0
    size = n * b * (4 + token) + n * (2 + b if case["keep8"] else 0)
    if case["train"]:
        size += n * b * (6 + 2 * token)
    return {"bytes": size, "flops": (40 if case["train"] else 12) * n}


# -- inputs ----------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _activations(g, t, c):
    """Normal values with a scale per channel: a few channels are far larger than the others."""
    return _randn(g, t, c) * torch.exp(_randn(g, 1, c))


def prepare(case, seed):
    g, dt, op = _gen(seed), TYPES[case["dtype"]], case["op"]
    s = {"case": case}
    if op in ("linear", "weights"):
        n, k = case["N"], case["K"]
        w = _randn(g, n, k) * torch.exp(0.3 * _randn(g, n, 1)) / math.sqrt(k)
    if op == "linear":
        # the weight as the optimizer step left it: codes and scale bytes, for one direction
        if case["back"]:
            s["codes"], s["scales"] = _encode(w.t(), 128)
            s["x"] = (1e-3 * _randn(g, case["T"], n) * torch.exp(_randn(g, case["T"], 1))).to(dt)
            s["dx"] = (1e-3 * _randn(g, case["T"], k)).to(dt)
        else:
            s["codes"], s["scales"] = _encode(w, 128)
            s["x"] = _activations(g, case["T"], k).to(dt)
    elif op == "weights":
        s["w"] = w.to(dt)
    else:
        t, c = case["T"], case["C"]
        s["seed"], s["offset"] = seed, 3
        if op == "dropout":
            s["x"], s["dy"] = _activations(g, t, c).to(dt), (1e-3 * _randn(g, t, c)).to(dt)
        else:
            s["x"] = (3.0 * _activations(g, t, c)).to(dt)
            s["h"] = _activations(g, t, c).to(dt)
            s["weight"] = 1.0 + 0.2 * _randn(g, c)
            s["post"] = 0.5 + 0.1 * _randn(g, c) if case["post"] else None
            s["gate"] = {"none": lambda: None, "channel": lambda: 0.5 + 0.2 * _randn(g, c),
                         "token": lambda: torch.tanh(_randn(g, t, c)).to(dt)}[case["gate"]]()
            s["dy"], s["dres"] = (1e-3 * _randn(g, t, c)).to(dt), (1e-3 * _randn(g, t, c)).to(dt)
    return s


# -- plain forms -----------------------------------------------------------------------

def _encode(x, rows):
    """[T, C] float -> codes e4m3 [T, P], scale exponents uint8 [T / rows up, S] (P: C up to 128s, S: P / 128 up to 4s).

    A block is `rows` rows of 128 columns; its scale is the smallest power of two that brings its largest value to
    at most 448, at least 2^-126."""
    t, c = x.shape
    up, p = (t + rows - 1) // rows * rows, (c + 127) // 128 * 128
    w = torch.zeros((up, p), device=x.device, dtype=torch.float32)
    w[:t, :c] = x.float()
    w = w.view(up // rows, rows, p // 128, 128)
    bits = w.abs().amax((1, 3)).view(torch.int32)
    e = (((bits + 0x1FFFFF) >> 23) - 8).clamp(min=1)
    v = w * ((254 - e) << 23).view(torch.float32)[:, None, :, None]
    # three bits behind the leading one, in steps of 2^-9 below 2^-6
    step = ((((v.abs().view(torch.int32) >> 23).clamp(min=121)) - 3) << 23).view(torch.float32)
    codes = (torch.round(v / step) * step).to(torch.float8_e4m3fn).view(up, p)[:t]
    scales = torch.ones((up // rows, (p + 511) // 512 * 4), device=x.device, dtype=torch.uint8)
    scales[:, :p // 128] = e.to(torch.uint8)
    return codes.contiguous(), scales


def _decode(codes, scales, rows, c):
    """float32 [T, c] of codes and scales."""
    t, p = codes.shape
    s = (scales[:, :p // 128].int() << 23).view(torch.float32).repeat_interleave(rows, 0)[:t]
    return (codes.float().view(t, p // 128, 128) * s[:, :, None]).view(t, p)[:, :c]


def _kept(seed, offset, t, c, p):
    """[t, c] truth values: which elements dropout keeps.

    Element (row, col) takes 16 bits of the ten-round Philox 4 x 32 generator with the key (seed low, high) and the
    counter (col / 8, row, offset low, high): the low half of word (col % 8) / 2 where col is even, else the high
    one.  It is kept unless they are below p, as a multiple of 2^-16."""
    m = 0xFFFFFFFF
    x0 = torch.arange((c + 7) // 8, device=DEV, dtype=torch.int64)[None, :].expand(t, -1)
    x1 = torch.arange(t, device=DEV, dtype=torch.int64)[:, None].expand_as(x0)
    x2, x3 = torch.full_like(x0, offset & m), torch.full_like(x0, offset >> 32)
    k0, k1 = seed & m, (seed >> 32) & m
    for _ in range(10):
        a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57          # 64-bit products, whatever their sign
        x0, x1, x2, x3 = ((b >> 32) & m) ^ x1 ^ k0, b & m, ((a >> 32) & m) ^ x3 ^ k1, a & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    words = torch.stack([x0, x1, x2, x3], -1)
    bits = torch.stack([words & 0xFFFF, words >> 16], -1).reshape(t, -1)[:, :c]
    return bits >= round(p * 65536)


def _keep_scale(p):
    return 65536.0 / (65536 - round(p * 65536))


def _plain_block(s):
    case = s["case"]
    t, c, dt, p = case["T"], case["C"], s["x"].dtype, case["p"]
    h = s["h"].float()
    one = torch.ones((), device=DEV)
    hh, post, gate = h, one, one
    if case["post"]:
        h_rstd = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
        hh, post = h * h_rstd, s["post"]
    if s["gate"] is not None:
        gate = s["gate"].float()
    drop = _kept(s["seed"], s["offset"], t, c, p).float() * _keep_scale(p) if p > 0 else one
    z = drop * (hh * post)
    x = (case["rho"] * s["x"].float() + gate * z).to(dt)
    xf = x.float()
    rstd = 1.0 / torch.sqrt((xf * xf).mean(1, keepdim=True) + EPS)
    xh = xf * rstd
    y = (xh * s["weight"]).to(dt)
    out = {"x": x, "y": y}
    if case["keep8"]:
        out["y8"] = _decode(*_encode(y, 1), 1, c).to(torch.bfloat16)
    if not case["train"]:
        return out
    dy = s["dy"].float()
    out["dweight"] = (dy * xh).sum(0)
    ty = dy * s["weight"]
    gx = s["dres"].float() + rstd * (ty - xh * (ty * xh).mean(1, keepdim=True))
    out["dx"] = (case["rho"] * gx).to(dt)
    if case["gate"] == "channel":
        out["dgate"] = (gx * z).sum(0)
    elif case["gate"] == "token":
        out["dgate"] = (gx * z).to(dt)
    dn = drop * (gx * gate)
    if case["post"]:
        out["dpost"] = (dn * hh).sum(0)
        u = dn * post
        dn = h_rstd * (u - hh * (u * hh).mean(1, keepdim=True))
    out["dh"] = dn.to(dt)
    return out


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "linear":
        inner, outer = (case["N"], case["K"]) if case["back"] else (case["K"], case["N"])
        x = _decode(*_encode(s["x"], 1), 1, inner)
        w = _decode(s["codes"], s["scales"], 128, inner)
        y = torch.matmul(x, w.t())
        if case["back"]:
            return {"dx": s["dx"].copy_(s["dx"].float() + y)}
        return {"y": y.to(s["x"].dtype)}
    if op == "weights":
        w, wt = _encode(s["w"], 128), _encode(s["w"].t(), 128)
        return {"w": _decode(*w, 128, case["K"]).to(torch.bfloat16),
                "wt": _decode(*wt, 128, case["N"]).to(torch.bfloat16)}
    if op == "block":
        return _plain_block(s)
    keep = _kept(s["seed"], s["offset"], case["T"], case["C"], case["p"])
    zero, scale = torch.zeros((), device=DEV), _keep_scale(case["p"])
    return {k: torch.where(keep, s[v].float() * scale, zero).to(s[v].dtype) for k, v in (("y", "x"), ("dx", "dy"))}


# -- the framework's operators -----------------------------------------------------------

def _own(s):
    import bit_quantized_shampoo_amd as s4
    case, op = s["case"], s["case"]["op"]
    if op == "linear":
        inner, outer = (case["N"], case["K"]) if case["back"] else (case["K"], case["N"])
        w8 = s4.Fp8(s["codes"], s["scales"], outer, inner, 128)
        if case["back"]:
            return {"dx": s4.fp8_linear(s["x"], w8, out=s["dx"], accumulate=True)}
        return {"y": s4.fp8_linear(s["x"], w8)}
    if op == "weights":
        w8, wt8 = s4.fp8_store_weight(s["w"], transposed=True)
        return {"w": s4.fp8_load(w8, dtype=torch.bfloat16), "wt": s4.fp8_load(wt8, dtype=torch.bfloat16)}
    drop = {"p": case["p"], "seed": s["seed"], "offset": s["offset"]}
    if op == "dropout":
        return {"y": s4.dropout(s["x"], **drop), "dx": s4.dropout(s["dy"], **drop)}
    x, y, y8, stats = s4.block_norm_forward(s["x"], s["weight"], s["h"], post_weight=s["post"], gate=s["gate"],
                                            residual_scale=case["rho"], eps=EPS, save8=case["keep8"], **drop)
    out = {"x": x, "y": y}
    if case["keep8"]:
        out["y8"] = s4.fp8_load(y8, dtype=torch.bfloat16)
    if not case["train"]:
        return out
    dx, dh, dweight, dpost, dgate = s4.block_norm_backward(s["dy"], s["dres"], x, s["weight"], stats, h=s["h"],
                                                           post_weight=s["post"], gate=s["gate"],
                                                           residual_scale=case["rho"], **drop)
    out.update(dx=dx, dh=dh, dweight=dweight)
    if dpost is not None:
        out["dpost"] = dpost
    if dgate is not None:
        out["dgate"] = dgate
    return out


def run(state):
    return _own(state) if own else _plain(state)


# -- the definitions in 64 bits ----------------------------------------------------------

def _blocks64(x, rows):
    """Values of x in e4m3 with a scale for each block of `rows` x 128, from the definition, in float64."""
    t, c = x.shape
    out = torch.empty((t, c), device=x.device, dtype=torch.float64)
    limit = max(1, (1 << 26) // max(1, c) // rows) * rows
    for r0 in range(0, t, limit):
        part = x[r0:r0 + limit].double()
        n = part.shape[0]
        w = torch.nn.functional.pad(part, (0, -c % 128, 0, -n % rows))
        w = w.view(-1, rows, (c + 127) // 128, 128)
        m, k = torch.frexp(w.abs().amax((1, 3), keepdim=True))
        # amax = m 2^k with m in [1/2, 1): m 2^9 <= 448, or else one power of two more
        k = k.double() - 9 + (m * 512 > 448).double()
        scale = torch.exp2(torch.where(m > 0, k, torch.full_like(k, -126.0)).clamp(min=-126.0))
        v = w / scale
        # e4m3: multiples of 2^(j - 4) for |v| in [2^(j - 1), 2^j), and of 2^-9 where that is finer
        unit = torch.exp2((torch.frexp(v)[1].double() - 4).clamp(min=-9.0))
        v = torch.round(v / unit) * unit * scale
        out[r0:r0 + limit] = v.reshape(-1, (c + 127) // 128 * 128)[:n, :c]
    return out


def _kept64(seed, offset, t, c, p):
    """_kept, with the products taken from 16-bit halves."""
    def product(x, const):
        xl, xh, cl, ch = x & 0xFFFF, x >> 16, const & 0xFFFF, const >> 16
        low, mid = xl * cl, xh * cl + ((xl * cl) >> 16)
        mid2 = xl * ch + (mid & 0xFFFF)
        return xh * ch + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | (low & 0xFFFF)

    cols, rows = torch.arange((c + 7) // 8, device=DEV), torch.arange(t, device=DEV)
    ctr = [cols.repeat(t), rows.repeat_interleave(len(cols)), torch.full((t * len(cols),), offset % 2 ** 32, device=DEV),
           torch.full((t * len(cols),), offset // 2 ** 32, device=DEV)]
    for r in range(10):
        key = [(seed % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32]
        hi0, lo0 = product(ctr[0], 0xD2511F53)
        hi1, lo1 = product(ctr[2], 0xCD9E8D57)
        ctr = [hi1 ^ ctr[1] ^ key[0], lo1, hi0 ^ ctr[3] ^ key[1], lo0]
    keep = torch.empty((t, len(cols), 8), device=DEV, dtype=torch.bool)
    for j in range(8):
        keep[:, :, j] = ((ctr[j // 2] // (65536 if j % 2 else 1)) % 65536 >= round(p * 65536)).view(t, -1)
    return keep.view(t, -1)[:, :c]


def _block64(s):
    case = s["case"]
    t, c, dt = case["T"], case["C"], s["x"].dtype
    outs = {"x": [], "y": [], "y8": [], "dx": [], "dh": [], "dgate": []}
    sums = {k: torch.zeros(c, device=DEV, dtype=torch.float64) for k in ("dweight", "dpost", "dgate")}
    keep = _kept64(s["seed"], s["offset"], t, c, case["p"]) if case["p"] > 0 else None
    one = torch.ones(c, device=DEV, dtype=torch.float64)
    w = s["weight"].double()
    post = s["post"].double() if case["post"] else one
    for r0 in range(0, t, 2048):
        row = slice(r0, r0 + 2048)
        h = s["h"][row].double()
        gate = one if case["gate"] == "none" else s["gate"].double() if case["gate"] == "channel" else s["gate"][row].double()
        hr = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) if case["post"] else torch.ones((), device=DEV).double()
        d = keep[row].double() * _keep_scale(case["p"]) if keep is not None else one
        z = h * hr * post * d
        x = case["rho"] * s["x"][row].double() + gate * z
        outs["x"].append(x)
        x = x.to(dt).double()                         # the norm reads what was written
        r = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
        y = x * r * w
        outs["y"].append(y)
        if case["keep8"]:
            outs["y8"].append(_blocks64(y.to(dt), 1))
        if not case["train"]:
            continue
        dy = s["dy"][row].double()
        sums["dweight"] += (dy * x * r).sum(0)
        back = r * w * dy - x * r ** 3 * (w * dy * x).mean(1, keepdim=True)
        gx = s["dres"][row].double() + back
        outs["dx"].append(case["rho"] * gx)
        if case["gate"] == "channel":
            sums["dgate"] += (gx * z).sum(0)
        elif case["gate"] == "token":
            outs["dgate"].append(gx * z)
        dn = gx * gate * d
        if case["post"]:
            sums["dpost"] += (dn * h * hr).sum(0)
            dn = hr * post * dn - h * hr ** 3 * (post * dn * h).mean(1, keepdim=True)
        outs["dh"].append(dn)
    out = {k: torch.cat(v) for k, v in outs.items() if v}
    if case["train"]:
        out["dweight"] = sums["dweight"]
        if case["post"]:
            out["dpost"] = sums["dpost"]
        if case["gate"] == "channel":
            out["dgate"] = sums["dgate"]
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "linear":
        inner = case["N"] if case["back"] else case["K"]
        scale = torch.exp2(s["scales"].double() - 127.0)[:, :s["codes"].shape[1] // 128]
        w = s["codes"].to(torch.float64).unflatten(1, (-1, 128))
        rows = torch.arange(len(w), device=DEV) // 128
        w = (w * scale[rows][:, :, None]).flatten(1)[:, :inner]
        y = torch.matmul(_blocks64(s["x"], 1), w.t().contiguous())
        return {"dx": s["dx"].double() + y} if case["back"] else {"y": y}
    if op == "weights":
        return {"w": _blocks64(s["w"], 128), "wt": _blocks64(s["w"].t(), 128)}
    if op == "block":
        return _block64(s)
    keep = _kept64(s["seed"], s["offset"], case["T"], case["C"], case["p"])
    scale = _keep_scale(case["p"])
    return {k: torch.where(keep, s[v].double() * scale, 0.0) for k, v in (("y", "x"), ("dx", "dy"))}
