"""The training operators that feed the 4-bit Shampoo step, as cases to time and compare.

Operators: activation checkpoints in 8 bits ("store": written and read back; "act": a gated or
plain activation whose backward pass reads its input from the checkpoint; "wgrad": the weight
gradient of a linear layer whose input is checkpointed), the embedding table ("lookup" and
"embgrad") and the clipped policy loss ("policy"; "logp" is its forward-only form).

`run` computes a case in plain torch, or (own = True) through bit_quantized_shampoo_amd.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
CLIP_LOW, CLIP_HIGH, KL = 0.2, 0.28, 0.04


# -- cases -----------------------------------------------------------------------------

def listed():
    return [
        # one micro-batch of 16 tokens of a 1024-wide layer: only the launches count
        {"name": "store_small", "op": "store", "dtype": "bf16", "T": 16, "C": 1024},
        # a 16384-token batch's input of a 4096-wide layer, the largest checkpoint
        {"name": "store_large", "op": "store", "dtype": "bf16", "T": 16384, "C": 4096},
        # the gated feed-forward activation of an 8192-token batch, forward and backward
        {"name": "act_large", "op": "act", "dtype": "bf16", "T": 8192, "C": 4096, "kind": "silu", "gated": True,
         "save": False},
        # float32 training with a plain activation, a ragged batch and an odd width, the output kept too
        {"name": "act_ragged", "op": "act", "dtype": "f32", "T": 1000, "C": 2309, "kind": "gelu", "gated": False,
         "save": True},
        # the weight gradient of a [4096, 4096] layer over a 16384-token batch, the largest product
        {"name": "wgrad_large", "op": "wgrad", "dtype": "bf16", "T": 16384, "N": 4096, "C": 4096,
         "accumulate": False},
        # a small ragged layer in float32, added to a gradient that is already there
        {"name": "wgrad_ragged", "op": "wgrad", "dtype": "f32", "T": 777, "N": 512, "C": 1153, "accumulate": True},
        # the first layer of a decoding step of eight sequences
        {"name": "lookup_small", "op": "lookup", "dtype": "bf16", "T": 8, "V": 32768, "D": 1024},
        # the embedding gradient of a 16384-token batch with a natural token distribution
        {"name": "embgrad_large", "op": "embgrad", "dtype": "bf16", "T": 16384, "V": 65536, "D": 1024,
         "accumulate": False},
        # a short float32 batch over a small odd table, added to a gradient that is already there
        {"name": "embgrad_odd", "op": "embgrad", "dtype": "f32", "T": 1000, "V": 5003, "D": 577, "accumulate": True},
        # the policy step of 4096 response tokens over a 65536-word vocabulary
        {"name": "policy_large", "op": "policy", "dtype": "bf16", "T": 4096, "V": 65536},
        # few rows of an odd vocabulary in float32: rows have to be split to fill the card
        {"name": "policy_few", "op": "policy", "dtype": "f32", "T": 8, "V": 40961},
        # scoring the last 16 tokens of a rollout under the old policy
        {"name": "logp_few", "op": "logp", "dtype": "bf16", "T": 16, "V": 131072},
    ]


def _size(rng, lo, hi):
    """A size in [lo, hi], spread over its logarithm; one in three a multiple of 64 where that fits."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    v = min(max(v, lo), hi)
    if rng.random() < 1 / 3 and v >= max(lo, 64):
        v = v // 64 * 64
    return v


def draw(rng):
    op = rng.choice(["store", "act", "wgrad", "lookup", "embgrad", "policy", "logp"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    b = BYTES[dtype] // 2
    c = {"op": op, "dtype": dtype}
    if op in ("store", "act"):
        c["T"] = _size(rng, 1, (16384 if op == "store" else 8192) // b)
        c["C"] = _size(rng, 16, 4096)
        if op == "act":
            c.update(kind=rng.choice(["silu", "gelu"]), gated=rng.random() < 0.6, save=rng.random() < 0.4)
    elif op == "wgrad":
        # float16 and float32 gradients take two and three matrix-core products per element
        c["T"] = _size(rng, 1, 16384 // {"bf16": 1, "f16": 2, "f32": 3}[dtype])
        c["N"] = _size(rng, 16, 4096)
        c["C"] = _size(rng, 16, 4096)
        c["accumulate"] = rng.random() < 0.4
    elif op in ("lookup", "embgrad"):
        c["T"] = _size(rng, 1, 16384 // b)
        c["V"] = _size(rng, 16, 65536)
        c["D"] = _size(rng, 16, 1024)
        if op == "embgrad":
            c["accumulate"] = rng.random() < 0.4
    else:
        c["V"] = _size(rng, 64, 131072)
        c["T"] = _size(rng, 1, min(8192, 4096 * 65536 // (c["V"] * b)))
    return c


def work(case):
    """Bytes and operations that a pass cannot do without: inputs read once, outputs written once."""
    op, b = case["op"], BYTES[case["dtype"]]
    t = case["T"]
    q = 1 + 1 / 32                       # bytes of a checkpointed value
    if op == "store":
        n = t * case["C"]
        return {"bytes": n * (b + q + q + b), "flops": 4 * n}
    if op == "act":
        n, k = t * case["C"], 2 if case["gated"] else 1
        fwd = k * b + b + k * q + (2 * q + b if case["save"] else 0)
        return {"bytes": n * (fwd + b + k * q + k * b), "flops": 30 * n}
    if op == "wgrad":
        n, c = case["N"], case["C"]
        return {"bytes": t * n * b + t * c * q + n * c * 4 * (2 if case["accumulate"] else 1), "flops": 2 * t * n * c}
    if op == "lookup":
        return {"bytes": t * (8 + 2 * b * case["D"]), "flops": t * case["D"]}
    if op == "embgrad":
        rows = 2 * min(t, case["V"]) if case["accumulate"] else case["V"]
        return {"bytes": t * (8 + b * case["D"]) + 4 * case["D"] * rows, "flops": t * case["D"]}
    n = t * case["V"]
    if op == "policy":
        return {"bytes": 2 * b * n + 32 * t, "flops": 8 * n}
    return {"bytes": b * n + 16 * t, "flops": 4 * n}


# -- inputs ----------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _activations(g, t, c):
    """Normal values with a scale per channel: a few channels are far larger than the others."""
    return _randn(g, t, c) * torch.exp(_randn(g, 1, c))


def _tokens(g, t, v):
    """Token ids whose frequency falls as 1 / rank (ranks in a shuffled order); one in 32 is padding (-1)."""
    u = torch.rand(t, generator=g, device=DEV, dtype=torch.float64)
    rank = (torch.exp(u * math.log(v + 1.0)) - 1.0).long().clamp_(0, v - 1)
    ids = torch.randperm(v, generator=g, device=DEV)[rank]
    pad = torch.rand(t, generator=g, device=DEV) < 1 / 32
    return torch.where(pad, torch.full_like(ids, -1), ids)


def prepare(case, seed):
    g, dt, op, t = _gen(seed), TYPES[case["dtype"]], case["op"], case["T"]
    s = {"case": case}
    if op == "store":
        s["x"] = _activations(g, t, case["C"]).to(dt)
    elif op == "act":
        s["gate"] = (1.5 * _activations(g, t, case["C"])).to(dt)
        s["up"] = _activations(g, t, case["C"]).to(dt) if case["gated"] else None
        s["dh"] = _randn(g, t, case["C"]).to(dt)
    elif op == "wgrad":
        # the layer's input as the forward pass left it: codes and scale bytes, 32 tokens a block
        s["codes"], s["scales"] = _encode(_activations(g, t, case["C"]))
        s["dy"] = (1e-3 * _randn(g, t, case["N"])).to(dt)
        s["grad"] = 1e-2 * _randn(g, case["N"], case["C"]) if case["accumulate"] else None
    elif op == "lookup":
        s["table"] = _randn(g, case["V"], case["D"]).to(dt)
        s["ids"] = _tokens(g, t, case["V"])
        s["scale"] = math.sqrt(case["D"])
    elif op == "embgrad":
        s["ids"] = _tokens(g, t, case["V"])
        s["dout"] = (1e-3 * _randn(g, t, case["D"])).to(dt)
        s["scale"] = math.sqrt(case["D"])
        s["grad"] = 1e-3 * _randn(g, case["V"], case["D"]) if case["accumulate"] else None
    else:
        v = case["V"]
        z = torch.empty((t, v), device=DEV, dtype=dt)
        for r0 in range(0, t, 512):
            z[r0:r0 + 512] = 2.0 * _randn(g, min(512, t - r0), v)
        y = torch.randint(0, v, (t,), generator=g, device=DEV)
        rows = torch.arange(t, device=DEV)
        # a sampled token is mostly a likely one
        z[rows, y] = (z[rows, y].float() + 8.0 * torch.rand(t, generator=g, device=DEV)).to(dt)
        s["logits"], s["targets"] = z, y
        if op == "policy":
            logp = torch.empty(t, device=DEV)
            for r0 in range(0, t, 512):
                zf = z[r0:r0 + 512].float()
                logp[r0:r0 + 512] = zf.gather(1, y[r0:r0 + 512, None])[:, 0] - torch.logsumexp(zf, 1)
            s["old"] = logp + 0.2 * _randn(g, t)
            s["ref"] = logp + 0.3 * _randn(g, t)
            # one advantage for each response, of 64 tokens
            s["adv"] = _randn(g, (t + 63) // 64).repeat_interleave(64)[:t].contiguous()
            keep = torch.rand(t, generator=g, device=DEV) > 0.1          # prompt and padding tokens do not count
            keep[0] = True
            s["weights"] = keep.float() / keep.sum()
    return s


# -- plain forms -----------------------------------------------------------------------

def _encode(x):
    """[T, C] float -> codes int8 [T32, P], scale exponents uint8 [T32 / 32, P] (T32: T up to 32s, P: C up to 16s).

    A block is 32 tokens of one channel; its scale is the smallest power of two that brings its largest value to at
    most 127, at least 2^-126."""
    t, c = x.shape
    t32, p = (t + 31) // 32 * 32, (c + 15) // 16 * 16
    w = torch.zeros((t32, p), device=x.device, dtype=torch.float32)
    w[:t, :c] = x.float()
    w = w.view(t32 // 32, 32, p)
    amax = w.abs().amax(1)
    bits = amax.view(torch.int32)
    e = (((bits + 0x1FFFF) >> 23) - 6).clamp(min=1)
    inv = ((254 - e) << 23).view(torch.float32)
    codes = torch.round(w * inv[:, None]).clamp(-127, 127)
    return codes.to(torch.int8).view(t32, p), e.to(torch.uint8)


def _decode(codes, scales, t, c):
    """float32 [t, c] of a checkpoint."""
    s = (scales.int() << 23).view(torch.float32)
    x = codes.view(scales.shape[0], 32, -1).float() * s[:, None]
    return x.view(codes.shape[0], -1)[:t, :c]


def _act(x, kind):
    """The activation and its derivative."""
    if kind == "silu":
        z, dz = x, 1.0
    else:
        k = math.sqrt(2.0 / math.pi)
        z = 2.0 * k * (x + 0.044715 * x * x * x)
        dz = 2.0 * k * (1.0 + 3 * 0.044715 * x * x)
    sig = 1.0 / (1.0 + torch.exp(-z))
    return x * sig, sig + x * sig * (1.0 - sig) * dz


def _plain_act(s):
    case = s["case"]
    dt, t, c = s["gate"].dtype, case["T"], case["C"]
    g = s["gate"].float()
    h = _act(g, case["kind"])[0]
    if s["up"] is not None:
        h = h * s["up"].float()
    h = h.to(dt)
    a, da = _act(_decode(*_encode(g), t, c), case["kind"])
    dh = s["dh"].float()
    out = {"h": h}
    if s["up"] is not None:
        u = _decode(*_encode(s["up"]), t, c)
        out["dup"] = (dh * a).to(dt)
        dh = dh * u
    out["dgate"] = (dh * da).to(dt)
    if case["save"]:
        out["h8"] = _decode(*_encode(h), t, c).to(torch.bfloat16)
    return out


def _plain_policy(s):
    z, y = s["logits"].float(), s["targets"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    logp = (z.gather(1, y[:, None]) - m - torch.log(total))[:, 0]
    if s["case"]["op"] == "logp":
        return {"logp": logp}
    w, adv = s["weights"], s["adv"]
    keep = w != 0
    r = torch.exp(logp - s["old"])
    plain = r * adv
    clipped = r.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * adv
    d = s["ref"] - logp
    ed = torch.exp(d)
    zero = torch.zeros_like(w)
    loss = torch.where(keep, w * (KL * (ed - d - 1.0) - torch.minimum(plain, clipped)), zero).sum()
    coef = torch.where(keep, w * (KL * (1.0 - ed) - torch.where(plain <= clipped, plain, zero)), zero)
    grad = e.mul_(-coef[:, None] / total)
    grad.scatter_add_(1, y[:, None], coef[:, None])
    return {"loss": loss, "logp": torch.where(keep, logp, zero), "dlogits": grad.to(s["logits"].dtype)}


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "store":
        return {"x": _decode(*_encode(s["x"]), case["T"], case["C"]).to(s["x"].dtype)}
    if op == "act":
        return _plain_act(s)
    if op == "wgrad":
        x = _decode(s["codes"], s["scales"], case["T"], case["C"])
        grad = torch.matmul(s["dy"].float().t(), x)
        return {"grad": grad if s["grad"] is None else s["grad"].add_(grad)}
    if op == "lookup":
        ids = s["ids"]
        keep = (ids >= 0) & (ids < case["V"])
        rows = s["table"][torch.where(keep, ids, torch.zeros_like(ids))].float() * s["scale"]
        return {"out": torch.where(keep[:, None], rows, torch.zeros_like(rows)).to(s["table"].dtype)}
    if op == "embgrad":
        ids = s["ids"]
        keep = (ids >= 0) & (ids < case["V"])
        rows = s["dout"].float() * s["scale"] * keep[:, None]
        grad = s["grad"]
        if grad is None:
            grad = torch.zeros((case["V"], case["D"]), device=DEV, dtype=torch.float32)
        return {"grad": grad.index_add_(0, torch.where(keep, ids, torch.zeros_like(ids)), rows)}
    return _plain_policy(s)


# -- the framework's operators -----------------------------------------------------------

def _own(s):
    import bit_quantized_shampoo_amd as s4
    case, op = s["case"], s["case"]["op"]
    if op == "store":
        return {"x": s4.act8_load(s4.act8_store(s["x"]), dtype=s["x"].dtype)}
    if op == "act":
        h, gate8, up8, h8 = s4.activation_forward(s["gate"], s["up"], kind=case["kind"], save_output=case["save"])
        dgate, dup = s4.activation_backward(s["dh"], gate8, up8, kind=case["kind"])
        out = {"h": h, "dgate": dgate}
        if dup is not None:
            out["dup"] = dup
        if h8 is not None:
            out["h8"] = s4.act8_load(h8, dtype=torch.bfloat16)
        return out
    if op == "wgrad":
        x8 = s4.Act8(s["codes"], s["scales"], case["T"], case["C"])
        return {"grad": s4.act8_weight_grad(s["dy"], x8, out=s["grad"], beta=0.0 if s["grad"] is None else 1.0)}
    if op == "lookup":
        return {"out": s4.embedding(s["table"], s["ids"], scale=s["scale"])}
    if op == "embgrad":
        return {"grad": s4.embedding_grad(s["dout"], s["ids"], case["V"], scale=s["scale"], out=s["grad"],
                                          accumulate=s["grad"] is not None)}
    if op == "logp":
        return {"logp": s4.token_logprobs(s["logits"], s["targets"])}
    loss, logp, dlogits = s4.policy_loss(s["logits"], s["targets"], s["old"], s["adv"], s["weights"], ref_logp=s["ref"],
                                         clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=KL)
    return {"loss": loss, "logp": logp, "dlogits": dlogits}


def run(state):
    return _own(state) if own else _plain(state)


# -- the definitions in 64 bits ----------------------------------------------------------

def _checkpoint64(x):
    """Values of the 8-bit checkpoint of x, from the definition, in float64."""
    t, c = x.shape
    out = torch.empty((t, c), device=x.device, dtype=torch.float64)
    limit = max(1, (1 << 27) // max(1, c) // 32) * 32
    for r0 in range(0, t, limit):
        w = torch.nn.functional.pad(x[r0:r0 + limit].double(), (0, 0, 0, -min(limit, t - r0) % 32))
        w = w.view(-1, 32, c)
        amax = w.abs().amax(1, keepdim=True)
        # amax = m 2^k with m in [1/2, 1): m 2^7 <= 127, or else one power of two more
        m, k = torch.frexp(amax)
        k = k.double() - 7 + (m * 128 > 127).double()
        step = torch.exp2(torch.where(amax > 0, k, torch.full_like(k, -126.0)).clamp(min=-126.0))
        out[r0:r0 + limit] = (torch.round(w / step) * step).view(-1, c)[:min(limit, t - r0)]
    return out


def _act64(x, kind):
    if kind == "silu":
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    k = math.sqrt(2 / math.pi)
    th = torch.tanh(k * (x + 0.044715 * x ** 3))
    return 0.5 * x * (1 + th), 0.5 * (1 + th) + 0.5 * x * (1 - th ** 2) * k * (1 + 3 * 0.044715 * x ** 2)


def _policy64(s):
    z, y = s["logits"], s["targets"]
    t = z.shape[0]
    loss = torch.zeros((), device=DEV, dtype=torch.float64)
    logp = torch.zeros(t, device=DEV, dtype=torch.float64)
    train = s["case"]["op"] == "policy"
    grad = torch.zeros(z.shape, device=DEV, dtype=torch.float64) if train else None
    for r0 in range(0, t, 256):
        row = slice(r0, r0 + 256)
        lp = torch.log_softmax(z[row].double(), 1)
        at = torch.arange(lp.shape[0], device=DEV)
        own_lp = lp[at, y[row]]
        if not train:
            logp[row] = own_lp
            continue
        w, a = s["weights"][row].double(), s["adv"][row].double()
        on = (w != 0).double()
        logp[row] = own_lp * on
        r = torch.exp(own_lp - s["old"][row].double())
        lo, hi = 1.0 - CLIP_LOW, 1.0 + CLIP_HIGH
        gain = torch.where(a >= 0, torch.minimum(r, torch.full_like(r, hi)), torch.maximum(r, torch.full_like(r, lo)))
        d = s["ref"][row].double() - own_lp
        loss += (w * (KL * (torch.expm1(d) - d) - gain * a)).sum()
        inside = torch.where(a >= 0, r <= hi, r >= lo).double()
        coef = w * (-KL * torch.expm1(d) - a * r * inside)
        grad[row] = -coef[:, None] * torch.exp(lp)
        grad[row].view(-1)[at * z.shape[1] + y[row]] += coef
    return {"loss": loss, "logp": logp, "dlogits": grad} if train else {"logp": logp}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "store":
        return {"x": _checkpoint64(s["x"])}
    if op == "act":
        gate = s["gate"].double()
        up = None if s["up"] is None else s["up"].double()
        h = _act64(gate, case["kind"])[0] * (1 if up is None else up)
        a, da = _act64(_checkpoint64(s["gate"]), case["kind"])
        dh = s["dh"].double()
        out = {"h": h, "dgate": dh * da}
        if up is not None:
            out["dgate"] = out["dgate"] * _checkpoint64(s["up"])
            out["dup"] = dh * a
        if case["save"]:
            out["h8"] = _checkpoint64(h.to(s["gate"].dtype))
        return out
    if op == "wgrad":
        x = s["codes"].double().view(-1, 32, s["codes"].shape[1])
        x = (x * torch.exp2(s["scales"].double() - 127.0)[:, None]).view(-1, x.shape[2])[:case["T"], :case["C"]]
        grad = torch.matmul(s["dy"].double().t().contiguous(), x.contiguous())
        return {"grad": grad if s["grad"] is None else grad + s["grad"].double()}
    if op in ("lookup", "embgrad"):
        ids, v = s["ids"], case["V"]
        t = torch.nonzero((ids >= 0) & (ids < v))[:, 0]
        if op == "lookup":
            out = torch.zeros((case["T"], case["D"]), device=DEV, dtype=torch.float64)
            out[t] = s["table"].double()[ids[t]] * s["scale"]
            return {"out": out}
        grad = torch.zeros((v, case["D"]), device=DEV, dtype=torch.float64) if s["grad"] is None else s["grad"].double()
        return {"grad": grad.index_add(0, ids[t], s["dout"].double()[t] * s["scale"])}
    return _policy64(s)
