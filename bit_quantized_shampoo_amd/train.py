"""Thin PyTorch-facing binding of the training operators (include/shampoo4_train.h): what
produces the gradients that the 4-bit Shampoo step reads.

Argument marshalling only, as in shampoo4.py: PyTorch provides device memory and streams,
every computation is a kernel of libshampoo4.so, and nothing falls back to the CPU.

Shapes are those of the tensors given; matrices may be strided views with unit column
stride.  Element types are float32, bfloat16 and float16.  Work is enqueued on `stream`
(default: the current stream), and tensors that a call allocates (outputs not passed in,
workspaces) belong to that stream, so the caching allocator reuses them in its order.
Inputs used on another stream than their own are the caller's to order, and to keep, as
with any PyTorch operator.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib as L

_DTYPES = {torch.float32: L.F32, torch.bfloat16: L.BF16, torch.float16: L.F16}
_KINDS = {"silu": L.ACT_SILU, "gelu": L.ACT_GELU}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}


class _On:
    """The device and stream of a call: allocations inside belong to the stream."""

    __slots__ = ("ptr", "_dev", "_stream")

    def __init__(self, device, stream):
        self._dev = torch.cuda.device(device) if device.index != torch.cuda.current_device() else None
        self._stream = torch.cuda.stream(stream) if stream is not None else None
        self.ptr = (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream

    def __enter__(self):
        if self._dev is not None:
            self._dev.__enter__()
        if self._stream is not None:
            self._stream.__enter__()
        return self.ptr

    def __exit__(self, *exc):
        if self._stream is not None:
            self._stream.__exit__(*exc)
        if self._dev is not None:
            self._dev.__exit__(*exc)


def _tensor(t, what: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA (HIP) tensor")


def _matrix(t, what: str, dtype=None, shape=None, device=None) -> int:
    """Checks a row-major matrix and returns its leading dimension."""
    _tensor(t, what)
    if dtype is None:
        if t.dtype not in _DTYPES:
            raise TypeError(f"{what} must be float32, bfloat16 or float16, got {t.dtype}")
    elif t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != shape):
        raise ValueError(f"{what} must have shape {shape or '[rows, cols]'}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{what} must be on {device}, got {t.device}")
    rows, cols = t.shape
    if cols < 1:
        raise ValueError(f"{what} needs at least one column")
    if rows == 0:
        return cols
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{what} must be row-major (unit column stride)")
    if rows > 1 and s0 < cols:
        raise ValueError(f"{what} must not have overlapping or broadcast rows")
    return s0 if rows > 1 else cols


def _vector(t, n: int, what: str, dtype, device):
    _tensor(t, what)
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous vector of {n}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}, got {t.device}")
    return t.data_ptr()


def _ids(t, n: int, what: str, device) -> int:
    _tensor(t, what)
    if t.dtype not in _ID_BYTES:
        raise TypeError(f"{what} must be int32 or int64, got {t.dtype}")
    return _vector(t, n, what, t.dtype, device)


def _workspace(ws, need: int, device):
    """(tensor or None, pointer, bytes): the caller's workspace if it is large enough."""
    if need == 0:
        return None, 0, 0
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        _tensor(ws, "workspace")
        if ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.numel() < need or ws.device != device:
            raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {need} bytes on {device}")
    return ws, ws.data_ptr(), ws.numel()


# -- 8-bit activation checkpoints --------------------------------------------------------

@dataclass
class Act8:
    """The 8-bit checkpoint of a [rows, cols] matrix: `codes` int8 [R, P] and `scales`
    uint8 [R / 32, P] (R: rows up to a multiple of 32, P: cols up to one of 16), the value
    of element (t, c) being codes[t, c] * 2 ** (scales[t // 32, c] - 127)."""

    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int

    @staticmethod
    def padded(rows: int, cols: int):
        return ((rows + L.ACT8_ROWS - 1) // L.ACT8_ROWS * L.ACT8_ROWS,
                (cols + L.ACT8_PITCH - 1) // L.ACT8_PITCH * L.ACT8_PITCH)

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda") -> "Act8":
        r, p = cls.padded(rows, cols)
        return cls(torch.empty((r, p), dtype=torch.int8, device=device),
                   torch.empty((r // L.ACT8_ROWS, p), dtype=torch.uint8, device=device), rows, cols)

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def _act8(a, what: str, shape=None, device=None):
    """Checks a checkpoint and returns its two pointers."""
    if not isinstance(a, Act8):
        raise TypeError(f"{what} must be an Act8")
    if shape is not None and (a.rows, a.cols) != shape:
        raise ValueError(f"{what} must hold {shape}, got {(a.rows, a.cols)}")
    r, p = Act8.padded(a.rows, a.cols)
    for t, dtype, want, nm in ((a.codes, torch.int8, (r, p), "codes"),
                               (a.scales, torch.uint8, (r // L.ACT8_ROWS, p), "scales")):
        _tensor(t, f"{what}.{nm}")
        if t.dtype != dtype or tuple(t.shape) != want or not t.is_contiguous():
            raise ValueError(f"{what}.{nm} must be a contiguous {dtype} tensor of shape {want}")
        if device is not None and t.device != device:
            raise ValueError(f"{what}.{nm} must be on {device}, got {t.device}")
    return a.codes.data_ptr(), a.scales.data_ptr()


def act8_store(x: torch.Tensor, out: Act8 | None = None, stream=None) -> Act8:
    """The 8-bit checkpoint of x."""
    ld = _matrix(x, "x")
    rows, cols = x.shape
    with _On(x.device, stream) as s:
        if out is None:
            out = Act8.empty(rows, cols, x.device)
        c, e = _act8(out, "out", (rows, cols), x.device)
        L.check(L.lib().shampoo4_act8_store(_DTYPES[x.dtype], rows, cols, x.data_ptr(), ld, c, e, s),
                "shampoo4_act8_store")
    return out


def act8_load(a: Act8, dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of a checkpoint, in `dtype` (or in `out`, of its own type)."""
    c, e = _act8(a, "a")
    device = a.codes.device
    with _On(device, stream) as s:
        if out is None:
            if dtype not in _DTYPES:
                raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
            out = torch.empty((a.rows, a.cols), dtype=dtype, device=device)
        ld = _matrix(out, "out", shape=(a.rows, a.cols), device=device)
        L.check(L.lib().shampoo4_act8_load(_DTYPES[out.dtype], a.rows, a.cols, c, e, out.data_ptr(), ld, s),
                "shampoo4_act8_load")
    return out


def activation_forward(gate: torch.Tensor, up: torch.Tensor | None = None, kind: str = "silu", checkpoint: bool = True,
                       save_output: bool = True, out: torch.Tensor | None = None, stream=None):
    """h = a(gate) * up (a(gate) without `up`), with the 8-bit checkpoints that training keeps.

    Returns (h, gate8, up8, h8): gate8 and up8 for activation_backward (None with
    checkpoint=False, as in inference), h8 for act8_weight_grad of the layer that reads h
    (None with save_output=False).  kind: "silu" or "gelu" (tanh form)."""
    if kind not in _KINDS:
        raise ValueError(f"kind must be one of {sorted(_KINDS)}, not {kind!r}")
    ldg = _matrix(gate, "gate")
    rows, cols = shape = tuple(gate.shape)
    dev = gate.device
    ldu = _matrix(up, "up", gate.dtype, shape, dev) if up is not None else 0
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty(shape, dtype=gate.dtype, device=dev)
        ldh = _matrix(out, "out", gate.dtype, shape, dev)
        g8 = Act8.empty(rows, cols, dev) if checkpoint else None
        u8 = Act8.empty(rows, cols, dev) if checkpoint and up is not None else None
        h8 = Act8.empty(rows, cols, dev) if save_output else None
        ptr = [p for a in (g8, u8, h8) for p in ((a.codes.data_ptr(), a.scales.data_ptr()) if a is not None else (0, 0))]
        L.check(L.lib().shampoo4_activation_forward(
            _KINDS[kind], _DTYPES[gate.dtype], rows, cols, gate.data_ptr(), ldg,
            up.data_ptr() if up is not None else 0, ldu, out.data_ptr(), ldh, *ptr, s), "shampoo4_activation_forward")
    return out, g8, u8, h8


def activation_backward(dh: torch.Tensor, gate8: Act8, up8: Act8 | None = None, kind: str = "silu",
                        dgate: torch.Tensor | None = None, dup: torch.Tensor | None = None, stream=None):
    """(dgate, dup) of activation_forward from its checkpoints (dup None without up8).  `dgate`
    may be dh."""
    if kind not in _KINDS:
        raise ValueError(f"kind must be one of {sorted(_KINDS)}, not {kind!r}")
    ldd = _matrix(dh, "dh")
    rows, cols = shape = tuple(dh.shape)
    dev = dh.device
    gc, ge = _act8(gate8, "gate8", shape, dev)
    uc, ue = _act8(up8, "up8", shape, dev) if up8 is not None else (0, 0)
    if up8 is None and dup is not None:
        raise ValueError("dup needs up8")
    with _On(dev, stream) as s:
        if dgate is None:
            dgate = torch.empty(shape, dtype=dh.dtype, device=dev)
        ldg = _matrix(dgate, "dgate", dh.dtype, shape, dev)
        ldu = 0
        if up8 is not None:
            if dup is None:
                dup = torch.empty(shape, dtype=dh.dtype, device=dev)
            ldu = _matrix(dup, "dup", dh.dtype, shape, dev)
        L.check(L.lib().shampoo4_activation_backward(
            _KINDS[kind], _DTYPES[dh.dtype], rows, cols, dh.data_ptr(), ldd, gc, ge, uc, ue, dgate.data_ptr(), ldg,
            dup.data_ptr() if dup is not None else 0, ldu, s), "shampoo4_activation_backward")
    return dgate, dup


def act8_weight_grad(dy: torch.Tensor, x8: Act8, out: torch.Tensor | None = None, alpha: float = 1.0,
                     beta: float = 0.0, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """alpha dy^T x^ + beta out, float32 [dy columns, x columns]: the weight gradient of
    y = x W^T from the checkpoint of x, as Shampoo4Blocks.step takes it."""
    ldd = _matrix(dy, "dy")
    rows, n = dy.shape
    dev = dy.device
    c, e = _act8(x8, "x8", (rows, x8.cols) if isinstance(x8, Act8) else None, dev)
    if out is None and beta != 0.0:
        raise ValueError("beta needs out")
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty((n, x8.cols), dtype=torch.float32, device=dev)
        ldo = _matrix(out, "out", torch.float32, (n, x8.cols), dev)
        lib = L.lib()
        ws, wp, wb = _workspace(workspace, lib.shampoo4_act8_weight_grad_workspace_bytes(rows, n, x8.cols), dev)
        L.check(lib.shampoo4_act8_weight_grad(_DTYPES[dy.dtype], rows, n, x8.cols, alpha, dy.data_ptr(), ldd, c, e,
                                              beta, out.data_ptr(), ldo, wp, wb, s), "shampoo4_act8_weight_grad")
    return out


# -- embedding -----------------------------------------------------------------------------

def embedding(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """scale * table[ids] ([tokens, dim], the table's type); an id outside the table, as -1
    for padding, gives a row of zeros."""
    ldt = _matrix(table, "table")
    vocab, dim = table.shape
    dev = table.device
    n = ids.numel() if isinstance(ids, torch.Tensor) else 0
    ip = _ids(ids, n, "ids", dev)
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty((n, dim), dtype=table.dtype, device=dev)
        ldo = _matrix(out, "out", table.dtype, (n, dim), dev)
        L.check(L.lib().shampoo4_embedding(_DTYPES[table.dtype], _ID_BYTES[ids.dtype], n, vocab, dim, table.data_ptr(),
                                           ldt, ip, scale, out.data_ptr(), ldo, s), "shampoo4_embedding")
    return out


def embedding_grad(dout: torch.Tensor, ids: torch.Tensor, num_embeddings: int, scale: float = 1.0,
                   out: torch.Tensor | None = None, accumulate: bool = False, workspace: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """The table's gradient in float32 [num_embeddings, dim], rows summed in the order of their
    tokens.  accumulate=True adds to `out` and touches only the rows of tokens that occur."""
    ldd = _matrix(dout, "dout")
    n, dim = dout.shape
    dev = dout.device
    ip = _ids(ids, n, "ids", dev)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty((num_embeddings, dim), dtype=torch.float32, device=dev)
        ldo = _matrix(out, "out", torch.float32, (num_embeddings, dim), dev)
        lib = L.lib()
        ws, wp, wb = _workspace(workspace, lib.shampoo4_embedding_grad_workspace_bytes(n, num_embeddings, dim), dev)
        L.check(lib.shampoo4_embedding_grad(_DTYPES[dout.dtype], _ID_BYTES[ids.dtype], n, num_embeddings, dim,
                                            dout.data_ptr(), ldd, ip, scale, int(accumulate), out.data_ptr(), ldo,
                                            wp, wb, s), "shampoo4_embedding_grad")
    return out


# -- policy loss ---------------------------------------------------------------------------

def policy_loss(logits: torch.Tensor, targets: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor,
                weights: torch.Tensor, ref_logp: torch.Tensor | None = None, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, grad_scale: float = 1.0, grad: bool = True,
                dlogits: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """(loss, logp, dlogits) of the clipped policy loss with a KL term (dlogits None with
    grad=False).  `weights` carries the mask and the normalisation of each token: a token
    with weight 0 is not read.  dlogits is grad_scale times the gradient, in the logits'
    type; it may be `logits` itself.  loss is a float32 scalar tensor."""
    ldz = _matrix(logits, "logits")
    rows, vocab = logits.shape
    dev = logits.device
    tp = _ids(targets, rows, "targets", dev)
    op = _vector(old_logp, rows, "old_logp", torch.float32, dev)
    ap = _vector(advantages, rows, "advantages", torch.float32, dev)
    wtp = _vector(weights, rows, "weights", torch.float32, dev)
    rp = _vector(ref_logp, rows, "ref_logp", torch.float32, dev) if ref_logp is not None else 0
    if kl_coef > 0 and ref_logp is None:
        raise ValueError("kl_coef needs ref_logp")
    if dlogits is not None and not grad:
        raise ValueError("dlogits given with grad=False")
    cfg = L.PolicyConfig(clip_low, clip_high, kl_coef, grad_scale)
    with _On(dev, stream) as s:
        loss = torch.empty((), dtype=torch.float32, device=dev)
        logp = torch.empty(rows, dtype=torch.float32, device=dev)
        ldd = 0
        if grad:
            if dlogits is None:
                dlogits = torch.empty((rows, vocab), dtype=logits.dtype, device=dev)
            ldd = _matrix(dlogits, "dlogits", logits.dtype, (rows, vocab), dev)
        lib = L.lib()
        dt = _DTYPES[logits.dtype]
        ws, wp, wb = _workspace(workspace, lib.shampoo4_policy_loss_workspace_bytes(dt, rows, vocab), dev)
        L.check(lib.shampoo4_policy_loss(ctypes.byref(cfg), dt, _ID_BYTES[targets.dtype], rows, vocab,
                                         logits.data_ptr(), ldz, tp, op, rp, ap, wtp, loss.data_ptr(),
                                         logp.data_ptr(), dlogits.data_ptr() if grad else 0, ldd, wp, wb, s),
                "shampoo4_policy_loss")
    return loss, logp, dlogits if grad else None


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """log softmax(logits)[targets] per row, float32; 0 for a target outside the vocabulary."""
    ldz = _matrix(logits, "logits")
    rows, vocab = logits.shape
    dev = logits.device
    tp = _ids(targets, rows, "targets", dev)
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty(rows, dtype=torch.float32, device=dev)
        op = _vector(out, rows, "out", torch.float32, dev)
        lib = L.lib()
        dt = _DTYPES[logits.dtype]
        ws, wp, wb = _workspace(workspace, lib.shampoo4_policy_loss_workspace_bytes(dt, rows, vocab), dev)
        L.check(lib.shampoo4_token_logprobs(dt, _ID_BYTES[targets.dtype], rows, vocab, logits.data_ptr(), ldz, tp, op,
                                            wp, wb, s), "shampoo4_token_logprobs")
    return out
