"""Thin PyTorch-facing binding of the training operators (include/shampoo4_train.h): what
produces the gradients that the 4-bit Shampoo step reads.

Argument marshalling only, as in shampoo4.py: PyTorch provides device memory and streams,
every computation is a kernel of libshampoo4.so, and nothing falls back to the CPU.

Shapes are those of the tensors given; matrices may be strided views with unit column
stride.  Element types are float32, bfloat16 and float16.  All tensors are on the current
device.  Work is enqueued on `stream` (default: the current stream), and tensors that a call
allocates (outputs not passed in, workspaces) belong to that stream, so the caching
allocator reuses them in its order.  Inputs used on another stream than their own are the
caller's to order, and to keep, as with any PyTorch operator.

None of these calls is recorded by autograd: an input that requires a gradient is read like
any other, and the result is detached from it.  Each backward pass is a call of its own
(activation_backward, act8_weight_grad, embedding_grad, the dlogits of policy_loss, fp8_linear with
the transposed weight, block_norm_backward, dropout on the gradient).
"""

from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib as L

_DTYPES = {torch.float32: L.F32, torch.bfloat16: L.BF16, torch.float16: L.F16}
_KINDS = {"silu": L.ACT_SILU, "gelu": L.ACT_GELU}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}
_F32, _I8, _U8, _E4M3 = torch.float32, torch.int8, torch.uint8, torch.float8_e4m3fn
_MASK64 = (1 << 64) - 1


def _on_stream(fn):
    """Adds the keyword `stream`: inside, it is the current stream."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _stream(device) -> int:
    """The current stream's handle; every tensor of a call is on `device`, the current one."""
    index = device.index
    if index != torch._C._cuda_getDevice():
        raise ValueError(f"tensors must be on the current device, got {device}")
    return torch._C._cuda_getCurrentRawStream(index)


def _tensor(t, what: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA (HIP) tensor")


def _matrix(t, what: str, dtype=None, rows=None, cols=None, device=None) -> int:
    """Checks a row-major matrix and returns its leading dimension."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA (HIP) tensor")
    if dtype is None:
        if t.dtype not in _DTYPES:
            raise TypeError(f"{what} must be float32, bfloat16 or float16, got {t.dtype}")
    elif t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.ndim != 2:
        raise ValueError(f"{what} must be a matrix, got shape {tuple(t.shape)}")
    r, c = t.shape
    if rows is not None and (r != rows or c != cols):
        raise ValueError(f"{what} must have shape {(rows, cols)}, got {(r, c)}")
    if device is not None and t.device != device:
        raise ValueError(f"{what} must be on {device}, got {t.device}")
    if c < 1:
        raise ValueError(f"{what} needs at least one column")
    if r == 0:
        return c
    s0, s1 = t.stride()
    if s1 != 1 and c > 1:
        raise ValueError(f"{what} must be row-major (unit column stride)")
    if r == 1:
        return c
    if s0 < c:
        raise ValueError(f"{what} must not have overlapping or broadcast rows")
    return s0


def _vector(t, n: int, what: str, dtype, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _tensor(t, what)
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {n}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}, got {t.device}")
    return t.data_ptr()


def _ids(t, n: int, what: str, device) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _tensor(t, what)
    if t.dtype not in _ID_BYTES:
        raise TypeError(f"{what} must be int32 or int64, got {t.dtype}")
    return _vector(t, n, what, t.dtype, device)


def _workspace(ws, need: int, like):
    """(tensor or None, pointer, bytes): the caller's workspace if it is large enough."""
    if need == 0:
        return None, 0, 0
    if ws is None:
        ws = like.new_empty(need, dtype=_U8)
        return ws, ws.data_ptr(), need
    _tensor(ws, "workspace")
    if ws.dtype is not _U8 or not ws.is_contiguous() or ws.numel() < need or ws.device != like.device:
        raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {need} bytes on {like.device}")
    return ws, ws.data_ptr(), ws.numel()


# -- 8-bit activation checkpoints --------------------------------------------------------

class Act8:
    """The 8-bit checkpoint of a [rows, cols] matrix: `codes` int8 [R, P] and `scales`
    uint8 [R / 32, P] (R: rows up to a multiple of 32, P: cols up to one of 16), the value
    of element (t, c) being codes[t, c] * 2 ** (scales[t // 32, c] - 127)."""

    # Two tensors, or one buffer with the scales behind the codes (one allocation where a call
    # makes the checkpoint), of which codes and scales are views made when asked for.
    __slots__ = ("_buf", "_codes", "_scales", "rows", "cols")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int):
        r, p = self.padded(rows, cols)
        for t, dtype, want, nm in ((codes, _I8, (r, p), "codes"), (scales, _U8, (r // L.ACT8_ROWS, p), "scales")):
            _tensor(t, nm)
            if t.dtype is not dtype or t.shape != want or not t.is_contiguous():
                raise ValueError(f"{nm} must be a contiguous {dtype} tensor of shape {want}")
        if codes.device != scales.device:
            raise ValueError("codes and scales must be on one device")
        self._buf, self._codes, self._scales, self.rows, self.cols = None, codes, scales, rows, cols

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            r, p = self.padded(self.rows, self.cols)
            self._codes = self._buf[:r * p].view(_I8).view(r, p)
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            r, p = self.padded(self.rows, self.cols)
            self._scales = self._buf[r * p:].view(r // L.ACT8_ROWS, p)
        return self._scales

    @property
    def device(self) -> torch.device:
        return (self._codes if self._buf is None else self._buf).device

    def _pointers(self):
        if self._buf is None:
            return self._codes.data_ptr(), self._scales.data_ptr()
        p = self._buf.data_ptr()
        return p, p + (-(-self.rows // 32) * 32) * (-(-self.cols // 16) * 16)

    @staticmethod
    def padded(rows: int, cols: int):
        return -(-rows // L.ACT8_ROWS) * L.ACT8_ROWS, -(-cols // L.ACT8_PITCH) * L.ACT8_PITCH

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda") -> "Act8":
        r, p = cls.padded(rows, cols)
        buf = torch.empty(r * p + r // L.ACT8_ROWS * p, dtype=_U8, device=device)
        _tensor(buf, "codes")
        return _of_buffer(buf, rows, cols)

    @property
    def nbytes(self) -> int:
        r, p = self.padded(self.rows, self.cols)
        return r * p + r // L.ACT8_ROWS * p


def _of_buffer(buf: torch.Tensor, rows: int, cols: int) -> Act8:
    a = Act8.__new__(Act8)
    a._buf, a._codes, a._scales, a.rows, a.cols = buf, None, None, rows, cols
    return a


def _new_act8(like: torch.Tensor, rows: int, cols: int) -> Act8:
    """Act8.empty on a tensor's device."""
    blocks = -(-rows // 32)
    return _of_buffer(like.new_empty(blocks * 33 * (-(-cols // 16) * 16), dtype=_U8), rows, cols)


def _act8(a, what: str, rows: int, cols: int, device):
    """Checks a checkpoint and returns its two pointers."""
    if not isinstance(a, Act8):
        raise TypeError(f"{what} must be an Act8")
    if a.rows != rows or a.cols != cols:
        raise ValueError(f"{what} must hold {(rows, cols)}, got {(a.rows, a.cols)}")
    if a.device != device:
        raise ValueError(f"{what} must be on {device}, got {a.device}")
    return a._pointers()


@_on_stream
def act8_store(x: torch.Tensor, out: Act8 | None = None) -> Act8:
    """The 8-bit checkpoint of x."""
    ld = _matrix(x, "x")
    rows, cols = x.shape
    dev = x.device
    s = _stream(dev)
    if out is None:
        out = _new_act8(x, rows, cols)
    c, e = _act8(out, "out", rows, cols, dev)
    L.check(L.lib().shampoo4_act8_store(_DTYPES[x.dtype], rows, cols, x.data_ptr(), ld, c, e, s),
            "shampoo4_act8_store")
    return out


@_on_stream
def act8_load(a: Act8, dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values of a checkpoint, in `dtype` (or in `out`, of its own type)."""
    if not isinstance(a, Act8):
        raise TypeError("a must be an Act8")
    held = a._codes if a._buf is None else a._buf
    rows, cols = a.rows, a.cols
    dev = held.device
    s = _stream(dev)
    c, e = a._pointers()
    if out is None:
        if dtype not in _DTYPES:
            raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
        out = held.new_empty((rows, cols), dtype=dtype)
        ld = cols
    else:
        ld = _matrix(out, "out", None, rows, cols, dev)
        dtype = out.dtype
    L.check(L.lib().shampoo4_act8_load(_DTYPES[dtype], rows, cols, c, e, out.data_ptr(), ld, s),
            "shampoo4_act8_load")
    return out


@_on_stream
def activation_forward(gate: torch.Tensor, up: torch.Tensor | None = None, kind: str = "silu", checkpoint: bool = True,
                       save_output: bool = True, out: torch.Tensor | None = None):
    """h = a(gate) * up (a(gate) without `up`), with the 8-bit checkpoints that training keeps.

    Returns (h, gate8, up8, h8): gate8 and up8 for activation_backward (None with
    checkpoint=False, as in inference), h8 for act8_weight_grad of the layer that reads h
    (None with save_output=False).  kind: "silu" or "gelu" (tanh form)."""
    if kind not in _KINDS:
        raise ValueError(f"kind must be one of {sorted(_KINDS)}, not {kind!r}")
    ldg = _matrix(gate, "gate")
    rows, cols = gate.shape
    dev, dtype = gate.device, gate.dtype
    s = _stream(dev)
    ldu = up_ptr = 0
    if up is not None:
        ldu = _matrix(up, "up", dtype, rows, cols, dev)
        up_ptr = up.data_ptr()
    if out is None:
        out = gate.new_empty((rows, cols))
        ldh = cols
    else:
        ldh = _matrix(out, "out", dtype, rows, cols, dev)
    g8 = u8 = h8 = None
    gc = ge = uc = ue = hc = he = 0
    if checkpoint:
        g8 = _new_act8(gate, rows, cols)
        gc, ge = g8._pointers()
        if up is not None:
            u8 = _new_act8(gate, rows, cols)
            uc, ue = u8._pointers()
    if save_output:
        h8 = _new_act8(gate, rows, cols)
        hc, he = h8._pointers()
    L.check(L.lib().shampoo4_activation_forward(_KINDS[kind], _DTYPES[dtype], rows, cols, gate.data_ptr(), ldg, up_ptr,
                                                ldu, out.data_ptr(), ldh, gc, ge, uc, ue, hc, he, s),
            "shampoo4_activation_forward")
    return out, g8, u8, h8


@_on_stream
def activation_backward(dh: torch.Tensor, gate8: Act8, up8: Act8 | None = None, kind: str = "silu",
                        dgate: torch.Tensor | None = None, dup: torch.Tensor | None = None):
    """(dgate, dup) of activation_forward from its checkpoints (dup None without up8).  `dgate`
    may be dh."""
    if kind not in _KINDS:
        raise ValueError(f"kind must be one of {sorted(_KINDS)}, not {kind!r}")
    ldd = _matrix(dh, "dh")
    rows, cols = dh.shape
    dev, dtype = dh.device, dh.dtype
    s = _stream(dev)
    gc, ge = _act8(gate8, "gate8", rows, cols, dev)
    if dgate is None:
        dgate = dh.new_empty((rows, cols))
        ldg = cols
    else:
        ldg = _matrix(dgate, "dgate", dtype, rows, cols, dev)
    uc = ue = ldu = dup_ptr = 0
    if up8 is not None:
        uc, ue = _act8(up8, "up8", rows, cols, dev)
        if dup is None:
            dup = dh.new_empty((rows, cols))
            ldu = cols
        else:
            ldu = _matrix(dup, "dup", dtype, rows, cols, dev)
        dup_ptr = dup.data_ptr()
    elif dup is not None:
        raise ValueError("dup needs up8")
    L.check(L.lib().shampoo4_activation_backward(_KINDS[kind], _DTYPES[dtype], rows, cols, dh.data_ptr(), ldd, gc, ge,
                                                 uc, ue, dgate.data_ptr(), ldg, dup_ptr, ldu, s),
            "shampoo4_activation_backward")
    return dgate, dup


@_on_stream
def act8_weight_grad(dy: torch.Tensor, x8: Act8, out: torch.Tensor | None = None, alpha: float = 1.0,
                     beta: float = 0.0, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """alpha dy^T x^ + beta out, float32 [dy columns, x columns]: the weight gradient of
    y = x W^T from the checkpoint of x, as Shampoo4Blocks.step takes it."""
    ldd = _matrix(dy, "dy")
    if not isinstance(x8, Act8):
        raise TypeError("x8 must be an Act8")
    rows, n = dy.shape
    cols = x8.cols
    dev = dy.device
    s = _stream(dev)
    c, e = _act8(x8, "x8", rows, cols, dev)
    if out is None:
        if beta != 0.0:
            raise ValueError("beta needs out")
        out = dy.new_empty((n, cols), dtype=_F32)
        ldo = cols
    else:
        ldo = _matrix(out, "out", _F32, n, cols, dev)
    lib = L.lib()
    ws, wp, wb = _workspace(workspace, lib.shampoo4_act8_weight_grad_workspace_bytes(rows, n, cols), dy)
    L.check(lib.shampoo4_act8_weight_grad(_DTYPES[dy.dtype], rows, n, cols, alpha, dy.data_ptr(), ldd, c, e, beta,
                                          out.data_ptr(), ldo, wp, wb, s), "shampoo4_act8_weight_grad")
    return out


# -- embedding -----------------------------------------------------------------------------

@_on_stream
def embedding(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """scale * table[ids] ([tokens, dim], the table's type); an id outside the table, as -1
    for padding, gives a row of zeros."""
    ldt = _matrix(table, "table")
    vocab, dim = table.shape
    dev = table.device
    s = _stream(dev)
    n = ids.numel() if isinstance(ids, torch.Tensor) else 0
    ip = _ids(ids, n, "ids", dev)
    if out is None:
        out = table.new_empty((n, dim))
        ldo = dim
    else:
        ldo = _matrix(out, "out", table.dtype, n, dim, dev)
    L.check(L.lib().shampoo4_embedding(_DTYPES[table.dtype], _ID_BYTES[ids.dtype], n, vocab, dim, table.data_ptr(), ldt,
                                       ip, scale, out.data_ptr(), ldo, s), "shampoo4_embedding")
    return out


@_on_stream
def embedding_grad(dout: torch.Tensor, ids: torch.Tensor, num_embeddings: int, scale: float = 1.0,
                   out: torch.Tensor | None = None, accumulate: bool = False,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The table's gradient in float32 [num_embeddings, dim], rows summed in the order of their
    tokens.  accumulate=True adds to `out` and touches only the rows of tokens that occur."""
    ldd = _matrix(dout, "dout")
    n, dim = dout.shape
    dev = dout.device
    s = _stream(dev)
    ip = _ids(ids, n, "ids", dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = dout.new_empty((num_embeddings, dim), dtype=_F32)
        ldo = dim
    else:
        ldo = _matrix(out, "out", _F32, num_embeddings, dim, dev)
    lib = L.lib()
    ws, wp, wb = _workspace(workspace, lib.shampoo4_embedding_grad_workspace_bytes(n, num_embeddings, dim), dout)
    L.check(lib.shampoo4_embedding_grad(_DTYPES[dout.dtype], _ID_BYTES[ids.dtype], n, num_embeddings, dim,
                                        dout.data_ptr(), ldd, ip, scale, int(accumulate), out.data_ptr(), ldo, wp, wb,
                                        s), "shampoo4_embedding_grad")
    return out


# -- policy loss ---------------------------------------------------------------------------

@_on_stream
def policy_loss(logits: torch.Tensor, targets: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor,
                weights: torch.Tensor, ref_logp: torch.Tensor | None = None, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, grad_scale: float = 1.0, grad: bool = True,
                dlogits: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """(loss, logp, dlogits) of the clipped policy loss with a KL term (dlogits None with
    grad=False).  `weights` carries the mask and the normalisation of each token: a token
    with weight 0 is not read.  dlogits is grad_scale times the gradient, in the logits'
    type; it may be `logits` itself.  loss is a float32 scalar tensor."""
    ldz = _matrix(logits, "logits")
    rows, vocab = logits.shape
    dev = logits.device
    s = _stream(dev)
    tp = _ids(targets, rows, "targets", dev)
    op = _vector(old_logp, rows, "old_logp", _F32, dev)
    ap = _vector(advantages, rows, "advantages", _F32, dev)
    wtp = _vector(weights, rows, "weights", _F32, dev)
    rp = 0
    if ref_logp is not None:
        rp = _vector(ref_logp, rows, "ref_logp", _F32, dev)
    elif kl_coef > 0:
        raise ValueError("kl_coef needs ref_logp")
    dp = ldd = 0
    if not grad:
        if dlogits is not None:
            raise ValueError("dlogits given with grad=False")
    else:
        if dlogits is None:
            dlogits = logits.new_empty((rows, vocab))
            ldd = vocab
        else:
            ldd = _matrix(dlogits, "dlogits", logits.dtype, rows, vocab, dev)
        dp = dlogits.data_ptr()
    loss = logits.new_empty((), dtype=_F32)
    logp = logits.new_empty(rows, dtype=_F32)
    lib = L.lib()
    dt = _DTYPES[logits.dtype]
    ws, wp, wb = _workspace(workspace, lib.shampoo4_policy_loss_workspace_bytes(dt, rows, vocab), logits)
    cfg = L.PolicyConfig(clip_low, clip_high, kl_coef, grad_scale)
    L.check(lib.shampoo4_policy_loss(ctypes.byref(cfg), dt, _ID_BYTES[targets.dtype], rows, vocab, logits.data_ptr(),
                                     ldz, tp, op, rp, ap, wtp, loss.data_ptr(), logp.data_ptr(), dp, ldd, wp, wb, s),
            "shampoo4_policy_loss")
    return loss, logp, dlogits


@_on_stream
def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """log softmax(logits)[targets] per row, float32; 0 for a target outside the vocabulary."""
    ldz = _matrix(logits, "logits")
    rows, vocab = logits.shape
    dev = logits.device
    s = _stream(dev)
    tp = _ids(targets, rows, "targets", dev)
    if out is None:
        out = logits.new_empty(rows, dtype=_F32)
        op = out.data_ptr()
    else:
        op = _vector(out, rows, "out", _F32, dev)
    lib = L.lib()
    dt = _DTYPES[logits.dtype]
    ws, wp, wb = _workspace(workspace, lib.shampoo4_token_logprobs_workspace_bytes(dt, rows, vocab), logits)
    L.check(lib.shampoo4_token_logprobs(dt, _ID_BYTES[targets.dtype], rows, vocab, logits.data_ptr(), ldz, tp, op, wp,
                                        wb, s), "shampoo4_token_logprobs")
    return out


# -- products in 8-bit floating point -------------------------------------------------------

class Fp8:
    """A [rows, cols] matrix in e4m3 with a scale for each block of 128 columns of `block_rows` rows (1:
    activations, 128: weights): `codes` float8_e4m3fn [rows, P] (P: cols up to a multiple of 128) and
    `scales` uint8 [rows / block_rows up, S] (S: P / 128 up to a multiple of 4), the value of element
    (t, c) being codes[t, c] * 2 ** (scales[t // block_rows, c // 128] - 127).  Columns of padding hold code
    0, and their scales 1."""

    # Two tensors, or one buffer with the scales behind the codes (one allocation where a call
    # makes it), of which codes and scales are views made when asked for.
    __slots__ = ("_buf", "_codes", "_scales", "rows", "cols", "block_rows")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int, block_rows: int = 1):
        if block_rows not in (1, L.FP8_BLOCK):
            raise ValueError(f"block_rows must be 1 or {L.FP8_BLOCK}, got {block_rows}")
        shapes = self.padded(rows, cols, block_rows)
        for t, dtype, want, nm in ((codes, _E4M3, shapes[0], "codes"), (scales, _U8, shapes[1], "scales")):
            _tensor(t, nm)
            if t.dtype is not dtype or t.shape != want or not t.is_contiguous():
                raise ValueError(f"{nm} must be a contiguous {dtype} tensor of shape {want}")
        if codes.device != scales.device:
            raise ValueError("codes and scales must be on one device")
        self._buf, self._codes, self._scales = None, codes, scales
        self.rows, self.cols, self.block_rows = rows, cols, block_rows

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            r, p = self.padded(self.rows, self.cols, self.block_rows)[0]
            self._codes = self._buf[:r * p].view(_E4M3).view(r, p)
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            (r, p), shape = self.padded(self.rows, self.cols, self.block_rows)
            self._scales = self._buf[r * p:].view(shape)
        return self._scales

    @property
    def device(self) -> torch.device:
        return self._held().device

    def _held(self) -> torch.Tensor:
        return self._codes if self._buf is None else self._buf

    def _pointers(self):
        if self._buf is None:
            return self._codes.data_ptr(), self._scales.data_ptr()
        p = self._buf.data_ptr()
        return p, p + self.rows * (-(-self.cols // 128) * 128)

    @staticmethod
    def padded(rows: int, cols: int, block_rows: int = 1):
        """The shapes of codes and scales."""
        return (rows, -(-cols // 128) * 128), (-(-rows // block_rows), -(-cols // 512) * 4)

    @classmethod
    def empty(cls, rows: int, cols: int, block_rows: int = 1, device="cuda") -> "Fp8":
        codes, scales = cls.padded(rows, cols, block_rows)
        return cls(torch.empty(codes, dtype=_E4M3, device=device), torch.empty(scales, dtype=_U8, device=device), rows,
                   cols, block_rows)

    @property
    def nbytes(self) -> int:
        (r, p), (sr, sp) = self.padded(self.rows, self.cols, self.block_rows)
        return r * p + sr * sp


def _new_fp8(like: torch.Tensor, rows: int, cols: int, block_rows: int) -> Fp8:
    """Fp8.empty on a tensor's device."""
    a = Fp8.__new__(Fp8)
    a._buf = like.new_empty(rows * (-(-cols // 128) * 128) + -(-rows // block_rows) * (-(-cols // 512) * 4), dtype=_U8)
    a._codes = a._scales = None
    a.rows, a.cols, a.block_rows = rows, cols, block_rows
    return a


def _fp8(a, what: str, rows, cols, block_rows: int, device):
    """Checks a quantised matrix (rows or cols None: any) and returns its two pointers."""
    if not isinstance(a, Fp8):
        raise TypeError(f"{what} must be an Fp8")
    if a.block_rows != block_rows:
        raise ValueError(f"{what} must have blocks of {block_rows} rows, got {a.block_rows}")
    if (rows is not None and a.rows != rows) or (cols is not None and a.cols != cols):
        raise ValueError(f"{what} must hold {(rows, cols)}, got {(a.rows, a.cols)}")
    if a.device != device:
        raise ValueError(f"{what} must be on {device}, got {a.device}")
    return a._pointers()


@_on_stream
def fp8_store(x: torch.Tensor, out: Fp8 | None = None) -> Fp8:
    """x in e4m3 with a scale for each 128 columns of a row (an operand of fp8_linear)."""
    ld = _matrix(x, "x")
    rows, cols = x.shape
    dev = x.device
    s = _stream(dev)
    if out is None:
        out = _new_fp8(x, rows, cols, 1)
    c, e = _fp8(out, "out", rows, cols, 1, dev)
    L.check(L.lib().shampoo4_fp8_store(_DTYPES[x.dtype], rows, cols, x.data_ptr(), ld, c, e, s), "shampoo4_fp8_store")
    return out


@_on_stream
def fp8_store_weight(w: torch.Tensor, transposed: bool = False, out: Fp8 | None = None, out_t: Fp8 | None = None):
    """w in e4m3 with a scale for each block of 128 x 128; with transposed=True (w8, wt8), wt8 being w^T
    in the same codes: fp8_linear(x, w8) is the layer, fp8_linear(dy, wt8) its input's gradient.  out and out_t
    are two."""
    ld = _matrix(w, "w")
    rows, cols = w.shape
    dev = w.device
    s = _stream(dev)
    if out is None:
        out = _new_fp8(w, rows, cols, L.FP8_BLOCK)
    c, e = _fp8(out, "out", rows, cols, L.FP8_BLOCK, dev)
    tc = te = 0
    if transposed:
        if out_t is None:
            out_t = _new_fp8(w, cols, rows, L.FP8_BLOCK)
        tc, te = _fp8(out_t, "out_t", cols, rows, L.FP8_BLOCK, dev)
    elif out_t is not None:
        raise ValueError("out_t needs transposed=True")
    L.check(L.lib().shampoo4_fp8_store_weight(_DTYPES[w.dtype], rows, cols, w.data_ptr(), ld, c, e, tc, te, s),
            "shampoo4_fp8_store_weight")
    return (out, out_t) if transposed else out


@_on_stream
def fp8_load(a: Fp8, dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values of a quantised matrix, in `dtype` (or in `out`, of its own type)."""
    if not isinstance(a, Fp8):
        raise TypeError("a must be an Fp8")
    rows, cols, held = a.rows, a.cols, a._held()
    dev = held.device
    s = _stream(dev)
    c, e = a._pointers()
    if out is None:
        if dtype not in _DTYPES:
            raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
        out = held.new_empty((rows, cols), dtype=dtype)
        ld = cols
    else:
        ld = _matrix(out, "out", None, rows, cols, dev)
        dtype = out.dtype
    L.check(L.lib().shampoo4_fp8_load(_DTYPES[dtype], rows, cols, a.block_rows, c, e, out.data_ptr(), ld, s),
            "shampoo4_fp8_load")
    return out


@_on_stream
def fp8_linear(x, w8: Fp8, out: torch.Tensor | None = None, accumulate: bool = False, dtype=None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """x w8^T, [x rows, w8 rows].  x is an Fp8 of fp8_store (or block_norm_forward), or a matrix, which the
    call quantises in the same way.  The result is of `dtype` (default: x's type, bfloat16 for an Fp8),
    or goes into `out`, of its own type; accumulate=True adds to `out`, which shares no memory with x or w8.

    A bfloat16 result's products are the 8-bit matrix cores', which cut a term off 13 bits below the largest
    of its eight neighbours: at most 7 * 2**-13 of the sum of the terms' sizes, which may be many steps of the
    result where they cancel; on ordinary operands 5e-5 of the results' root mean square, a fortieth of
    bfloat16's rounding.  Those of a float32 or float16 result are exact, with float32 sums, at about a third of the
    rate; a bfloat16 result of float32 sums is a float32 one, rounded by the caller."""
    if isinstance(x, Fp8):
        rows, k, held = x.rows, x.cols, x._held()
        dev = held.device
        s = _stream(dev)
        xc, xe = _fp8(x, "x", None, None, 1, dev)
        xp = ld = 0
        xdt = torch.bfloat16
    else:
        ld = _matrix(x, "x")
        rows, k = x.shape
        dev, held, xdt = x.device, x, x.dtype
        s = _stream(dev)
        xp, xc, xe = x.data_ptr(), 0, 0
    wc, we = _fp8(w8, "w8", None, k, L.FP8_BLOCK, dev)
    n = w8.rows
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        odt = xdt if dtype is None else dtype
        if odt not in _DTYPES:
            raise TypeError(f"dtype must be float32, bfloat16 or float16, got {odt}")
        out = held.new_empty((rows, n), dtype=odt)
        ldo = n
    else:
        ldo = _matrix(out, "out", dtype, rows, n, dev)
        odt = out.dtype
        if rows and out.data_ptr() == (xp or xc):
            raise ValueError("out must not be x")
    lib = L.lib()
    o = _DTYPES[odt]
    ws, wp, wb = _workspace(workspace, lib.shampoo4_fp8_linear_workspace_bytes(o, rows, n, k, not xp), held)
    L.check(lib.shampoo4_fp8_linear(_DTYPES[xdt], o, rows, n, k, xp, ld, xc, xe, wc, we, int(accumulate), out.data_ptr(),
                                    ldo, wp, wb, s), "shampoo4_fp8_linear")
    return out


# -- dropout -------------------------------------------------------------------------------

def _dropout_config(p: float, seed: int, offset: int, counter, device) -> L.DropoutConfig:
    cp = 0
    if counter is not None:
        cp = _vector(counter, 1, "counter", torch.int64, device)
    return L.DropoutConfig(p, 0, seed & _MASK64, offset & _MASK64, cp)


@_on_stream
def dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0, counter: torch.Tensor | None = None,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """x with each element dropped with probability p (in steps of 2**-16) and the others divided by what is
    kept of 1.  Which are dropped follows from (seed, offset + counter, row, column) alone, so that the
    backward pass is the same call on the gradient, and no mask is stored.  `counter` is an int64 tensor of
    one element that the kernel reads: a captured graph whose program advances it drops others in each
    replay.  `out` may be x."""
    ld = _matrix(x, "x")
    rows, cols = x.shape
    dev = x.device
    s = _stream(dev)
    if out is None:
        out = x.new_empty((rows, cols))
        ldo = cols
    else:
        ldo = _matrix(out, "out", x.dtype, rows, cols, dev)
    cfg = _dropout_config(p, seed, offset, counter, dev)
    L.check(L.lib().shampoo4_dropout(ctypes.byref(cfg), _DTYPES[x.dtype], rows, cols, x.data_ptr(), ld, out.data_ptr(),
                                     ldo, s), "shampoo4_dropout")
    return out


# -- the ends of a residual block ------------------------------------------------------------

def _gate(gate, dtype, rows: int, cols: int, device, what: str = "gate"):
    """(pointer, is a matrix, leading dimension) of a gate: float32 [cols], or [rows, cols] of `dtype`."""
    if gate is None:
        return 0, 0, 0
    _tensor(gate, what)
    if gate.ndim == 1:
        return _vector(gate, cols, what, _F32, device), 0, 0
    ld = _matrix(gate, what, dtype, rows, cols, device)
    return gate.data_ptr(), 1, ld


def _out(t, what: str, like: torch.Tensor):
    """A result's tensor, made where it is not given, and its leading dimension."""
    rows, cols = like.shape
    if t is None:
        return like.new_empty((rows, cols)), cols
    return t, _matrix(t, what, like.dtype, rows, cols, like.device)


@_on_stream
def block_norm_forward(x: torch.Tensor, weight: torch.Tensor | None = None, h: torch.Tensor | None = None,
                       post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                       residual_scale: float = 1.0, eps: float = 1e-6, p: float = 0.0, seed: int = 0, offset: int = 0,
                       counter: torch.Tensor | None = None, save8: bool = False, out: torch.Tensor | None = None,
                       y: torch.Tensor | None = None):
    """The end of a block and the norm before the next one:

        x' = residual_scale x + gate dropout(h rstd(h) post_weight)
        y  = x' rstd(x') weight                          rstd(v) = 1 / sqrt(mean(v^2) + eps)

    Returns (x', y, y8, stats): y8 is y quantised as by fp8_store (None without save8), stats is what
    block_norm_backward needs.  Without `h`, x' is x (the norm alone); without `weight` there is no y;
    without `post_weight` the block's end is h as it is.  gate: float32 [cols], a matrix like x, or None
    for 1.  Weights are float32 [cols].  p, seed, offset, counter: as of dropout (which h is needed for).
    `out` may be x or h, and `y` may be h, but not `out`."""
    ldx = _matrix(x, "x")
    rows, cols = x.shape
    dev, dtype = x.device, x.dtype
    s = _stream(dev)
    hp = ldh = ldo = op = pp = hr = ldy = yp = yc = ye = wp = rr = 0
    stats = x.new_empty((2, rows), dtype=_F32)
    gp, grows, ldg = _gate(gate, dtype, rows, cols, dev)
    if h is not None:
        ldh = _matrix(h, "h", dtype, rows, cols, dev)
        hp = h.data_ptr()
        out, ldo = _out(out, "out", x)
        op = out.data_ptr()
        if post_weight is not None:
            pp = _vector(post_weight, cols, "post_weight", _F32, dev)
            hr = stats.data_ptr()
    elif post_weight is not None or gate is not None or out is not None or residual_scale != 1.0:
        raise ValueError("post_weight, gate, out and residual_scale need h")
    y8 = None
    if weight is not None:
        wp = _vector(weight, cols, "weight", _F32, dev)
        y, ldy = _out(y, "y", x)
        yp = y.data_ptr()
        rr = stats.data_ptr() + 4 * rows
        if save8:
            y8 = _new_fp8(x, rows, cols, 1)
            yc, ye = y8._pointers()
    elif y is not None or save8 or h is None:
        raise ValueError("y and save8 need weight, and so does a call without h")
    cfg = L.BlockNormConfig(eps, residual_scale, _dropout_config(p, seed, offset, counter, dev))
    L.check(L.lib().shampoo4_block_norm_forward(ctypes.byref(cfg), _DTYPES[dtype], rows, cols, x.data_ptr(), ldx, hp, ldh,
                                                pp, gp, grows, ldg, wp, op, ldo, yp, ldy, yc, ye, hr, rr, s),
            "shampoo4_block_norm_forward")
    return x if h is None else out, y, y8, stats


@_on_stream
def block_norm_backward(dy: torch.Tensor | None, dres: torch.Tensor | None, x: torch.Tensor,
                        weight: torch.Tensor | None, stats: torch.Tensor, h: torch.Tensor | None = None,
                        post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                        residual_scale: float = 1.0, eps: float = 1e-6, p: float = 0.0, seed: int = 0,
                        offset: int = 0, counter: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                        dh: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """(dx, dh, dweight, dpost_weight, dgate) of block_norm_forward, from the gradients of y (`dy`, None without
    `weight`) and of x' (`dres`, None for 0).  `x` is x', what the forward call returned first; the other
    arguments are as there.  Gradients of vectors are float32 [cols]; what has no input is None.
    dx may be dres or dy, and dh may be h or the other of the two."""
    ldx = _matrix(x, "x")
    rows, cols = x.shape
    dev, dtype = x.device, x.dtype
    s = _stream(dev)
    ldy = yp = ldr = rp = wp = rr = hp = ldh = hr = pp = ldh2 = dhp = dwp = dpp = dgp = lddg = 0
    _tensor(stats, "stats")
    if stats.dtype is not _F32 or stats.shape != (2, rows) or not stats.is_contiguous() or stats.device != dev:
        raise ValueError(f"stats must be a contiguous float32 tensor of shape {(2, rows)} on {dev}")
    if dres is not None:
        ldr = _matrix(dres, "dres", dtype, rows, cols, dev)
        rp = dres.data_ptr()
    dweight = dpost = dgate = None
    sums = x.new_empty((3, cols), dtype=_F32).unbind(0)      # of the vectors' gradients
    if weight is not None:
        if dy is None:
            raise ValueError("weight needs dy")
        ldy = _matrix(dy, "dy", dtype, rows, cols, dev)
        yp = dy.data_ptr()
        wp = _vector(weight, cols, "weight", _F32, dev)
        rr = stats.data_ptr() + 4 * rows
        dweight = sums[0]
        dwp = dweight.data_ptr()
    elif dy is not None:
        raise ValueError("dy needs weight")
    elif dres is None:
        raise ValueError("one of dy and dres is needed")
    gp, grows, ldg = _gate(gate, dtype, rows, cols, dev)
    if h is not None:
        ldh = _matrix(h, "h", dtype, rows, cols, dev)
        hp = h.data_ptr()
        if post_weight is not None:
            pp = _vector(post_weight, cols, "post_weight", _F32, dev)
            hr = stats.data_ptr()
            dpost = sums[1]
            dpp = dpost.data_ptr()
        if gate is not None:
            dgate, lddg = x.new_empty((rows, cols)) if grows else sums[2], cols
            dgp = dgate.data_ptr()
        dh, ldh2 = _out(dh, "dh", x)
        dhp = dh.data_ptr()
    elif post_weight is not None or gate is not None or dh is not None or residual_scale != 1.0:
        raise ValueError("post_weight, gate, dh and residual_scale need h")
    dx, ldd = _out(dx, "dx", x)
    lib = L.lib()
    ws, wsp, wb = _workspace(workspace, lib.shampoo4_block_norm_workspace_bytes(rows, cols), x)
    cfg = L.BlockNormConfig(eps, residual_scale, _dropout_config(p, seed, offset, counter, dev))
    L.check(lib.shampoo4_block_norm_backward(ctypes.byref(cfg), _DTYPES[dtype], rows, cols, yp, ldy, rp, ldr,
                                             x.data_ptr(), ldx, rr, wp, hp, ldh, hr, pp, gp, grows, ldg, dx.data_ptr(),
                                             ldd, dhp, ldh2, dwp, dpp, dgp, lddg, wsp, wb, s),
            "shampoo4_block_norm_backward")
    return dx, dh, dweight, dpost, dgate
