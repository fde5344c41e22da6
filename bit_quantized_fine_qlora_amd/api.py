"""Torch-facing binding of the QLoRA library.

Only marshals tensors into pointers and sizes and passes the current HIP
stream; every step of the computation runs in the HIP kernels of
libqlora.so.  Torch supplies device memory (outputs and workspaces).
"""

from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _lib

QLORA_OP_FWD = 0
QLORA_OP_BWD = 1
QLORA_OP_BWD_DROPOUT = 2


@dataclasses.dataclass
class QuantizedWeight:
    """NF4 + double-quantized m x n weight: codes, absmax8 (E4M3) and c2."""
    codes: torch.Tensor     # uint8 [m*n/2]
    absmax8: torch.Tensor   # uint8 [m*n/64]
    c2: torch.Tensor        # float32 [ceil(m*n/16384)]
    m: int
    n: int

    def nbytes(self) -> int:
        return self.codes.numel() + self.absmax8.numel() + 4 * self.c2.numel()


@dataclasses.dataclass
class Checkpoint8:
    """A bf16 [M, n] tensor kept in 8 bits: codes and one scale byte per 32 values of a row."""
    codes: torch.Tensor     # int8 [M, n]
    scales: torch.Tensor    # uint8 [M, 4 ceil(n / 128)]

    @property
    def shape(self):
        return self.codes.shape

    @property
    def device(self):
        return self.codes.device

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()

    def check(self, name: str) -> None:
        M, n = self.codes.shape
        _need(self.codes, torch.int8, (M, n), name + ".codes")
        _need(self.scales, torch.uint8, (M, checkpoint_pitch(n)), name + ".scales")


def checkpoint_pitch(n: int) -> int:
    """Bytes in a row of a Checkpoint8's scales."""
    return (n + 127) // 128 * 4


def _ptr(t):
    return None if t is None else t.data_ptr()


# torch's own short way to a device's current stream, 0.1 us where the stream
# object takes 1.9; not part of its documented interface, so not relied on.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device=None):
    if _raw_stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    index = device.index if device is not None else None
    return _raw_stream(torch.cuda.current_device() if index is None else index)


def _need(t: torch.Tensor, dtype, shape, name: str):
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


QTYPE_NF4 = 0
QTYPE_UNIFORM4 = 1
QTYPE_EDGE_MEAN4 = 2
QTYPE_INT4 = 3


def level_table(qtype: int = QTYPE_NF4):
    """(levels[16], thresholds[15]) of a level table as the library derived them (host)."""
    lib = _lib.load()
    lv = (ctypes.c_float * 16)()
    th = (ctypes.c_float * 15)()
    _lib.check(lib.qlora_level_table(int(qtype), ctypes.cast(lv, ctypes.c_void_p), ctypes.cast(th, ctypes.c_void_p)),
               "qlora_level_table")
    return list(lv), list(th)


def quantize_dq(W: torch.Tensor, qtype: int = QTYPE_NF4, out: QuantizedWeight | None = None) -> QuantizedWeight:
    """Blockwise 4-bit quantization with double quantization on a chosen level table."""
    m, n = W.shape
    _need(W, torch.float32, (m, n), "W")
    q = out if out is not None else alloc_quantized(m, n, W.device)
    st = _lib.load().qlora_quantize_dq(int(qtype), _ptr(W), m, n, _ptr(q.codes), _ptr(q.absmax8), _ptr(q.c2),
                                       _stream(W.device))
    _lib.check(st, "qlora_quantize_dq")
    return q


def quantize_dq_grouped(Ws, qtype: int = QTYPE_NF4, outs=None):
    """Quantize several fp32 weights in one launch, each as quantize_dq would.

    Ws: sequence of up to 8 m x n fp32 tensors on one device; outs: matching
    QuantizedWeights to write, or None to allocate.  Returns the list of
    QuantizedWeights.
    """
    if not Ws:
        return []
    dev = Ws[0].device
    arr = (_lib.QuantWeight * len(Ws))()
    qs = []
    for i, W in enumerate(Ws):
        m, n = W.shape
        _need(W, torch.float32, (m, n), "W")
        if W.device != dev:
            raise ValueError("quantize_dq_grouped: all weights must be on one device")
        q = outs[i] if outs is not None else alloc_quantized(m, n, dev)
        arr[i] = _lib.QuantWeight(_ptr(W), m, n, _ptr(q.codes), _ptr(q.absmax8), _ptr(q.c2))
        qs.append(q)
    st = _lib.load().qlora_quantize_dq_grouped(int(qtype), len(Ws), arr, _stream(dev))
    _lib.check(st, "qlora_quantize_dq_grouped")
    return qs


def dequant_dq(q: QuantizedWeight, qtype: int = QTYPE_NF4) -> torch.Tensor:
    out = torch.empty((q.m, q.n), dtype=torch.bfloat16, device=q.codes.device)
    st = _lib.load().qlora_dequant_dq(int(qtype), _ptr(q.codes), _ptr(q.absmax8), _ptr(q.c2), q.m, q.n, _ptr(out),
                                      _stream(q.codes.device))
    _lib.check(st, "qlora_dequant_dq")
    return out


def nf4_table():
    """(levels[16], thresholds[15]) as the library derived them (host)."""
    lib = _lib.load()
    lv = (ctypes.c_float * 16)()
    th = (ctypes.c_float * 15)()
    lib.qlora_nf4_table(ctypes.cast(lv, ctypes.c_void_p), ctypes.cast(th, ctypes.c_void_p))
    return list(lv), list(th)


def workspace_bytes(op: int, M: int, n: int, m: int, r: int) -> int:
    return int(_lib.load().qlora_workspace_bytes(op, M, n, m, r))


def alloc_quantized(m: int, n: int, device="cuda") -> QuantizedWeight:
    numel = m * n
    return QuantizedWeight(
        codes=torch.empty(numel // 2, dtype=torch.uint8, device=device),
        absmax8=torch.empty(numel // 64, dtype=torch.uint8, device=device),
        c2=torch.empty((numel // 64 + 255) // 256, dtype=torch.float32, device=device),
        m=m, n=n)


def quantize_nf4_dq(W: torch.Tensor, out: QuantizedWeight | None = None) -> QuantizedWeight:
    m, n = W.shape
    _need(W, torch.float32, (m, n), "W")
    q = out if out is not None else alloc_quantized(m, n, W.device)
    st = _lib.load().qlora_quantize_nf4_dq(_ptr(W), m, n, _ptr(q.codes), _ptr(q.absmax8), _ptr(q.c2),
                                           _stream(W.device))
    _lib.check(st, "qlora_quantize_nf4_dq")
    return q


def dequant_nf4_dq(q: QuantizedWeight) -> torch.Tensor:
    out = torch.empty((q.m, q.n), dtype=torch.bfloat16, device=q.codes.device)
    st = _lib.load().qlora_dequant_nf4_dq(_ptr(q.codes), _ptr(q.absmax8), _ptr(q.c2), q.m, q.n, _ptr(out),
                                          _stream(q.codes.device))
    _lib.check(st, "qlora_dequant_nf4_dq")
    return out


class AdamStep:
    """Prepared optimizer step over a fixed list of adapter tensors.

    tensors: list of (param fp32, param_bf16 bf16 or None, grad bf16, exp_avg fp32, exp_avg_sq fp32), each
    contiguous with the same number of elements, on the GPU or (param and moments) in pinned host memory.
    The tensor table is marshalled once; run() launches the step.
    """

    def __init__(self, tensors):
        self._keep = list(tensors)
        self._arr = (_lib.AdamTensor * len(self._keep))()
        self._dev = None
        for i, (p, p16, g, m, v) in enumerate(self._keep):
            n = p.numel()
            if p.dtype != torch.float32 or m.dtype != torch.float32 or v.dtype != torch.float32:
                raise TypeError("param, exp_avg and exp_avg_sq must be float32")
            if g.dtype != torch.bfloat16 or (p16 is not None and p16.dtype != torch.bfloat16):
                raise TypeError("grad and param_bf16 must be bfloat16")
            named = [(p, "param"), (g, "grad"), (m, "exp_avg"), (v, "exp_avg_sq")]
            if p16 is not None:
                named.append((p16, "param_bf16"))
            for t, nm in named:
                if t.numel() != n or not t.is_contiguous():
                    raise ValueError(f"{nm}: expected {n} contiguous elements")
            if g.is_cuda:
                self._dev = g.device
            self._arr[i] = _lib.AdamTensor(n, p.data_ptr(), p16.data_ptr() if p16 is not None else None,
                                           g.data_ptr(), m.data_ptr(), v.data_ptr())

    def run(self, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
            weight_decay: float = 0.0, step: int = 1) -> None:
        st = _lib.load().qlora_adam_step(self._arr, len(self._keep), float(lr), float(beta1), float(beta2),
                                         float(eps), float(weight_decay), int(step), _stream(self._dev))
        _lib.check(st, "qlora_adam_step")


def adam_step(tensors, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
              weight_decay: float = 0.0, step: int = 1) -> None:
    """Adam step with decoupled weight decay on adapter tensors, in place (see AdamStep)."""
    AdamStep(tensors).run(lr, beta1, beta2, eps, weight_decay, step)


def merge_adapter(q: QuantizedWeight, A: torch.Tensor, B: torch.Tensor, s: float) -> torch.Tensor:
    """bf16(W' + s B A): the adapter folded into the dequantized weight (m x n bf16)."""
    r = A.shape[0]
    _need(A, torch.bfloat16, (r, q.n), "A")
    _need(B, torch.bfloat16, (q.m, r), "B")
    out = torch.empty((q.m, q.n), dtype=torch.bfloat16, device=q.codes.device)
    st = _lib.load().qlora_merge_adapter(_ptr(q.codes), _ptr(q.absmax8), _ptr(q.c2), q.m, q.n, r, float(s),
                                         _ptr(A), _ptr(B), _ptr(out), _stream(q.codes.device))
    _lib.check(st, "qlora_merge_adapter")
    return out


def _room(need: int, device, workspace):
    """A workspace of `need` bytes: the given one where it is large enough, or a new one."""
    if workspace is not None:
        if workspace.device != device:
            raise ValueError(f"workspace: must be on {device}, got one on {workspace.device}")
        if not workspace.is_contiguous():
            raise ValueError("workspace: must be contiguous")
        if workspace.numel() >= need:
            return workspace
    return torch.empty(max(need, 256), dtype=torch.uint8, device=device)


def _workspace(op, M, n, m, r, device, workspace):
    return _room(workspace_bytes(op, M, n, m, r), device, workspace)


def _dropout(dropout):
    """(p, seed, offset) or None -> a qlora_dropout pointer (None: plain layer)."""
    if dropout is None:
        return None
    p, seed, offset = dropout
    return ctypes.pointer(_lib.Dropout(float(p), int(seed) & (2 ** 64 - 1), int(offset) & (2 ** 64 - 1)))


def linear_fwd(x: torch.Tensor, q: QuantizedWeight, A: torch.Tensor, B: torch.Tensor, s: float,
               h: torch.Tensor | None = None, u: torch.Tensor | None = None, want_u: bool = True,
               workspace: torch.Tensor | None = None, dropout=None):
    """h = x W'^T + s (x A^T) B^T.  Returns (h bf16 [M, m], u fp32 [M, r] or None).

    dropout: (p, seed, offset) for dropout on the adapter input (the adapter
    reads x * keep / (1 - p)), or None.
    """
    M, n = x.shape
    m = q.m
    r = A.shape[0]
    _need(x, torch.bfloat16, (M, q.n), "x")
    _need(A, torch.bfloat16, (r, q.n), "A")
    _need(B, torch.bfloat16, (m, r), "B")
    if h is None:
        h = torch.empty((M, m), dtype=torch.bfloat16, device=x.device)
    if u is None and want_u:
        u = torch.empty((M, r), dtype=torch.float32, device=x.device)
    ws = _workspace(QLORA_OP_FWD, M, n, m, r, x.device, workspace)
    if dropout is None:
        st = _lib.load().qlora_linear_fwd(M, n, m, r, float(s), _ptr(x), _ptr(q.codes), _ptr(q.absmax8),
                                          _ptr(q.c2), _ptr(A), _ptr(B), _ptr(h), _ptr(u), _ptr(ws), ws.numel(),
                                          _stream(x.device))
        _lib.check(st, "qlora_linear_fwd")
    else:
        st = _lib.load().qlora_linear_fwd_ex(M, n, m, r, float(s), _ptr(x), _ptr(q.codes), _ptr(q.absmax8),
                                             _ptr(q.c2), _ptr(A), _ptr(B), _ptr(h), _ptr(u), _dropout(dropout),
                                             _ptr(ws), ws.numel(), _stream(x.device))
        _lib.check(st, "qlora_linear_fwd_ex")
    return h, u


def linear_fwd_static(x: torch.Tensor, q: QuantizedWeight, A: torch.Tensor, B: torch.Tensor, s: float,
                      h: torch.Tensor, u: torch.Tensor | None = None):
    """qlora_linear_fwd_static: the forward with the library's own device scratch
    (no workspace).  h (and u, if wanted) must be given: nothing is allocated."""
    M, n = x.shape
    m = q.m
    r = A.shape[0]
    _need(x, torch.bfloat16, (M, q.n), "x")
    _need(A, torch.bfloat16, (r, q.n), "A")
    _need(B, torch.bfloat16, (m, r), "B")
    _need(h, torch.bfloat16, (M, m), "h")
    if u is not None:
        _need(u, torch.float32, (M, r), "u")
    st = _lib.load().qlora_linear_fwd_static(M, n, m, r, float(s), _ptr(x), _ptr(q.codes), _ptr(q.absmax8),
                                             _ptr(q.c2), _ptr(A), _ptr(B), _ptr(h), _ptr(u), _stream(x.device))
    _lib.check(st, "qlora_linear_fwd_static")
    return h, u


class GroupedForward:
    """A reusable grouped forward: outputs, descriptors and workspace are made once.

    layers: sequence of (x, q, A, B, s) as for linear_fwd, all with the same
    token count M.  run() launches the forward of every layer (one launch
    pair for M <= 32) and returns the list of (h, u) output tensors.
    """

    def __init__(self, layers):
        if not layers:
            raise ValueError("no layers")
        self.M = layers[0][0].shape[0]
        self.device = layers[0][0].device
        self.keep = list(layers)
        self.descs = (_lib.LinearLayer * len(layers))()
        self.outs = []
        for i, (x, q, A, B, s) in enumerate(layers):
            r = A.shape[0]
            _need(x, torch.bfloat16, (self.M, q.n), "x")
            _need(A, torch.bfloat16, (r, q.n), "A")
            _need(B, torch.bfloat16, (q.m, r), "B")
            h = torch.empty((self.M, q.m), dtype=torch.bfloat16, device=self.device)
            u = torch.empty((self.M, r), dtype=torch.float32, device=self.device)
            self.outs.append((h, u))
            self.descs[i] = _lib.LinearLayer(q.n, q.m, r, float(s), x.data_ptr(), q.codes.data_ptr(),
                                             q.absmax8.data_ptr(), q.c2.data_ptr(), A.data_ptr(), B.data_ptr(),
                                             h.data_ptr(), u.data_ptr())
        need = _lib.load().qlora_grouped_workspace_bytes(self.M, len(layers), self.descs)
        if need == 0:
            raise ValueError("invalid grouped forward arguments")
        self.workspace = torch.empty(need, dtype=torch.uint8, device=self.device)

    def run(self):
        st = _lib.load().qlora_linear_fwd_grouped(self.M, len(self.keep), self.descs, _ptr(self.workspace),
                                                  self.workspace.numel(), _stream(self.device))
        _lib.check(st, "qlora_linear_fwd_grouped")
        return self.outs


def linear_fwd_grouped(layers):
    """Forward of several layers sharing the token count M, in one call.

    layers: sequence of (x, q, A, B, s) as for linear_fwd.  Returns a list of
    (h, u) pairs.  For M <= 32 all layers are streamed by one launch.
    """
    if not layers:
        return []
    return GroupedForward(layers).run()


def linear_bwd(x: torch.Tensor, g: torch.Tensor, q: QuantizedWeight, A: torch.Tensor, B: torch.Tensor, s: float,
               u: torch.Tensor | None = None, need_grad_x: bool = True, out=None,
               workspace: torch.Tensor | None = None, dropout=None):
    """Returns (grad_x bf16 [M, n] or None, grad_A bf16 [r, n], grad_B bf16 [m, r]).

    dropout: the forward's (p, seed, offset), or None; u, when given, is the
    forward's u (with the mask).  x may be the saved input's Checkpoint8; u is
    then required.
    """
    ckpt = isinstance(x, Checkpoint8)
    M, n = x.shape
    m = q.m
    r = A.shape[0]
    if ckpt:
        if u is None:
            raise ValueError("u: required with a checkpointed input")
        if n != q.n:
            raise ValueError(f"x: expected a checkpoint of {(M, q.n)}, got one of {(M, n)}")
        x.check("x")
    else:
        _need(x, torch.bfloat16, (M, q.n), "x")
    _need(g, torch.bfloat16, (M, m), "g")
    _need(A, torch.bfloat16, (r, n), "A")
    _need(B, torch.bfloat16, (m, r), "B")
    if u is not None:
        _need(u, torch.float32, (M, r), "u")
    if out is None:
        gx = torch.empty((M, n), dtype=torch.bfloat16, device=x.device) if need_grad_x else None
        gA = torch.empty((r, n), dtype=torch.bfloat16, device=x.device)
        gB = torch.empty((m, r), dtype=torch.bfloat16, device=x.device)
    else:
        gx, gA, gB = out
        if gx is not None:
            _need(gx, torch.bfloat16, (M, n), "out[0]")
        _need(gA, torch.bfloat16, (r, n), "out[1]")
        _need(gB, torch.bfloat16, (m, r), "out[2]")
    if ckpt:
        op = QLORA_OP_BWD if dropout is None else QLORA_OP_BWD_DROPOUT
        ws = _workspace(op, M, n, m, r, x.device, workspace)
        st = _lib.load().qlora_linear_bwd_ckpt(M, n, m, r, float(s), _ptr(x.codes), _ptr(x.scales), _ptr(g),
                                               _ptr(q.codes), _ptr(q.absmax8), _ptr(q.c2), _ptr(A), _ptr(B), _ptr(u),
                                               _ptr(gx), _ptr(gA), _ptr(gB), _dropout(dropout), _ptr(ws), ws.numel(),
                                               _stream(x.device))
        _lib.check(st, "qlora_linear_bwd_ckpt")
    elif dropout is None:
        ws = _workspace(QLORA_OP_BWD, M, n, m, r, x.device, workspace)
        st = _lib.load().qlora_linear_bwd(M, n, m, r, float(s), _ptr(x), _ptr(g), _ptr(q.codes), _ptr(q.absmax8),
                                          _ptr(q.c2), _ptr(A), _ptr(B), _ptr(u), _ptr(gx), _ptr(gA), _ptr(gB),
                                          _ptr(ws), ws.numel(), _stream(x.device))
        _lib.check(st, "qlora_linear_bwd")
    else:
        ws = _workspace(QLORA_OP_BWD_DROPOUT, M, n, m, r, x.device, workspace)
        st = _lib.load().qlora_linear_bwd_ex(M, n, m, r, float(s), _ptr(x), _ptr(g), _ptr(q.codes),
                                             _ptr(q.absmax8), _ptr(q.c2), _ptr(A), _ptr(B), _ptr(u), _ptr(gx),
                                             _ptr(gA), _ptr(gB), _dropout(dropout), _ptr(ws), ws.numel(),
                                             _stream(x.device))
        _lib.check(st, "qlora_linear_bwd_ex")
    return gx, gA, gB


def linear_check(op: int, M: int, n: int, m: int, r: int, workspace: torch.Tensor | None) -> None:
    """Raise if the last call of `op` on `workspace` had a bounded wait run out
    (qlora_linear_check; synchronizes the current stream).  workspace None with
    the forward op: the scratch of linear_fwd_static."""
    dev = workspace.device if workspace is not None else None
    st = _lib.load().qlora_linear_check(int(op), M, n, m, r, _ptr(workspace), _stream(dev))
    _lib.check(st, "qlora_linear_check")


def alloc_checkpoint(M: int, n: int, device="cuda") -> Checkpoint8:
    return Checkpoint8(torch.empty((M, n), dtype=torch.int8, device=device),
                       torch.empty((M, checkpoint_pitch(n)), dtype=torch.uint8, device=device))


def checkpoint_pack(x: torch.Tensor, out: Checkpoint8 | None = None) -> Checkpoint8:
    """The 8-bit checkpoint of a bf16 [M, n] tensor (qlora_checkpoint_pack)."""
    M, n = x.shape
    _need(x, torch.bfloat16, (M, n), "x")
    if out is None:
        out = alloc_checkpoint(M, n, x.device)
    else:
        _need(out.codes, torch.int8, (M, n), "out.codes")
        out.check("out")
    st = _lib.load().qlora_checkpoint_pack(M, n, _ptr(x), _ptr(out.codes), _ptr(out.scales), _stream(x.device))
    _lib.check(st, "qlora_checkpoint_pack")
    return out


def checkpoint_unpack(c: Checkpoint8, out: torch.Tensor | None = None) -> torch.Tensor:
    """The bf16 [M, n] tensor that a checkpoint stands for."""
    M, n = c.shape
    c.check("c")
    if out is None:
        out = torch.empty((M, n), dtype=torch.bfloat16, device=c.device)
    else:
        _need(out, torch.bfloat16, (M, n), "out")
    st = _lib.load().qlora_checkpoint_unpack(M, n, _ptr(c.codes), _ptr(c.scales), _ptr(out), _stream(c.device))
    _lib.check(st, "qlora_checkpoint_unpack")
    return out


NORM_LAYER = 0
NORM_RMS = 1
_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_CKPT8 = 2


def _type_of(t: torch.Tensor, name: str) -> int:
    ty = _TYPES.get(t.dtype)
    if ty is None:
        raise TypeError(f"{name}: expected torch.bfloat16 or torch.float32, got {t.dtype}")
    return ty


def norm_fwd(x: torch.Tensor, w: torch.Tensor, b: torch.Tensor | None = None, kind: int = NORM_RMS,
             eps: float = 1e-5, checkpoint: bool = False, out: torch.Tensor | None = None):
    """Layer norm (NORM_LAYER) or RMS norm (NORM_RMS) of the rows of x, bf16 or fp32 [M, n].

    w, b: bf16 or fp32 [n] (fp32 with an fp32 x).  Returns (y, mean, rstd): y like x, mean (None for
    NORM_RMS) and rstd fp32 [M]; with checkpoint=True (bf16 only) also the
    Checkpoint8 of y.
    """
    M, n = x.shape
    xt, wt = _type_of(x, "x"), _type_of(w, "w")
    _need(x, x.dtype, (M, n), "x")
    _need(w, w.dtype, (n,), "w")
    if b is not None:
        _need(b, w.dtype, (n,), "b")
    if out is None:
        out = torch.empty_like(x)
    else:
        _need(out, x.dtype, (M, n), "out")
    mean = torch.empty(M, dtype=torch.float32, device=x.device) if kind == NORM_LAYER else None
    rstd = torch.empty(M, dtype=torch.float32, device=x.device)
    y8 = alloc_checkpoint(M, n, x.device) if checkpoint else None
    st = _lib.load().qlora_norm_fwd(int(kind), xt, wt, M, n, float(eps), _ptr(x), _ptr(w), _ptr(b), _ptr(out),
                                    _ptr(mean), _ptr(rstd), _ptr(y8.codes) if y8 else None,
                                    _ptr(y8.scales) if y8 else None, _stream(x.device))
    _lib.check(st, "qlora_norm_fwd")
    return (out, mean, rstd, y8) if checkpoint else (out, mean, rstd)


def norm_bwd(x, g: torch.Tensor, w: torch.Tensor, rstd: torch.Tensor, mean: torch.Tensor | None = None,
             bias: bool = False, need_grad_w: bool = True, out: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, kind: int | None = None):
    """Backward of norm_fwd: (grad_x like g, grad_w, grad_b like w).

    x: the forward's input or its Checkpoint8 (g is bf16 then).  mean: the
    forward's, None for NORM_RMS.  kind: the forward's; a mean that does not
    go with it, missing or too many, is refused.  Without kind a mean means
    NORM_LAYER and none NORM_RMS.  grad_b is None without bias, both weights'
    gradients without need_grad_w.
    """
    M, n = x.shape
    if kind is None:
        kind = NORM_RMS if mean is None else NORM_LAYER
    elif kind == NORM_LAYER and mean is None:
        raise ValueError("mean: required with NORM_LAYER")
    elif kind == NORM_RMS and mean is not None:
        raise ValueError("mean: NORM_RMS has none")
    if isinstance(x, Checkpoint8):
        x.check("x")
        xt, xp, xs, gtype = _CKPT8, _ptr(x.codes), _ptr(x.scales), torch.bfloat16
    else:
        xt, xp, xs, gtype = _type_of(x, "x"), _ptr(x), None, x.dtype
        _need(x, x.dtype, (M, n), "x")
    wt = _type_of(w, "w")
    _need(g, gtype, (M, n), "g")
    _need(w, w.dtype, (n,), "w")
    _need(rstd, torch.float32, (M,), "rstd")
    if mean is not None:
        _need(mean, torch.float32, (M,), "mean")
    if out is None:
        out = torch.empty_like(g)
    else:
        _need(out, gtype, (M, n), "out")
    gw = torch.empty_like(w) if need_grad_w else None
    gb = torch.empty_like(w) if need_grad_w and bias else None
    lib = _lib.load()
    need = int(lib.qlora_norm_workspace_bytes(int(kind), M, n, 2 if gb is not None else 1 if gw is not None else 0))
    workspace = _room(need, g.device, workspace) if need else None
    st = lib.qlora_norm_bwd(int(kind), xt, wt, M, n, xp, xs, _ptr(g), _ptr(w),
                            _ptr(mean), _ptr(rstd), _ptr(out), _ptr(gw), _ptr(gb), _ptr(workspace),
                            workspace.numel() if workspace is not None else 0, _stream(g.device))
    _lib.check(st, "qlora_norm_bwd")
    return out, gw, gb


@dataclasses.dataclass
class PreferenceResult:
    """What preference_fwd returns; preference_bwd reads lse and coef."""
    loss: torch.Tensor      # float32 [], mean over pairs
    logps: torch.Tensor     # float32 [2 pairs]
    lse: torch.Tensor       # float32 [T]
    coef: torch.Tensor      # float32 [T], dloss / dlog-probability of each token


def _packed(logits, labels, offsets):
    T, V = logits.shape
    ty = _type_of(logits, "logits")
    _need(logits, logits.dtype, (T, V), "logits")
    _need(labels, torch.int64, (T,), "labels")
    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError(f"offsets: expected sequences + 1 values, got shape {tuple(offsets.shape)}")
    _need(offsets, torch.int32, tuple(offsets.shape), "offsets")
    return ty, T, V, offsets.numel() - 1


def _preference_workspace(T, V, pairs, device, workspace):
    return _room(int(_lib.load().qlora_preference_workspace_bytes(T, V, pairs)), device, workspace)


def sequence_logps(logits: torch.Tensor, labels: torch.Tensor, offsets: torch.Tensor,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Log-probability of each packed sequence (fp32 [sequences]).

    logits: bf16 or fp32 [T, V], row t predicting labels[t] (int64 [T]; a
    negative label takes its token out); sequence s is the tokens offsets[s]
    .. offsets[s + 1] - 1 (int32 [sequences + 1], on the device).
    """
    ty, T, V, S = _packed(logits, labels, offsets)
    dev = logits.device
    logps = torch.empty(S, dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    ws = _preference_workspace(T, V, 0, dev, workspace)
    st = _lib.load().qlora_sequence_logps(ty, T, V, S, _ptr(logits), _ptr(labels), _ptr(offsets), _ptr(logps),
                                          _ptr(lse), _ptr(ws), ws.numel(), _stream(dev))
    _lib.check(st, "qlora_sequence_logps")
    return logps


def preference_fwd(logits: torch.Tensor, labels: torch.Tensor, offsets: torch.Tensor,
                   ref_logps: torch.Tensor | None = None, beta: float = 0.1, label_smoothing: float = 0.0,
                   workspace: torch.Tensor | None = None) -> PreferenceResult:
    """Preference loss of packed pairs: sequence 2i is preferred to sequence 2i + 1.

    logits, labels, offsets as for sequence_logps; ref_logps: fp32 [2 pairs],
    the reference model's log-probabilities (None: zeros).
    """
    ty, T, V, S = _packed(logits, labels, offsets)
    if S % 2:
        raise ValueError(f"offsets: pairs need an even number of sequences, got {S}")
    if ref_logps is not None:
        _need(ref_logps, torch.float32, (S,), "ref_logps")
    dev = logits.device
    loss = torch.empty((), dtype=torch.float32, device=dev)
    logps = torch.empty(S, dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    coef = torch.empty(T, dtype=torch.float32, device=dev)
    ws = _preference_workspace(T, V, S // 2, dev, workspace)
    st = _lib.load().qlora_preference_fwd(ty, T, V, S // 2, _ptr(logits), _ptr(labels), _ptr(offsets),
                                          _ptr(ref_logps), float(beta), float(label_smoothing), _ptr(loss),
                                          _ptr(logps), _ptr(lse), _ptr(coef), _ptr(ws), ws.numel(), _stream(dev))
    _lib.check(st, "qlora_preference_fwd")
    return PreferenceResult(loss, logps, lse, coef)


def preference_bwd(logits: torch.Tensor, labels: torch.Tensor, saved: PreferenceResult, grad_scale: float = 1.0,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """grad_scale times the loss's gradient with respect to the logits (out may be the logits themselves)."""
    T, V = logits.shape
    ty = _type_of(logits, "logits")
    _need(logits, logits.dtype, (T, V), "logits")
    _need(labels, torch.int64, (T,), "labels")
    _need(saved.lse, torch.float32, (T,), "saved.lse")
    _need(saved.coef, torch.float32, (T,), "saved.coef")
    if out is None:
        out = torch.empty_like(logits)
    else:
        _need(out, logits.dtype, (T, V), "out")
    st = _lib.load().qlora_preference_bwd(ty, T, V, _ptr(logits), _ptr(labels), _ptr(saved.lse), _ptr(saved.coef),
                                          float(grad_scale), _ptr(out), _stream(logits.device))
    _lib.check(st, "qlora_preference_bwd")
    return out


def profile_enable(on: bool = True) -> None:
    _lib.check(_lib.load().qlora_profile_enable(1 if on else 0), "qlora_profile_enable")


def profile_query(name: str):
    """(launches, total_ms) of a kernel recorded while profiling was on."""
    n = ctypes.c_int64(0)
    ms = ctypes.c_double(0.0)
    _lib.check(_lib.load().qlora_profile_query(name.encode(), ctypes.byref(n), ctypes.byref(ms)),
               "qlora_profile_query")
    return int(n.value), float(ms.value)
