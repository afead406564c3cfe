"""The expert FFN in 8-bit floating point: e4m3 values with one fp32 scale for each block of
128 (include/moe.h, "8-bit floating point").

Thin binding like the rest of the package: the calls carry the C names and write into tensors
that the caller owns.  They also check types, shapes and devices, since a quantised tensor is
a pair whose halves have to match; what does not fit raises ValueError before anything is
enqueued.  The calls run on the tensors' device, on `stream` (None: its current stream).
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass, field
from typing import Optional

import torch

from . import LayerBuffers, MoELayer, _abi, alloc_workspace
from ._abi import MoeConfig, MoeFp8Buffers, MoeFp8Experts, MoeLayerInputs, check

E4M3 = torch.float8_e4m3fn
_CODE = {torch.float32: 0, torch.bfloat16: 1}  # moe_dtype_t
_DTYPE = {v: k for k, v in _CODE.items()}

__all__ = ["moe_fp8_quantize_rows", "moe_fp8_permute_rows", "moe_fp8_quantize_weights",
           "fp8_workspace_size", "alloc_fp8_workspace", "moe_fp8_workspace_init",
           "moe_fp8_grouped_gemm", "moe_expert_ffn_fp8", "moe_layer_forward_fp8",
           "fp8_scale_shape", "Fp8Experts", "Fp8LayerBuffers", "MoELayerFp8"]


def _blocks(n: int) -> int:
    return (n + 127) >> 7


def fp8_scale_shape(shape) -> tuple:
    """Shape of the scales of a quantised tensor: [rows, cols] -> [rows, ceil(cols / 128)],
    [E, N, K] -> [E, ceil(N / 128), ceil(K / 128)]."""
    if len(shape) == 2:
        return (shape[0], _blocks(shape[1]))
    if len(shape) == 3:
        return (shape[0], _blocks(shape[1]), _blocks(shape[2]))
    raise ValueError(f"rows have 2 axes and expert weights 3, got {tuple(shape)}")


def _need(t, name: str, dtype, shape, device) -> int:
    """The address of a contiguous tensor of this type, shape and device."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                     f"{device}, got {t.dtype} {tuple(t.shape)} on {t.device}"
                     f"{'' if t.is_contiguous() else ', not contiguous'}")


def _source(t, name: str, axes: int) -> int:
    if t.dtype not in _CODE or t.dim() != axes or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 or bf16 tensor with {axes} axes, got "
                         f"{t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


# The handle of a device's current stream; torch.cuda.current_stream takes some 2 us to say it,
# as long as a launch.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _handle(device: torch.device, stream) -> int:
    """The handle of `stream` (None: the device's current stream)."""
    if device.type != "cuda":
        raise ValueError(f"the tensors must be on a CUDA device, got {device}")
    if stream is None:
        return _raw_stream(device.index)
    if isinstance(stream, torch.cuda.Stream):
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        return stream.cuda_stream
    return int(stream)


def _call(fn, device: torch.device, stream, *args) -> None:
    """fn(*args, stream) with the tensors' device current."""
    raw = _handle(device, stream)
    if device.index == _current_device():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device.index):
            status = fn(*args, raw)
    if status:
        check(status)


def _allocating_on(stream, device):
    """New tensors' memory comes from work that `stream`, one of `device`, has already been given
    (another stream's may still be in use there when `stream` writes to it)."""
    if stream is None:
        return torch.cuda.device(device)
    if isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    return torch.cuda.stream(torch.cuda.ExternalStream(int(stream), device=device))


def _max_rows(cfg: MoeConfig) -> int:
    return _max_rows_of(bytes(cfg))


@functools.lru_cache(maxsize=256)  # a function of the configuration's values; 1 us to ask for
def _max_rows_of(values: bytes) -> int:
    r = _abi.lib().moe_max_rows(ctypes.byref(MoeConfig.from_buffer_copy(values)))
    if r < 0:
        raise _abi.MoEError(1, _abi.lib().moe_last_error().decode())
    return r


# ------------------------------------------------------------------ quantisation
def moe_fp8_quantize_rows(x, q, scale, stream=None) -> None:
    """x [rows, cols] fp32 or bf16 -> q [rows, cols] e4m3, scale [rows, ceil(cols / 128)]."""
    px = _source(x, "x", 2)
    rows, cols = x.shape
    pq = _need(q, "q", E4M3, x.shape, x.device)
    ps = _need(scale, "scale", torch.float32, (rows, _blocks(cols)), x.device)
    _call(_abi.lib().moe_fp8_quantize_rows, x.device, stream, _CODE[x.dtype], rows, cols, px, pq,
          ps)


def moe_fp8_permute_rows(cfg, x, assign_row, x_q, x_scale, stream=None) -> None:
    """Quantise each token's row of x [T, d_model] once and write it to the bucket rows of its
    kept picks: assign_row [T, k] int32 as moe_dispatch (with x_perm None) wrote it, x_q
    [max_rows, d_model] e4m3, x_scale [max_rows, ceil(d_model / 128)]."""
    d, dev, rows = cfg.d_model, x.device, _max_rows(cfg)
    px = _need(x, "x", _DTYPE[cfg.dtype], (cfg.T, d), dev)
    pa = _need(assign_row, "assign_row", torch.int32, (cfg.T, cfg.k), dev)
    pq = _need(x_q, "x_q", E4M3, (rows, d), dev)
    ps = _need(x_scale, "x_scale", torch.float32, (rows, _blocks(d)), dev)
    _call(_abi.lib().moe_fp8_permute_rows, dev, stream, ctypes.byref(cfg), px, pa, pq, ps)


def moe_fp8_quantize_weights(w, q, scale, stream=None) -> None:
    """w [E, N, K] fp32 or bf16 -> q [E, N, K] e4m3, scale [E, ceil(N / 128), ceil(K / 128)]."""
    pw = _source(w, "w", 3)
    pq = _need(q, "q", E4M3, w.shape, w.device)
    ps = _need(scale, "scale", torch.float32, fp8_scale_shape(w.shape), w.device)
    _call(_abi.lib().moe_fp8_quantize_weights, w.device, stream, _CODE[w.dtype], *w.shape, pw, pq,
          ps)


# ------------------------------------------------------------------ products
def fp8_workspace_size(device="cuda") -> int:
    """Bytes of workspace moe_fp8_grouped_gemm and moe_expert_ffn_fp8 need on the device."""
    n = ctypes.c_size_t(0)
    with torch.cuda.device(device):
        check(_abi.lib().moe_fp8_workspace_size(ctypes.byref(n)))
    return n.value


def alloc_fp8_workspace(device="cuda", stream=None) -> torch.Tensor:
    """A workspace, initialised.  Calls on one workspace must not overlap: one for each stream,
    and for each captured graph that may run beside another."""
    n = fp8_workspace_size(device)
    with _allocating_on(stream, device):
        ws = torch.empty(n, dtype=torch.uint8, device=device)
    moe_fp8_workspace_init(ws, stream)
    return ws


def moe_fp8_workspace_init(ws, stream=None) -> None:
    _call(_abi.lib().moe_fp8_workspace_init, ws.device, stream, ws.data_ptr(), ws.numel())


def _workspace(ws, device) -> tuple:
    if ws.dtype != torch.uint8 or ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on {device}, got {ws.dtype} on "
                         f"{ws.device}")
    return ws.data_ptr(), ws.numel()


def moe_fp8_grouped_gemm(a_q, a_scale, seg_start, seg_count, w_q, w_scale, out, ws,
                         stream=None) -> None:
    """out[r] = a[r] . w[e]^T for the rows r of bucket e = [seg_start[e], + seg_count[e]):
    a_q [rows, K] and w_q [E, N, K] e4m3 with their scales, out [rows, N] bf16; seg_start may
    be dispatch's expert_offsets (its first E entries are read)."""
    if a_q.dim() != 2 or w_q.dim() != 3:
        raise ValueError(f"a_q has 2 axes and w_q 3, got {tuple(a_q.shape)} and "
                         f"{tuple(w_q.shape)}")
    dev, (rows, K), (E, N, Kw) = a_q.device, a_q.shape, w_q.shape
    pa = _need(a_q, "a_q", E4M3, (rows, Kw), dev)
    pas = _need(a_scale, "a_scale", torch.float32, (rows, _blocks(K)), dev)
    pw = _need(w_q, "w_q", E4M3, (E, N, K), dev)
    pws = _need(w_scale, "w_scale", torch.float32, (E, _blocks(N), _blocks(K)), dev)
    pc = _need(seg_count, "seg_count", torch.int32, (E,), dev)
    po = _need(out, "out", torch.bfloat16, (rows, N), dev)
    ps = _starts(seg_start, "seg_start", E, dev)
    wp, wn = _workspace(ws, dev)
    _call(_abi.lib().moe_fp8_grouped_gemm, dev, stream, E, rows, N, K, pa, pas, ps, pc, pw, pws,
          po, wp, wn)


def _starts(t, name: str, E: int, dev) -> int:
    """[E] bucket starts, or [E + 1] offsets."""
    return _need(t, name, torch.int32, (E + 1,) if t.shape == (E + 1,) else (E,), dev)


@dataclass(frozen=True)
class Fp8Experts:
    """The quantised weights of a layer's experts: w_gate, w_up [E, d_ff, d_model], w_down
    [E, d_model, d_ff] e4m3, each with its [E, ceil(N / 128), ceil(K / 128)] fp32 scales."""
    w_gate: torch.Tensor
    gate_scale: torch.Tensor
    w_up: torch.Tensor
    up_scale: torch.Tensor
    w_down: torch.Tensor
    down_scale: torch.Tensor
    struct: MoeFp8Experts = field(init=False, repr=False, compare=False)

    def __post_init__(self):
        if self.w_gate.dim() != 3:
            raise ValueError(f"w_gate has 3 axes, got {tuple(self.w_gate.shape)}")
        E, f, d = self.w_gate.shape
        dev, p = self.w_gate.device, {}
        for name, scale, shape in (("w_gate", "gate_scale", (E, f, d)),
                                   ("w_up", "up_scale", (E, f, d)),
                                   ("w_down", "down_scale", (E, d, f))):
            p[name] = _need(getattr(self, name), name, E4M3, shape, dev)
            p[scale] = _need(getattr(self, scale), scale, torch.float32, fp8_scale_shape(shape),
                             dev)
        object.__setattr__(self, "struct", MoeFp8Experts(**p))

    @staticmethod
    def quantize(w_gate, w_up, w_down, stream=None) -> "Fp8Experts":
        """Quantise a layer's fp32 or bf16 weights."""
        parts = []
        for w in (w_gate, w_up, w_down):
            with _allocating_on(stream, w.device):
                q = torch.empty(w.shape, dtype=E4M3, device=w.device)
                s = torch.empty(fp8_scale_shape(w.shape), dtype=torch.float32, device=w.device)
            moe_fp8_quantize_weights(w, q, s, stream)
            parts += [q, s]
        return Fp8Experts(*parts)


def _fits(cfg, experts: Fp8Experts) -> None:
    if experts.w_gate.shape != (cfg.E, cfg.d_ff, cfg.d_model):
        raise ValueError(f"experts have weights of shape {tuple(experts.w_gate.shape)}, the "
                         f"layer {(cfg.E, cfg.d_ff, cfg.d_model)}")


def moe_expert_ffn_fp8(cfg, x_q, x_scale, expert_offsets, kept_counts, experts: Fp8Experts, h_q,
                       h_scale, y_perm, ws, stream=None) -> None:
    """moe_expert_ffn on quantised rows (moe_fp8_permute_rows) and weights: h_q [max_rows, d_ff]
    e4m3 and h_scale hold the quantised hidden rows, y_perm [max_rows, d_model] bf16."""
    _fits(cfg, experts)
    d, f, E, dev, rows = cfg.d_model, cfg.d_ff, cfg.E, experts.w_gate.device, _max_rows(cfg)
    px = _need(x_q, "x_q", E4M3, (rows, d), dev)
    pxs = _need(x_scale, "x_scale", torch.float32, (rows, _blocks(d)), dev)
    po = _starts(expert_offsets, "expert_offsets", E, dev)
    pk = _need(kept_counts, "kept_counts", torch.int32, (E,), dev)
    ph = _need(h_q, "h_q", E4M3, (rows, f), dev)
    phs = _need(h_scale, "h_scale", torch.float32, (rows, _blocks(f)), dev)
    py = _need(y_perm, "y_perm", torch.bfloat16, (rows, d), dev)
    wp, wn = _workspace(ws, dev)
    _call(_abi.lib().moe_expert_ffn_fp8, dev, stream, ctypes.byref(cfg), px, pxs, po, pk,
          ctypes.byref(experts.struct), ph, phs, py, wp, wn)


# ------------------------------------------------------------------ whole layer
@dataclass
class Fp8LayerBuffers:
    """Every output and intermediate of one layer forward: the layer's own (without x_perm and
    h) and the quantised rows."""
    layer: LayerBuffers
    x_q: torch.Tensor
    x_scale: torch.Tensor
    h_q: torch.Tensor
    h_scale: torch.Tensor

    @staticmethod
    def allocate(cfg: MoeConfig, device="cuda") -> "Fp8LayerBuffers":
        R = max(_max_rows(cfg), 1)
        layer = LayerBuffers.allocate(cfg, device, gather=True, hidden=False)

        def pair(width):
            return (torch.empty((R, width), dtype=E4M3, device=device),
                    torch.empty((R, _blocks(width)), dtype=torch.float32, device=device))

        return Fp8LayerBuffers(layer, *pair(cfg.d_model), *pair(cfg.d_ff))

    def as_struct(self) -> MoeFp8Buffers:
        return MoeFp8Buffers(x_q=self.x_q.data_ptr(), x_scale=self.x_scale.data_ptr(),
                             h_q=self.h_q.data_ptr(), h_scale=self.h_scale.data_ptr())


def moe_layer_forward_fp8(cfg, inputs: MoeLayerInputs, experts: Fp8Experts, bufs, fp8_bufs, ws,
                          fp8_ws, stream=None) -> None:
    """moe_layer_forward with the experts in 8-bit floating point; bufs and fp8_bufs are the
    structs of Fp8LayerBuffers (layer.as_struct(), as_struct())."""
    _fits(cfg, experts)
    dev = experts.w_gate.device
    lp, ln = _workspace(ws, dev)
    wp, wn = _workspace(fp8_ws, dev)
    _call(_abi.lib().moe_layer_forward_fp8, dev, stream, ctypes.byref(cfg), ctypes.byref(inputs),
          ctypes.byref(experts.struct), ctypes.byref(bufs), ctypes.byref(fp8_bufs), lp, ln, wp,
          wn)


class MoELayerFp8(MoELayer):
    """MoELayer with its experts in 8-bit floating point: the same routing, dispatch, combine
    and statistics (bf16 layers), on the experts' device.  forward(x) enqueues the whole layer
    and returns the output, a view of the layer's own buffer that the next call overwrites."""

    def __init__(self, cfg: MoeConfig, w_router, experts: Fp8Experts, logit_bias=None):
        _fits(cfg, experts)
        dev = experts.w_gate.device
        _need(w_router, "w_router", torch.float32, (cfg.d_model, cfg.E), dev)
        if logit_bias is not None:
            one = logit_bias.dim() == 1
            _need(logit_bias, "logit_bias", torch.float32,
                  (cfg.E,) if one else (cfg.T, max(cfg.E, logit_bias.shape[-1])), dev)
        self.cfg, self.w_router, self.experts, self.logit_bias = cfg, w_router, experts, logit_bias
        with torch.cuda.device(dev):
            self.ws = alloc_workspace(cfg, dev)
            self.fp8_ws = alloc_fp8_workspace(dev)
            self.fp8_bufs = Fp8LayerBuffers.allocate(cfg, dev)
            self.bufs = self.fp8_bufs.layer
            self._structs = self.bufs.as_struct(True), self.fp8_bufs.as_struct()
            self.resplit_router()

    def resplit_router(self, stream=None) -> None:
        dev = self.experts.w_gate.device
        raw = _handle(dev, stream)
        with _allocating_on(stream, dev):
            super().resplit_router(raw)

    def pick_rank_counts(self, group_of_expert=None, stream=None):
        dev = self.experts.w_gate.device
        raw = _handle(dev, stream)
        with _allocating_on(stream, dev):
            return super().pick_rank_counts(group_of_expert, raw)

    def inputs(self, x) -> MoeLayerInputs:
        b, split = self.logit_bias, self.w_router_split
        px = _need(x, "x", torch.bfloat16, (self.cfg.T, self.cfg.d_model),
                   self.experts.w_gate.device)
        return MoeLayerInputs(
            x=px, w_router=self.w_router.data_ptr(),
            logit_bias=None if b is None else b.data_ptr(),
            bias_row_stride=0 if (b is None or b.dim() == 1) else b.shape[1],
            w_router_split=None if split is None else split.data_ptr())

    def forward(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        moe_layer_forward_fp8(self.cfg, self.inputs(x), self.experts, *self._structs, self.ws,
                              self.fp8_ws, stream)
        return self.bufs.out

    __call__ = forward

    def check_device_error(self, stream: Optional[torch.cuda.Stream] = None) -> None:
        """Report (MoEError) and clear the kernel-side errors of the forwards so far: of both
        workspaces, the first one's error first.  Any error of the products' workspace has it
        initialised again: a wait that ran out leaves counters behind, and the status, which
        keeps the first error alone, may show another."""
        check_error = _abi.lib().moe_check_device_error
        found = []
        for ws in (self.ws, self.fp8_ws):
            try:
                _call(check_error, ws.device, stream, ws.data_ptr(), ws.numel())
            except _abi.MoEError as e:
                found.append(e)
                if ws is self.fp8_ws:
                    try:
                        moe_fp8_workspace_init(ws, stream)
                    except _abi.MoEError as failed:
                        found.append(failed)
        if found:
            raise found[0]
