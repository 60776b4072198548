"""Thin Python binding of include/moe_decode.h (ctypes; argument marshalling only).

Every step of the block runs in libmoe_decode.so.  PyTorch supplies device memory and streams.
If the library is missing this module raises; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import os
import struct
import threading

import numpy as np
import torch

from . import synth
from .workloads import Shape

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_decode.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_OOM, MOE_ERR_BAD_ID = (
    0, -1, -2, -3, -4, -5)
DTYPE_BF16, DTYPE_F32, DTYPE_F16 = 0, 1, 2
TREE_MAX_Q = 64
PART_GATE_UP, PART_DOWN = 1, 2
KERNELS_FUSED, KERNELS_SEPARATE, KERNELS_COLUMNS, KERNELS_COLUMNS_AHEAD, KERNELS_POOL = 0, 1, 2, 3, 4
KERNELS_MMA = 5
NOALLOC_MAX_ACT_FLOATS = 65536
_STATUS = {0: "MOE_OK", -1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_UNSUPPORTED", -3: "MOE_ERR_CUDA",
           -4: "MOE_ERR_OOM", -5: "MOE_ERR_BAD_ID", -6: "MOE_ERR_TIMEOUT",
           -7: "MOE_ERR_PLAN"}

EXPORTS = ["moe_decode_create", "moe_decode_forward", "moe_decode_get_error", "moe_decode_destroy",
           "moe_decode_routes",
           "moe_decode_forward_noalloc",
           "moe_gemv_bf16",
           "moe_stack_create", "moe_stack_create_chained", "moe_stack_step",
           "moe_stack_step_parts", "moe_stack_step_host",
           "moe_stack_get_error",
           "moe_stack_destroy", "moe_pack_codes", "moe_unpack_codes", "moe_unpack_codes_device",
           "moe_synth_codes", "moe_synth_scales", "moe_synth_biases", "moe_route_invert_device",
           "moe_debug_wait_timeout", "moe_router_topk", "moe_debug_col_pieces",
           "moe_debug_col_plan", "moe_qk_norm_rope", "moe_tree_attention_workspace",
           "moe_tree_attention", "moe_prompt_attention_workspace", "moe_prompt_attention",
           "moe_prefix_attention_workspace", "moe_prefix_attention", "moe_page_bounds",
           "moe_select_pages_workspace", "moe_select_pages",
           "moe_sparse_attention_workspace", "moe_sparse_attention",
           "moe_debug_attention_wait_cycles"]


class MoeError(RuntimeError):
    def __init__(self, fn, rc):
        super().__init__(f"{fn} returned {_STATUS.get(rc, rc)}")
        self.rc = rc


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "din", "dff", "n_experts", "top_k", "max_tokens", "bits_gate", "bits_up", "bits_down",
        "n_shared", "dff_shared", "bits_shared", "shared_gate", "resid_dtype", "out_dtype",
        "kernel_mode")]


class Proj(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("biases", ctypes.c_void_p)]


class LayerWeights(ctypes.Structure):
    _fields_ = [("gate", Proj), ("up", Proj), ("down", Proj), ("sh_gate", Proj), ("sh_up", Proj),
                ("sh_down", Proj), ("gate_vec", ctypes.c_void_p)]


# The structs of the attention calls as packed bytes (native alignment, the C layout): one pack() is
# much cheaper than filling a ctypes.Structure field by field, and these calls take microseconds.
_pack_kv_cache = struct.Struct("@2P3q5i").pack
_pack_norm_rope = struct.Struct("@3P6qP2q6P5if").pack
_pack_attention = struct.Struct("@2P4q3Pq4ifP").pack


_lock = threading.Lock()
_lib = None
_timeline = False


def use_timeline_build() -> None:
    """Load libmoe_decode_timeline.so (the column-split kernel records per-CTA, per-layer time
    stamps, read by MoeStack.timeline) instead of the product library.  Call before lib()."""
    global LIB_PATH, _timeline
    with _lock:
        if _lib is not None:
            raise RuntimeError("the library is already loaded")
        LIB_PATH = os.path.join(_HERE, "libmoe_decode_timeline.so")
        _timeline = True


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it was not built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: run __graft_entry__.build() or "
                                   "python -m quantized_moe_expert_dequant_gb300.build")
            L = ctypes.CDLL(LIB_PATH)
            vp, i32, i64, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
            sig = {
                "moe_decode_create": [ctypes.POINTER(Config), ctypes.POINTER(LayerWeights),
                                      ctypes.POINTER(vp)],
                "moe_decode_forward": [vp, vp, i32, vp, vp, vp, vp, vp],
                "moe_decode_get_error": [vp, ctypes.POINTER(i32)],
                "moe_decode_routes": [vp, vp, vp, vp],
                "moe_decode_destroy": [vp],
                "moe_decode_forward_noalloc": [ctypes.POINTER(Config), ctypes.POINTER(LayerWeights),
                                               vp, i32, vp, vp, vp, vp, vp, vp],
                "moe_stack_create": [ctypes.POINTER(Config), i32, ctypes.POINTER(LayerWeights),
                                     ctypes.POINTER(vp)],
                "moe_gemv_bf16": [vp, vp, ctypes.c_int64, vp, i32, i32, i32, i32, vp],
                "moe_stack_create_chained": [ctypes.POINTER(Config), i32,
                                             ctypes.POINTER(LayerWeights), vp, ctypes.c_float,
                                             ctypes.POINTER(vp)],
                "moe_stack_step": [vp, vp, i32, vp, vp, vp, vp, vp],
                "moe_stack_step_parts": [vp, i32, vp, i32, vp, vp, vp, vp, vp],
                "moe_stack_step_host": [vp, vp, i32, vp, vp, vp, vp, vp],
                "moe_stack_get_error": [vp, ctypes.POINTER(i32)],
                "moe_stack_destroy": [vp],
                "moe_pack_codes": [vp, i64, i64, i32, vp],
                "moe_unpack_codes": [vp, i64, i64, i32, vp],
                "moe_unpack_codes_device": [vp, i64, i64, i32, vp, vp],
                "moe_synth_codes": [vp, u64, i32, i32, i64, vp],
                "moe_synth_scales": [vp, u64, i32, i32, i64, vp],
                "moe_synth_biases": [vp, vp, u64, i32, i32, i64, i32, vp],
                "moe_route_invert_device": [vp, i32, i32, i32, vp, vp],
                "moe_debug_wait_timeout": [i32, vp, vp, vp],
                "moe_router_topk": [vp, i32, i32, i32, vp, vp, vp],
                "moe_debug_col_pieces": [i32, i32, i32, i32, i32, i32, i32, i32, vp, i32],
                "moe_debug_col_plan": [ctypes.POINTER(Config), i32, i32, vp, vp],
                "moe_qk_norm_rope": [vp, vp, vp],
                "moe_tree_attention_workspace": [vp, vp, i32, vp],
                "moe_tree_attention": [vp, vp, vp, i32, vp, i64, vp],
                "moe_prefix_attention_workspace": [vp, vp, i32, i32, vp],
                "moe_prefix_attention": [vp, vp, vp, vp, i32, vp, i32, vp, i64, vp],
                "moe_page_bounds": [vp, vp, vp, vp],
                "moe_select_pages_workspace": [vp, vp, vp],
                "moe_select_pages": [vp, vp, vp, i32, i32, i32, vp, vp, i64, vp],
                "moe_sparse_attention_workspace": [vp, vp, i32, vp],
                "moe_sparse_attention": [vp, vp, vp, i32, vp, i64, vp],
                "moe_prompt_attention_workspace": [vp, vp, vp],
                "moe_prompt_attention": [vp, vp, vp, i64, vp],
                "moe_debug_attention_wait_cycles": [i64],
            }
            if _timeline:
                sig["moe_stack_timeline"] = [vp, vp, i64, ctypes.POINTER(i32)]
            for name, args in sig.items():
                f = getattr(L, name)
                f.argtypes = args
                f.restype = None if name.endswith("_destroy") else ctypes.c_int
            _lib = L
    return _lib


def check(fn: str, rc: int) -> None:
    if rc != MOE_OK:
        raise MoeError(fn, rc)


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _p(t) -> int | None:
    return None if t is None else t.data_ptr()


def config(shape: Shape, max_tokens: int = 1, resid_dtype: int = DTYPE_BF16,
           out_dtype: int = DTYPE_F32, kernel_mode: int = KERNELS_FUSED) -> Config:
    return Config(shape.din, shape.dff, shape.n_experts, shape.top_k, max_tokens, shape.bits_gate,
                  shape.bits_up, shape.bits_down, shape.n_shared, shape.dff_shared,
                  shape.bits_shared, shape.shared_gate, resid_dtype, out_dtype, kernel_mode)


# ---------------------------------------------------------------- device weights

@dataclasses.dataclass
class DeviceProj:
    codes: torch.Tensor   # uint8 [E, rows, rowbytes]
    scales: torch.Tensor  # fp16 [E, rows, cols/64]
    biases: torch.Tensor  # fp16 [E, rows, cols/64]

    def struct(self) -> Proj:
        return Proj(self.codes.data_ptr(), self.scales.data_ptr(), self.biases.data_ptr())

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.codes, self.scales, self.biases))


@dataclasses.dataclass
class DeviceLayer:
    shape: Shape
    gate: DeviceProj | None
    up: DeviceProj | None
    down: DeviceProj | None
    sh_gate: DeviceProj | None = None
    sh_up: DeviceProj | None = None
    sh_down: DeviceProj | None = None
    gate_vec: torch.Tensor | None = None   # bf16 [din]

    def struct(self) -> LayerWeights:
        z = Proj(None, None, None)
        f = lambda p: p.struct() if p is not None else z
        return LayerWeights(f(self.gate), f(self.up), f(self.down), f(self.sh_gate),
                            f(self.sh_up), f(self.sh_down), _p(self.gate_vec))


def _empty_proj(n, rows, cols, bits, device) -> DeviceProj:
    return DeviceProj(torch.empty((n, rows, cols * bits // 8), dtype=torch.uint8, device=device),
                      torch.empty((n, rows, cols // 64), dtype=torch.float16, device=device),
                      torch.empty((n, rows, cols // 64), dtype=torch.float16, device=device))


def synth_proj_device(seed, layer, proj, n, rows, cols, bits, device="cuda", stream=None):
    """All n experts of one projection drawn in HBM by the device generator."""
    p = _empty_proj(n, rows, cols, bits, device)
    L, st = lib(), _stream(stream)
    words = rows * cols * bits // 8 // 8
    groups = rows * (cols // 64)
    check("moe_synth_codes", L.moe_synth_codes(
        p.codes.data_ptr(), synth.tensor_key(seed, layer, proj, synth.CODES), 0, n, words, st))
    check("moe_synth_scales", L.moe_synth_scales(
        p.scales.data_ptr(), synth.tensor_key(seed, layer, proj, synth.SCALES), 0, n, groups, st))
    check("moe_synth_biases", L.moe_synth_biases(
        p.biases.data_ptr(), p.scales.data_ptr(), synth.tensor_key(seed, layer, proj, synth.BIASES),
        0, n, groups, bits, st))
    return p


def synth_layer_device(shape: Shape, layer: int, device="cuda", stream=None) -> DeviceLayer:
    s, E = shape.seed, shape.n_experts
    mk = lambda proj, n, r, c, b: synth_proj_device(s, layer, proj, n, r, c, b, device, stream)
    dl = DeviceLayer(shape, None, None, None)
    if shape.top_k > 0:
        dl.gate = mk(synth.GATE, E, shape.dff, shape.din, shape.bits_gate)
        dl.up = mk(synth.UP, E, shape.dff, shape.din, shape.bits_up)
        dl.down = mk(synth.DOWN, E, shape.din, shape.dff, shape.bits_down)
    if shape.n_shared:
        n, d, b = shape.n_shared, shape.dff_shared, shape.bits_shared
        dl.sh_gate = mk(synth.SH_GATE, n, d, shape.din, b)
        dl.sh_up = mk(synth.SH_UP, n, d, shape.din, b)
        dl.sh_down = mk(synth.SH_DOWN, n, shape.din, d, b)
        if shape.shared_gate:
            dl.gate_vec = torch.from_numpy(
                synth.gate_vector(s, layer, shape.din).view(np.int16)).view(torch.bfloat16).to(device)
    return dl


def proj_from_host(codes, scales, biases, device="cuda") -> DeviceProj:
    """Stacked host arrays (uint8 codes, uint16 fp16 bits) copied to the device."""
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).view(dt).to(device)
    return DeviceProj(t(codes, torch.uint8), t(scales.view(np.int16), torch.float16),
                      t(biases.view(np.int16), torch.float16))


# ---------------------------------------------------------------- the block

class MoeDecode:
    """One prepared layer: moe_decode_create once, moe_decode_forward per token batch."""

    def __init__(self, layer: DeviceLayer, max_tokens: int = 1, resid_dtype=DTYPE_BF16,
                 out_dtype=DTYPE_F32, kernel_mode: int = KERNELS_FUSED):
        self.layer = layer
        self.cfg = config(layer.shape, max_tokens, resid_dtype, out_dtype, kernel_mode)
        self._w = layer.struct()
        h = ctypes.c_void_p()
        check("moe_decode_create", lib().moe_decode_create(ctypes.byref(self.cfg),
                                                           ctypes.byref(self._w), ctypes.byref(h)))
        self.handle = h

    def forward(self, x: torch.Tensor, ids: torch.Tensor | None, scores: torch.Tensor | None,
                resid: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """x bf16 [m, din]; ids int32 [m, K]; scores fp32 [m, K]; resid [m, din]; out [m, din]."""
        m = x.shape[0] if x.dim() == 2 else 1
        if out is None:
            dt = torch.float32 if self.cfg.out_dtype == DTYPE_F32 else torch.bfloat16
            out = torch.empty((m, self.cfg.din), dtype=dt, device=x.device)
        check("moe_decode_forward", lib().moe_decode_forward(
            self.handle, _p(x), m, _p(ids), _p(scores), _p(resid), _p(out), _stream(stream)))
        return out

    def routes(self, m: int, slots: bool = False, stream=None):
        """The ids the last forward's kernels read, int32 [m, top_k], and (pool mode, slots=True)
        each slot's and shared expert's down output before its coefficient, fp32
        [m, top_k + n_shared, din]; device tensors (moe_decode_routes)."""
        sh = self.layer.shape
        ids = torch.empty((m, max(sh.top_k, 1)), dtype=torch.int32, device="cuda")
        y = (torch.empty((m, sh.top_k + sh.n_shared, sh.din), dtype=torch.float32, device="cuda")
             if slots else None)
        check("moe_decode_routes", lib().moe_decode_routes(self.handle, _p(ids), _p(y),
                                                           _stream(stream)))
        return (ids[:, :sh.top_k], y) if slots else ids[:, :sh.top_k]

    def get_error(self) -> int:
        v = ctypes.c_int32()
        check("moe_decode_get_error", lib().moe_decode_get_error(self.handle, ctypes.byref(v)))
        return v.value

    def close(self):
        if self.handle:
            lib().moe_decode_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def forward_noalloc(layer: "DeviceLayer", x: torch.Tensor, ids: torch.Tensor | None,
                    scores: torch.Tensor | None, resid: torch.Tensor, out: torch.Tensor,
                    device_error: torch.Tensor | None = None, max_tokens: int | None = None,
                    resid_dtype=DTYPE_BF16, out_dtype=DTYPE_F32, stream=None) -> torch.Tensor:
    """moe_decode_forward_noalloc: one layer without a handle, activations in the library's
    fixed scratch array (two-kernel mode).  `out` must be given; `device_error` is an int32
    device tensor of one element that must start at 0."""
    m = x.shape[0] if x.dim() == 2 else 1
    cfg = config(layer.shape, max_tokens or m, resid_dtype, out_dtype, KERNELS_SEPARATE)
    w = layer.struct()
    check("moe_decode_forward_noalloc", lib().moe_decode_forward_noalloc(
        ctypes.byref(cfg), ctypes.byref(w), _p(x), m, _p(ids), _p(scores), _p(resid), _p(out),
        _p(device_error), _stream(stream)))
    return out


class MoeStack:
    """A stack of layers replayed as one CUDA graph per decode step.

    norm_weight (bf16 [L - 1, din] on the device) folds the next layer's RMSNorm in
    (moe_stack_create_chained): layer l >= 1 then reads RMSNorm(out of layer l - 1) instead of x,
    and step() reads x as [m, din]."""

    def __init__(self, layers: list[DeviceLayer], max_tokens: int = 1, resid_dtype=DTYPE_BF16,
                 kernel_mode: int = KERNELS_FUSED, norm_weight=None, eps: float = 1e-6):
        self.layers = layers
        self.cfg = config(layers[0].shape, max_tokens, resid_dtype, DTYPE_F32, kernel_mode)
        arr = (LayerWeights * len(layers))()
        for i, l in enumerate(layers):
            arr[i] = l.struct()
        self._w = arr
        self._norm = norm_weight
        h = ctypes.c_void_p()
        if norm_weight is None:
            check("moe_stack_create", lib().moe_stack_create(ctypes.byref(self.cfg), len(layers),
                                                             arr, ctypes.byref(h)))
        else:
            check("moe_stack_create_chained", lib().moe_stack_create_chained(
                ctypes.byref(self.cfg), len(layers), arr, _p(norm_weight), eps, ctypes.byref(h)))
        self.handle = h

    def step(self, x, ids, scores, resid0, out, stream=None):
        """x bf16 [L, m, din]; ids int32 [L, m, K]; scores fp32 [L, m, K]; resid0 [m, din];
        out fp32 [m, din]; all on the device."""
        m = resid0.shape[0]
        check("moe_stack_step", lib().moe_stack_step(self.handle, _p(x), m, _p(ids), _p(scores),
                                                     _p(resid0), _p(out), _stream(stream)))
        return out

    def step_parts(self, parts, x, ids, scores, resid0, out, stream=None):
        """Only kernel A (parts=1) or only kernel B (parts=2) of every layer: a timing aid."""
        m = resid0.shape[0]
        check("moe_stack_step_parts", lib().moe_stack_step_parts(
            self.handle, parts, _p(x), m, _p(ids), _p(scores), _p(resid0), _p(out),
            _stream(stream)))
        return out

    def step_host(self, x, ids, scores, resid0, out, stream=None):
        """The same step from host (ideally pinned) tensors; returns after out is on the host."""
        m = resid0.shape[0]
        check("moe_stack_step_host", lib().moe_stack_step_host(
            self.handle, _p(x), m, _p(ids), _p(scores), _p(resid0), _p(out), _stream(stream)))
        return out

    def get_error(self) -> int:
        v = ctypes.c_int32()
        check("moe_stack_get_error", lib().moe_stack_get_error(self.handle, ctypes.byref(v)))
        return v.value

    def timeline(self) -> np.ndarray:
        """Timeline build only: the column-split kernel's stamps of the last step,
        uint64 [grid, L, points] (see moe_timeline.cuh)."""
        P = 64  # kTlPoints
        buf = np.zeros(512 * len(self.layers) * P, np.uint64)
        g = ctypes.c_int32()
        check("moe_stack_timeline", lib().moe_stack_timeline(
            self.handle, buf.ctypes.data, buf.nbytes, ctypes.byref(g)))
        return buf[:g.value * len(self.layers) * P].reshape(g.value, len(self.layers), P)

    def close(self):
        if self.handle:
            lib().moe_stack_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------- packing

def pack_codes(codes: np.ndarray, bits: int) -> np.ndarray:
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    rows, cols = codes.shape
    out = np.empty((rows, cols * bits // 8), dtype=np.uint8)
    check("moe_pack_codes", lib().moe_pack_codes(codes.ctypes.data, rows, cols, bits,
                                                 out.ctypes.data))
    return out


def unpack_codes(packed: np.ndarray, cols: int, bits: int) -> np.ndarray:
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    rows = packed.shape[0]
    out = np.empty((rows, cols), dtype=np.uint8)
    check("moe_unpack_codes", lib().moe_unpack_codes(packed.ctypes.data, rows, cols, bits,
                                                     out.ctypes.data))
    return out


def unpack_codes_device(packed: torch.Tensor, cols: int, bits: int, stream=None) -> torch.Tensor:
    rows = packed.shape[0]
    out = torch.empty((rows, cols), dtype=torch.uint8, device=packed.device)
    check("moe_unpack_codes_device", lib().moe_unpack_codes_device(
        packed.data_ptr(), rows, cols, bits, out.data_ptr(), _stream(stream)))
    return out


def route_invert_device(ids: torch.Tensor, n_experts: int, stream=None):
    """The kernels' route inversion of ids int32 [m, k] (device): (uniq, offs, pairs) as numpy."""
    m, k = ids.shape
    out = torch.full((2 + 3 * m * k,), -7, dtype=torch.int32, device=ids.device)
    check("moe_route_invert_device", lib().moe_route_invert_device(
        _p(ids.contiguous()), m, k, n_experts, _p(out), _stream(stream)))
    o = out.cpu().numpy()
    u = int(o[0])
    uniq = o[1:1 + u]
    offs = o[1 + u:2 + 2 * u]
    pairs = o[2 + 2 * u:2 + 2 * u + int(offs[-1])]
    return uniq.copy(), offs.copy(), pairs.copy()


def debug_wait_timeout(kind: int, device_error: torch.Tensor, stream=None) -> None:
    """Runs the kernels' bounded wait on a condition nothing satisfies (kind 0: grid-barrier
    count, 1: mbarrier stage); the time-out bit lands in device_error (int32 [1], device)."""
    scratch = torch.zeros(1, dtype=torch.int32, device=device_error.device)
    check("moe_debug_wait_timeout", lib().moe_debug_wait_timeout(kind, _p(scratch), _p(device_error),
                                                                 _stream(stream)))


def debug_attention_wait_cycles(cycles: int) -> None:
    """The limit in cycles of the waits in attention kernels launched from now on (0: the usual)."""
    check("moe_debug_attention_wait_cycles", lib().moe_debug_attention_wait_cycles(cycles))


def router_topk(logits: torch.Tensor, top_k: int, stream=None):
    """moe_router_topk on fp32 logits [m, E] (device): (ids int32 [m, top_k], scores fp32)."""
    m, E = logits.shape
    ids = torch.empty((m, top_k), dtype=torch.int32, device=logits.device)
    scores = torch.empty((m, top_k), dtype=torch.float32, device=logits.device)
    check("moe_router_topk", lib().moe_router_topk(_p(logits.contiguous()), m, E, top_k, _p(ids),
                                                   _p(scores), _stream(stream)))
    return ids, scores


def col_pieces(top_k: int, dff: int, n_shared: int, dff_shared: int, bits_down: int,
               bits_shared: int, u0: int, u1: int, max_pieces: int = 64):
    """The column split's pieces of the activation columns [u0, u1) (host only):
    [(seg, j0, j1, a0, blk0, nb, pb, grp), ...]."""
    import numpy as np
    out = np.zeros(8 * max_pieces, dtype=np.int32)
    rc = lib().moe_debug_col_pieces(top_k, dff, n_shared, dff_shared, bits_down, bits_shared, u0,
                                    u1, out.ctypes.data, max_pieces)
    check("moe_debug_col_pieces", min(rc, 0))
    return [tuple(int(v) for v in out[8 * q:8 + 8 * q]) for q in range(rc)]


def col_plan(shape, grid: int, ring_bytes: int) -> dict:
    """The column split's launch plan for a workload shape (host only); "bounds": the CTAs'
    column ranges, CTA c owning [bounds[c], bounds[c + 1])."""
    import numpy as np
    cfg = config(shape, 1, DTYPE_BF16, DTYPE_F32, KERNELS_COLUMNS)
    out = np.zeros(10, dtype=np.int32)
    bounds = np.zeros(grid + 1, dtype=np.int32)
    check("moe_debug_col_plan", lib().moe_debug_col_plan(ctypes.byref(cfg), grid, ring_bytes,
                                                         out.ctypes.data, bounds.ctypes.data))
    keys = ("stages", "stage_bytes", "nbs", "ro", "cb_r", "cb_s", "rows_a_r", "rows_a_s", "pack",
            "prefetch")
    plan = dict(zip(keys, (int(v) for v in out)))
    plan["bounds"] = [int(v) for v in bounds]
    return plan


# ---------------------------------------------------------------- dense bf16 decode GEMV

def gemv_bf16(W, x, y=None, shared_x: bool = True, stream=None):
    """y [n_mats, m, n_out] fp32 = x W^T for every matrix of W (bf16 [n_mats, n_out, n_in] on
    the device).  x is bf16 [m, n_in] (shared_x) or [n_mats, m, n_in]."""
    import torch
    n_mats, n_out, n_in = W.shape
    m = x.shape[-2]
    if y is None:
        y = torch.empty((n_mats, m, n_out), dtype=torch.float32, device=W.device)
    x_stride = 0 if shared_x else m * n_in
    check("moe_gemv_bf16", lib().moe_gemv_bf16(_p(W), _p(x), x_stride, _p(y), n_mats, m, n_out,
                                               n_in, _stream(stream)))
    return y


# ---------------------------------------------------------------- the attention half of a layer

_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32, torch.float16: DTYPE_F16}


def _vector(t, dtype, n, dev, name) -> int:
    """The address of a contiguous tensor of n elements (at least) on GPU `dev`; 0 for None."""
    if t is None:
        return 0
    if t.dtype != dtype or t.numel() < n or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of {n} elements on cuda:{dev} is "
                         f"wanted, not {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(t, shape, dtype, dev, name):
    """(address, row stride, head stride) of a tensor [rows, heads, dim]."""
    st = t.stride()
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev or st[2] != 1:
        raise ValueError(f"{name}: {dtype} {shape} on cuda:{dev} with elements side by side is "
                         f"wanted, not {t.dtype} {tuple(t.shape)} on {t.device}, strides {st}")
    return t.data_ptr(), st[0] if shape[0] > 1 else 0, st[1] if shape[1] > 1 else 0


def _empty_on(shape, dtype, device, stream):
    """An uninitialised tensor whose memory is ordered on `stream` (None: the current one)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


@functools.lru_cache(maxsize=None)
def _entry(fn: str):
    return getattr(lib(), fn)


def _on(dev: int, fn: str, *args) -> None:
    """One library call with GPU `dev` current: launches and plans go by the current one."""
    if torch._C._cuda_getDevice() == dev:
        rc = _entry(fn)(*args)
    else:
        with torch.cuda.device(dev):
            rc = _entry(fn)(*args)
    if rc != MOE_OK:
        raise MoeError(fn, rc)


def _call(fn: str, dev: int, stream, *args) -> None:
    """One library call on `stream` (None: the current one of GPU `dev`) with that GPU current."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    _on(dev, fn, *args, stream)


class KvCache:
    """The pages of a key/value cache: k and v are [n_pages, n_kv_heads, page_size, head_dim],
    bf16 or fp16, with the same strides (the last 1, the others multiples of 8); a permuted
    [n_pages, page_size, n_kv_heads, head_dim] does as well."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if not (k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype
                and k.stride() == v.stride() and k.stride(3) == 1 and k.device == v.device
                and k.is_cuda):
            raise ValueError("k and v: [n_pages, n_kv_heads, page_size, head_dim] alike, on a GPU")
        if k.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("k and v: bf16 or fp16")
        self.k, self.v = k, v
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.device, self.dtype = k.device, k.dtype
        self._dev = k.get_device()
        self._heads = (self.n_kv_heads, self.head_dim)
        st = [k.stride(i) if k.shape[i] > 1 else 0 for i in range(3)]
        self._sizes = {}  # of workspaces, by what they go by
        self._bounds = torch.Size((self.n_pages, self.n_kv_heads, 2, self.head_dim))
        self._shape = (self.n_pages, self.n_kv_heads, self.page_size, self.head_dim, _DTYPES[k.dtype])
        self._c = _pack_kv_cache(k.data_ptr(), v.data_ptr(), *st, self.n_pages, self.page_size,
                                 self.n_kv_heads, self.head_dim, _DTYPES[k.dtype])


def qk_norm_rope(cache: KvCache, q, k, v, positions, slots, inv_freq, q_weight=None, k_weight=None,
                 eps: float = 1e-6, interleaved: bool = False, q_out=None, device_error=None,
                 stream=None):
    """moe_qk_norm_rope: norms and rotates the heads of q [T, Hq, D] and k [T, Hkv, D] (fp32 or the
    cache's dtype), writes k and v [T, Hkv, D] to their slots (int32 [T]; negative: padding) in
    the cache and returns q_out [T, Hq, D] in the cache's dtype.  positions int32 [T], inv_freq fp64
    [rot_dim / 2] (None: no rotation), weights [D] in the cache's dtype or None: no norm.  The rows of
    padding are not written: in a q_out made here they are uninitialised memory.  device_error: int32
    [1], whose bit 1 a slot outside the cache sets (its key and value are not written)."""
    shape = q.shape
    T, Hq, D = shape
    dev, dt, to, kv, i32 = cache._dev, q.dtype, cache.dtype, (T, *cache._heads), torch.int32
    if D != cache.head_dim or dt not in _DTYPES:
        raise ValueError(f"q: fp32 or {to} heads of {cache.head_dim} are wanted")
    if q_out is None:
        q_out = _empty_on(shape, to, cache.device, stream)
    # the checks of _rows and _vector in one expression for the calls that pass them: on small
    # batches the host is what takes time
    a, b, c, o = q.stride(), k.stride(), v.stride(), q_out.stride()
    if (a[2] == b[2] == c[2] == o[2] == 1 and k.shape == kv and v.shape == kv and k.dtype is dt
            and v.dtype is dt and q_out.dtype is to and q_out.shape == shape
            and q.get_device() == k.get_device() == v.get_device() == q_out.get_device() == dev
            and slots.dtype is i32 and slots.numel() >= T and slots.is_contiguous()
            and slots.get_device() == dev):
        ptrs = q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), slots.data_ptr()
    else:
        ptrs = (*(_rows(t, n, d, dev, name)[0] for t, n, d, name in (
            (q, shape, dt, "q"), (k, kv, dt, "k"), (v, kv, dt, "v"), (q_out, shape, to, "q_out"))),
            _vector(slots, i32, T, dev, "slots"))
    many, heads, kv_heads = T > 1, Hq > 1, kv[1] > 1  # a dimension of extent 1 may have any stride
    args = _pack_norm_rope(
        ptrs[0], ptrs[1], ptrs[2], a[0] if many else 0, a[1] if heads else 0, b[0] if many else 0,
        b[1] if kv_heads else 0, c[0] if many else 0, c[1] if kv_heads else 0, ptrs[3],
        o[0] if many else 0, o[1] if heads else 0,
        0 if q_weight is None else _vector(q_weight, to, D, dev, "q_weight"),
        0 if k_weight is None else _vector(k_weight, to, D, dev, "k_weight"),
        0 if inv_freq is None else _vector(inv_freq, torch.float64, 1, dev, "inv_freq"),
        _vector(positions, i32, T, dev, "positions"), ptrs[4],
        0 if device_error is None else _vector(device_error, i32, 1, dev, "device_error"), T, Hq,
        0 if inv_freq is None else 2 * inv_freq.numel(), interleaved, _DTYPES[dt], eps)
    _call("moe_qk_norm_rope", dev, stream, cache._c, args)
    return q_out


_NONE = (0, 0, 0)  # for a tensor that a call does not use


def _batch_args(cache, a, b, T, Hq, scale, cu_q, ctx_len, page_table, device_error):
    """moe_attention of q and out as _rows gives them; T rows of Hq query heads."""
    dev, i32 = cache._dev, torch.int32
    n, width = page_table.shape
    st = page_table.stride()
    if page_table.dtype is not i32 or page_table.get_device() != dev or (st[1] != 1 and width > 1):
        raise ValueError(f"page_table: int32 [n_seqs, width] on cuda:{dev} is wanted")
    # the checks of _vector in one expression for the calls that pass them: on small batches the host is
    # what takes time
    if (cu_q.dtype is i32 and ctx_len.dtype is i32 and cu_q.get_device() == dev
            and ctx_len.get_device() == dev and cu_q.numel() > n and ctx_len.numel() >= n
            and cu_q.is_contiguous() and ctx_len.is_contiguous()):
        cu, ctx = cu_q.data_ptr(), ctx_len.data_ptr()
    else:
        cu = _vector(cu_q, i32, n + 1, dev, "cu_q")
        ctx = _vector(ctx_len, i32, n, dev, "ctx_len")
    return _pack_attention(
        a[0], b[0], a[1], a[2], b[1], b[2], cu, ctx, page_table.data_ptr(), st[0] if n > 1 else width,
        width, n, T, Hq, scale,
        0 if device_error is None else _vector(device_error, i32, 1, dev, "device_error"))


def _attention_args(cache, q, cu_q, ctx_len, page_table, scale, out, device_error, stream):
    dev, D, dt = cache._dev, cache.head_dim, cache.dtype
    T, Hq, dim = shape = q.shape
    if dim != D:
        raise ValueError(f"q: heads of {D} are wanted")
    a = _rows(q, shape, dt, dev, "q")
    if out is None:
        out = _empty_on(shape, dt, cache.device, stream)
        b = out.data_ptr(), Hq * D, D
    else:
        b = _rows(out, shape, dt, dev, "out")
    return _batch_args(cache, a, b, T, Hq, D ** -0.5 if scale is None else scale, cu_q, ctx_len,
                       page_table, device_error), out


def _workspace_bytes(fn: str, cache, table, shape, more) -> int:
    """What fn answers for a page table and queries of these shapes: it goes by nothing else, and no address is
    read.  The cache keeps the answers."""
    n_pages, kv_heads, page, dim, dtype = cache._shape
    c = _pack_kv_cache(16, 16, 0, 0, 0, n_pages, page, kv_heads, dim, dtype)
    a = _pack_attention(16, 16, 0, 0, 0, 0, 16, 16, 16, table[1], table[1], table[0], shape[0], shape[1],
                        1.0, 0)
    size = ctypes.c_int64()
    _on(cache._dev, fn + "_workspace", c, a, *more, ctypes.byref(size))
    if len(cache._sizes) >= 4096:
        cache._sizes.clear()
    cache._sizes[fn, table, shape, more] = size.value
    return size.value


def _run(fn: str, cache, stream, workspace, table, shape, more, *args) -> None:
    """fn(cache, *args, workspace, its bytes, stream) for a page table and queries of these shapes; `more`: what else
    its workspace goes by.  Without the caller's workspace, memory of torch's allocator, given back behind the
    call in the order of its stream as a tensor's is that goes out of scope (making a tensor takes as long as a
    launch)."""
    dev = cache._dev
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    ptr = 0
    if workspace is None:
        n = cache._sizes.get((fn, table, shape, more))
        if n is None:
            n = _workspace_bytes(fn, cache, table, shape, more)
    else:
        n = workspace.numel()
        ptr = _vector(workspace, torch.uint8, n, dev, "workspace")
    if n == 0 or ptr:
        _on(dev, fn, cache._c, *args, ptr, n, stream)
        return
    if torch._C._cuda_getDevice() == dev:
        ptr = torch._C._cuda_cudaCachingAllocator_raw_alloc(n, int(stream))
    else:
        with torch.cuda.device(dev):
            ptr = torch._C._cuda_cudaCachingAllocator_raw_alloc(n, int(stream))
    try:
        _on(dev, fn, cache._c, *args, ptr, n, stream)
    finally:
        torch._C._cuda_cudaCachingAllocator_raw_delete(ptr)


def _workspace(fn: str, cache, workspace, stream, *args):
    """(address, bytes, tensor) of the caller's workspace, or of a new one as large as fn says."""
    if workspace is None:
        n = ctypes.c_int64()
        _on(cache._dev, fn, cache._c, *args, ctypes.byref(n))
        if n.value == 0:
            return 0, 0, None
        workspace = _empty_on(n.value, torch.uint8, cache.device, stream)
        return workspace.data_ptr(), n.value, workspace
    n = workspace.numel()
    return _vector(workspace, torch.uint8, n, cache._dev, "workspace"), n, workspace


def _tree_mask(tree_mask, rows, dev) -> int:
    if tree_mask is None:
        return 0
    if tree_mask.dtype not in (torch.int64, torch.uint64):
        raise ValueError("tree_mask: 64-bit integers are wanted")
    return _vector(tree_mask, tree_mask.dtype, rows, dev, "tree_mask")


def tree_attention(cache: KvCache, q, cu_q, ctx_len, page_table, max_q: int, tree_mask=None,
                   scale: float | None = None, out=None, device_error=None, workspace=None,
                   stream=None):
    """moe_tree_attention: decoded tokens (max_q = 1) or trees of up to max_q <= 64 drafted tokens a
    sequence.  q [T, Hq, D]; cu_q int32 [n + 1]; ctx_len int32 [n]; page_table int32 [n, width];
    tree_mask int64 [T], bit j of a row: it sees drafted token j of its sequence (None: causal);
    scale None: 1 / sqrt(D).  workspace: uint8 tensor to use instead of a new one.

    A sequence that is not within its bounds (more than max_q rows, more positions than its pages) is
    skipped on the device: its rows of out, like those that belong to no sequence, are not written, and
    in an out made here they are uninitialised memory.  device_error (int32 [1], zeroed by the caller)
    shows that without a wait on this call: bit 1 of it is set, for a page outside the cache too."""
    dev = cache._dev
    args, out = _attention_args(cache, q, cu_q, ctx_len, page_table, scale, out, device_error,
                                stream)
    mask = _tree_mask(tree_mask, q.shape[0], dev)
    ws = _workspace("moe_tree_attention_workspace", cache, workspace, stream, args, max_q)
    _call("moe_tree_attention", dev, stream, cache._c, args, mask, max_q, *ws[:2])
    return out


def prompt_attention(cache: KvCache, q, cu_q, ctx_len, page_table, scale: float | None = None,
                     out=None, device_error=None, workspace=None, stream=None):
    """moe_prompt_attention: causal attention of packed prompts, or of chunks behind ctx_len cached
    positions; arguments and device_error as for tree_attention, without a limit on the rows of a
    sequence."""
    args, out = _attention_args(cache, q, cu_q, ctx_len, page_table, scale, out, device_error,
                                stream)
    ws = _workspace("moe_prompt_attention_workspace", cache, workspace, stream, args)
    _call("moe_prompt_attention", cache._dev, stream, cache._c, args, *ws[:2])
    return out


# ---------------------------------------------------------------- without reading the whole cache

def prefix_attention(cache: KvCache, q, cu_q, ctx_len, page_table, cu_group, prefix_len, max_q: int,
                     tree_mask=None, scale: float | None = None, out=None, device_error=None,
                     workspace=None, stream=None):
    """moe_prefix_attention: tree_attention of sequences that share their first positions, group by group:
    sequences cu_group[g] .. cu_group[g + 1] - 1 (int32 [n_groups + 1]) the first prefix_len[g] (int32
    [n_groups]), which are read once for the group, by its first sequence's row of page_table.  The other
    arguments, and what happens to sequences out of range, as for tree_attention."""
    dev, groups = cache._dev, prefix_len.numel()
    args, out = _attention_args(cache, q, cu_q, ctx_len, page_table, scale, out, device_error,
                                stream)
    shape = q.shape
    _run("moe_prefix_attention", cache, stream, workspace, page_table.shape, shape, (groups, max_q), args,
         _vector(cu_group, torch.int32, groups + 1, dev, "cu_group"),
         _vector(prefix_len, torch.int32, groups, dev, "prefix_len"), groups,
         _tree_mask(tree_mask, shape[0], dev), max_q)
    return out


def _bounds(cache, bounds) -> int:
    if bounds.shape != cache._bounds:
        raise ValueError(f"bounds: {tuple(cache._bounds)} is wanted, not {tuple(bounds.shape)}")
    return _vector(bounds, cache.dtype, 0, cache._dev, "bounds")


def page_bounds(cache: KvCache, bounds, cu_q, ctx_len, page_table, n_rows: int, device_error=None,
                stream=None):
    """moe_page_bounds: writes the least and the largest key of every page that holds one of the batch's
    new positions to bounds [n_pages, Hkv, 2, D] (the cache's dtype) and returns it.  Called when the
    new keys are in the cache; n_rows: the batch's rows, as of q; the other arguments as for
    tree_attention."""
    args = _batch_args(cache, _NONE, _NONE, n_rows, 0, 0.0, cu_q, ctx_len, page_table, device_error)
    _call("moe_page_bounds", cache._dev, stream, cache._c, args, _bounds(cache, bounds))
    return bounds


def select_pages(cache: KvCache, bounds, q, cu_q, ctx_len, page_table, n_select: int, sink: int = 1,
                 recent: int = 1, out=None, device_error=None, workspace=None, stream=None):
    """moe_select_pages: for each row of q [T, Hq, D] and key/value head the n_select pages to read, int32
    [T, Hkv, n_select]: places in the row of page_table, ascending, -1 behind the last.  All that the row
    sees when they are no more; else the first `sink`, the last `recent` and those whose bounds
    (page_bounds) allow the largest scores.  Rows of no sequence are not written."""
    dev = cache._dev
    T, Hq, D = shape = q.shape
    if D != cache.head_dim:
        raise ValueError(f"q: heads of {cache.head_dim} are wanted")
    pages = (T, cache.n_kv_heads, n_select)
    if out is None:
        out = _empty_on(pages, torch.int32, cache.device, stream)
        to = out.data_ptr()
    elif out.shape != pages:
        raise ValueError(f"out: {pages} is wanted, not {tuple(out.shape)}")
    else:
        to = _vector(out, torch.int32, 0, dev, "out")
    args = _batch_args(cache, _rows(q, shape, cache.dtype, dev, "q"), _NONE, T, Hq, 0.0, cu_q, ctx_len,
                       page_table, device_error)
    _run("moe_select_pages", cache, stream, workspace, page_table.shape, shape, (), args,
         _bounds(cache, bounds), n_select, sink, recent, to)
    return out


def sparse_attention(cache: KvCache, q, cu_q, ctx_len, page_table, pages,
                     scale: float | None = None, out=None, device_error=None, workspace=None,
                     stream=None):
    """moe_sparse_attention: causal attention of each row of q over the pages listed for it, pages int32
    [T, Hkv, n_select] as select_pages gives them; the other arguments as for prompt_attention."""
    if pages.dim() != 3 or pages.shape[:2] != (q.shape[0], cache.n_kv_heads):
        raise ValueError(f"pages: [{q.shape[0]}, {cache.n_kv_heads}, n_select] is wanted, not "
                         f"{tuple(pages.shape)}")
    args, out = _attention_args(cache, q, cu_q, ctx_len, page_table, scale, out, device_error,
                                stream)
    n = pages.shape[2]
    _run("moe_sparse_attention", cache, stream, workspace, page_table.shape, q.shape, (n,), args,
         _vector(pages, torch.int32, 0, cache._dev, "pages"), n)
    return out
