"""PyTorch-facing wrappers of the C ABI: device tensors in, device tensors out.

PyTorch supplies device memory and the current stream; each call passes raw pointers to
libtq.so, which enqueues the gfx950 kernels on that stream. No computation happens here.
"""

import ctypes
from dataclasses import dataclass

import numpy as np
import torch

from . import _lib
from ._lib import (TQ_AUTO, TQ_COMBINE, TQ_GEMM, TQ_GEMV, TQ_LAYOUT_GEMV,  # noqa: F401
                   TQ_LAYOUT_STORE, TQ_LAYOUT_UNIT128, TQ_OUT_BF16, TQ_ROTATE, TQ_FP8, TQ_FP4,
                   TQ_SCORE_SOFTMAX, TQ_SCORE_SIGMOID, TQ_LOGITS_BF16, TQ_CODEBOOK_T16,
                   TQ_CODEBOOK_MUL1, TQ_CODEBOOK_PMCGX, check)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _require_cuda(*tensors):
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must be on the GPU")


@dataclass
class TrellisLayer:
    """A trellis expert layer in device memory (see tq_trellis_layer in include/tq.h)."""
    E: int
    out: int
    in_: int
    bits: torch.Tensor       # uint8 [E]
    code_off: torch.Tensor   # int64 [E], byte offsets
    codes: torch.Tensor      # int32 [words] (uint32 bit patterns)
    scales: torch.Tensor     # int16 [E, out] (fp16 bit patterns)
    signs: torch.Tensor = None  # int8 [in] rotation signs (TQ_ROTATE), or None
    layout: int = TQ_LAYOUT_STORE
    out_signs: torch.Tensor = None  # int8 [out] output-side rotation signs, or None
    codebook: int = 0               # TQ_CODEBOOK_T16, _MUL1 or _PMCGX

    @classmethod
    def from_host(cls, layer, device="cuda"):
        signs = layer.get("signs")
        out_signs = layer.get("out_signs")
        return cls(
            E=int(layer["E"]), out=int(layer["out"]), in_=int(layer["in"]),
            bits=torch.from_numpy(np.ascontiguousarray(layer["bits"], dtype=np.uint8)).to(device),
            code_off=torch.from_numpy(np.ascontiguousarray(layer["code_off"], dtype=np.int64)).to(device),
            codes=torch.from_numpy(np.ascontiguousarray(layer["codes"]).view(np.int32)).to(device),
            scales=torch.from_numpy(np.ascontiguousarray(layer["scales"]).view(np.int16)).to(device),
            signs=None if signs is None else
            torch.from_numpy(np.ascontiguousarray(signs, dtype=np.int8)).to(device),
            layout=int(layer.get("layout", TQ_LAYOUT_STORE)),
            out_signs=None if out_signs is None else
            torch.from_numpy(np.ascontiguousarray(out_signs, dtype=np.int8)).to(device),
            codebook=int(layer.get("codebook", 0)),
        )

    def with_codes(self, codes):
        """The same layer reading its units from another copy of the code buffer."""
        return TrellisLayer(self.E, self.out, self.in_, self.bits, self.code_off, codes,
                            self.scales, self.signs, self.layout, self.out_signs, self.codebook)

    def repacked(self):
        """The same layer with its units copied into TQ_LAYOUT_GEMV (see trellis_repack in
        include/tq.h)."""
        _require_cuda(self.codes)
        dst = torch.zeros_like(self.codes)
        c = self.c_struct()
        check(_lib.load().trellis_repack(ctypes.byref(c), _ptr(dst), _stream(self.codes.device)))
        return TrellisLayer(self.E, self.out, self.in_, self.bits, self.code_off, dst,
                            self.scales, self.signs, TQ_LAYOUT_GEMV, self.out_signs,
                            self.codebook)

    def c_struct(self):
        return _lib.TrellisLayerC(self.E, self.out, self.in_, self.layout, self.bits.data_ptr(),
                                  self.code_off.data_ptr(), self.codes.data_ptr(),
                                  self.scales.data_ptr(),
                                  None if self.signs is None else self.signs.data_ptr(),
                                  self.codes.numel() * self.codes.element_size(),
                                  None if self.out_signs is None else self.out_signs.data_ptr(),
                                  self.codebook)


@dataclass
class Mxfp4Layer:
    """An MXFP4 expert layer in device memory (see tq_mxfp4_layer in include/tq.h)."""
    E: int
    out: int
    in_: int
    units: torch.Tensor      # uint8 [E * unit_bytes]
    layout: int = TQ_LAYOUT_STORE

    @classmethod
    def from_host(cls, layer, device="cuda"):
        return cls(E=int(layer["E"]), out=int(layer["out"]), in_=int(layer["in"]),
                   units=torch.from_numpy(np.ascontiguousarray(layer["units"], dtype=np.uint8)).to(device))

    def with_units(self, units):
        return Mxfp4Layer(self.E, self.out, self.in_, units, self.layout)

    def c_struct(self):
        return _lib.Mxfp4LayerC(self.E, self.out, self.in_, self.layout, self.units.data_ptr())

    def repacked(self):
        """The same layer with its units copied into TQ_LAYOUT_GEMV (see mxfp4_repack in
        include/tq.h)."""
        _require_cuda(self.units)
        dst = torch.empty_like(self.units)
        c = self.c_struct()
        check(_lib.load().mxfp4_repack(ctypes.byref(c), _ptr(dst), _stream(self.units.device)))
        return Mxfp4Layer(self.E, self.out, self.in_, dst, TQ_LAYOUT_GEMV)


@dataclass
class Fp8b32Layer:
    """An fp8b32 expert layer in device memory (see tq_fp8b32_layer in include/tq.h)."""
    E: int
    out: int
    in_: int
    units: torch.Tensor      # uint8 [E * unit_bytes]
    layout: int = TQ_LAYOUT_STORE

    @classmethod
    def from_host(cls, layer, device="cuda"):
        return cls(E=int(layer["E"]), out=int(layer["out"]), in_=int(layer["in"]),
                   units=torch.from_numpy(np.ascontiguousarray(layer["units"], dtype=np.uint8)).to(device))

    def with_units(self, units):
        return Fp8b32Layer(self.E, self.out, self.in_, units, self.layout)

    def c_struct(self):
        return _lib.Mxfp4LayerC(self.E, self.out, self.in_, self.layout, self.units.data_ptr())

    def repacked(self):
        """The same layer with its units copied into TQ_LAYOUT_GEMV (see fp8b32_repack in
        include/tq.h)."""
        _require_cuda(self.units)
        dst = torch.empty_like(self.units)
        c = self.c_struct()
        check(_lib.load().fp8b32_repack(ctypes.byref(c), _ptr(dst), _stream(self.units.device)))
        return Fp8b32Layer(self.E, self.out, self.in_, dst, TQ_LAYOUT_GEMV)


def workspace_bytes(T, topk, E, out, in_, flags=TQ_AUTO):
    return int(_lib.load().tq_workspace_bytes(T, topk, E, out, in_, flags))


def workspace(T, topk, E, out, in_, flags=TQ_AUTO, device="cuda"):
    """A zero-filled workspace (the library requires zeros before the first use)."""
    n = max(256, workspace_bytes(T, topk, E, out, in_, flags))
    return torch.zeros(n, dtype=torch.uint8, device=device)


def hadamard128(x, signs=None, out=None):
    """bf16 [rows, n] -> bf16 [rows, n], 128-wide rotation (x may be bf16/int16/uint16)."""
    _require_cuda(x, signs, out)
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [rows, n] tensor")
    y = torch.empty_like(x) if out is None else out
    check(_lib.load().hadamard128(_ptr(x), _ptr(y), x.shape[0], x.shape[1], _ptr(signs),
                                  _stream(x.device)))
    return y


def mxfp8_quantize(x):
    """(codes uint8 [rows, n], scales uint8 [rows, n / 32]): the MXFP8 form of bf16 rows (see
    mxfp8_quantize in include/tq.h)."""
    _require_cuda(x)
    rows, n = x.shape
    codes = torch.empty((rows, n), dtype=torch.uint8, device=x.device)
    scales = torch.empty((rows, n // 32), dtype=torch.uint8, device=x.device)
    check(_lib.load().mxfp8_quantize(_ptr(x), rows, n, _ptr(codes), _ptr(scales),
                                     _stream(x.device)))
    return codes, scales


def _gemm(fn, layer_c, E, out_ch, in_, x, topk_ids, topk_w, flags, out, ws, mxfp4):
    _require_cuda(x, topk_ids, topk_w, out, ws)
    T, topk = topk_ids.shape
    if out is None:
        shape = (T, out_ch) if flags & TQ_COMBINE else (T, topk, out_ch)
        out = torch.empty(shape, dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(T, topk, E, out_ch, in_, flags, device=x.device)
    _call_on(x.device, fn, ctypes.byref(layer_c), x.data_ptr(), T, topk_ids.data_ptr(),
             None if topk_w is None else topk_w.data_ptr(), topk, out.data_ptr(), flags,
             ws.data_ptr(), ws.numel())
    return out


def trellis_expert_gemm(layer, x, topk_ids, topk_w=None, flags=TQ_AUTO, out=None, ws=None):
    """fp32 per-slot outputs [T, topk, out] (or [T, out] with TQ_COMBINE)."""
    return _gemm(_lib.load().trellis_expert_gemm, layer.c_struct(), layer.E, layer.out,
                 layer.in_, x, topk_ids, topk_w, flags, out, ws, False)


def trellis_expert_gemm_noalloc(layer, x, topk_ids, topk_w=None, flags=TQ_AUTO, out=None):
    """trellis_expert_gemm with the library's static device scratch as its workspace (see
    trellis_expert_gemm_noalloc in include/tq.h). `out` must be given for the call itself
    to allocate nothing."""
    _require_cuda(x, topk_ids, topk_w, out)
    T, topk = topk_ids.shape
    if out is None:
        shape = (T, layer.out) if flags & TQ_COMBINE else (T, topk, layer.out)
        out = torch.empty(shape, dtype=torch.float32, device=x.device)
    layer_c = layer.c_struct()
    check(_lib.load().trellis_expert_gemm_noalloc(ctypes.byref(layer_c), _ptr(x), T,
                                                  _ptr(topk_ids), _ptr(topk_w), topk, _ptr(out),
                                                  flags, _stream(x.device)))
    return out


def mxfp4_expert_gemm(layer, x, topk_ids, topk_w=None, flags=TQ_AUTO, out=None, ws=None):
    """fp32 per-slot outputs [T, topk, out] (or [T, out] with TQ_COMBINE) of bf16 x [T, in]; TQ_FP4
    multiplies in 4 bits on both sides (see mxfp4_expert_gemm in include/tq.h)."""
    if flags & TQ_FP4:
        _check_fp4(layer, x, topk_ids, topk_w, flags, out, ws)
    return _gemm(_lib.load().mxfp4_expert_gemm, layer.c_struct(), layer.E, layer.out,
                 layer.in_, x, topk_ids, topk_w, flags, out, ws, True)


def fp8b32_expert_gemm(layer, x, topk_ids, topk_w=None, flags=TQ_AUTO, out=None, ws=None):
    return _gemm(_lib.load().fp8b32_expert_gemm, layer.c_struct(), layer.E, layer.out,
                 layer.in_, x, topk_ids, topk_w, flags, out, ws, True)


def route_bucket(topk_ids, E, ws=None):
    """(counts [E], offsets [E+1], pairs [T*topk]) as int32 device tensors."""
    _require_cuda(topk_ids, ws)
    T, topk = topk_ids.shape
    dev = topk_ids.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    pairs = torch.full((max(1, T * topk),), -1, dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(T, topk, E, 16, 256, TQ_GEMM, device=dev)
    check(_lib.load().route_bucket(_ptr(topk_ids), T, topk, E, _ptr(counts), _ptr(offsets),
                                   _ptr(pairs), _ptr(ws), ws.numel(), _stream(dev)))
    return counts, offsets, pairs[:T * topk]


def trellis_decode(codes, K, out_ch, in_, path=0):
    """int16 q [out, in] of one unit, via the GEMV (path 0) or prefill (path 1) decoder; path
    2 gives the E4M3 codes of the FP8 prefill's decoder."""
    _require_cuda(codes)
    q = torch.empty((out_ch, in_), dtype=torch.int16, device=codes.device)
    check(_lib.load().trellis_decode(_ptr(codes), K, out_ch, in_, _ptr(q), path,
                                     _stream(codes.device)))
    return q


def mxfp4_decode(unit, out_ch, in_):
    """bf16 bit patterns (int16) [out, in] of one MXFP4 unit."""
    _require_cuda(unit)
    w = torch.empty((out_ch, in_), dtype=torch.int16, device=unit.device)
    _call_on(unit.device, _lib.load().mxfp4_decode, unit.data_ptr(), out_ch, in_, w.data_ptr())
    return w


def fp8b32_decode(unit, out_ch, in_):
    """bf16 bit patterns (int16) [out, in] of one fp8b32 unit."""
    _require_cuda(unit)
    w = torch.empty((out_ch, in_), dtype=torch.int16, device=unit.device)
    check(_lib.load().fp8b32_decode(_ptr(unit), out_ch, in_, _ptr(w), _stream(unit.device)))
    return w


def ffn_workspace(T, topk, E, H, I, flags=TQ_AUTO, device="cuda"):
    n = max(256, int(_lib.load().tq_ffn_workspace_bytes(T, topk, E, H, I, flags)))
    return torch.zeros(n, dtype=torch.uint8, device=device)


def trellis_expert_ffn(gate_up, down, x, topk_ids, topk_w=None, flags=TQ_AUTO, out=None,
                       ws=None):
    """fp32 [T, H]: the routed expert FFN over a fused trellis gate/up layer (out = 2I) and a
    trellis down layer (see trellis_expert_ffn in include/tq.h)."""
    _require_cuda(x, topk_ids, topk_w, out, ws)
    T, topk = topk_ids.shape
    if out is None:
        out = torch.empty((T, gate_up.in_), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = ffn_workspace(T, topk, gate_up.E, gate_up.in_, gate_up.out // 2, flags,
                           device=x.device)
    gu, d = gate_up.c_struct(), down.c_struct()
    check(_lib.load().trellis_expert_ffn(ctypes.byref(gu), ctypes.byref(d), _ptr(x), T,
                                         _ptr(topk_ids), _ptr(topk_w), topk, _ptr(out), flags,
                                         _ptr(ws), ws.numel(), _stream(x.device)))
    return out


def mxfp4_to_nvfp4(layer, codes=None, scales=None, scale2=None, status=None):
    """NVFP4 form of an MXFP4 layer: (codes uint8 [E, out*in/2], scales uint8 [E, out, in/16],
    scale2 fp32 [E], status uint8 [E]) (see mxfp4_to_nvfp4 in include/tq.h)."""
    _require_cuda(layer.units, codes, scales, scale2, status)
    dev = layer.units.device
    E, out_ch, in_ = layer.E, layer.out, layer.in_
    if codes is None:
        codes = torch.empty((E, out_ch * in_ // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((E, out_ch, in_ // 16), dtype=torch.uint8, device=dev)
    if scale2 is None:
        scale2 = torch.empty(E, dtype=torch.float32, device=dev)
    if status is None:
        status = torch.empty(E, dtype=torch.uint8, device=dev)
    c = layer.c_struct()
    check(_lib.load().mxfp4_to_nvfp4(ctypes.byref(c), _ptr(codes), _ptr(scales), _ptr(scale2),
                                     _ptr(status), _stream(dev)))
    return codes, scales, scale2, status


@dataclass(frozen=True)
class Fp8b128Layer:
    """A dense projection in the fp8b128 store (see tq_fp8b128_layer in include/tq.h)."""
    codes: torch.Tensor      # uint8 or float8_e4m3fn [out, in]
    scales: torch.Tensor     # fp32 [ceil(out / 128), ceil(in / 128)]

    def __post_init__(self):
        state = self._state()
        codes_at, scales_at, shape, scales_shape, dtype, scales_dtype, dev, scales_dev, whole, scales_whole = state
        out, in_ = shape if len(shape) == 2 else (0, 0)
        fit = (-(-out // 128), -(-in_ // 128))
        if not (len(shape) == 2 and dtype in _E4M3 and scales_dtype == torch.float32
                and scales_shape == fit and whole and scales_whole and scales_dev == dev
                and self.codes.is_cuda):  # the same checks, with their messages
            _check_rows("codes", self.codes, _E4M3)
            _check_rows("scales", self.scales, _F32, dev, fit)
        c = _lib.Fp8b128LayerC(out, in_, codes_at, scales_at)
        d = self.__dict__
        d["out"], d["in_"], d["blocks"], d["device"] = out, in_, fit[1], dev
        d["_c"], d["_ref"], d["_checked"] = c, ctypes.byref(c), state

    def _state(self):
        """All that the checks and the C struct depend on."""
        c, s = self.codes, self.scales
        return (c.data_ptr(), s.data_ptr(), c.shape, s.shape, c.dtype, s.dtype, c.device, s.device,
                c.is_contiguous(), s.is_contiguous())

    def renew(self):
        """Checks the layer again if a tensor has been given other memory, another shape or
        another type (set_, resize_, t_, an assignment to .data), also at the same address; the
        fields themselves cannot be assigned again. Every call does this before it uses the C
        struct."""
        if self._state() != self._checked:
            self.__post_init__()

    def __reduce__(self):
        return Fp8b128Layer, (self.codes, self.scales)  # copies and pickles hold the tensors alone

    @classmethod
    def from_host(cls, layer, device="cuda"):
        return cls(torch.from_numpy(np.ascontiguousarray(layer["codes"], dtype=np.uint8)).to(device),
                   torch.from_numpy(np.ascontiguousarray(layer["scales"], dtype=np.float32)).to(device))


_E4M3 = (torch.uint8, torch.float8_e4m3fn)
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_F32 = (torch.float32,)


def _check_rows(name, t, dtypes, device=None, shape=None):
    """The kernels read raw pointers: a tensor has to be on the GPU, contiguous, of one of
    `dtypes` and, where they are given, on `device` and of `shape`."""
    if (t.dtype in dtypes and t.is_cuda and t.is_contiguous()
            and (device is None or t.device == device)
            and (t.dim() == 2 if shape is None else t.shape == shape)):
        return
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    if t.dtype not in dtypes:
        raise ValueError("%s is %s, not %s" % (name, t.dtype, dtypes[0]))
    dims = 2 if shape is None else len(shape)
    if t.dim() != dims or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %d-D tensor" % (name, dims))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, not %s" % (name, t.device, device))
    raise ValueError("%s is %s, not %s" % (name, tuple(t.shape), shape))


def _call_on(device, fn, *args):
    """fn(*args, stream) on the device's current stream, with that device current (a kernel
    launched while another device is current would not run on it). The stream's handle is read
    without making a Stream object: 0.1 us instead of 1.8, in calls of a few microseconds."""
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc:
        check(rc)


def _check_ws(ws, device, nbytes):
    """The given workspace, or a new one (the fp8b128 calls need no cleared memory)."""
    if ws is None:
        return torch.empty(max(256, nbytes), dtype=torch.uint8, device=device)
    if not ws.is_cuda or ws.device != device or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor on %s" % device)
    return ws


def _check_fp8b128(layer, codes, scales):
    """(T, device) of activations that fit the layer."""
    layer.renew()
    dev = layer.device
    shape = codes.shape
    T = shape[0] if shape else 0
    if not (codes.dtype in _E4M3 and scales.dtype == torch.float32 and codes.device == dev
            and scales.device == dev and shape == (T, layer.in_)
            and scales.shape == (T, layer.blocks) and codes.is_contiguous()
            and scales.is_contiguous()):  # the same checks, with their messages
        _check_rows("codes", codes, _E4M3, dev, (T, layer.in_))
        _check_rows("scales", scales, _F32, dev, (T, layer.blocks))
    return T, dev


def fp8b128_quantize(x, codes=None, scales=None):
    """(codes uint8 [rows, n], scales fp32 [rows, ceil(n / 128)]): the 8-bit form of bf16 rows
    with one power-of-two scale per 128 inputs (see fp8b128_quantize in include/tq.h)."""
    _check_rows("x", x, _BF16)
    rows, n = x.shape
    dev = x.device
    nb = -(-n // 128)
    if codes is None:
        codes = x.new_empty((rows, n), dtype=torch.uint8)
    else:
        _check_rows("codes", codes, _E4M3, dev, (rows, n))
    if scales is None:
        scales = x.new_empty((rows, nb), dtype=torch.float32)
    else:
        _check_rows("scales", scales, _F32, dev, (rows, nb))
    _call_on(dev, _lib.load().fp8b128_quantize, x.data_ptr(), rows, n, codes.data_ptr(),
             scales.data_ptr())
    return codes, scales


def fp8b128_gemm(layer, codes, scales, flags=0, out=None):
    """[T, out]: quantized activations times an fp8b128 projection, fp32 or (TQ_OUT_BF16) bf16
    (see fp8b128_gemm in include/tq.h)."""
    T, dev = _check_fp8b128(layer, codes, scales)
    dtype = torch.bfloat16 if flags & TQ_OUT_BF16 else torch.float32
    if out is None:
        out = codes.new_empty((T, layer.out), dtype=dtype)
    else:
        _check_rows("out", out, (dtype,), dev, (T, layer.out))
    _call_on(dev, _lib.load().fp8b128_gemm, layer._ref, codes.data_ptr(),
             scales.data_ptr(), T, out.data_ptr(), flags)
    return out


def fp8b128_gated(layer, codes, scales, out=None):
    """bf16 [T, I]: silu(gate) * up of quantized activations over a fused gate/up projection
    (out = 2I) (see fp8b128_gated in include/tq.h)."""
    T, dev = _check_fp8b128(layer, codes, scales)
    if out is None:
        out = codes.new_empty((T, layer.out // 2), dtype=torch.bfloat16)
    else:
        _check_rows("out", out, _BF16, dev, (T, layer.out // 2))
    _call_on(dev, _lib.load().fp8b128_gated, layer._ref, codes.data_ptr(),
             scales.data_ptr(), T, out.data_ptr())
    return out


def fp8b128_workspace(T, out, in_, device="cuda"):
    """A workspace of the two backward calls (it need not be cleared)."""
    n = int(_lib.load().tq_fp8b128_workspace_bytes(T, out, in_))
    return torch.empty(max(256, n), dtype=torch.uint8, device=device)


def _fp8b128_backward(fn, layer, codes, scales, dy, parts, need_dx, need_dw, dx, dw, ws):
    T, dev = _check_fp8b128(layer, codes, scales)
    _check_rows("the output's gradient", dy, _BF16, dev, (T, layer.out // parts))
    if dx is not None:
        _check_rows("dx", dx, _BF16, dev, (T, layer.in_))
    elif need_dx:
        dx = dy.new_empty((T, layer.in_), dtype=torch.bfloat16)
    if dw is not None:
        _check_rows("dw", dw, _BF16, dev, (layer.out, layer.in_))
    elif need_dw:
        dw = dy.new_empty((layer.out, layer.in_), dtype=torch.bfloat16)
    lib = _lib.load()
    ws = _check_ws(ws, dev, lib.tq_fp8b128_workspace_bytes(T, layer.out, layer.in_))
    _call_on(dev, getattr(lib, fn), layer._ref, codes.data_ptr(),
             scales.data_ptr(), T, dy.data_ptr(), None if dx is None else dx.data_ptr(),
             None if dw is None else dw.data_ptr(), ws.data_ptr(), ws.numel())
    return dx, dw


def fp8b128_gemm_backward(layer, codes, scales, dy, need_dx=True, need_dw=True, dx=None, dw=None,
                          ws=None):
    """(dx bf16 [T, in], dw bf16 [out, in]): the gradients of fp8b128_gemm from dy [T, out];
    None for one that is not needed (see fp8b128_gemm_backward in include/tq.h)."""
    return _fp8b128_backward("fp8b128_gemm_backward", layer, codes, scales, dy, 1,
                             need_dx, need_dw, dx, dw, ws)


def fp8b128_gated_backward(layer, codes, scales, dh, need_dx=True, need_dw=True, dx=None, dw=None,
                           ws=None):
    """(dx bf16 [T, in], dw bf16 [2I, in]): the gradients of fp8b128_gated from dh [T, I] and
    the 8-bit activations; None for one that is not needed (see fp8b128_gated_backward in
    include/tq.h)."""
    return _fp8b128_backward("fp8b128_gated_backward", layer, codes, scales, dh, 2,
                             need_dx, need_dw, dx, dw, ws)


def fp8b128_ffn(gate_up, down, x, flags=0, out=None, ws=None):
    """[T, H]: a dense gated FFN over two fp8b128 projections, fp32 or (TQ_OUT_BF16) bf16 (see
    fp8b128_ffn in include/tq.h)."""
    gate_up.renew()
    down.renew()
    dev = gate_up.device
    _check_rows("x", x, _BF16, dev)
    if down.device != dev:
        raise ValueError("the two layers are on different devices")
    T, H = x.shape
    if H != gate_up.in_:
        raise ValueError("x has %d inputs, the layer %d" % (H, gate_up.in_))
    dtype = torch.bfloat16 if flags & TQ_OUT_BF16 else torch.float32
    if out is None:
        out = torch.empty((T, H), dtype=dtype, device=dev)
    else:
        _check_rows("out", out, (dtype,), dev, (T, H))
    lib = _lib.load()
    ws = _check_ws(ws, dev, lib.tq_fp8b128_ffn_workspace_bytes(T, H, gate_up.out // 2))
    _call_on(dev, lib.fp8b128_ffn, gate_up._ref, down._ref,
             x.data_ptr(), T, out.data_ptr(), flags, ws.data_ptr(), ws.numel())
    return out


def _check_fp4(layer, x, topk_ids, topk_w, flags, out, ws):
    dev = layer.units.device
    _check_rows("topk_ids", topk_ids, _I32, dev)
    T, topk = topk_ids.shape
    _check_rows("x", x, _BF16, dev, (T, layer.in_))
    if topk_w is not None:
        _check_rows("topk_w", topk_w, _F32, dev, (T, topk))
    if out is not None:
        _check_rows("out", out, _F32, dev,
                    (T, layer.out) if flags & TQ_COMBINE else (T, topk, layer.out))
    if ws is not None:
        _check_ws(ws, dev, 0)


def mxfp4_quantize(x, codes=None, scales=None):
    """(codes uint8 [rows, n / 2], scales uint8 [rows, n / 32]): the MXFP4 form of bf16 rows (see
    mxfp4_quantize in include/tq.h)."""
    _check_rows("x", x, _BF16)
    rows, n = x.shape
    dev = x.device
    if codes is None:
        codes = x.new_empty((rows, n // 2), dtype=torch.uint8)
    else:
        _check_rows("codes", codes, _U8, dev, (rows, n // 2))
    if scales is None:
        scales = x.new_empty((rows, n // 32), dtype=torch.uint8)
    else:
        _check_rows("scales", scales, _U8, dev, (rows, n // 32))
    _call_on(dev, _lib.load().mxfp4_quantize, x.data_ptr(), rows, n, codes.data_ptr(),
             scales.data_ptr())
    return codes, scales


@dataclass(frozen=True)
class Router:
    """How a token's logits choose its experts (see tq_router in include/tq.h)."""
    E: int
    topk: int
    score: str = "softmax"       # or "sigmoid"
    bias: torch.Tensor = None    # fp32 [E], added to the scores for the choice alone
    groups: int = 1
    group_topk: int = 1
    group_top: int = 1
    renorm: bool = True
    scale: float = 1.0

    def __post_init__(self):
        if self.score not in _SCORES:
            raise ValueError("score is %r, not 'softmax' or 'sigmoid'" % (self.score,))
        b = self.bias
        if b is not None:
            if not b.is_cuda:
                raise ValueError("tensors must be on the GPU")
            if b.dtype != torch.float32 or b.shape != (self.E,) or not b.is_contiguous():
                raise ValueError("bias must be a contiguous float32 tensor of %d values" % self.E)
        c = _lib.RouterC(self.E, self.topk, _SCORES[self.score], self.groups, self.group_topk,
                         self.group_top, 1 if self.renorm else 0, self.scale,
                         None if b is None else b.data_ptr())
        d = self.__dict__
        d["_c"], d["_ref"], d["_checked"] = c, ctypes.byref(c), self._state()

    def _state(self):
        """All that the checks of the bias and its pointer depend on."""
        b = self.bias
        return None if b is None else (b.data_ptr(), b.shape, b.dtype, b.device, b.is_contiguous())

    def renew(self):
        """Checks the bias again if it has been given other memory, another shape or another
        type. Every call does this before it uses the C struct."""
        if self.bias is not None and self._state() != self._checked:
            self.__post_init__()

    def __reduce__(self):
        return Router, (self.E, self.topk, self.score, self.bias, self.groups, self.group_topk,
                        self.group_top, self.renorm, self.scale)


_SCORES = {"softmax": TQ_SCORE_SOFTMAX, "sigmoid": TQ_SCORE_SIGMOID}
_U8 = (torch.uint8,)
_I32 = (torch.int32,)
_LOGITS = (torch.float32, torch.bfloat16)


def _check_logits(router, logits):
    """(T, device, flags) of logits that fit the router."""
    router.renew()
    _check_rows("logits", logits, _LOGITS)
    T, E = logits.shape
    dev = logits.device
    if E != router.E:
        raise ValueError("logits have %d experts, the router %d" % (E, router.E))
    if router.bias is not None and router.bias.device != dev:
        raise ValueError("bias is on %s, not %s" % (router.bias.device, dev))
    return T, dev, TQ_LOGITS_BF16 if logits.dtype == torch.bfloat16 else 0


def expert_route(router, logits, ids=None, w=None):
    """(topk_ids int32 [T, topk], topk_w fp32 [T, topk]) of fp32 or bf16 logits [T, E] (see
    expert_route in include/tq.h). The weights are not connected to logits that require a gradient:
    expert_route_backward computes it."""
    T, dev, flags = _check_logits(router, logits)
    shape = (T, router.topk)
    if ids is None:
        ids = logits.new_empty(shape, dtype=torch.int32)
    else:
        _check_rows("ids", ids, _I32, dev, shape)
    if w is None:
        w = logits.new_empty(shape, dtype=torch.float32)
    else:
        _check_rows("w", w, _F32, dev, shape)
    _call_on(dev, _lib.load().expert_route, router._ref, logits.data_ptr(), T, ids.data_ptr(),
             w.data_ptr(), flags)
    return ids, w


def expert_route_backward(router, logits, ids, dw, dlogits=None):
    """The gradient [T, E] of expert_route's weights with respect to the logits, of their type, from
    dw [T, topk], the gradient with respect to the weights (see expert_route_backward in
    include/tq.h)."""
    T, dev, flags = _check_logits(router, logits)
    shape = (T, router.topk)
    _check_rows("ids", ids, _I32, dev, shape)
    _check_rows("dw", dw, _F32, dev, shape)
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    else:
        _check_rows("dlogits", dlogits, (logits.dtype,), dev, logits.shape)
    _call_on(dev, _lib.load().expert_route_backward, router._ref, logits.data_ptr(), T,
             ids.data_ptr(), dw.data_ptr(), dlogits.data_ptr(), flags)
    return dlogits


def device_status(ws):
    """Synchronise, read and clear the workspace status bits."""
    v = ctypes.c_uint32(0)
    check(_lib.load().tq_device_status(_ptr(ws), _stream(ws.device), ctypes.byref(v)))
    return v.value


def version():
    return int(_lib.load().tq_version())


def time_kernel(start, stop):
    """Measurement hook: the next expert GEMM or FFN call on this thread sets the
    torch.cuda.Event pair (start, stop) to its main kernel's own start and end
    (tq_time_kernel)."""
    if start is None:
        check(_lib.load().tq_time_kernel(None, None))
        return
    check(_lib.load().tq_time_kernel(ctypes.c_void_p(start.cuda_event),
                                      ctypes.c_void_p(stop.cuda_event)))
