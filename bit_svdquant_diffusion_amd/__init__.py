"""MI355X (gfx950) SVDQuant W4A4 linear layer.

A thin ctypes binding over libsvdq.so (C ABI in include/svdq.h): argument
marshalling only. Every step of the runtime path runs in the library's HIP
kernels; PyTorch is used for device memory and streams. The library must be
built (``python -m bit_svdquant_diffusion_amd.build``); without it every call
raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import functools
import os
import warnings
from dataclasses import dataclass

import numpy as np

__all__ = [
    "SvdqError", "FMT_INT4", "FMT_MXFP4", "LayerDesc", "lib", "lib_path", "status_string",
    "packed_bytes", "pack_weights", "quantize_residual", "lora_extend", "unpack_weights", "workspace_bytes",
    "to_device", "linear_forward", "linear_forward_noalloc", "stage1", "gemm", "unpack_workspace", "debug_int4_group_sums",
    "SVDQLinear", "EXPORTED_SYMBOLS", "Layer", "measure_mfma_peak", "measure_copy",
    "awq_packed_bytes", "awq_pack", "awq_unpack", "awq_to_device", "awq_forward",
    "pack_weights_gpu", "calibrate_alpha", "to_host", "mlp_workspace_bytes", "mlp_fused", "mlp_forward",
    "MLP_AUTO", "MLP_UNFUSED", "stage1_outputs",
    "layer_norm_forward", "layer_norm_backward",
    "fp8_packed_bytes", "fp8_pack", "fp8_forward", "fp8_norm_forward", "fp8_backward", "fp8_quantize",
    "fp8_workspace_bytes", "fp8_norm_workspace_bytes", "fp8_backward_workspace_bytes", "Fp8Linear",
]

FMT_INT4 = 0
FMT_MXFP4 = 1
FORMATS = {"int4": FMT_INT4, "mxfp4": FMT_MXFP4}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libsvdq.so"

EXPORTED_SYMBOLS = [
    "svdq_status_string", "svdq_version", "svdq_packed_bytes", "svdq_pack_weights",
    "svdq_quantize_residual", "svdq_unpack_weights", "svdq_workspace_bytes",
    "svdq_linear_forward", "svdq_stage1", "svdq_stage1_outputs", "svdq_unpack_workspace",
    "svdq_debug_int4_group_sums", "svdq_gemm", "svdq_linear_forward_noalloc", "svdq_lora_extend",
    "svdq_measure_mfma_peak", "svdq_measure_copy",
    "svdq_awq_packed_bytes", "svdq_awq_pack", "svdq_awq_unpack", "svdq_awq_forward",
    "svdq_pack_gpu_workspace_bytes", "svdq_pack_weights_gpu", "svdq_calibrate_workspace_bytes",
    "svdq_calibrate_alpha", "svdq_mlp_workspace_bytes", "svdq_mlp_fused", "svdq_mlp_forward",
    "svdq_layer_norm_forward", "svdq_layer_norm_backward_workspace_bytes", "svdq_layer_norm_backward",
    "svdq_fp8_packed_bytes", "svdq_fp8_pack", "svdq_fp8_workspace_bytes", "svdq_fp8_forward",
    "svdq_fp8_norm_workspace_bytes", "svdq_fp8_norm_forward", "svdq_fp8_backward_workspace_bytes",
    "svdq_fp8_backward", "svdq_fp8_quantize",
]

# svdq_mlp_forward modes
MLP_AUTO = 0
MLP_UNFUSED = 1

# bytes of the library-owned device workspace of svdq_linear_forward_noalloc
NOALLOC_SCRATCH_BYTES = 256 << 20


class SvdqError(RuntimeError):
    def __init__(self, status: int, fn: str):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)}")


class LayerDesc(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int32), ("N", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("format", ctypes.c_int32)]


class PackedSizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("mu", "l1", "l2", "qw", "sw", "bias")]


class Packed(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("mu", "l1", "l2", "qw", "sw", "bias")]


PACKED_FIELDS = ("mu", "l1", "l2", "qw", "sw", "bias")


class AwqDesc(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int32), ("N", ctypes.c_int32)]


AWQ_FIELDS = ("inv_s", "qw", "scales", "zeros", "bias")


class AwqSizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in AWQ_FIELDS]


class AwqPacked(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in AWQ_FIELDS]


class NormDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("channels", "dtype", "param_dtype", "one_plus", "groups")] + \
               [("eps", ctypes.c_float), ("rows_per_group", ctypes.c_int64)]


class Fp8Desc(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int32), ("N", ctypes.c_int32)]


FP8_FIELDS = ("q", "s", "qt", "st", "bias")


class Fp8Sizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in FP8_FIELDS]


class Fp8Packed(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in FP8_FIELDS]


_lib = None


def lib_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def lib() -> ctypes.CDLL:
    """Load libsvdq.so (built in-tree). Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m bit_svdquant_diffusion_amd.build`")
    L = ctypes.CDLL(path)
    P = ctypes.POINTER
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    D = P(LayerDesc)
    L.svdq_status_string.restype = ctypes.c_char_p
    L.svdq_status_string.argtypes = [ctypes.c_int]
    L.svdq_version.restype = ctypes.c_int32
    L.svdq_version.argtypes = []
    sigs = {
        "svdq_packed_bytes": [D, P(PackedSizes)],
        "svdq_pack_weights": [D, vp, vp, vp, ctypes.c_uint64, P(Packed)],
        "svdq_quantize_residual": [D, vp, vp, vp, vp, vp, P(Packed)],
        "svdq_unpack_weights": [D, P(Packed), vp, vp, vp, vp, vp],
        "svdq_lora_extend": [D, P(Packed), ctypes.c_int32, vp, vp, ctypes.c_float, P(Packed)],
        "svdq_measure_mfma_peak": [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P(ctypes.c_double), vp],
        "svdq_measure_copy": [vp, vp, sz, vp],
        "svdq_awq_packed_bytes": [P(AwqDesc), P(AwqSizes)],
        "svdq_awq_pack": [P(AwqDesc), vp, vp, vp, i64, ctypes.c_float, P(ctypes.c_double), vp, P(AwqPacked)],
        "svdq_awq_unpack": [P(AwqDesc), P(AwqPacked), vp, vp, vp],
        "svdq_awq_forward": [P(AwqDesc), P(AwqPacked), vp, i64, vp, vp],
        "svdq_pack_gpu_workspace_bytes": [D, P(sz)],
        "svdq_pack_weights_gpu": [D, vp, vp, vp, ctypes.c_float, ctypes.c_uint64, P(Packed), vp, sz, vp],
        "svdq_calibrate_workspace_bytes": [D, i64, P(sz)],
        "svdq_calibrate_alpha": [D, vp, vp, vp, i64, vp, ctypes.c_int32, ctypes.c_uint64, P(ctypes.c_float),
                                 vp, P(Packed), vp, sz, vp],
        "svdq_workspace_bytes": [D, i64, P(sz)],
        "svdq_linear_forward": [D, P(Packed), vp, i64, vp, vp, sz, vp],
        "svdq_linear_forward_noalloc": [D, P(Packed), vp, i64, vp, vp],
        "svdq_stage1": [D, P(Packed), vp, i64, vp, sz, vp],
        "svdq_stage1_outputs": [D, P(Packed), vp, i64, vp, vp, vp, vp, sz, vp],
        "svdq_gemm": [D, P(Packed), vp, sz, i64, vp, vp],
        "svdq_unpack_workspace": [D, i64, vp, sz, vp, vp, vp],
        "svdq_debug_int4_group_sums": [D, P(Packed), vp, sz, i64, i64, i64, i64, i64, vp, vp],
        "svdq_layer_norm_forward": [P(NormDesc), vp, i64, vp, i64, vp, i64, i64, vp, i64, vp, vp, vp],
        "svdq_layer_norm_backward_workspace_bytes": [P(NormDesc), i64, P(sz)],
        "svdq_layer_norm_backward": [P(NormDesc), vp, i64, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp,
                                     ctypes.c_int32, vp, sz, vp],
        "svdq_fp8_packed_bytes": [P(Fp8Desc), P(Fp8Sizes)],
        "svdq_fp8_pack": [P(Fp8Desc), vp, ctypes.c_int32, P(Fp8Packed), vp],
        "svdq_fp8_workspace_bytes": [P(Fp8Desc), i64, P(sz)],
        "svdq_fp8_forward": [P(Fp8Desc), P(Fp8Packed), vp, i64, vp, vp, sz, vp],
        "svdq_fp8_norm_workspace_bytes": [P(Fp8Desc), i64, P(sz)],
        "svdq_fp8_norm_forward": [P(NormDesc), vp, i64, vp, i64, P(Fp8Desc), P(Fp8Packed), vp, i64, vp, vp, vp, vp, sz,
                                  vp],
        "svdq_fp8_backward_workspace_bytes": [P(Fp8Desc), i64, P(sz)],
        "svdq_fp8_backward": [P(Fp8Desc), P(Fp8Packed), vp, vp, i64, vp, vp, vp, vp, sz, vp],
        "svdq_fp8_quantize": [vp, i64, ctypes.c_int32, vp, vp, vp],
        "svdq_mlp_workspace_bytes": [D, D, i64, P(sz), P(sz)],
        "svdq_mlp_fused": [D, D, i64, P(ctypes.c_int32)],
        "svdq_mlp_forward": [D, P(Packed), D, P(Packed), vp, i64, vp, vp, sz, ctypes.c_int32, vp],
    }
    for name, args in sigs.items():
        f = getattr(L, name)
        f.restype = ctypes.c_int
        f.argtypes = args
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().svdq_status_string(int(status)).decode()


def _check(status: int, fn: str):
    if status != 0:
        raise SvdqError(status, fn)


def _desc(K: int, N: int, rank: int, fmt) -> LayerDesc:
    f = FORMATS[fmt] if isinstance(fmt, str) else int(fmt)
    return LayerDesc(int(K), int(N), int(rank), f)


def _ptr(a) -> int | None:
    if a is None:
        return None
    if isinstance(a, np.ndarray):
        assert a.flags["C_CONTIGUOUS"]
        return a.ctypes.data
    return a.data_ptr()   # torch tensor


@dataclass
class Layer:
    """Shape and format of one SVDQuant linear."""
    K: int
    N: int
    rank: int
    fmt: str

    @property
    def desc(self) -> LayerDesc:
        return _desc(self.K, self.N, self.rank, self.fmt)


def packed_bytes(layer: Layer) -> dict:
    s = PackedSizes()
    d = layer.desc
    _check(lib().svdq_packed_bytes(ctypes.byref(d), ctypes.byref(s)), "svdq_packed_bytes")
    return {n: getattr(s, n) for n in PACKED_FIELDS}


def _alloc_host(layer: Layer) -> tuple[dict, Packed]:
    sizes = packed_bytes(layer)
    bufs = {n: np.zeros(max(sizes[n], 1), dtype=np.uint8) for n in PACKED_FIELDS}
    p = Packed(*[bufs[n].ctypes.data if sizes[n] else None for n in PACKED_FIELDS])
    return bufs, p


def pack_weights(layer: Layer, w_lin: np.ndarray, bias: np.ndarray | None,
                 act_absmax: np.ndarray, seed: int = 0) -> dict:
    """svdq_pack_weights on host numpy arrays; returns host buffers (uint8 arrays)."""
    w = np.ascontiguousarray(w_lin, dtype=np.float32)
    ax = np.ascontiguousarray(act_absmax, dtype=np.float32)
    b = None if bias is None else np.ascontiguousarray(bias, dtype=np.float32)
    bufs, p = _alloc_host(layer)
    d = layer.desc
    _check(lib().svdq_pack_weights(ctypes.byref(d), _ptr(w), _ptr(b), _ptr(ax), int(seed),
                                   ctypes.byref(p)), "svdq_pack_weights")
    return bufs


def quantize_residual(layer: Layer, w_lin, bias, mu, l1_bits, l2_bits) -> dict:
    """svdq_quantize_residual: host buffers from given mu (fp32 [K]) and bf16 factors."""
    w = np.ascontiguousarray(w_lin, dtype=np.float32)
    b = None if bias is None else np.ascontiguousarray(bias, dtype=np.float32)
    mu = np.ascontiguousarray(mu, dtype=np.float32)
    l1 = np.ascontiguousarray(l1_bits, dtype=np.uint16)
    l2 = np.ascontiguousarray(l2_bits, dtype=np.uint16)
    bufs, p = _alloc_host(layer)
    d = layer.desc
    _check(lib().svdq_quantize_residual(ctypes.byref(d), _ptr(w), _ptr(b), _ptr(mu),
                                        _ptr(l1) if layer.rank else None,
                                        _ptr(l2) if layer.rank else None, ctypes.byref(p)),
           "svdq_quantize_residual")
    return bufs


def lora_extend(layer: Layer, host: dict, lora_a, lora_b, scale: float, share_base: bool = False):
    """svdq_lora_extend: (extended Layer, host buffers) of `layer` with the LoRA
    adapter scale * X A B (A fp32 [K][r_a], B fp32 [r_a][N]) in its 16-bit
    branch. With share_base, only l1 and l2 are returned (the rest of the base
    layer's buffers are used as they are)."""
    a = np.ascontiguousarray(lora_a, dtype=np.float32)
    b = np.ascontiguousarray(lora_b, dtype=np.float32)
    ra = a.shape[1]
    assert a.shape == (layer.K, ra) and b.shape == (ra, layer.N)
    ext = Layer(layer.K, layer.N, layer.rank + ra, layer.fmt)
    bufs, p = _alloc_host(ext)
    if share_base:
        for n in ("mu", "qw", "sw", "bias"):
            setattr(p, n, None)
    base = _packed_struct(layer, host)
    _check(lib().svdq_lora_extend(ctypes.byref(layer.desc), ctypes.byref(base), int(ra), _ptr(a), _ptr(b),
                                  float(scale), ctypes.byref(p)), "svdq_lora_extend")
    if share_base:
        bufs = {n: (bufs[n] if n in ("l1", "l2") else host[n]) for n in PACKED_FIELDS}
    return ext, bufs


def _packed_struct(layer: Layer, bufs: dict) -> Packed:
    sizes = packed_bytes(layer)
    return Packed(*[_ptr(bufs[n]) if sizes[n] else None for n in PACKED_FIELDS])


def unpack_weights(layer: Layer, host: dict) -> dict:
    """Logical codes [N][K], scales [N][K/g], l1 [K][r] / l2 [r][N] / bias bf16 bits."""
    K, N, r = layer.K, layer.N, layer.rank
    g = 64 if layer.fmt == "int4" else 32
    codes = np.zeros((N, K), np.int8)
    scales = np.zeros((N, K // g), np.float32 if layer.fmt == "int4" else np.uint8)
    l1 = np.zeros((K, r), np.uint16)
    l2 = np.zeros((r, N), np.uint16)
    bias = np.zeros(N, np.uint16)
    p = _packed_struct(layer, host)
    d = layer.desc
    _check(lib().svdq_unpack_weights(ctypes.byref(d), ctypes.byref(p), _ptr(codes), _ptr(scales),
                                     _ptr(l1) if r else None, _ptr(l2) if r else None, _ptr(bias)),
           "svdq_unpack_weights")
    mu = host["mu"].view(np.float32)[:K].copy()
    return dict(codes=codes, scales=scales, l1=l1, l2=l2, bias=bias, mu=mu)


def workspace_bytes(layer: Layer, M: int) -> int:
    out = ctypes.c_size_t()
    d = layer.desc
    _check(lib().svdq_workspace_bytes(ctypes.byref(d), int(M), ctypes.byref(out)),
           "svdq_workspace_bytes")
    return out.value


def to_device(layer: Layer, host: dict, device="cuda"):
    """Copy host buffers into torch device tensors (byte for byte)."""
    import torch
    sizes = packed_bytes(layer)
    return {n: torch.from_numpy(host[n][:max(sizes[n], 1)].copy()).to(device) for n in PACKED_FIELDS}


def _stream(stream):
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def linear_forward(layer: Layer, dev: dict, x, y=None, workspace=None, stream=None):
    """y[M][N] (bf16 tensor) = layer(x[M][K] bf16 tensor) via svdq_linear_forward."""
    import torch
    assert x.dtype == torch.bfloat16 and x.is_contiguous() and x.shape[-1] == layer.K
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, layer.N), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(max(workspace_bytes(layer, M), 1), dtype=torch.uint8, device=x.device)
    p = _packed_struct(layer, dev)
    d = layer.desc
    _check(lib().svdq_linear_forward(ctypes.byref(d), ctypes.byref(p), _ptr(x), M, _ptr(y),
                                     _ptr(workspace), workspace.numel(), _stream(stream)),
           "svdq_linear_forward")
    return y


def linear_forward_noalloc(layer: Layer, dev: dict, x, y, stream=None):
    """svdq_linear_forward_noalloc: y (caller's bf16 tensor [M][N]) = layer(x),
    with the library's own device workspace (no allocation by the call)."""
    import torch
    assert x.dtype == torch.bfloat16 and x.is_contiguous() and x.shape[-1] == layer.K
    assert y.dtype == torch.bfloat16 and y.is_contiguous() and tuple(y.shape) == (x.shape[0], layer.N)
    p = _packed_struct(layer, dev)
    d = layer.desc
    _check(lib().svdq_linear_forward_noalloc(ctypes.byref(d), ctypes.byref(p), _ptr(x), x.shape[0],
                                             _ptr(y), _stream(stream)),
           "svdq_linear_forward_noalloc")
    return y


def mlp_workspace_bytes(up: Layer, down: Layer, M: int):
    """(total bytes, offset of the down layer's part) of svdq_mlp_forward's workspace."""
    out, off = ctypes.c_size_t(), ctypes.c_size_t()
    du, dd = up.desc, down.desc
    _check(lib().svdq_mlp_workspace_bytes(ctypes.byref(du), ctypes.byref(dd), int(M), ctypes.byref(out),
                                          ctypes.byref(off)), "svdq_mlp_workspace_bytes")
    return out.value, off.value


def mlp_fused(up: Layer, down: Layer, M: int) -> bool:
    """Whether svdq_mlp_forward in MLP_AUTO mode takes the fused path for M tokens."""
    f = ctypes.c_int32()
    du, dd = up.desc, down.desc
    _check(lib().svdq_mlp_fused(ctypes.byref(du), ctypes.byref(dd), int(M), ctypes.byref(f)), "svdq_mlp_fused")
    return bool(f.value)


def mlp_forward(up: Layer, dev_up: dict, down: Layer, dev_down: dict, x, y=None, workspace=None,
                mode: int = MLP_AUTO, stream=None):
    """y[M][down N] = down(GELU(up(x))) via svdq_mlp_forward (bf16 tensors)."""
    import torch
    assert x.dtype == torch.bfloat16 and x.is_contiguous() and x.shape[-1] == up.K
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, down.N), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(max(mlp_workspace_bytes(up, down, M)[0], 1), dtype=torch.uint8, device=x.device)
    pu, pd = _packed_struct(up, dev_up), _packed_struct(down, dev_down)
    du, dd = up.desc, down.desc
    _check(lib().svdq_mlp_forward(ctypes.byref(du), ctypes.byref(pu), ctypes.byref(dd), ctypes.byref(pd), _ptr(x), M, _ptr(y), _ptr(workspace), workspace.numel(),
                                  int(mode), _stream(stream)), "svdq_mlp_forward")
    return y


def stage1(layer: Layer, dev: dict, x, workspace=None, stream=None):
    import torch
    M = x.shape[0]
    if workspace is None:
        workspace = torch.empty(max(workspace_bytes(layer, M), 1), dtype=torch.uint8, device=x.device)
    p = _packed_struct(layer, dev)
    d = layer.desc
    _check(lib().svdq_stage1(ctypes.byref(d), ctypes.byref(p), _ptr(x), M, _ptr(workspace),
                             workspace.numel(), _stream(stream)), "svdq_stage1")
    return workspace


def stage1_outputs(layer: Layer, dev: dict, x, workspace=None, codes=None, scales=None, z=None,
                   stream=None) -> dict:
    """Kernel (1) with its outputs in logical layouts as device tensors:
    codes int8 [M][K], scales float32 [M][K/64] (INT4) or uint8 [M][K/32]
    (MXFP4), z float32 [M][rank]; allocated here unless given."""
    import torch
    M = x.shape[0]
    if workspace is None:
        workspace = torch.empty(max(workspace_bytes(layer, M), 1), dtype=torch.uint8, device=x.device)
    g = 64 if layer.fmt == "int4" else 32
    if codes is None:
        codes = torch.empty((M, layer.K), dtype=torch.int8, device=x.device)
    if scales is None:
        scales = torch.empty((M, layer.K // g), dtype=torch.float32 if layer.fmt == "int4" else torch.uint8,
                             device=x.device)
    if z is None:
        z = torch.empty((M, layer.rank), dtype=torch.float32, device=x.device)
    assert codes.shape == (M, layer.K) and codes.dtype == torch.int8 and codes.is_contiguous()
    assert scales.shape == (M, layer.K // g) and scales.is_contiguous()
    assert scales.dtype == (torch.float32 if layer.fmt == "int4" else torch.uint8)
    assert z.shape == (M, layer.rank) and z.dtype == torch.float32 and z.is_contiguous()
    p = _packed_struct(layer, dev)
    d = layer.desc
    _check(lib().svdq_stage1_outputs(ctypes.byref(d), ctypes.byref(p), _ptr(x), M, _ptr(codes), _ptr(scales),
                                     _ptr(z) if layer.rank else None, _ptr(workspace), workspace.numel(),
                                     _stream(stream)), "svdq_stage1_outputs")
    return {"codes": codes, "scales": scales, "z": z, "workspace": workspace}


def gemm(layer: Layer, dev: dict, workspace, M: int, y, stream=None):
    """Kernel (2) alone on a workspace filled by stage1() for the same M."""
    p = _packed_struct(layer, dev)
    d = layer.desc
    _check(lib().svdq_gemm(ctypes.byref(d), ctypes.byref(p), _ptr(workspace), workspace.numel(),
                           int(M), _ptr(y), _stream(stream)), "svdq_gemm")
    return y


def unpack_workspace(layer: Layer, M: int, ws_host: np.ndarray) -> dict:
    K, r = layer.K, layer.rank
    g = 64 if layer.fmt == "int4" else 32
    codes = np.zeros((M, K), np.int8)
    scales = np.zeros((M, K // g), np.float32 if layer.fmt == "int4" else np.uint8)
    z = np.zeros((M, r), np.float32)
    ws = np.ascontiguousarray(ws_host, dtype=np.uint8)
    d = layer.desc
    _check(lib().svdq_unpack_workspace(ctypes.byref(d), int(M), _ptr(ws), ws.nbytes, _ptr(codes),
                                       _ptr(scales), _ptr(z) if r else None),
           "svdq_unpack_workspace")
    return dict(codes=codes, scales=scales, z=z)


def debug_int4_group_sums(layer: Layer, dev: dict, workspace, M: int, m0: int, mc: int,
                          n0: int, nc: int, stream=None, out=None):
    """int32 group sums P [mc][nc][K/64] of the window, from the GEMM kernel the
    forward runs for this M. ``out`` (int32 device tensor of that shape) is
    written in place when given."""
    import torch
    p_out = out if out is not None else torch.empty((mc, nc, layer.K // 64), dtype=torch.int32,
                                                    device=workspace.device)
    assert p_out.dtype == torch.int32 and p_out.is_contiguous() and p_out.numel() == mc * nc * (layer.K // 64)
    p = _packed_struct(layer, dev)
    d = layer.desc
    _check(lib().svdq_debug_int4_group_sums(ctypes.byref(d), ctypes.byref(p), _ptr(workspace),
                                            workspace.numel(), int(M), int(m0), int(mc), int(n0),
                                            int(nc), _ptr(p_out), _stream(stream)),
           "svdq_debug_int4_group_sums")
    return p_out


MFMA_KINDS = {"mxfp4": 0, "int8": 1, "bf16": 2}


def measure_mfma_peak(kind: str, iters: int, constant: bool = False, stream=None) -> float:
    """Enqueue the MFMA-only loop of `kind` on the current stream; returns its
    flop count (time it with events on the same stream)."""
    f = ctypes.c_double()
    _check(lib().svdq_measure_mfma_peak(MFMA_KINDS[kind], 1 if constant else 0, int(iters), ctypes.byref(f),
                                        _stream(stream)), "svdq_measure_mfma_peak")
    return f.value


def measure_copy(src, dst, stream=None):
    """Enqueue dst = src (device tensors of the same byte size) on the stream."""
    nbytes = src.numel() * src.element_size()
    assert dst.numel() * dst.element_size() == nbytes
    _check(lib().svdq_measure_copy(_ptr(src), _ptr(dst), nbytes, _stream(stream)), "svdq_measure_copy")


# ----------------------------------------------------------------------------
# GPU-side pack and the calibrated smoothing strength
# ----------------------------------------------------------------------------
def _alloc_device(layer: Layer, device="cuda") -> dict:
    import torch
    sizes = packed_bytes(layer)
    return {n: torch.zeros(max(sizes[n], 1), dtype=torch.uint8, device=device) for n in PACKED_FIELDS}


def pack_weights_gpu(layer: Layer, w_lin, bias, act_absmax, alpha: float = 0.5, seed: int = 0, stream=None):
    """svdq_pack_weights_gpu: device tensors in (fp32 w_lin [N][K], bias [N] or
    None, act_absmax [K]); returns the packed layer as device uint8 tensors."""
    import torch
    dev = _alloc_device(layer, w_lin.device)
    d = layer.desc
    n = ctypes.c_size_t()
    _check(lib().svdq_pack_gpu_workspace_bytes(ctypes.byref(d), ctypes.byref(n)), "svdq_pack_gpu_workspace_bytes")
    ws = torch.empty(max(n.value, 1), dtype=torch.uint8, device=w_lin.device)
    p = _packed_struct(layer, dev)
    _check(lib().svdq_pack_weights_gpu(ctypes.byref(d), _ptr(w_lin), _ptr(bias), _ptr(act_absmax), float(alpha),
                                       int(seed), ctypes.byref(p), _ptr(ws), ws.numel(), _stream(stream)),
           "svdq_pack_weights_gpu")
    return dev


def calibrate_alpha(layer: Layer, w_lin, bias, x_cal, alphas, seed: int = 0, stream=None):
    """svdq_calibrate_alpha: (packed device layer of the best alpha, alpha, losses)."""
    import torch
    dev = _alloc_device(layer, w_lin.device)
    d = layer.desc
    M = x_cal.shape[0]
    n = ctypes.c_size_t()
    _check(lib().svdq_calibrate_workspace_bytes(ctypes.byref(d), M, ctypes.byref(n)),
           "svdq_calibrate_workspace_bytes")
    ws = torch.empty(max(n.value, 1), dtype=torch.uint8, device=w_lin.device)
    al = np.ascontiguousarray(alphas, dtype=np.float32)
    losses = np.zeros(len(al), np.float64)
    a_out = ctypes.c_float()
    p = _packed_struct(layer, dev)
    _check(lib().svdq_calibrate_alpha(ctypes.byref(d), _ptr(w_lin), _ptr(bias), _ptr(x_cal), M, _ptr(al), len(al),
                                      int(seed), ctypes.byref(a_out), _ptr(losses), ctypes.byref(p), _ptr(ws),
                                      ws.numel(), _stream(stream)), "svdq_calibrate_alpha")
    return dev, a_out.value, losses


def to_host(dev: dict) -> dict:
    """Device packed buffers back to host uint8 arrays (byte for byte)."""
    return {n: t.cpu().numpy() for n, t in dev.items()}


# ----------------------------------------------------------------------------
# AWQ-style W4A16 linear (adaptive-normalization and modulation layers)
# ----------------------------------------------------------------------------
def awq_packed_bytes(K: int, N: int) -> dict:
    s = AwqSizes()
    d = AwqDesc(int(K), int(N))
    _check(lib().svdq_awq_packed_bytes(ctypes.byref(d), ctypes.byref(s)), "svdq_awq_packed_bytes")
    return {n: getattr(s, n) for n in AWQ_FIELDS}


def awq_pack(w_lin: np.ndarray, bias, x_cal: np.ndarray, alpha: float | None = None):
    """svdq_awq_pack on host arrays: (host buffers, chosen alpha, s float64 [K])."""
    w = np.ascontiguousarray(w_lin, dtype=np.float32)
    N, K = w.shape
    xc = np.ascontiguousarray(x_cal, dtype=np.float32)
    b = None if bias is None else np.ascontiguousarray(bias, dtype=np.float32)
    sizes = awq_packed_bytes(K, N)
    bufs = {n: np.zeros(max(sizes[n], 1), np.uint8) for n in AWQ_FIELDS}
    p = AwqPacked(*[bufs[n].ctypes.data for n in AWQ_FIELDS])
    a_out = ctypes.c_double()
    s_out = np.zeros(K, np.float64)
    d = AwqDesc(K, N)
    _check(lib().svdq_awq_pack(ctypes.byref(d), _ptr(w), _ptr(b), _ptr(xc), xc.shape[0],
                               -1.0 if alpha is None else float(alpha), ctypes.byref(a_out), _ptr(s_out),
                               ctypes.byref(p)), "svdq_awq_pack")
    return bufs, a_out.value, s_out


def _awq_struct(bufs: dict) -> AwqPacked:
    return AwqPacked(*[_ptr(bufs[n]) for n in AWQ_FIELDS])


def awq_unpack(K: int, N: int, host: dict) -> dict:
    codes = np.zeros((N, K), np.uint8)
    scales = np.zeros((N, K // 128), np.float32)
    zeros = np.zeros((N, K // 128), np.uint8)
    d = AwqDesc(int(K), int(N))
    p = _awq_struct(host)
    _check(lib().svdq_awq_unpack(ctypes.byref(d), ctypes.byref(p), _ptr(codes), _ptr(scales), _ptr(zeros)),
           "svdq_awq_unpack")
    return dict(codes=codes, scales=scales, zeros=zeros, inv_s=host["inv_s"].view(np.float32)[:K].copy(),
                bias=host["bias"].view(np.uint16)[:N].copy())


def awq_to_device(host: dict, device="cuda") -> dict:
    import torch
    return {n: torch.from_numpy(host[n].copy()).to(device) for n in AWQ_FIELDS}


def awq_forward(K: int, N: int, dev: dict, x, y=None, stream=None):
    """y[M][N] bf16 = AWQ layer(x[M][K] bf16) via svdq_awq_forward."""
    import torch
    assert x.dtype == torch.bfloat16 and x.is_contiguous() and x.shape[-1] == K
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    d = AwqDesc(int(K), int(N))
    p = _awq_struct(dev)
    _check(lib().svdq_awq_forward(ctypes.byref(d), ctypes.byref(p), _ptr(x), M, _ptr(y), _stream(stream)),
           "svdq_awq_forward")
    return y


class SVDQLinear:
    """A packed SVDQuant W4A4 linear held in device memory; call it on bf16 input."""

    def __init__(self, layer: Layer, host: dict, device="cuda"):
        self.layer = layer
        self.dev = to_device(layer, host, device)
        self._ws = None

    @classmethod
    def from_float(cls, w_lin, bias, act_absmax, rank: int, fmt: str, seed: int = 0, device="cuda"):
        N, K = w_lin.shape
        layer = Layer(K, N, rank, fmt)
        return cls(layer, pack_weights(layer, w_lin, bias, act_absmax, seed), device)

    def __call__(self, x, y=None, stream=None):
        import torch
        need = max(workspace_bytes(self.layer, x.shape[0]), 1)
        if self._ws is None or self._ws.numel() < need or self._ws.device != x.device:
            self._ws = torch.empty(need, dtype=torch.uint8, device=x.device)
        return linear_forward(self.layer, self.dev, x, y=y, workspace=self._ws, stream=stream)


# ----------------------------------------------------------------------------
# Layer norm and the FP8 linear, forward and backward. The gradients are calls
# of their own: no call records an autograd graph, and one whose input requires
# grad (in grad mode) warns that its outputs do not.
# ----------------------------------------------------------------------------
_t = None         # torch, imported on first use
_DT_CODES = {}    # svdq_dtype of the torch dtypes
_raw_stream = None   # the current stream's handle on a GPU
_current_device = None


def _torch():
    global _t, _raw_stream, _current_device
    if _t is None:
        import torch
        _DT_CODES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
        # (without a Stream object where this torch has the call)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda at: torch.cuda.current_stream(at).cuda_stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _t = torch
    return _t


def _dt(dtype) -> int:
    """svdq_dtype of a torch dtype."""
    code = _DT_CODES.get(dtype)
    if code is None:
        _torch()
        if dtype not in _DT_CODES:
            raise ValueError(f"unsupported dtype {dtype}: bfloat16, float16 or float32")
        code = _DT_CODES[dtype]
    return code


def _need(ok, what: str):
    if not ok:
        raise ValueError(what)


def _on_device(x, *tensors) -> int:
    """The index of the GPU that x and every other given tensor live on."""
    at = x.get_device()
    if at < 0:
        raise ValueError("the tensors must be on a GPU")
    _same_device(at, *tensors)
    return at


def _same_device(at: int, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != at:
            raise ValueError(f"tensors on GPU {at} and on {t.device}")


def _no_graph(name: str):
    """Tells a caller who differentiates with torch that the outputs of a call
    with an input that requires grad are outside of its graph."""
    if _torch().is_grad_enabled():
        warnings.warn(f"{name} records no autograd graph, and an input requires grad: its outputs do not. Call it in a "
                      "torch.autograd.Function with the matching backward call, or under torch.no_grad()", stacklevel=3)


def _empty(shape, dtype, like, stream):
    """A tensor for a call on `stream`, allocated under it, so that the
    allocator does not hand its memory to other work while the call runs."""
    torch = _torch()
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _under(stream, like.device):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _under(stream, device):
    """The context of a stream, given as torch's object or as its handle."""
    if isinstance(stream, int):
        stream = _t.cuda.ExternalStream(stream, device=device)
    return _t.cuda.stream(stream)


def _call(name: str, at: int, stream, *args):
    """The library's function on GPU `at` and the given stream (by default the
    GPU's current one)."""
    f = getattr(lib(), name)
    s = _raw_stream(at) if stream is None else _stream(stream)
    if _current_device() == at:
        st = f(*args, s)
    else:
        with _t.cuda.device(at):
            st = f(*args, s)
    if st != 0:
        raise SvdqError(st, name)


def _rows(t, what: str):
    """(pointer, row stride) of a matrix whose rows are contiguous and apart."""
    shape = t.shape
    if len(shape) == 2:
        cols = shape[1]
        if t.is_contiguous():
            return t.data_ptr(), cols
        ld, step = t.stride()
        if (step == 1 or cols <= 1) and (ld >= cols or shape[0] <= 1):
            return t.data_ptr(), max(ld, cols)
    raise ValueError(f"{what}: a matrix with contiguous rows")


def _param(t, C, groups, dtype, what):
    """(pointer, group stride) of a [C] or [groups][C] parameter."""
    shape = t.shape
    if t.dtype is dtype:
        if len(shape) == 1:
            if groups == 1 and shape[0] == C and t.is_contiguous():
                return t.data_ptr(), C
        elif len(shape) == 2 and shape[0] == groups and shape[1] == C:
            if t.is_contiguous():
                return t.data_ptr(), C
            ld, step = t.stride()
            if (step == 1 or C == 1) and (ld >= C or groups == 1):
                return t.data_ptr(), max(ld, C)
    raise ValueError(f"{what}: [channels] or [groups][channels], contiguous channels, both of one type")


@functools.lru_cache(maxsize=1024)
def _norm_desc(C, dt, pdt, one_plus, groups, eps, rows_per_group):
    """A reference to the descriptor (the library only reads it) and itself."""
    d = NormDesc(C, dt, pdt, one_plus, groups, eps, rows_per_group)
    return ctypes.byref(d), d


@functools.lru_cache(maxsize=4096)
def _norm_ws(C, dt, groups, rows_per_group, M) -> int:
    """Workspace bytes of the gradients (the parameters' type does not matter)."""
    need = ctypes.c_size_t()
    _check(lib().svdq_layer_norm_backward_workspace_bytes(_norm_desc(C, dt, 0, 0, groups, 0.0, rows_per_group)[0], M,
                                                          ctypes.byref(need)),
           "svdq_layer_norm_backward_workspace_bytes")
    return need.value


def _norm_params(C, weight, bias, one_plus, eps, rows_per_group, M, dtype, groups=None):
    """(NormDesc reference, groups, weight pointer, stride, bias pointer,
    stride) of [C] or [groups][C] parameters."""
    wp = bp = shape = None
    ldw = ldb = C
    pdt = dtype
    some = weight if weight is not None else bias
    if some is not None:
        shape, pdt = some.shape, some.dtype
        groups = shape[0] if len(shape) == 2 else 1
        plain = (C,) if len(shape) == 1 else (groups, C)
        if weight is not None:
            if shape == plain and weight.is_contiguous():
                wp = weight.data_ptr()
            else:
                wp, ldw = _param(weight, C, groups, pdt, "weight")
        if bias is not None:
            if bias.shape == plain and bias.dtype is pdt and bias.is_contiguous():
                bp = bias.data_ptr()
            else:
                bp, ldb = _param(bias, C, groups, pdt, "bias")
    elif groups is None:
        groups = 1
    if rows_per_group is None:
        rows_per_group = M if groups == 1 and M > 0 else max(1, -(-M // max(1, groups)))
    dt = _dt(dtype)
    return (_norm_desc(C, dt, dt if pdt is dtype else _dt(pdt), 1 if one_plus else 0, groups, eps, rows_per_group)[0], groups,
            wp, ldw, bp, ldb)


def _rows_like(x, shape, stream):
    """An uninitialised matrix of x's type."""
    if stream is None and x.is_contiguous():
        return _t.empty_like(x)
    return _empty(shape, x.dtype, x, stream)


def _stats(M, x, stream):
    """Uninitialised mean and rstd of M rows."""
    if stream is None:
        mean = x.new_empty((M,), dtype=_t.float32)
        return mean, _t.empty_like(mean)
    return _empty((M,), _t.float32, x, stream), _empty((M,), _t.float32, x, stream)


def layer_norm_forward(x, weight=None, bias=None, eps: float = 1e-6, one_plus: bool = False, rows_per_group=None,
                       y=None, stream=None):
    """svdq_layer_norm_forward: (y, mean, rstd) of the rows of x [M][C]
    (bfloat16, float16 or float32; rows contiguous, any row stride).

    weight and bias: [C], or [groups][C] for rows in groups of rows_per_group
    (default: the rows split evenly); the gain is weight, or 1 + weight with
    one_plus. mean and rstd are float32 [M], for layer_norm_backward."""
    at = _on_device(x, weight, bias, y)
    if x.requires_grad or (weight is not None and weight.requires_grad) or (bias is not None and bias.requires_grad):
        _no_graph("layer_norm_forward")
    xp, ldx = _rows(x, "x")
    M, C = x.shape
    d, _, wp, ldw, bp, ldb = _norm_params(C, weight, bias, one_plus, eps, rows_per_group, M, x.dtype)
    if y is None:
        y = _rows_like(x, (M, C), stream)
    elif y.dtype != x.dtype or y.shape != x.shape:
        raise ValueError("y: the shape and type of x")
    mean, rstd = _stats(M, x, stream)
    yp, ldy = _rows(y, "y")
    _call("svdq_layer_norm_forward", at, stream, d, xp, ldx, wp, ldw, bp, ldb, M, yp, ldy, mean.data_ptr(),
          rstd.data_ptr())
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, one_plus: bool = False, rows_per_group=None, groups=None,
                        grad_dtype=None, param_grads: bool = True, dx=None, stream=None):
    """svdq_layer_norm_backward: (dx, dweight, dbias) for dy [M][C], from the
    forward's x, mean, rstd, weight and grouping. dweight and dbias are
    [groups][C] ([C] for a [C] or absent weight) of grad_dtype (default: the
    weight's type, float32 without one); None without param_grads."""
    at = _on_device(x, dy, mean, rstd, weight, dx)
    if dy.requires_grad:
        _no_graph("layer_norm_backward")
    M, C = x.shape
    _need(dy.shape == x.shape and dy.dtype == x.dtype, "dy: the shape and type of x")
    f32 = _torch().float32
    for t in (mean, rstd):
        _need(t.dtype == f32 and t.shape == (M,) and t.is_contiguous(), "mean, rstd: float32 [rows]")
    flat = groups is None if weight is None else weight.dim() == 1
    d, G, wp, ldw, _, _ = _norm_params(C, weight, None, one_plus, 0.0, rows_per_group, M, x.dtype, groups)
    rpg = rows_per_group if rows_per_group is not None else max(1, -(-M // max(1, G)))
    gdt = grad_dtype if grad_dtype is not None else (weight.dtype if weight is not None else f32)
    if dx is None:
        dx = _rows_like(x, (M, C), stream)
    elif dx.dtype != x.dtype or dx.shape != x.shape:
        raise ValueError("dx: the shape and type of x")
    dw = db = wsp = ws = None
    size = 0
    if param_grads:
        size = _norm_ws(C, _dt(x.dtype), G, rpg, M)
        dw = _empty((C,) if flat else (G, C), gdt, x, stream)
        db = _t.empty_like(dw) if stream is None else _empty(dw.shape, gdt, x, stream)
        if size:
            ws = _empty((size,), _t.uint8, x, stream)
            wsp = ws.data_ptr()
    (dyp, lddy), (xp, ldx), (dxp, lddx) = _rows(dy, "dy"), _rows(x, "x"), _rows(dx, "dx")
    _call("svdq_layer_norm_backward", at, stream, d, dyp, lddy, xp, ldx, wp, ldw, mean.data_ptr(),
          rstd.data_ptr(), M, dxp, lddx, None if dw is None else dw.data_ptr(), None if db is None else db.data_ptr(),
          _dt(gdt), wsp, size)
    return dx, dw, db


@functools.lru_cache(maxsize=4096)
def _fp8_bytes(name: str, K: int, N: int, M: int) -> int:
    out = ctypes.c_size_t()
    _check(getattr(lib(), name)(ctypes.byref(Fp8Desc(K, N)), M, ctypes.byref(out)), name)
    return out.value


def fp8_workspace_bytes(K: int, N: int, M: int) -> int:
    return _fp8_bytes("svdq_fp8_workspace_bytes", K, N, M)


def fp8_norm_workspace_bytes(K: int, N: int, M: int) -> int:
    return _fp8_bytes("svdq_fp8_norm_workspace_bytes", K, N, M)


def fp8_backward_workspace_bytes(K: int, N: int, M: int) -> int:
    return _fp8_bytes("svdq_fp8_backward_workspace_bytes", K, N, M)


def fp8_packed_bytes(K: int, N: int) -> dict:
    s = Fp8Sizes()
    _check(lib().svdq_fp8_packed_bytes(ctypes.byref(Fp8Desc(int(K), int(N))), ctypes.byref(s)), "svdq_fp8_packed_bytes")
    return {n: getattr(s, n) for n in FP8_FIELDS}


def fp8_pack(w, bias=None, transposed: bool = True, out: dict | None = None, stream=None) -> dict:
    """svdq_fp8_pack of a weight [N][K] (bfloat16, float16 or float32, on the
    GPU): {"q", "s", "qt", "st", "bias"}, device tensors of the layer's own (qt
    and st, which the gradient of x reads, are None without `transposed`; bias
    is a bfloat16 copy of `bias`, None without one). `out`: a dict of an earlier
    call, whose tensors are overwritten, as after an update of w: its bias by
    `bias`, which stays as it is without one. A call that is refused changes
    nothing."""
    torch = _torch()
    at = _on_device(w, bias)
    _need(w.dim() == 2 and w.is_contiguous(), "w: a contiguous matrix [N][K]")
    N, K = w.shape
    _need(bias is None or bias.shape == (N,), "bias: [N]")
    sizes = fp8_packed_bytes(K, N)
    if out is None:
        def new(rows, name):
            return _empty((rows, sizes[name] // rows), torch.uint8, w, stream)
        out = {"q": new(N, "q"), "s": new(-(-N // 128), "s"), "qt": new(K, "qt") if transposed else None,
               "st": new(-(-K // 128), "st") if transposed else None, "bias": None}
    d, p = _fp8_struct(K, N, out, at)
    own = out.get("bias")
    if bias is not None and own is None:
        own = _empty((N,), torch.bfloat16, w, stream)
    _call("svdq_fp8_pack", at, stream, d, w.data_ptr(), _dt(w.dtype), p)
    if bias is not None:
        if stream is None:
            own.copy_(bias.detach())
        else:
            with _under(stream, w.device):   # on the call's stream, as the codes
                own.copy_(bias.detach())
        out["bias"] = own
    return out


@functools.lru_cache(maxsize=1024)
def _fp8_desc(K: int, N: int):
    """(descriptor reference, itself, shapes of q, s, qt, st)"""
    d, rk, rn = Fp8Desc(K, N), (K + 127) // 128, (N + 127) // 128
    return (ctypes.byref(d), d, (N, K), (rn, (rk + 3) // 4 * 4), (K, N), (rk, (rn + 3) // 4 * 4))


def _fp8_buffer(t, shape: tuple, name: str, at: int):
    """The address of a layer's buffer of bytes on GPU `at`: of this shape, or,
    as plain bytes, of at least as many."""
    if t is None:
        return None
    if (t.shape != shape and (t.dim() != 1 or t.shape[0] < shape[0] * shape[1])) or t.element_size() != 1 or \
            not t.is_contiguous():
        raise ValueError(f"fp8 layer: {name} must be contiguous bytes {list(shape)}")
    if t.get_device() != at:
        raise ValueError(f"tensors on GPU {at} and on {t.device}")
    return t.data_ptr()


def _fp8_struct(K: int, N: int, dev: dict, at: int = -1, forward: bool = True, backward: bool = True):
    """(reference to the descriptor, reference to the buffers) of a layer on
    GPU `at`: those that the forward or the backward read, or all."""
    ref, _, nq, ns, nqt, nst = _fp8_desc(K, N)
    p = Fp8Packed()
    if forward:
        p.q, p.s = _fp8_buffer(dev.get("q"), nq, "q", at), _fp8_buffer(dev.get("s"), ns, "s", at)
        bias = dev.get("bias")
        if bias is not None:
            if bias.dtype != _torch().bfloat16 or bias.numel() != N or not bias.is_contiguous():
                raise ValueError(f"fp8 layer: bias must be contiguous bfloat16 [{N}]")
            if bias.get_device() != at:
                raise ValueError(f"tensors on GPU {at} and on {bias.device}")
            p.bias = bias.data_ptr()
    if backward:
        p.qt, p.st = _fp8_buffer(dev.get("qt"), nqt, "qt", at), _fp8_buffer(dev.get("st"), nst, "st", at)
    return ref, ctypes.byref(p)


def _bf16_rows(t, cols: int, what: str):
    shape = t.shape
    if t.dtype != _torch().bfloat16 or len(shape) != 2 or shape[1] != cols or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous bfloat16 matrix of {cols} columns")


def _scratch(workspace, size: int, like, stream):
    """(tensor to keep, pointer, bytes) of the caller's workspace or a new one."""
    if workspace is None:
        if not size:
            return None, None, 0
        workspace = _empty((size,), _t.uint8, like, stream)
        return workspace, workspace.data_ptr(), size
    _need(workspace.is_contiguous(), "workspace: contiguous")
    return workspace, workspace.data_ptr(), workspace.nbytes


def fp8_forward(K: int, N: int, dev: dict, x, y=None, workspace=None, stream=None):
    """y[M][N] bf16 = FP8 layer(x[M][K] bf16) via svdq_fp8_forward. y may be x
    itself or overlap it except with a few tokens (fp8_workspace_bytes is 0)."""
    at = _on_device(x, y, workspace)
    if x.requires_grad:
        _no_graph("fp8_forward")
    _bf16_rows(x, K, "x")
    M = x.shape[0]
    if y is None:
        y = _empty((M, N), _t.bfloat16, x, stream)
    else:
        _bf16_rows(y, N, "y")
        _need(y.shape[0] == M, "y: as many rows as x")
    ws, wsp, size = _scratch(workspace, fp8_workspace_bytes(K, N, M), x, stream)
    d, p = _fp8_struct(K, N, dev, at, backward=False)
    _call("svdq_fp8_forward", at, stream, d, p, x.data_ptr(), M, y.data_ptr(), wsp, size)
    return y


def fp8_norm_forward(K: int, N: int, dev: dict, x, weight=None, bias=None, eps: float = 1e-6, one_plus: bool = False,
                     rows_per_group=None, y=None, workspace=None, stats: bool = False, stream=None):
    """y[M][N] = FP8 layer(layer norm(x)) via svdq_fp8_norm_forward, the norm's
    parameters as in layer_norm_forward (`bias` is the norm's; the layer's own
    is in dev). With stats: (y, mean, rstd)."""
    at = _on_device(x, weight, bias, y, workspace)
    if x.requires_grad or (weight is not None and weight.requires_grad) or (bias is not None and bias.requires_grad):
        _no_graph("fp8_norm_forward")
    _bf16_rows(x, K, "x")
    M = x.shape[0]
    d, _, wp, ldw, bp, ldb = _norm_params(K, weight, bias, one_plus, eps, rows_per_group, M, x.dtype)
    if y is None:
        y = _empty((M, N), _t.bfloat16, x, stream)
    else:
        _bf16_rows(y, N, "y")
        _need(y.shape[0] == M, "y: as many rows as x")
    ws, wsp, size = _scratch(workspace, fp8_norm_workspace_bytes(K, N, M), x, stream)
    mean = rstd = None
    if stats:
        mean, rstd = _stats(M, x, stream)
    fd, p = _fp8_struct(K, N, dev, at, backward=False)
    _call("svdq_fp8_norm_forward", at, stream, d, wp, ldw, bp, ldb, fd, p, x.data_ptr(), M, y.data_ptr(), _ptr(mean),
          _ptr(rstd), wsp, size)
    return (y, mean, rstd) if stats else y


def fp8_backward(K: int, N: int, dev: dict, x, dy, need=(True, True, True), workspace=None, stream=None):
    """svdq_fp8_backward: (dx [M][K], dw [N][K], db [N]), bf16, of fp8_forward
    for dy [M][N] bf16; None where `need` says no. Without dx, dev may lack qt
    and st; without dw, x may be None."""
    at = _on_device(dy, x, workspace)
    if dy.requires_grad:
        _no_graph("fp8_backward")
    _bf16_rows(dy, N, "dy")
    M = dy.shape[0]
    if x is not None:
        _bf16_rows(x, K, "x")
        _need(x.shape[0] == M, "x: as many rows as dy")
    bf16 = _t.bfloat16
    dx = _empty((M, K), bf16, dy, stream) if need[0] else None
    dw = _empty((N, K), bf16, dy, stream) if need[1] else None
    db = _empty((N,), bf16, dy, stream) if need[2] else None
    ws, wsp, size = _scratch(workspace, fp8_backward_workspace_bytes(K, N, M), dy, stream)
    d, p = _fp8_struct(K, N, dev, at, forward=False)
    _call("svdq_fp8_backward", at, stream, d, p, _ptr(x), dy.data_ptr(), M, _ptr(dx), _ptr(dw), _ptr(db), wsp, size)
    return dx, dw, db


def fp8_quantize(x, stream=None):
    """svdq_fp8_quantize: (codes uint8 [M][K padded to 128], scale bytes uint8
    [blocks / 4][M][4]) of x bf16 [M][K]."""
    at = _on_device(x)
    _bf16_rows(x, x.shape[-1], "x")
    M, K = x.shape
    nb = -(-K // 128)
    q = _empty((M, nb * 128), _t.uint8, x, stream)
    s = _empty((-(-nb // 4), M, 4), _t.uint8, x, stream)
    _call("svdq_fp8_quantize", at, stream, x.data_ptr(), M, K, q.data_ptr(), s.data_ptr())
    return q, s


class Fp8Linear:
    """An FP8 linear in device memory: call it on bf16 input; `backward` gives
    its gradients; `update` quantizes a new weight (and copies a new bias) into
    the same buffers, which captured graphs of the layer then read."""

    def __init__(self, w, bias=None, trainable: bool = True):
        self.N, self.K = w.shape
        self.dev = fp8_pack(w, bias, transposed=trainable)

    def __call__(self, x, y=None, stream=None):
        return fp8_forward(self.K, self.N, self.dev, x, y=y, stream=stream)

    def after_norm(self, x, weight=None, bias=None, eps: float = 1e-6, one_plus: bool = False, rows_per_group=None,
                   stats: bool = False, stream=None):
        """The layer on layer_norm_forward(x, weight, bias, ...), in one call."""
        return fp8_norm_forward(self.K, self.N, self.dev, x, weight, bias, eps, one_plus, rows_per_group, stats=stats,
                                stream=stream)

    def backward(self, x, dy, need=(True, True, True), stream=None):
        return fp8_backward(self.K, self.N, self.dev, x, dy, need, stream=stream)

    def update(self, w, bias=None, stream=None):
        _need(w.shape == (self.N, self.K), "w: the layer's shape")
        fp8_pack(w, bias, out=self.dev, stream=stream)
