"""Low-bit all-reduce activation codec for AMD Instinct MI355X (gfx950).

A thin ctypes binding over the C ABI in `include/fc.h` and `include/fc/layer.h`
(libfc.so, built from `csrc/` by `build.py`). Every step of the codec runs in the library's HIP
kernels; this module only checks tensor metadata, allocates outputs with
torch on the input's device, and passes raw device pointers and the current
HIP stream. There is no fallback: if the library cannot be loaded, calls
raise.

Method: "Flash Communication: Reducing Tensor Parallelization Bottleneck for
Fast Large Language Model Inference" -- quantize the R partial sums before
the Reduce-Scatter, reduce and requantize each hidden chunk before the
All-Gather, dequantize after it (Figure 5, right; groups as in Figure 4).
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

__all__ = [
    "FcError", "lib", "library_path",
    "fc_quantize_groups", "fc_dequant_sum_requant", "fc_dequantize", "fc_allreduce_emulated",
    "fc_workspace_bytes", "fc_workspace_layout", "fc_stage2_group", "fc_status_string",
    "fc_sum_uncompressed", "fc_dequantize_residual", "fc_linear_quantize", "workspace_views",
    "fc_allreduce_emulated_noalloc", "NOALLOC_SCRATCH_BYTES",
    "EXPORTED_SYMBOLS",
    "fc_residual_norm", "fc_dequantize_residual_norm", "fc_allreduce_emulated_norm",
    "fc_quantize_mxfp4", "fc_dequantize_mxfp4", "fc_matmul_mxfp4", "fc_linear_mxfp4",
    "fc_linear_mxfp4_workspace_bytes", "LAYER_SYMBOLS",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_PKG, "libfc.so")

FC_F16, FC_BF16 = 0, 1
_DTYPES = {torch.float16: FC_F16, torch.bfloat16: FC_BF16}
EXPORTED_SYMBOLS = (
    "fc_quantize_groups", "fc_dequant_sum_requant", "fc_dequantize", "fc_allreduce_emulated",
    "fc_workspace_bytes", "fc_workspace_layout", "fc_stage2_group", "fc_status_string",
    "fc_sum_uncompressed", "fc_dequant_sum_requant_mixed", "fc_allreduce_emulated_mixed",
    "fc_workspace_bytes_mixed", "fc_workspace_layout_mixed",
    "fc_dequantize_residual", "fc_allreduce_emulated_residual", "fc_linear_quantize",
    "fc_allreduce_emulated_noalloc",
)
# the operators of include/fc/layer.h
LAYER_SYMBOLS = (
    "fc_residual_norm", "fc_dequantize_residual_norm", "fc_allreduce_emulated_norm",
    "fc_quantize_mxfp4", "fc_dequantize_mxfp4", "fc_matmul_mxfp4", "fc_linear_mxfp4",
    "fc_linear_mxfp4_workspace_bytes",
)
# FC_NOALLOC_SCRATCH_BYTES of include/fc.h: the payload scratch the library holds per device
NOALLOC_SCRATCH_BYTES = 64 << 20

_lock = threading.Lock()
_lib = None


class FcError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib().fc_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{where}: {msg}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libfc.so (building it with hipcc first if it is absent)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(library_path):
                from . import build as _build
                _build.build()
            L = ctypes.CDLL(library_path)
            P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            L.fc_quantize_groups.argtypes = [P, I, I, I, I, I, I, P, P, P, P]
            L.fc_dequant_sum_requant.argtypes = [P, P, P, I, I, I, I, I, P, P, P, P]
            L.fc_dequantize.argtypes = [P, P, P, I, I, I, I, I, P, P]
            L.fc_allreduce_emulated.argtypes = [P, I, I, I, I, I, I, P, P, Z, P]
            L.fc_sum_uncompressed.argtypes = [P, I, I, I, I, P, P]
            L.fc_dequant_sum_requant_mixed.argtypes = [P, P, P, I, I, I, I, I, I, P, P, P, P]
            L.fc_allreduce_emulated_mixed.argtypes = [P, I, I, I, I, I, I, I, P, P, Z, P]
            L.fc_dequantize_residual.argtypes = [P, P, P, I, I, I, I, I, P, P, P]
            L.fc_allreduce_emulated_residual.argtypes = [P, I, I, I, I, I, I, I, P, P, P, Z, P]
            L.fc_linear_quantize.argtypes = [P, P, I, I, I, I, I, I, I, P, P, P, P, P]
            L.fc_allreduce_emulated_noalloc.argtypes = [P, I, I, I, I, I, I, P, P]
            for f in (L.fc_linear_quantize, L.fc_quantize_groups, L.fc_dequant_sum_requant, L.fc_dequantize,
                      L.fc_allreduce_emulated, L.fc_sum_uncompressed,
                      L.fc_dequant_sum_requant_mixed, L.fc_allreduce_emulated_mixed,
                      L.fc_dequantize_residual, L.fc_allreduce_emulated_residual,
                      L.fc_allreduce_emulated_noalloc):
                f.restype = I
            F = ctypes.c_float
            norm = [P, P, I, P, F, F, F, P, P]   # w_post, gate, gate_tokens, w_pre, scales, eps, h, y
            L.fc_residual_norm.argtypes = [P, P, I, I, I, *norm, P]
            L.fc_dequantize_residual_norm.argtypes = [P, P, P, I, I, I, I, I, P, *norm, P]
            L.fc_allreduce_emulated_norm.argtypes = [P, I, I, I, I, I, I, I, P, *norm, P, Z, P]
            L.fc_quantize_mxfp4.argtypes = [P, I, I, I, I, P, P, P]
            L.fc_dequantize_mxfp4.argtypes = [P, P, I, I, I, I, P, P]
            L.fc_matmul_mxfp4.argtypes = [P, P, P, P, I, I, I, I, I, P, P]
            L.fc_linear_mxfp4.argtypes = [P, P, P, I, I, I, I, I, P, P, Z, P]
            for f in (L.fc_residual_norm, L.fc_dequantize_residual_norm, L.fc_allreduce_emulated_norm,
                      L.fc_quantize_mxfp4, L.fc_dequantize_mxfp4, L.fc_matmul_mxfp4,
                      L.fc_linear_mxfp4):
                f.restype = I
            L.fc_linear_mxfp4_workspace_bytes.argtypes = [I, I, I]
            L.fc_linear_mxfp4_workspace_bytes.restype = Z
            L.fc_workspace_bytes_mixed.argtypes = [I, I, I, I, I, I]
            L.fc_workspace_bytes_mixed.restype = Z
            L.fc_workspace_layout_mixed.argtypes = [I, I, I, I, I, I, ctypes.POINTER(Z),
                                                    ctypes.POINTER(Z)]
            L.fc_workspace_layout_mixed.restype = I
            L.fc_workspace_bytes.argtypes = [I, I, I, I, I]
            L.fc_workspace_bytes.restype = Z
            L.fc_workspace_layout.argtypes = [I, I, I, I, I, ctypes.POINTER(Z), ctypes.POINTER(Z)]
            L.fc_workspace_layout.restype = I
            L.fc_stage2_group.argtypes = [I, I, I]
            L.fc_stage2_group.restype = I
            L.fc_status_string.argtypes = [I]
            L.fc_status_string.restype = ctypes.c_char_p
            _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status != 0:
        raise FcError(status, where)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# torch's current stream as a raw handle without building a Stream object
# (a few microseconds per call, which matters for decode-sized calls); the
# public route where this accessor does not exist
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device) -> ctypes.c_void_p:
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if _raw_current_stream is not None:
        idx = device.index if device.index is not None else torch.cuda.current_device()
        return ctypes.c_void_p(_raw_current_stream(idx))
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dev_tensor(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dt(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float16 or bfloat16, not {t.dtype}")
    return _DTYPES[t.dtype]


def _room(t: torch.Tensor, name: str, nbytes: int, device) -> None:
    """A caller's buffer: a contiguous tensor on `device` of at least `nbytes`
    bytes (the library writes or reads that many through a raw pointer)."""
    _dev_tensor(t, name)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name} holds {have} bytes, {nbytes} needed")


def fc_status_string(status: int) -> str:
    return lib().fc_status_string(status).decode()


def fc_stage2_group(R: int, H: int, group: int) -> int:
    return lib().fc_stage2_group(R, H, group)


def fc_workspace_bytes(R: int, T: int, H: int, bits: int, group: int,
                       bits2: int | None = None) -> int:
    if bits2 is None or bits2 == bits:
        return lib().fc_workspace_bytes(R, T, H, bits, group)
    return lib().fc_workspace_bytes_mixed(R, T, H, bits, bits2, group)


def fc_workspace_layout(R: int, T: int, H: int, bits: int, group: int, bits2: int | None = None):
    """[(offset, size)] of the six workspace slices: codes1, s1, z1, codes2, s2, z2."""
    off = (ctypes.c_size_t * 6)()
    size = (ctypes.c_size_t * 6)()
    if bits2 is None or bits2 == bits:
        _check(lib().fc_workspace_layout(R, T, H, bits, group, off, size), "fc_workspace_layout")
    else:
        _check(lib().fc_workspace_layout_mixed(R, T, H, bits, bits2, group, off, size),
               "fc_workspace_layout_mixed")
    return [(off[i], size[i]) for i in range(6)]


def fc_quantize_groups(x: torch.Tensor, bits: int, group: int, codes1=None, s1=None, z1=None,
                       stream=None):
    """x [R, T, H] fp16/bf16 -> (codes1 [R, T, H*bits/8] u8, s1, z1 [R, T, H/group] fp16 bits)."""
    _dev_tensor(x, "x")
    R, T, H = x.shape
    dev = x.device
    if codes1 is None:
        codes1 = torch.empty((R, T, H * bits // 8), dtype=torch.uint8, device=dev)
    if s1 is None:
        s1 = torch.empty((R, T, max(H // group, 0)), dtype=torch.uint16, device=dev)
    if z1 is None:
        z1 = torch.empty_like(s1)
    _room(codes1, "codes1", R * T * H * bits // 8, dev)
    _room(s1, "s1", R * T * (H // group) * 2, dev)
    _room(z1, "z1", R * T * (H // group) * 2, dev)
    _check(lib().fc_quantize_groups(_ptr(x), _dt(x, "x"), R, T, H, bits, group, _ptr(codes1),
                                    _ptr(s1), _ptr(z1), _stream(stream, dev)), "fc_quantize_groups")
    return codes1, s1, z1


def fc_dequant_sum_requant(codes1, s1, z1, R: int, T: int, H: int, bits: int, group: int,
                           codes2=None, s2=None, z2=None, stream=None, bits2: int | None = None):
    """Stage-1 payload -> (codes2 [T, H*bits2/8], s2, z2 [T, H/g2]); bits2 defaults to bits."""
    bits2 = bits if bits2 is None else bits2
    for n, t in (("codes1", codes1), ("s1", s1), ("z1", z1)):
        _dev_tensor(t, n)
    dev = codes1.device
    g2 = fc_stage2_group(R, H, group)
    if codes2 is None:
        codes2 = torch.empty((T, H * bits2 // 8), dtype=torch.uint8, device=dev)
    if s2 is None:
        s2 = torch.empty((T, H // g2 if g2 else 0), dtype=torch.uint16, device=dev)
    if z2 is None:
        z2 = torch.empty_like(s2)
    _room(codes1, "codes1", R * T * H * bits // 8, dev)
    _room(s1, "s1", R * T * (H // group) * 2, dev)
    _room(z1, "z1", R * T * (H // group) * 2, dev)
    _room(codes2, "codes2", T * H * bits2 // 8, dev)
    _room(s2, "s2", T * (H // g2 if g2 else 0) * 2, dev)
    _room(z2, "z2", T * (H // g2 if g2 else 0) * 2, dev)
    if bits2 == bits:
        st = lib().fc_dequant_sum_requant(_ptr(codes1), _ptr(s1), _ptr(z1), R, T, H, bits, group,
                                          _ptr(codes2), _ptr(s2), _ptr(z2), _stream(stream, dev))
    else:
        st = lib().fc_dequant_sum_requant_mixed(_ptr(codes1), _ptr(s1), _ptr(z1), R, T, H, bits,
                                                bits2, group, _ptr(codes2), _ptr(s2), _ptr(z2),
                                                _stream(stream, dev))
    _check(st, "fc_dequant_sum_requant")
    return codes2, s2, z2


def fc_dequantize(codes2, s2, z2, T: int, H: int, bits: int, group2: int, dtype: torch.dtype,
                  out=None, stream=None):
    """Stage-2 payload -> out [T, H] of `dtype`."""
    for n, t in (("codes2", codes2), ("s2", s2), ("z2", z2)):
        _dev_tensor(t, n)
    dev = codes2.device
    if out is None:
        out = torch.empty((T, H), dtype=dtype, device=dev)
    _room(codes2, "codes2", T * H * bits // 8, dev)
    _room(s2, "s2", T * (H // group2 if group2 > 0 else 0) * 2, dev)
    _room(z2, "z2", T * (H // group2 if group2 > 0 else 0) * 2, dev)
    _room(out, "out", T * H * 2, dev)
    _check(lib().fc_dequantize(_ptr(codes2), _ptr(s2), _ptr(z2), T, H, bits, group2,
                               _dt(out, "out"), _ptr(out), _stream(stream, dev)), "fc_dequantize")
    return out


def fc_linear_quantize(a: torch.Tensor, w: torch.Tensor, bits: int, group: int, codes1=None,
                       s1=None, z1=None, y=None, stream=None):
    """Row-parallel linear layer of every rank with the stage-1 quantization in its
    epilogue: a [R, T, K], w [R, H, K] (fp16/bf16) -> (codes1, s1, z1, y) for the
    layer output y [R, T, H] = a @ w^T rounded to the dtype. y is written only when
    a tensor (or True, to allocate one) is passed; otherwise None is returned."""
    _dev_tensor(a, "a")
    _dev_tensor(w, "w")
    if a.dtype != w.dtype or a.dim() != 3 or w.dim() != 3 or a.shape[0] != w.shape[0] \
            or a.shape[2] != w.shape[2]:
        raise ValueError("a must be [R, T, K] and w [R, H, K] of one dtype")
    R, T, K = a.shape
    H = w.shape[1]
    dev = a.device
    if w.device != dev:
        raise ValueError(f"w is on {w.device}, a on {dev}")
    if codes1 is None:
        codes1 = torch.empty((R, T, H * bits // 8), dtype=torch.uint8, device=dev)
    if s1 is None:
        s1 = torch.empty((R, T, max(H // group, 0)), dtype=torch.uint16, device=dev)
    if z1 is None:
        z1 = torch.empty_like(s1)
    if y is True:
        y = torch.empty((R, T, H), dtype=a.dtype, device=dev)
    if y is not None and y.dtype != a.dtype:
        raise ValueError(f"y must have a's dtype ({a.dtype}), not {y.dtype}")
    _room(codes1, "codes1", R * T * H * bits // 8, dev)
    _room(s1, "s1", R * T * (H // group) * 2, dev)
    _room(z1, "z1", R * T * (H // group) * 2, dev)
    if y is not None:
        _room(y, "y", R * T * H * 2, dev)
    _check(lib().fc_linear_quantize(_ptr(a), _ptr(w), _dt(a, "a"), R, T, K, H, bits, group,
                                    _ptr(codes1), _ptr(s1), _ptr(z1), _ptr(y),
                                    _stream(stream, dev)), "fc_linear_quantize")
    return codes1, s1, z1, y


def fc_dequantize_residual(codes2, s2, z2, T: int, H: int, bits: int, group2: int,
                           residual: torch.Tensor, out=None, stream=None):
    """Stage-2 payload + residual [T, H] -> out [T, H] = residual + dequantized result
    (`out` may be `residual` itself for an in-place update)."""
    for n, t in (("codes2", codes2), ("s2", s2), ("z2", z2), ("residual", residual)):
        _dev_tensor(t, n)
    dev = codes2.device
    if out is None:
        out = torch.empty((T, H), dtype=residual.dtype, device=dev)
    if out.dtype != residual.dtype:
        raise ValueError("out and residual must have the same dtype")
    _room(codes2, "codes2", T * H * bits // 8, dev)
    _room(s2, "s2", T * (H // group2 if group2 > 0 else 0) * 2, dev)
    _room(z2, "z2", T * (H // group2 if group2 > 0 else 0) * 2, dev)
    _room(residual, "residual", T * H * 2, dev)
    _room(out, "out", T * H * 2, dev)
    _check(lib().fc_dequantize_residual(_ptr(codes2), _ptr(s2), _ptr(z2), T, H, bits, group2,
                                        _dt(residual, "residual"), _ptr(residual), _ptr(out),
                                        _stream(stream, dev)), "fc_dequantize_residual")
    return out


def fc_allreduce_emulated(x: torch.Tensor, bits: int, group: int, out=None, workspace=None,
                          stream=None, bits2: int | None = None, residual=None):
    """x [R, T, H] -> out [T, H]: the whole emulated all-reduce (three kernels).
    `bits` codes the reduce-scatter payload, `bits2` (default: the same) the all-gather one.
    With `residual` [T, H], out = residual + the all-reduce (the last kernel adds it)."""
    _dev_tensor(x, "x")
    bits2 = bits if bits2 is None else bits2
    R, T, H = x.shape
    dev = x.device
    if out is None:
        out = torch.empty((T, H), dtype=x.dtype, device=dev)
    if workspace is None:
        workspace = torch.empty(max(fc_workspace_bytes(R, T, H, bits, group, bits2), 1),
                                dtype=torch.uint8, device=dev)
    if out.dtype != x.dtype:
        raise ValueError("out must have x's dtype")
    _room(out, "out", T * H * 2, dev)
    _room(workspace, "workspace", 0, dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    if residual is not None:
        _room(residual, "residual", T * H * 2, dev)
        if residual.dtype != x.dtype or tuple(residual.shape) != (T, H):
            raise ValueError("residual must be [T, H] of x's dtype")
        st = lib().fc_allreduce_emulated_residual(_ptr(x), _dt(x, "x"), R, T, H, bits, bits2,
                                                  group, _ptr(residual), _ptr(out),
                                                  _ptr(workspace), ws_bytes, _stream(stream, dev))
    elif bits2 == bits:
        st = lib().fc_allreduce_emulated(_ptr(x), _dt(x, "x"), R, T, H, bits, group, _ptr(out),
                                         _ptr(workspace), ws_bytes, _stream(stream, dev))
    else:
        st = lib().fc_allreduce_emulated_mixed(_ptr(x), _dt(x, "x"), R, T, H, bits, bits2, group,
                                               _ptr(out), _ptr(workspace), ws_bytes,
                                               _stream(stream, dev))
    _check(st, "fc_allreduce_emulated")
    return out, workspace


def fc_allreduce_emulated_noalloc(x: torch.Tensor, bits: int, group: int, out=None,
                                  stream=None):
    """x [R, T, H] -> out [T, H]: fc_allreduce_emulated with both payloads in the library's
    own per-device scratch (the C call allocates nothing; pass `out` to allocate nothing
    here either). Raises FcError (FC_ERR_SCRATCH) when the payloads exceed
    NOALLOC_SCRATCH_BYTES. Calls that overlap in time on one device race on the scratch."""
    _dev_tensor(x, "x")
    R, T, H = x.shape
    dev = x.device
    if out is None:
        out = torch.empty((T, H), dtype=x.dtype, device=dev)
    if out.dtype != x.dtype:
        raise ValueError("out must have x's dtype")
    _room(out, "out", T * H * 2, dev)
    _check(lib().fc_allreduce_emulated_noalloc(_ptr(x), _dt(x, "x"), R, T, H, bits, group,
                                               _ptr(out), _stream(stream, dev)),
           "fc_allreduce_emulated_noalloc")
    return out


def fc_sum_uncompressed(x: torch.Tensor, out=None, stream=None):
    """x [R, T, H] fp16/bf16 -> out [T, H]: the uncompressed all-reduce result (binary32 sum)."""
    _dev_tensor(x, "x")
    R, T, H = x.shape
    if out is None:
        out = torch.empty((T, H), dtype=x.dtype, device=x.device)
    if out.dtype != x.dtype:
        raise ValueError("out must have x's dtype")
    _room(out, "out", T * H * 2, x.device)
    _check(lib().fc_sum_uncompressed(_ptr(x), _dt(x, "x"), R, T, H, _ptr(out),
                                     _stream(stream, x.device)), "fc_sum_uncompressed")
    return out


def workspace_views(workspace: torch.Tensor, R: int, T: int, H: int, bits: int, group: int,
                    bits2: int | None = None) -> dict:
    """Views of the payloads inside an fc_allreduce_emulated workspace."""
    bits2 = bits if bits2 is None else bits2
    lay = fc_workspace_layout(R, T, H, bits, group, bits2)
    g2 = fc_stage2_group(R, H, group)
    names = ("codes1", "s1", "z1", "codes2", "s2", "z2")
    shapes = ((R, T, H * bits // 8), (R, T, H // group), (R, T, H // group),
              (T, H * bits2 // 8), (T, H // g2), (T, H // g2))
    out = {}
    for name, (off, size), shape in zip(names, lay, shapes):
        raw = workspace[off:off + size]
        out[name] = raw.view(torch.uint16).view(shape) if name[0] in "sz" else raw.view(shape)
    return out


# --- transformer-block operators (include/fc/layer.h) ------------------------
# Their calls are often short next to a launch, so the checks of a call that is
# in order are a few attribute reads; what is wrong is found out afterwards.

# the current device without torch.cuda's lazy-initialization check
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


_INT_MAX = 2**31 - 1


def _ints(**values) -> None:
    """The library takes 32-bit integers, and ctypes would cut longer ones down to them."""
    for name, v in values.items():
        if not -_INT_MAX <= v <= _INT_MAX:
            raise ValueError(f"{name} must fit 32 bits, not {v}")


def _launch(name: str, device, stream, *args) -> None:
    """Calls the library on `device` (it launches on the current one) and `stream`."""
    fn = getattr(_lib or lib(), name)
    index = device.index
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the call runs on {device}")
        raw = stream.cuda_stream
    elif _raw_current_stream is not None:
        raw = _raw_current_stream(index)
    else:
        raw = torch.cuda.current_stream(device).cuda_stream
    if index == _current_device():
        st = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            st = fn(*args, raw)
    if st != 0:
        raise FcError(st, name)


def _empty(like: torch.Tensor, shape, dtype, stream):
    """A new tensor on like's device for a call on `stream` (None: torch's current one).
    It belongs to that stream: memory that other streams still use cannot come back in
    it, and it is not handed on before the call's work is done."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _like(t: torch.Tensor, name: str, shape: tuple, dtype, device) -> int:
    """The address of an operand of exactly this shape and dtype on `device`."""
    if t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.is_cuda and t.device == device:
        return t.data_ptr()
    _dev_tensor(t, name)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")
    raise ValueError(f"{name} must be {list(shape)} of {dtype}, not {list(t.shape)} of {t.dtype}")


def _norm_operands(T, H, residual, w_post, gate, gate_tokens, w_pre, h, y, stream):
    """Checks what the block-norm calls share; -> (dtype code, the addresses of
    residual, w_post, gate, then gate_tokens, the addresses of w_pre, h, y, and h, y)."""
    dev, dt = residual.device, residual.dtype
    code = _dt(residual, "residual")
    if T > _INT_MAX or H > _INT_MAX:
        _ints(T=T, H=H)
    rows = (T, H)
    pr = _like(residual, "residual", rows, dt, dev)
    pg = py = None
    pw = None if w_post is None else _like(w_post, "w_post", (H,), dt, dev)
    pv = None if w_pre is None else _like(w_pre, "w_pre", (H,), dt, dev)
    if gate is not None:
        if gate_tokens is None:
            gate_tokens = max(T, 1) if gate.dim() == 1 else 1
        if gate_tokens < 1:
            raise ValueError(f"gate_tokens must be at least 1, not {gate_tokens}")
        gate_tokens = min(gate_tokens, max(T, 1))   # beyond T they mean the same
        n = -(-T // gate_tokens)
        pg = _like(gate, "gate", (H,) if gate.dim() == 1 and n <= 1 else (n, H), dt, dev)
    else:
        gate_tokens = 1
    if h is None:
        h = torch.empty_like(residual) if stream is None else _empty(residual, rows, dt, stream)
        ph = h.data_ptr()
    else:
        ph = _like(h, "h", rows, dt, dev)
    if w_pre is not None:
        if y is None:
            y = torch.empty_like(residual) if stream is None else _empty(residual, rows, dt, stream)
            py = y.data_ptr()
        else:
            py = _like(y, "y", rows, dt, dev)
    elif y is not None:
        raise ValueError("y needs w_pre")
    return code, pr, pw, pg, gate_tokens, pv, ph, py, h, y


def fc_residual_norm(x: torch.Tensor, residual: torch.Tensor, w_post=None, w_pre=None, gate=None,
                     gate_tokens: int | None = None, eps: float = 1e-5, res_scale: float = 1.0,
                     out_scale: float = 1.0, h=None, y=None, stream=None):
    """Block norms of a block output x [T, H] and the residual stream [T, H] (fp16/bf16):
        h = res_scale * residual + out_scale * gate * post_norm(x),  y = pre_norm(h)
    -> (h, y), y None without w_pre. w_post and w_pre [H] are RMS-norm weights; without
    w_post x is not normed. gate: [H], or a row for every gate_tokens consecutive tokens
    (default: a row per token). `h` may be `residual` itself (in-place update)."""
    if residual.dim() != 2:
        raise ValueError("residual must be [T, H]")
    T, H = residual.shape
    code, pr, pw, pg, gate_tokens, pv, ph, py, h, y = _norm_operands(
        T, H, residual, w_post, gate, gate_tokens, w_pre, h, y, stream)
    dev = residual.device
    _launch("fc_residual_norm", dev, stream, _like(x, "x", (T, H), residual.dtype, dev), pr, code, T, H, pw, pg,
            gate_tokens, pv, res_scale, out_scale, eps, ph, py)
    return h, y


def fc_dequantize_residual_norm(codes2, s2, z2, T: int, H: int, bits: int, group2: int,
                                residual: torch.Tensor, w_post=None, w_pre=None, gate=None,
                                gate_tokens: int | None = None, eps: float = 1e-5,
                                res_scale: float = 1.0, out_scale: float = 1.0, h=None, y=None,
                                stream=None):
    """fc_residual_norm of the dequantized stage-2 payload (as for fc_dequantize_residual,
    but not rounded to 16 bits before the norms) -> (h, y)."""
    _ints(bits=bits, group2=group2)
    code, pr, pw, pg, gate_tokens, pv, ph, py, h, y = _norm_operands(
        T, H, residual, w_post, gate, gate_tokens, w_pre, h, y, stream)
    dev = residual.device
    meta = T * (H // group2 if group2 > 0 else 0) * 2
    _room(codes2, "codes2", T * H * bits // 8, dev)
    _room(s2, "s2", meta, dev)
    _room(z2, "z2", meta, dev)
    _launch("fc_dequantize_residual_norm", dev, stream, codes2.data_ptr(), s2.data_ptr(), z2.data_ptr(), T, H, bits,
            group2, code, pr, pw, pg, gate_tokens, pv, res_scale, out_scale, eps, ph, py)
    return h, y


def fc_allreduce_emulated_norm(x: torch.Tensor, bits: int, group: int, residual: torch.Tensor,
                               w_post=None, w_pre=None, gate=None, gate_tokens: int | None = None,
                               eps: float = 1e-5, res_scale: float = 1.0, out_scale: float = 1.0,
                               h=None, y=None, workspace=None, stream=None, bits2: int | None = None):
    """x [R, T, H] -> (h, y, workspace): the emulated all-reduce whose last step is
    fc_dequantize_residual_norm. Payloads as fc_allreduce_emulated leaves them."""
    _dev_tensor(x, "x")
    bits2 = bits if bits2 is None else bits2
    R, T, H = x.shape
    _ints(R=R, bits=bits, bits2=bits2, group=group)
    dev = x.device
    _like(residual, "residual", (T, H), x.dtype, dev)
    code, pr, pw, pg, gate_tokens, pv, ph, py, h, y = _norm_operands(
        T, H, residual, w_post, gate, gate_tokens, w_pre, h, y, stream)
    if workspace is None:
        workspace = _empty(x, max(fc_workspace_bytes(R, T, H, bits, group, bits2), 1), torch.uint8, stream)
    _room(workspace, "workspace", 0, dev)
    _launch("fc_allreduce_emulated_norm", dev, stream, x.data_ptr(), code, R, T, H, bits, bits2, group, pr, pw, pg,
            gate_tokens, pv, res_scale, out_scale, eps, ph, py, workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    return h, y, workspace


def _mx_padded(K: int) -> int:
    return (K + 127) // 128 * 128


def _rows3(t: torch.Tensor, name: str):
    """(R, rows, n) of a 3-D tensor, (1, rows, n) of a 2-D one."""
    s = t.shape
    if len(s) == 2:
        s = (1, *s)
    elif len(s) != 3:
        raise ValueError(f"{name} must have 2 or 3 dimensions")
    if max(s) > _INT_MAX:
        raise ValueError(f"the dimensions of {name} must fit 32 bits, not {list(s)}")
    return s


def _mx_operand(codes, scales, name: str, device):
    """MXFP4 codes [..., rows, Kp/2] with scales [..., rows, Kp/32] -> (R, rows, Kp, their addresses)."""
    s = codes.shape
    R, rows, half = _rows3(codes, name + "codes")
    if half == 0 or half % 64 != 0:
        raise ValueError(f"{name}codes must hold a positive multiple of 64 bytes a row, not {half}")
    return (R, rows, 2 * half, _like(codes, name + "codes", s, torch.uint8, device),
            _like(scales, name + "scales", (*s[:-1], half // 16), torch.uint8, device))


def fc_quantize_mxfp4(x: torch.Tensor, codes=None, scales=None, stream=None):
    """x [..., K] fp16/bf16 (2 or 3 dimensions) -> MXFP4 (codes [..., Kp/2], scales
    [..., Kp/32]) uint8, Kp = K rounded up to a multiple of 128 (the padding is zeros)."""
    _dev_tensor(x, "x")
    R, T, K = _rows3(x, "x")
    dev, Kp, lead = x.device, _mx_padded(K), x.shape[:-1]
    if codes is None:
        codes = _empty(x, (*lead, Kp // 2), torch.uint8, stream)
        pc = codes.data_ptr()
    else:
        pc = _like(codes, "codes", (*lead, Kp // 2), torch.uint8, dev)
    if scales is None:
        scales = _empty(x, (*lead, Kp // 32), torch.uint8, stream)
        ps = scales.data_ptr()
    else:
        ps = _like(scales, "scales", (*lead, Kp // 32), torch.uint8, dev)
    _launch("fc_quantize_mxfp4", dev, stream, x.data_ptr(), _dt(x, "x"), R, T, K, pc, ps)
    return codes, scales


def fc_dequantize_mxfp4(codes, scales, K: int, dtype: torch.dtype, out=None, stream=None):
    """MXFP4 codes [..., Kp/2] and scales [..., Kp/32] -> out [..., K] of `dtype`."""
    dev = codes.device
    R, T, Kp, pc, ps = _mx_operand(codes, scales, "", dev)
    if K < 1 or _mx_padded(K) != Kp:
        raise ValueError(f"codes hold rows of {Kp} values, K is {K}")
    shape = (*codes.shape[:-1], K)
    if out is None:
        out = _empty(codes, shape, dtype, stream)
        po = out.data_ptr()
    else:
        po = _like(out, "out", shape, dtype, dev)
    _launch("fc_dequantize_mxfp4", dev, stream, pc, ps, R, T, K, _dt(out, "out"), po)
    return out


def fc_matmul_mxfp4(a_codes, a_scales, w_codes, w_scales, dtype: torch.dtype, y=None, stream=None):
    """MXFP4 a [R, T, K] and w [R, H, K] (or both without R) -> y [R, T, H] = a @ w^T of
    `dtype`, accumulated in binary32."""
    dev = a_codes.device
    R, T, Kp, pa, pas = _mx_operand(a_codes, a_scales, "a_", dev)
    Rw, H, Kw, pw, pws = _mx_operand(w_codes, w_scales, "w_", dev)
    if R != Rw or Kp != Kw or a_codes.dim() != w_codes.dim():
        raise ValueError("a must be [R, T, K] and w [R, H, K]")
    shape = (*a_codes.shape[:-1], H)
    if y is None:
        y = _empty(a_codes, shape, dtype, stream)
        py = y.data_ptr()
    else:
        py = _like(y, "y", shape, dtype, dev)
    _launch("fc_matmul_mxfp4", dev, stream, pa, pas, pw, pws, R, T, Kp, H, _dt(y, "y"), py)
    return y


def fc_linear_mxfp4_workspace_bytes(R: int, T: int, K: int) -> int:
    _ints(R=R, T=T, K=K)
    return (_lib or lib()).fc_linear_mxfp4_workspace_bytes(R, T, K)


def fc_linear_mxfp4(a: torch.Tensor, w_codes, w_scales, y=None, workspace=None, stream=None):
    """a [R, T, K] fp16/bf16 (quantized to MXFP4 in the call) times MXFP4 weights
    w [R, H, K] (or both without R) -> y [R, T, H] = a @ w^T of a's dtype."""
    _dev_tensor(a, "a")
    R, T, K = _rows3(a, "a")
    dev = a.device
    Rw, H, Kw, pw, pws = _mx_operand(w_codes, w_scales, "w_", dev)
    if R != Rw or _mx_padded(K) != Kw or a.dim() != w_codes.dim():
        raise ValueError("a must be [R, T, K] and w [R, H, K]")
    shape = (*a.shape[:-1], H)
    if y is None:
        y = _empty(a, shape, a.dtype, stream)
        py = y.data_ptr()
    else:
        py = _like(y, "y", shape, a.dtype, dev)
    have, pk = 0, None
    if workspace is None:
        need = (_lib or lib()).fc_linear_mxfp4_workspace_bytes(R, T, K)   # integers checked by _rows3
        if need:
            workspace = _empty(a, need, torch.uint8, stream)
            have, pk = need, workspace.data_ptr()
    else:
        _room(workspace, "workspace", 0, dev)
        have, pk = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    _launch("fc_linear_mxfp4", dev, stream, a.data_ptr(), pw, pws, _dt(a, "a"), R, T, K, H, py, pk, have)
    return y
