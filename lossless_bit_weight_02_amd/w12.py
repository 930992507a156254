"""Python binding of libw12.so (ctypes): argument marshalling over torch device tensors.

Every step runs in the HIP library; this module only allocates the output tensors with torch,
passes raw device pointers and the current stream, and turns non-zero statuses into W12Error.
If the library is missing, loading fails loudly: there is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw12.so")

W12_OK = 0
W12_ERR_ARG = -1
W12_ERR_SHAPE = -2
W12_ERR_ALIGN = -3
W12_ERR_CAPACITY = -4
W12_ERR_RANGE = -5
W12_ERR_HIP = -6

PATH_AUTO, PATH_GEMV, PATH_MFMA, PATH_STREAM = 0, 1, 2, 3
Q8_MIDPOINT = 0x10
OUT_BF16 = 0x20
IDS_I64 = 0x40
LOGITS_BF16 = 0x80
IN_F32 = 0x100
ROPE_PAIRS = 0x200
KV_E4M3 = 0x1
_PATHS = {None: PATH_AUTO, "auto": PATH_AUTO, "gemv": PATH_GEMV, "mfma": PATH_MFMA, "stream": PATH_STREAM}


class W12Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"w12 status {status}: {msg}")
        self.status = status


class _W12Weight(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("base", ctypes.c_void_p), ("ae", ctypes.c_void_p), ("lo", ctypes.c_void_p),
                ("esc_ptr", ctypes.c_void_p), ("esc_col", ctypes.c_void_p),
                ("esc_val", ctypes.c_void_p), ("esc_cap", ctypes.c_uint64)]


class _W12I8(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("q", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class _W12MX4(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("k", ctypes.c_int64), ("q", ctypes.c_void_p),
                ("nz_ptr", ctypes.c_void_p), ("nz_end", ctypes.c_void_p), ("nz_col", ctypes.c_void_p),
                ("nz_val", ctypes.c_void_p), ("nz_cap", ctypes.c_uint64)]


class _W12KV(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int64), ("heads", ctypes.c_int64), ("page", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("flags", ctypes.c_uint32)]


class _W12KVBatch(ctypes.Structure):
    _fields_ = [("seqs", ctypes.c_int64), ("table", ctypes.c_void_p), ("table_cols", ctypes.c_int64),
                ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("tree", ctypes.c_void_p)]


_lib = None
_lock = threading.Lock()

# name -> (restype, argtypes)
EXPORTS = {
    "w12_abi_version": (ctypes.c_int, []),
    "w12_release_workspace": (ctypes.c_int, [ctypes.c_void_p]),
    "w12_last_error": (ctypes.c_char_p, []),
    "w12_encode": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(_W12Weight),
                                  ctypes.POINTER(ctypes.c_uint64), ctypes.c_void_p]),
    "w12_decode": (ctypes.c_int, [ctypes.POINTER(_W12Weight), ctypes.c_void_p, ctypes.c_void_p]),
    "w12_gemm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_W12Weight),
                                ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p]),
    "w12_gemm_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_W12Weight),
                                        ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p]),
    "w12_q8_gemm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_W12Weight),
                                   ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p]),
    "w12_q8_top1": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_W12Weight),
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p]),
    "w12_gemm_top1": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_W12Weight),
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p]),
    "w12_gemm_silu_mul": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_W12Weight),
                                         ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p]),
    "w12_interleave_rows": (ctypes.c_int, [ctypes.POINTER(_W12Weight), ctypes.POINTER(_W12Weight),
                                           ctypes.POINTER(_W12Weight), ctypes.POINTER(ctypes.c_uint64),
                                           ctypes.c_void_p]),
    "w12_i8_build": (ctypes.c_int, [ctypes.POINTER(_W12Weight), ctypes.POINTER(_W12I8), ctypes.c_void_p]),
    "w12_i8_gemm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_W12I8),
                                   ctypes.POINTER(_W12Weight), ctypes.c_void_p, ctypes.c_uint32,
                                   ctypes.c_void_p]),
    "w12_i8_top1": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_W12I8),
                                   ctypes.POINTER(_W12Weight), ctypes.c_void_p, ctypes.c_void_p,
                                   ctypes.c_uint32, ctypes.c_void_p]),
    "w12_concat_rows": (ctypes.c_int, [ctypes.POINTER(_W12Weight), ctypes.c_int,
                                       ctypes.POINTER(_W12Weight), ctypes.POINTER(ctypes.c_uint64),
                                       ctypes.c_void_p]),
    "w12_mx4_build": (ctypes.c_int, [ctypes.POINTER(_W12Weight), ctypes.POINTER(_W12MX4), ctypes.c_void_p]),
    "w12_mx4_decode": (ctypes.c_int, [ctypes.POINTER(_W12MX4), ctypes.POINTER(_W12Weight), ctypes.c_void_p,
                                      ctypes.c_void_p]),
    "w12_mx4_gemm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_W12MX4),
                                    ctypes.POINTER(_W12Weight), ctypes.c_void_p, ctypes.c_uint32,
                                    ctypes.c_void_p]),
    "w12_mx4_top1": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_W12MX4),
                                    ctypes.POINTER(_W12Weight), ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_uint32, ctypes.c_void_p]),
    "w12_embed": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(_W12Weight), ctypes.c_float,
                                 ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p]),
    "w12_logprobs_scratch": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_uint32,
                                            ctypes.POINTER(ctypes.c_uint64)]),
    "w12_logprobs": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                    ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_uint64, ctypes.c_uint32, ctypes.c_void_p]),
    "w12_kv_append": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                     ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                     ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(_W12KV),
                                     ctypes.POINTER(_W12KVBatch), ctypes.c_void_p, ctypes.c_uint32,
                                     ctypes.c_void_p]),
    "w12_attention_scratch": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(_W12KV),
                                             ctypes.POINTER(_W12KVBatch), ctypes.POINTER(ctypes.c_uint64)]),
    "w12_attention": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                     ctypes.POINTER(_W12KV), ctypes.POINTER(_W12KVBatch), ctypes.c_float,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32,
                                     ctypes.c_void_p]),
    "w12_sample_scratch": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_uint32,
                                          ctypes.POINTER(ctypes.c_uint64)]),
    "w12_sample": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                  ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_void_p]),
    "w12_bf16_gemm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                     ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                     ctypes.c_uint32, ctypes.c_void_p]),
    "w12_bf16_to_tiles": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_void_p, ctypes.c_void_p]),
    "w12_read_probe": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p,
                                      ctypes.c_void_p]),
}


def padded_rows(n: int) -> int:
    """Rows of the tiled plane storage (16-row tiles)."""
    return 16 * ((int(n) + 15) // 16)


def lib():
    """The loaded library (raises if it was never built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m lossless_bit_weight_02_amd.build`")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in EXPORTS.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            if L.w12_abi_version() != 1:
                raise RuntimeError("libw12.so ABI version mismatch")
            _lib = L
    return _lib


def _check(status: int):
    if status != W12_OK:
        raise W12Error(status, lib().w12_last_error().decode(errors="replace"))


def _stream_handle(device) -> int:
    """The raw handle of the device's current stream."""
    if device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


_HERE = contextlib.nullcontext()


def _on_device(device):
    """Makes a tensor's device the current one for a call, at no cost where it already is."""
    return _HERE if torch._C._cuda_getDevice() == device.index else torch.cuda.device(device)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _bits16(t: torch.Tensor) -> torch.Tensor:
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return t
    raise TypeError(f"expected bfloat16 (or 16-bit raw bits), got {t.dtype}")


class W12Weight:
    """A W12 record held as torch device tensors (layout of include/w12.h; ``ae`` and ``lo`` are
    in the tiled storage order, padded_rows(n) rows)."""

    def __init__(self, n, k, base, ae, lo, esc_ptr, esc_col, esc_val):
        self.n, self.k = int(n), int(k)
        self.base, self.ae, self.lo = base, ae, lo
        self.esc_ptr, self.esc_col, self.esc_val = esc_ptr, esc_col, esc_val

    @property
    def n_esc(self) -> int:
        return int(self.esc_col.numel())

    @property
    def device(self):
        return self.ae.device

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.base, self.ae, self.lo, self.esc_ptr, self.esc_col, self.esc_val))

    def bits_per_weight(self) -> float:
        return 8.0 * self.nbytes() / (self.n * self.k)

    def c_struct(self) -> _W12Weight:
        return _W12Weight(self.n, self.k, _ptr(self.base), _ptr(self.ae), _ptr(self.lo),
                          _ptr(self.esc_ptr), _ptr(self.esc_col), _ptr(self.esc_val),
                          self.esc_col.numel())

    def clone(self) -> "W12Weight":
        return W12Weight(self.n, self.k, *(t.clone() for t in
                                           (self.base, self.ae, self.lo, self.esc_ptr,
                                            self.esc_col, self.esc_val)))

    def to_numpy(self) -> dict:
        """Host copies of every array as stored (uint8/uint32/uint16 numpy arrays; ``ae_s`` and
        ``lo_s`` flat, in the tiled storage order)."""
        def host(t, dt):
            return t.cpu().numpy().view(dt)
        import numpy as np
        return dict(n=self.n, k=self.k, base=host(self.base, np.uint8),
                    ae_s=host(self.ae, np.uint8), lo_s=host(self.lo, np.uint8),
                    esc_ptr=host(self.esc_ptr, np.uint32), esc_col=host(self.esc_col, np.uint32),
                    esc_val=host(self.esc_val, np.uint16))


def encode(w: torch.Tensor, esc_guess: int | None = None) -> W12Weight:
    """bfloat16 W [n, k] on the GPU -> W12Weight (one host synchronisation for the escape total)."""
    w = _bits16(w)
    if w.dim() != 2 or not w.is_cuda:
        raise ValueError("w must be a 2-D CUDA tensor")
    w = w.contiguous()
    n, k = w.shape
    dev = w.device
    u8, i32, i16 = torch.uint8, torch.int32, torch.int16
    base = torch.empty(n, dtype=u8, device=dev)
    npad = padded_rows(n)
    ae = torch.empty(npad * k, dtype=u8, device=dev)
    lo = torch.empty(npad * k // 2, dtype=u8, device=dev)
    esc_ptr = torch.empty(n + 1, dtype=i32, device=dev)
    cap = max(1024, (n * k) // 256) if esc_guess is None else max(1, int(esc_guess))
    esc_col = torch.empty(cap, dtype=i32, device=dev)
    esc_val = torch.empty(cap, dtype=i16, device=dev)
    n_esc = ctypes.c_uint64(0)
    L = lib()
    def run():
        s = _W12Weight(n, k, base.data_ptr(), ae.data_ptr(), lo.data_ptr(),
                       esc_ptr.data_ptr(), esc_col.data_ptr(), esc_val.data_ptr(), esc_col.numel())
        return L.w12_encode(w.data_ptr(), ctypes.byref(s), ctypes.byref(n_esc), _stream_handle(dev))

    st = run()
    if st == W12_ERR_CAPACITY:  # the first guess was too small: size exactly and encode again
        esc_col = torch.empty(max(1, n_esc.value), dtype=i32, device=dev)
        esc_val = torch.empty(max(1, n_esc.value), dtype=i16, device=dev)
        st = run()
    _check(st)
    ne = n_esc.value
    return W12Weight(n, k, base, ae, lo, esc_ptr, esc_col[:ne], esc_val[:ne])


def concat_rows(parts) -> W12Weight:
    """Record of the row-stacked matrix [W_0; W_1; ...] from the parts' records (same k; every part
    but the last with n % 16 == 0), built on the device without re-encoding."""
    parts = list(parts)
    if not parts:
        raise ValueError("no parts")
    dev = parts[0].device
    k = parts[0].k
    n = sum(p.n for p in parts)
    ne = sum(p.n_esc for p in parts)
    npad = padded_rows(n)
    u8 = torch.uint8
    out = W12Weight(n, k, torch.empty(n, dtype=u8, device=dev), torch.empty(npad * k, dtype=u8, device=dev),
                    torch.empty(npad * k // 2, dtype=u8, device=dev),
                    torch.empty(n + 1, dtype=torch.int32, device=dev),
                    torch.empty(max(1, ne), dtype=torch.int32, device=dev)[:ne],
                    torch.empty(max(1, ne), dtype=torch.int16, device=dev)[:ne])
    arr = (_W12Weight * len(parts))(*[p.c_struct() for p in parts])
    s = out.c_struct()
    s.esc_cap = ne
    n_esc = ctypes.c_uint64(0)
    _check(lib().w12_concat_rows(arr, len(parts), ctypes.byref(s), ctypes.byref(n_esc), _stream_handle(dev)))
    return out


def interleave_rows(gate: W12Weight, up: W12Weight) -> W12Weight:
    """Record of the gate and up projections with rows interleaved in groups of 8 (rows 16t..16t+7
    gate rows 8t..8t+7, rows 16t+8..16t+15 up rows 8t..8t+7), built on the device without
    re-encoding; the input of gemm_silu_mul."""
    dev, k, n = gate.device, gate.k, 2 * gate.n
    ne = gate.n_esc + up.n_esc
    npad = padded_rows(n)
    u8 = torch.uint8
    out = W12Weight(n, k, torch.empty(n, dtype=u8, device=dev), torch.empty(npad * k, dtype=u8, device=dev),
                    torch.empty(npad * k // 2, dtype=u8, device=dev),
                    torch.empty(n + 1, dtype=torch.int32, device=dev),
                    torch.empty(max(1, ne), dtype=torch.int32, device=dev)[:ne],
                    torch.empty(max(1, ne), dtype=torch.int16, device=dev)[:ne])
    g, u, o = gate.c_struct(), up.c_struct(), out.c_struct()
    o.esc_cap = ne
    n_esc = ctypes.c_uint64(0)
    _check(lib().w12_interleave_rows(ctypes.byref(g), ctypes.byref(u), ctypes.byref(o), ctypes.byref(n_esc),
                                     _stream_handle(dev)))
    return out


def decode_into(wt: W12Weight, out: torch.Tensor) -> torch.Tensor:
    """Decode into a preallocated contiguous bfloat16 [n, k] tensor."""
    if out.numel() != wt.n * wt.k or not out.is_contiguous() or out.element_size() != 2:
        raise ValueError("out must be a contiguous 16-bit tensor with n*k elements")
    s = wt.c_struct()
    _check(lib().w12_decode(ctypes.byref(s), out.data_ptr(), _stream_handle(wt.device)))
    return out


def decode(wt: W12Weight) -> torch.Tensor:
    """W12Weight -> bfloat16 W [n, k] (bit-exact)."""
    return decode_into(wt, torch.empty((wt.n, wt.k), dtype=torch.bfloat16, device=wt.device))


def _prep_x(x: torch.Tensor, k: int, device) -> torch.Tensor:
    """x as the kernels read it: 2-D, 16-bit (bfloat16 bits), contiguous, on the weights' device,
    with k columns.  A wrong x raises here, before anything is launched."""
    x = _bits16(x)
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError("x must be a 2-D CUDA tensor")
    if x.device != device:
        raise ValueError(f"x is on {x.device}, the weights on {device}")
    if x.shape[1] != k:
        raise ValueError(f"x has {x.shape[1]} columns, the weights have k={k}")
    return x.contiguous()


def _check_out(out: torch.Tensor, shape, dtypes, device, what="out"):
    """A caller-provided output: contiguous, on the weights' device, of the given shape, and of
    one of the given dtypes (a wrong one would be written past its end or misread)."""
    if not isinstance(out, torch.Tensor):
        raise TypeError(f"{what} must be a torch tensor")
    if out.device != device:
        raise ValueError(f"{what} is on {out.device}, the weights on {device}")
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(out.shape)}, expected {tuple(shape)}")
    if out.dtype not in dtypes:
        raise ValueError(f"{what} has dtype {out.dtype}, expected one of {dtypes}")
    if not out.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _gemm_io(x, n, k, device, out, out_bf16):
    """Checked (x, out) of a GEMM call: out [m, n] float32, or bfloat16 (OUT_BF16: the float
    result rounded to nearest even), allocated when not given."""
    x = _prep_x(x, k, device)
    if out is None:
        dt = torch.bfloat16 if out_bf16 else torch.float32
        out = torch.empty((x.shape[0], n), dtype=dt, device=device)
    else:
        _check_out(out, (x.shape[0], n), (torch.float32, torch.bfloat16), device)
    return x, out


def _out_flag(out):
    """float32 outputs, or bfloat16 ones (OUT_BF16: the float result rounded to nearest even)."""
    return OUT_BF16 if out.dtype == torch.bfloat16 else 0


def gemm(x: torch.Tensor, wt: W12Weight, path: str | None = None, out: torch.Tensor | None = None,
         out_bf16: bool = False):
    """Exact pass: y = x W^T (fp32, or bfloat16 with ``out_bf16`` / a bfloat16 ``out``) with W
    read from its W12 record."""
    x, out = _gemm_io(x, wt.n, wt.k, wt.device, out, out_bf16)
    if x.shape[0] == 0:
        return out
    s = wt.c_struct()
    _check(lib().w12_gemm(x.data_ptr(), x.shape[0], ctypes.byref(s), out.data_ptr(),
                          _PATHS[path] | _out_flag(out), _stream_handle(x.device)))
    return out


def gemm_silu_mul(x: torch.Tensor, wt: W12Weight, path: str | None = None, out: torch.Tensor | None = None,
                  out_bf16: bool = False):
    """Exact pass on row-interleaved gate+up weights (interleave_rows) with SiLU(gate) * up
    applied where the outputs are stored: h [m, n / 2] float32 (or bfloat16)."""
    x, out = _gemm_io(x, wt.n // 2, wt.k, wt.device, out, out_bf16)
    if x.shape[0] == 0:
        return out
    s = wt.c_struct()
    _check(lib().w12_gemm_silu_mul(x.data_ptr(), x.shape[0], ctypes.byref(s), out.data_ptr(),
                                   _PATHS[path] | _out_flag(out), _stream_handle(x.device)))
    return out


def gemm_noalloc(x: torch.Tensor, wt: W12Weight, out: torch.Tensor, path: str | None = None):
    """gemm into a caller-provided ``out`` (float32 or bfloat16 [m, n]) through the allocation-free
    entry point: the library allocates nothing; its scratch is a fixed per-GPU array shared by
    every call on that GPU (calls overlapping in time on one GPU race)."""
    x, out = _gemm_io(x, wt.n, wt.k, wt.device, out, False)
    if x.shape[0] == 0:
        return out
    s = wt.c_struct()
    _check(lib().w12_gemm_noalloc(x.data_ptr(), x.shape[0], ctypes.byref(s), out.data_ptr(),
                                  _PATHS[path] | _out_flag(out), _stream_handle(x.device)))
    return out


def q8_gemm(x: torch.Tensor, wt: W12Weight, path: str | None = None, out: torch.Tensor | None = None,
            midpoint: bool = False, out_bf16: bool = False):
    """Q pass: y = x W_q^T with W_q the 8-bit view (B plane taken as 0, or as 8 with
    ``midpoint``), escapes exact; outputs as in gemm."""
    x, out = _gemm_io(x, wt.n, wt.k, wt.device, out, out_bf16)
    if x.shape[0] == 0:
        return out
    s = wt.c_struct()
    s.lo = None
    flags = _PATHS[path] | (Q8_MIDPOINT if midpoint else 0) | _out_flag(out)
    _check(lib().w12_q8_gemm(x.data_ptr(), x.shape[0], ctypes.byref(s), out.data_ptr(),
                             flags, _stream_handle(x.device)))
    return out


def _top1(fn, x, wt, lo, out, flags=0):
    x = _prep_x(x, wt.k, wt.device)
    m = x.shape[0]
    if out is None:
        out = (torch.empty(m, dtype=torch.int32, device=x.device),
               torch.empty(m, dtype=torch.float32, device=x.device))
    else:
        if len(out) != 2:
            raise ValueError("out must be a pair (index int32 [m], value float32 [m])")
        _check_out(out[0], (m,), (torch.int32,), wt.device, "out[0]")
        _check_out(out[1], (m,), (torch.float32,), wt.device, "out[1]")
    if m == 0:
        return out
    s = wt.c_struct()
    if not lo:
        s.lo = None
    _check(fn(x.data_ptr(), m, ctypes.byref(s), out[0].data_ptr(), out[1].data_ptr(), flags,
              _stream_handle(x.device)))
    return out


def q8_top1(x: torch.Tensor, wt: W12Weight, out=None, midpoint: bool = False):
    """Top-1 of the Q pass per row of x: (index int32 [m], value float32 [m]), no logits written;
    ``midpoint`` reads the dropped nibble as 8 as in q8_gemm."""
    return _top1(lib().w12_q8_top1, x, wt, False, out, Q8_MIDPOINT if midpoint else 0)


def gemm_top1(x: torch.Tensor, wt: W12Weight, out=None):
    """Top-1 of the exact pass per row of x: (index int32 [m], value float32 [m])."""
    return _top1(lib().w12_gemm_top1, x, wt, True, out)


class I8Copy:
    """The separate 8-bit Q-pass copy of a W12 record: int8 codes in the AE plane's storage order
    (padded_rows(n) * k) and a float32 scale per row; it shares ``rec``'s escape list."""

    def __init__(self, rec: W12Weight, q, scale):
        self.rec, self.q, self.scale = rec, q, scale
        self.n, self.k = rec.n, rec.k

    @property
    def device(self):
        return self.q.device

    def nbytes(self) -> int:
        return self.q.numel() + self.scale.numel() * 4

    def c_struct(self) -> _W12I8:
        return _W12I8(self.n, self.k, self.q.data_ptr(), self.scale.data_ptr())

    def to_numpy(self) -> dict:
        import numpy as np
        return dict(q_s=self.q.cpu().numpy().view(np.int8), scale=self.scale.cpu().numpy())


def i8_build(rec: W12Weight) -> I8Copy:
    """The 8-bit Q-pass copy of ``rec`` (per-row scale from the largest in-window magnitude / 127,
    codes rounded to nearest even, escaped slots 0), built on the device."""
    q = torch.empty(padded_rows(rec.n) * rec.k, dtype=torch.int8, device=rec.device)
    scale = torch.empty(rec.n, dtype=torch.float32, device=rec.device)
    cp = I8Copy(rec, q, scale)
    s, c = rec.c_struct(), cp.c_struct()
    _check(lib().w12_i8_build(ctypes.byref(s), ctypes.byref(c), _stream_handle(rec.device)))
    return cp


def i8_gemm(x: torch.Tensor, cp: I8Copy, path: str | None = None, out: torch.Tensor | None = None,
            out_bf16: bool = False):
    """Q pass on the 8-bit copy: y = x (s q)^T with the record's escapes exact; outputs as in gemm."""
    x, out = _gemm_io(x, cp.n, cp.k, cp.device, out, out_bf16)
    if x.shape[0] == 0:
        return out
    c, s = cp.c_struct(), cp.rec.c_struct()
    s.ae = None
    s.lo = None
    _check(lib().w12_i8_gemm(x.data_ptr(), x.shape[0], ctypes.byref(c), ctypes.byref(s), out.data_ptr(),
                             _PATHS[path] | _out_flag(out), _stream_handle(x.device)))
    return out


def i8_top1(x: torch.Tensor, cp: I8Copy, out=None):
    """Top-1 of the Q pass on the 8-bit copy per row of x: (index int32 [m], value float32 [m])."""
    c = cp.c_struct()
    return _top1(lambda xp, m, s, ip, vp, fl, st: lib().w12_i8_top1(xp, m, ctypes.byref(c), s, ip, vp, fl, st),
                 x, cp.rec, False, out)


class Mx4Copy:
    """The microscaled 4-bit Q-pass copy of a W12 record: tile records of 32-column blocks and the list of
    the record's escapes that are not zero (layout of include/w12.h); it shares ``rec``'s window
    bottoms."""

    def __init__(self, rec: W12Weight, q, nz_ptr, nz_end, nz_col, nz_val):
        self.rec, self.q = rec, q
        self.nz_ptr, self.nz_end, self.nz_col, self.nz_val = nz_ptr, nz_end, nz_col, nz_val
        self.n, self.k = rec.n, rec.k

    @property
    def device(self):
        return self.q.device

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.q, self.nz_ptr, self.nz_end, self.nz_col, self.nz_val))

    def c_struct(self) -> _W12MX4:
        return _W12MX4(self.n, self.k, _ptr(self.q), _ptr(self.nz_ptr), _ptr(self.nz_end), _ptr(self.nz_col),
                       _ptr(self.nz_val), self.nz_col.numel())

    def to_numpy(self) -> dict:
        import numpy as np
        return dict(q_s=self.q.cpu().numpy(), nz_ptr=self.nz_ptr.cpu().numpy().view(np.uint32),
                    nz_end=self.nz_end.cpu().numpy().view(np.uint32),
                    nz_col=self.nz_col.cpu().numpy().view(np.uint32),
                    nz_val=self.nz_val.cpu().numpy().view(np.uint16))


def mx4_build(rec: W12Weight) -> Mx4Copy:
    """The microscaled 4-bit Q-pass copy of ``rec`` (blocks of 32 columns, power-of-two scales, E2M1 codes
    rounded to nearest even, escaped slots 0), built on the device."""
    dev, i32 = rec.device, torch.int32
    cap = rec.n_esc
    cp = Mx4Copy(rec, torch.empty(padded_rows(rec.n) * rec.k // 32 * 17, dtype=torch.uint8, device=dev),
                 torch.empty(rec.n + 1, dtype=i32, device=dev), torch.empty(rec.n, dtype=i32, device=dev),
                 torch.empty(cap, dtype=i32, device=dev), torch.empty(cap, dtype=torch.int16, device=dev))
    s, c = rec.c_struct(), cp.c_struct()
    with _on_device(dev):
        _check(lib().w12_mx4_build(ctypes.byref(s), ctypes.byref(c), _stream_handle(dev)))
    return cp


def mx4_decode(cp: Mx4Copy, out: torch.Tensor | None = None) -> torch.Tensor:
    """The bfloat16 matrix [n, k] the Q pass on the copy multiplies (escaped slots exact)."""
    if out is None:
        out = torch.empty((cp.n, cp.k), dtype=torch.bfloat16, device=cp.device)
    else:
        _check_out(out, (cp.n, cp.k), (torch.bfloat16,), cp.device)
    c, s = cp.c_struct(), cp.rec.c_struct()
    with _on_device(cp.device):
        _check(lib().w12_mx4_decode(ctypes.byref(c), ctypes.byref(s), out.data_ptr(), _stream_handle(cp.device)))
    return out


def mx4_gemm(x: torch.Tensor, cp: Mx4Copy, path: str | None = None, out: torch.Tensor | None = None,
             out_bf16: bool = False):
    """Q pass on the 4-bit copy: y = x Wq^T with Wq = mx4_decode(cp); outputs as in gemm."""
    x, out = _gemm_io(x, cp.n, cp.k, cp.device, out, out_bf16)
    if x.shape[0] == 0:
        return out
    c, s = cp.c_struct(), _W12Weight(cp.n, cp.k, _ptr(cp.rec.base))   # (the record's other arrays are not read)
    with _on_device(x.device):
        _check(lib().w12_mx4_gemm(x.data_ptr(), x.shape[0], ctypes.byref(c), ctypes.byref(s), out.data_ptr(),
                                  _PATHS[path] | _out_flag(out), _stream_handle(x.device)))
    return out


def mx4_top1(x: torch.Tensor, cp: Mx4Copy, out=None):
    """Top-1 of the Q pass on the 4-bit copy per row of x: (index int32 [m], value float32 [m])."""
    c = cp.c_struct()
    with _on_device(cp.device):
        return _top1(lambda xp, m, s, ip, vp, fl, st: lib().w12_mx4_top1(xp, m, ctypes.byref(c), s, ip, vp, fl, st),
                     x, cp.rec, False, out)


def _ids_flag(ids: torch.Tensor, device, what: str):
    if not isinstance(ids, torch.Tensor):
        raise TypeError(f"{what} must be a torch tensor")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"{what} must be int32 or int64, got {ids.dtype}")
    if ids.device != device:
        raise ValueError(f"{what} is on {ids.device}, expected {device}")
    return IDS_I64 if ids.dtype == torch.int64 else 0


def embed(ids: torch.Tensor, wt: W12Weight, scale: float = 1.0, out: torch.Tensor | None = None,
          out_f32: bool = False):
    """Embedding lookup: scale * W[ids], W read from its W12 record.  ids: int32 or int64 of any shape
    on the weights' device; returns [*ids.shape, k] bfloat16 (scale 1: the weight's own bits), or
    float32 with ``out_f32`` / a float32 ``out``.  An id outside 0 .. n-1 gives a row of zeros."""
    dev = wt.device
    flag = _ids_flag(ids, dev, "ids")
    shape = (*ids.shape, wt.k)
    if out is None:
        out = wt.ae.new_empty(shape, dtype=torch.float32 if out_f32 else torch.bfloat16)
    else:
        _check_out(out, shape, (torch.float32, torch.bfloat16), dev)
    if ids.numel() == 0:
        return out
    ids = ids.contiguous()
    s = wt.c_struct()
    with _on_device(dev):
        _check(lib().w12_embed(ids.data_ptr(), ids.numel(), ctypes.byref(s), float(scale), out.data_ptr(),
                               flag | _out_flag(out), _stream_handle(dev)))
    return out


class LogProbs(NamedTuple):
    """Result of logprobs: ``logp`` (the shape of tokens; [m, 0] without), ``entropy`` [m],
    ``top_index`` int32 [m, top] and ``top_logp`` [m, top], descending."""
    logp: torch.Tensor
    entropy: torch.Tensor
    top_index: torch.Tensor
    top_logp: torch.Tensor


_lp_sizes: dict = {}       # (device, m, n, top, flags) -> bytes
_lp_buffers: dict = {}     # (device, stream) -> zero-counter scratch of the stream's calls


def _lp_scratch(m, n, top, flags, device, stream):
    """(scratch or None, bytes) of a logprobs call on `stream`.  Calls of one stream follow each other,
    so they share one buffer, kept until release_workspace; a call under graph capture gets its own,
    cleared by the graph, since graphs may be replayed on any stream."""
    key = (device.index, m, n, top, flags)
    need = _lp_sizes.get(key)
    if need is None:
        b = ctypes.c_uint64(0)
        _check(lib().w12_logprobs_scratch(m, n, top, flags, ctypes.byref(b)))
        if len(_lp_sizes) > 4096:
            _lp_sizes.clear()
        need = _lp_sizes[key] = b.value
    if need == 0:
        return None, 0
    if torch.cuda.is_current_stream_capturing():
        return torch.zeros(need, dtype=torch.uint8, device=device), need
    buf = _lp_buffers.get((device.index, stream))
    if buf is None or buf.numel() < need:
        buf = torch.zeros(max(need, 1 << 18), dtype=torch.uint8, device=device)
        _lp_buffers[(device.index, stream)] = buf
    return buf, need


def logprobs(y: torch.Tensor, tokens: torch.Tensor | None = None, top: int = 0) -> LogProbs:
    """Log probabilities of given tokens, entropy and the ``top`` (0..64) best alternatives of rows of
    logits, in one pass.  y [m, n] float32 or bfloat16 on the GPU, rows at any stride, columns
    contiguous (others are copied); tokens int32 or int64, [m] or [m, t] (a token outside 0 .. n-1 has
    log probability -Inf).  Equal logits go by the lower index; a row of -Inf alone gives -Inf and
    entropy 0; a row with NaN or +Inf gives NaN.  Calls that cut rows in parts keep a scratch buffer
    per stream (256 KiB and up); release_workspace frees it."""
    if not isinstance(y, torch.Tensor) or y.dim() != 2 or not y.is_cuda:
        raise ValueError("y must be a 2-D CUDA tensor")
    if y.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"y must be float32 or bfloat16, got {y.dtype}")
    m, n = y.shape
    top = int(top)
    if not 0 <= top <= min(64, n):
        raise ValueError(f"top must be 0..{min(64, n)}, got {top}")
    if n > 0 and (y.stride(1) != 1 and n > 1 or y.stride(0) < n and m > 1):
        y = y.contiguous()
    flags = LOGITS_BF16 if y.dtype == torch.bfloat16 else 0
    nt = 0
    if tokens is not None:
        flags |= _ids_flag(tokens, y.device, "tokens")
        if tokens.dim() not in (1, 2) or tokens.shape[0] != m:
            raise ValueError(f"tokens must be [{m}] or [{m}, t], got {tuple(tokens.shape)}")
        nt = 1 if tokens.dim() == 1 else tokens.shape[1]
        tokens = tokens.contiguous()
    f32 = torch.float32
    r = LogProbs(y.new_empty((m, 0) if tokens is None else tokens.shape, dtype=f32), y.new_empty(m, dtype=f32),
                 y.new_empty((m, top), dtype=torch.int32), y.new_empty((m, top), dtype=f32))
    if m == 0:
        return r
    if n == 0:
        raise ValueError("y has no columns")
    with _on_device(y.device):
        stream = _stream_handle(y.device)
        scratch, nbytes = _lp_scratch(m, n, top, flags, y.device, stream)
        _check(lib().w12_logprobs(y.data_ptr(), m, n, y.stride(0) if m > 1 else n,
                                  tokens.data_ptr() if nt else None, nt, top,
                                  r.logp.data_ptr() if nt else None, r.entropy.data_ptr(),
                                  r.top_index.data_ptr() if top else None,
                                  r.top_logp.data_ptr() if top else None, _ptr(scratch), nbytes, flags, stream))
    return r


def _kept(name: str):
    """A tensor that a structure of the library holds the address of: read-only."""
    return property(lambda self: self._tensors[name])


class KVCache:
    """A paged key/value cache: k and v [pages, heads, page, dim], bfloat16 or float8_e4m3fn (then standing
    for value * scale of the head, k_scale and v_scale float32 [heads]), with equal strides, columns
    contiguous.  The memory order of pages, heads and places is free (a transposed [pages, page, heads, dim]
    tensor will do).  page is a multiple of 16, dim 64, 128 or 256.  The tensors are the cache's for its life: their
    values may change, other tensors make another KVCache."""

    k, v, k_scale, v_scale = (_kept(n) for n in ("k", "v", "k_scale", "v_scale"))

    def __init__(self, k, v, k_scale=None, v_scale=None):
        for t, what in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor) or t.dim() != 4 or not t.is_cuda:
                raise ValueError(f"{what} must be a 4-D CUDA tensor [pages, heads, page, dim]")
            if t.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
                raise TypeError(f"{what} must be bfloat16 or float8_e4m3fn, got {t.dtype}")
            if t.stride(3) != 1:
                raise ValueError(f"the columns of {what} must be contiguous")
        if k.dtype != v.dtype or k.shape != v.shape or k.stride() != v.stride() or k.device != v.device:
            raise ValueError("k and v differ in type, shape, strides or device")
        e4m3 = k.dtype == torch.float8_e4m3fn
        for t, what in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is None:
                continue
            if not e4m3:
                raise ValueError(f"{what} belongs to a float8_e4m3fn cache")
            if t.dtype != torch.float32:
                raise TypeError(f"{what} must be float32, got {t.dtype}")
            if t.shape != (k.shape[1],) or not t.is_contiguous() or t.device != k.device:
                raise ValueError(f"{what} must be contiguous [{k.shape[1]}] on {k.device}")
        self._tensors = dict(k=k, v=v, k_scale=k_scale, v_scale=v_scale)
        self.pages, self.heads, self.page, self.dim = k.shape
        self.device, self.dtype = k.device, k.dtype
        # (in sizes of 1 a stride says nothing, and torch lets it be anything)
        st = [k.stride(i) if k.shape[i] > 1 else 0 for i in range(3)]
        self._c = _W12KV(self.pages, self.heads, self.page, self.dim, k.data_ptr(), v.data_ptr(), *st,
                         _ptr(k_scale), _ptr(v_scale), KV_E4M3 if e4m3 else 0)
        self._ref = ctypes.byref(self._c)

    def nbytes(self) -> int:
        return 2 * self.k.numel() * self.k.element_size()


def kv_cache(pages: int, heads: int, dim: int, page: int = 64, dtype: torch.dtype = torch.bfloat16, k_scale=None,
             v_scale=None, device="cuda") -> KVCache:
    """A zeroed cache, a page's places of one head side by side."""
    k, v = (torch.zeros((pages, heads, page, dim), dtype=dtype, device=device) for _ in range(2))
    return KVCache(k, v, k_scale, v_scale)


class KVBatch:
    """The new tokens of a step, for every layer's kv_append and attention.  Sequence s has lens[s] places in
    the cache, the last q_start[s + 1] - q_start[s] of them (without q_start: one) its new tokens, rows
    q_start[s] .. of the step; place c is on page table[s, c // page].  All int32 on the device and read when
    the work runs: table [seqs, pages of the longest], lens [seqs], q_start [seqs + 1], positions
    [rows] for the rotation (default: the place).  tree int64 [rows]: bit b of a row's mask lets it see its
    sequence's b-th new token (default: those up to its own).  The tensors are the batch's for its life: update
    them in place from step to step, other tensors make another KVBatch."""

    table, lens, q_start, positions, tree = (_kept(n) for n in ("table", "lens", "q_start", "positions", "tree"))

    def __init__(self, table, lens, q_start=None, positions=None, tree=None):
        i32 = torch.int32
        if not isinstance(table, torch.Tensor) or table.dim() != 2 or not table.is_cuda:
            raise ValueError("table must be a 2-D CUDA tensor")
        if table.shape[0] == 0 or table.shape[1] == 0:
            raise ValueError("table is empty")
        seqs = table.shape[0]
        for t, what, dt, n in ((table, "table", i32, None), (lens, "lens", i32, seqs),
                               (q_start, "q_start", i32, seqs + 1), (positions, "positions", i32, None),
                               (tree, "tree", torch.int64, None)):
            if t is None and what != "lens":
                continue
            if not isinstance(t, torch.Tensor) or t.dtype != dt:
                raise TypeError(f"{what} must be a tensor of {dt}")
            if t.device != table.device:
                raise ValueError(f"{what} is on {t.device}, expected {table.device}")
            if t is not table and (t.dim() != 1 or not t.is_contiguous() or (n is not None and t.shape[0] != n)):
                raise ValueError(f"{what} must be contiguous [{'rows' if n is None else n}]")
        if table.stride(1) != 1 and table.shape[1] > 1 or table.stride(0) < table.shape[1] and seqs > 1:
            raise ValueError("the rows of table must be contiguous and apart")
        self._tensors = dict(table=table, lens=lens, q_start=q_start, positions=positions, tree=tree)
        self.seqs = seqs
        self.device = table.device
        self._c = _W12KVBatch(seqs, table.data_ptr(), table.shape[1], table.stride(0) if seqs > 1 else table.shape[1],
                              lens.data_ptr(), _ptr(q_start), _ptr(positions), _ptr(tree))
        self._ref = ctypes.byref(self._c)
        self._sizes = {}        # scratch of attention calls
        self._fixed = [(n, what) for n, what in ((seqs if q_start is None else None, "lens"),
                                                 (None if positions is None else positions.shape[0], "positions"),
                                                 (None if tree is None else tree.shape[0], "tree")) if n is not None]

    def _rows(self, m: int):
        for n, what in self._fixed:
            if n != m:
                raise ValueError(f"{m} rows for {n} sequences of one new token each" if what == "lens" else
                                 f"{what} has {n} entries for {m} rows")


def _check_step(kv: KVCache, batch: KVBatch):
    if kv.device != batch.device:
        raise ValueError(f"the batch is on {batch.device}, the cache on {kv.device}")


def _step_rows(t, m, cols, device, what):
    """(pointer, row stride) of rows of `cols` values whose columns are contiguous."""
    if t.dim() != 2 or t.shape[1] != cols or (m is not None and t.shape[0] != m):
        raise ValueError(f"{what} must be [{'rows' if m is None else m}, {cols}], got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    if t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < cols:
        raise ValueError(f"the rows of {what} must be contiguous and apart")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else cols


def _check_apart(out, what, at, m, cols, ld, size, same=False):
    """Refuses an output that overlaps rows it is computed from; with ``same`` it may be those rows themselves (every
    value is read before it is written)."""
    to = out.data_ptr()
    if to < at + ((m - 1) * ld + cols) * size and at < to + out.numel() * out.element_size():
        if not (same and to == at and size == out.element_size() and (m == 1 or ld == cols)):
            raise ValueError(f"out overlaps {what}")


def kv_append(qkv, kv: KVCache, batch: KVBatch, rope: torch.Tensor | None = None, interleaved: bool = False,
              out: torch.Tensor | None = None):
    """Rotates the new tokens' q and k by position and puts k and v into the cache; returns the rotated q
    [m, hq * dim] bfloat16.  qkv: the stacked product's rows [m, (hq + 2 heads) * dim], bfloat16 or
    float32, or a tuple of q, k and v rows (q None: only k and v, returns None).  rope float32 [positions,
    rot]: the cosines of a position's rot / 2 angles, then their sines; pairs are (i, i + rot / 2), or
    (2 i, 2 i + 1) with ``interleaved``.  A token without a place in the cache, or with a position outside
    the table, is not appended (the latter's q is zero); rows behind the last sequence are left alone.  out may be
    the rows of q themselves, and else must not overlap q, k or v."""
    _check_step(kv, batch)
    dev, dim, heads = kv.device, kv.dim, kv.heads
    if isinstance(qkv, torch.Tensor):
        if qkv.dim() != 2 or qkv.shape[1] % dim or qkv.shape[1] // dim <= 2 * heads:
            raise ValueError(f"qkv must be [rows, (hq + {2 * heads}) * {dim}], got {tuple(qkv.shape)}")
        m, hq = qkv.shape[0], qkv.shape[1] // dim - 2 * heads
        dt = qkv.dtype
        k, ldk = _step_rows(qkv, m, qkv.shape[1], dev, "qkv")
        q, ldq = k, ldk
        k += hq * dim * qkv.element_size()
        v, ldv = k + heads * dim * qkv.element_size(), ldk
    else:
        tq, tk, tv = qkv
        m, dt = tk.shape[0], tk.dtype
        if tv.dtype != dt or tq is not None and tq.dtype != dt:
            raise TypeError("q, k and v differ in type")
        k, ldk = _step_rows(tk, m, heads * dim, dev, "k")
        v, ldv = _step_rows(tv, m, heads * dim, dev, "v")
        q, ldq, hq = None, 0, 0
        if tq is not None:
            if tq.dim() != 2 or tq.shape[1] % dim or tq.shape[1] == 0:
                raise ValueError(f"q must be [rows, hq * {dim}], got {tuple(tq.shape)}")
            hq = tq.shape[1] // dim
            q, ldq = _step_rows(tq, m, hq * dim, dev, "q")
    if dt not in (torch.bfloat16, torch.float32):
        raise TypeError(f"q, k and v must be bfloat16 or float32, got {dt}")
    batch._rows(m)
    rows = rot = 0
    if rope is not None:
        if rope.dtype != torch.float32 or rope.dim() != 2 or not rope.is_contiguous() or rope.device != dev:
            raise ValueError(f"rope must be contiguous float32 [positions, rot] on {dev}")
        rows, rot = rope.shape
    if out is not None:
        if hq == 0:
            raise ValueError("out without q")
        _check_out(out, (m, hq * dim), (torch.bfloat16,), dev)
        if m:
            size = 4 if dt == torch.float32 else 2
            _check_apart(out, "q", q, m, hq * dim, ldq, size, same=True)
            _check_apart(out, "k", k, m, heads * dim, ldk, size)
            _check_apart(out, "v", v, m, heads * dim, ldv, size)
    elif hq:
        out = batch.lens.new_empty((m, hq * dim), dtype=torch.bfloat16)
    if m == 0:
        return out
    flags = (IN_F32 if dt == torch.float32 else 0) | (ROPE_PAIRS if interleaved else 0)
    with _on_device(dev):
        _check(lib().w12_kv_append(q, ldq, k, ldk, v, ldv, m, hq, _ptr(rope), rows, rot, kv._ref, batch._ref,
                                   _ptr(out), flags, _stream_handle(dev)))
    return out


_step_buffers: dict = {}   # (operator, device, stream) -> scratch of the stream's calls
_step_lock = threading.Lock()


def _step_scratch(what, need, device, stream):
    """Scratch of an attention or sample call on `stream`, kept for the stream's next one until
    release_workspace; a call under graph capture gets its own, since graphs may be replayed on any stream."""
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(need, dtype=torch.uint8, device=device)
    buf = _step_buffers.get((what, device.index, stream))
    if buf is None or buf.numel() < need:
        buf = torch.empty(max(need, 1 << 18), dtype=torch.uint8, device=device)
        _step_buffers[(what, device.index, stream)] = buf
    return buf


def _step_call(what, need, device, stream, call):
    """call(address of scratch) with no other call between its launches: two threads on one stream share
    its buffer, which holds for one call's kernels at a time."""
    with _step_lock:
        _check(call(_step_scratch(what, need, device, stream).data_ptr()))


def attention(q: torch.Tensor, kv: KVCache, batch: KVBatch, scale: float | None = None,
              out: torch.Tensor | None = None):
    """Attention of the new tokens over the cache: q [m, hq * dim] bfloat16 (kv_append's result), hq a
    multiple of the cache's heads; returns [m, hq * dim] bfloat16, the output projection's x.  A row sees
    its sequence's places before the new tokens and the new ones up to its own (or those of its tree mask).
    scale: of the scores, default 1 / sqrt(dim).  A row that sees nothing gives zeros; rows behind the last
    sequence are left alone.  out may be q itself, and else must not overlap it.  Keeps a scratch buffer per stream; release_workspace frees it."""
    _check_step(kv, batch)
    dev, dim = kv.device, kv.dim
    if q.dtype != torch.bfloat16:
        raise TypeError(f"q must be bfloat16, got {q.dtype}")
    if q.dim() != 2 or q.shape[1] == 0 or q.shape[1] % (dim * kv.heads):
        raise ValueError(f"q must be [rows, hq * {dim}] with hq a multiple of {kv.heads}, got {tuple(q.shape)}")
    m, hq = q.shape[0], q.shape[1] // dim
    qp, ldq = _step_rows(q, m, hq * dim, dev, "q")
    batch._rows(m)
    if out is None:
        out = q.new_empty((m, hq * dim))
    else:
        _check_out(out, (m, hq * dim), (torch.bfloat16,), dev)
        if m:
            _check_apart(out, "q", qp, m, hq * dim, ldq, 2, same=True)
    if m == 0:
        return out
    L = lib()
    with _on_device(dev):
        stream = _stream_handle(dev)
        key = (m, hq, kv.heads, dim, kv.page, kv.dtype)
        need = batch._sizes.get(key)
        if need is None:
            n = ctypes.c_uint64(0)
            _check(L.w12_attention_scratch(m, hq, kv._ref, batch._ref, ctypes.byref(n)))
            need = batch._sizes[key] = n.value
        scale = dim ** -0.5 if scale is None else float(scale)
        _step_call("attention", need, dev, stream, lambda buf: L.w12_attention(
            qp, ldq, m, hq, kv._ref, batch._ref, scale, out.data_ptr(), buf, need, 0, stream))
    return out


class Samples(NamedTuple):
    """Result of sample: ``token`` int32 [m], ``logp`` float32 [m] among the kept tokens, ``kept`` int32 [m]."""
    token: torch.Tensor
    logp: torch.Tensor
    kept: torch.Tensor


_sample_sizes: dict = {}   # (m, n, flags) -> bytes of scratch


def sample(y: torch.Tensor, u: torch.Tensor, temperature: torch.Tensor | None = None,
           top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
           min_p: torch.Tensor | None = None) -> Samples:
    """A token per row of logits y [m, n] (float32 or bfloat16, rows at any stride) from the uniform numbers
    u float32 [m].  Per row, each [m] or None: temperature float32 (0 or less: the largest logit), top_k
    int32 (0: off), top_p and min_p float32.  top_k comes first, then the shortest run of what it leaves
    with top_p of its mass, then those of at least min_p times the best one's probability; the token is the
    first in column order at which the kept mass passes u of it.  Equal logits go by the lower index.  A row
    of -Inf alone gives -1, log probability -Inf and 0 kept, one with NaN or +Inf -1, NaN and 0.  Calls
    may keep a scratch buffer per stream; release_workspace frees it."""
    if not isinstance(y, torch.Tensor) or y.dim() != 2 or not y.is_cuda:
        raise ValueError("y must be a 2-D CUDA tensor")
    if y.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"y must be float32 or bfloat16, got {y.dtype}")
    m, n = y.shape
    dev = y.device
    if u is None:
        raise TypeError("u must be a tensor of torch.float32")
    for t, what, dt in ((u, "u", torch.float32), (temperature, "temperature", torch.float32),
                        (top_k, "top_k", torch.int32), (top_p, "top_p", torch.float32), (min_p, "min_p", torch.float32)):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or t.dtype != dt:
            raise TypeError(f"{what} must be a tensor of {dt}")
        if t.shape != (m,) or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous [{m}] on {dev}")
    if n > 0 and (y.stride(1) != 1 and n > 1 or y.stride(0) < n and m > 1):
        y = y.contiguous()
    r = Samples(y.new_empty(m, dtype=torch.int32), y.new_empty(m, dtype=torch.float32),
                y.new_empty(m, dtype=torch.int32))
    if m == 0:
        return r
    if n == 0:
        raise ValueError("y has no columns")
    flags = LOGITS_BF16 if y.dtype == torch.bfloat16 else 0
    L = lib()
    with _on_device(dev):
        stream = _stream_handle(dev)
        need = _sample_sizes.get((m, n, flags))
        if need is None:
            nb = ctypes.c_uint64(0)
            _check(L.w12_sample_scratch(m, n, flags, ctypes.byref(nb)))
            if len(_sample_sizes) > 4096:
                _sample_sizes.clear()
            need = _sample_sizes[m, n, flags] = nb.value
        _step_call("sample", need, dev, stream, lambda buf: L.w12_sample(
            y.data_ptr(), m, n, y.stride(0) if m > 1 else n, _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p),
            u.data_ptr(), r.token.data_ptr(), r.logp.data_ptr(), r.kept.data_ptr(), buf, need, flags, stream))
    return r


class Bf16Tiles:
    """Dense bfloat16 W in the tiled storage order of the baseline kernels."""

    def __init__(self, n, k, data):
        self.n, self.k, self.data = int(n), int(k), data

    def nbytes(self) -> int:
        return self.data.numel() * 2


def bf16_tiles(w: torch.Tensor) -> Bf16Tiles:
    """bfloat16 W [n, k] (row-major, on the GPU) -> the baseline's tiled storage."""
    w = _bits16(w).contiguous()
    n, k = w.shape
    out = torch.empty(padded_rows(n) * k, dtype=torch.bfloat16, device=w.device)
    _check(lib().w12_bf16_to_tiles(w.data_ptr(), n, k, out.data_ptr(), _stream_handle(w.device)))
    return Bf16Tiles(n, k, out)


def bf16_gemm(x: torch.Tensor, wt: Bf16Tiles, path: str | None = None, out: torch.Tensor | None = None,
              out_bf16: bool = False):
    """Same-build dense baseline: y = x W^T with W plain bfloat16 (tiled storage); outputs as in
    gemm."""
    x, out = _gemm_io(x, wt.n, wt.k, wt.data.device, out, out_bf16)
    if x.shape[0] == 0:
        return out
    _check(lib().w12_bf16_gemm(x.data_ptr(), x.shape[0], wt.data.data_ptr(), wt.n, wt.k,
                               out.data_ptr(), _PATHS[path] | _out_flag(out), _stream_handle(x.device)))
    return out


def read_probe(buf: torch.Tensor, sink: torch.Tensor | None = None):
    """Stream every byte of ``buf`` through the read-bandwidth probe kernel."""
    if sink is None:
        sink = torch.zeros(4096, dtype=torch.int32, device=buf.device)
    _check(lib().w12_read_probe(buf.data_ptr(), buf.numel() * buf.element_size(), sink.data_ptr(),
                                _stream_handle(buf.device)))
    return sink


def release_workspace(stream: "torch.cuda.Stream | None" = None, device=None):
    """Free what calls on ``stream`` (default: the current stream of ``device``) have left allocated for
    the next ones: the library's GEMM workspace and the scratch of logprobs, attention and sample; waits for
    the stream's work first.  A later call on the stream allocates anew.  To be called before a stream that either
    ran on is destroyed: a new stream may get its handle."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    with torch.cuda.device(stream.device):
        _check(lib().w12_release_workspace(stream.cuda_stream))
    key = (stream.device.index, stream.cuda_stream)
    with _step_lock:
        held = [d for d in ((_lp_buffers, key), *((_step_buffers, (w, *key)) for w in ("attention", "sample"))) if d[1] in d[0]]
        if held:
            stream.synchronize()
            for bufs, k in held:
                bufs.pop(k, None)
