"""Python binding of libq4gemv (weight-only 4-bit dequant-in-GEMV for sm_103a).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libq4gemv.so``; this module checks tensor dtypes and devices,
passes raw pointers and the current CUDA stream, and raises on a non-OK
status.  PyTorch provides device memory and streams, nothing else.  There is
no CPU fallback: if the library is missing the calls raise.

Entry points (same names as the C ABI in ``include/q4gemv.h``):
``q4_gemv``, ``q4_nrm_gemv``, ``q4_dual_gemv``, ``q4_gus_nrm``,
``q4_res_gemv``, ``q4_argmax``, ``q4_group_sums``, ``q4_pack_half``,
``q4_gemv_half``, ``q4_gemm``, ``q4_decode_step``, ``q4_attn_decode``,
``q4_kv_append``, ``q4_attn_prefill``, ``q4_attn_paged``, ``q4_logprobs``,
``q4_mx_quant``, ``q4_mx_dequant``, ``q4_mx_gemm``, ``q4_moe``; plus ``Q4Weight``
for repacking host weights into the device layout, ``KVPages`` (a paged KV cache),
``MXMatrix`` (a matrix of microscaled 4-bit values), ``MoELayer`` (a layer of experts)
and ``rope_table``.
"""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
LIB_PATH = os.path.join(_HERE, "libq4gemv.so")
HEADER_PATH = os.path.join(_ROOT, "include", "q4gemv.h")

Q4_FMT_Q4_0 = 0
Q4_FMT_AFFINE = 1
Q4_FMT_Q8_0 = 2
Q4_FMT_Q4_K = 3
Q4_FMT_Q1 = 4
MAX_NB = 16
Q4_MX_MXFP4 = 0
Q4_MX_NVFP4 = 1

STATUS = {0: "Q4_OK", 1: "Q4_ERR_NULL", 2: "Q4_ERR_SHAPE", 3: "Q4_ERR_ALIGN",
          4: "Q4_ERR_UNSUPPORTED", 5: "Q4_ERR_WORKSPACE", 6: "Q4_ERR_CUDA"}


class Q4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed: %s" % (what, STATUS.get(status, status)))


class _CWeight(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32),
                ("dev", ctypes.c_void_p), ("bytes", ctypes.c_size_t)]


class _CDecodeLayer(ctypes.Structure):
    _fields_ = [("Wq", _CWeight), ("Wk", _CWeight), ("Wv", _CWeight), ("Wo", _CWeight), ("Wg", _CWeight),
                ("Wu", _CWeight), ("Wd", _CWeight), ("gamma_in", ctypes.c_void_p),
                ("gamma_post", ctypes.c_void_p), ("attn", ctypes.c_void_p)]


class _CStepAttention(ctypes.Structure):
    _fields_ = [("k_caches", ctypes.c_void_p), ("v_caches", ctypes.c_void_p), ("rope_cos", ctypes.c_void_p),
                ("rope_sin", ctypes.c_void_p), ("out", ctypes.c_void_p), ("max_seq", ctypes.c_int32),
                ("position", ctypes.c_int32), ("window", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("scale", ctypes.c_float)]


class _CKvPages(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("dtype", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("nseq", ctypes.c_int32),
                ("width", ctypes.c_int32)]


class _CMx(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("rows", ctypes.c_int32), ("k", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("dev", ctypes.c_void_p), ("bytes", ctypes.c_size_t), ("scale", ctypes.c_float)]


class _CMxSrc(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("up", ctypes.c_void_p), ("gamma", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("rows", ctypes.c_int32), ("k", ctypes.c_int32), ("eps", ctypes.c_float)]


class _CMoELayer(ctypes.Structure):
    _fields_ = [("gate_up", _CMx), ("down", _CMx), ("router", ctypes.c_void_p), ("experts", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("renormalize", ctypes.c_int32)]


_lib = None


def build(force: bool = False) -> str:
    """Compile libq4gemv.so in-tree (nvcc, sm_103a)."""
    from . import _build
    return _build.build(force=force)


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libq4gemv.so is not built (run __graft_entry__.build() or "
                               "bit_weight_quantized_q4_gb300.build())")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
        W, KV = ctypes.POINTER(_CWeight), ctypes.POINTER(_CKvPages)
        MX, SRC, MOE = ctypes.POINTER(_CMx), ctypes.POINTER(_CMxSrc), ctypes.POINTER(_CMoELayer)
        sig = {
            "q4_packed_bytes": (SZ, [I32, I32, I32]),
            "q4_weight_bytes": (SZ, [I32, I32, I32]),
            "q4_repack_q4_0": (I32, [P, I32, I32, P, SZ]),
            "q4_repack_affine": (I32, [P, P, P, I32, I32, P, SZ]),
            "q4_repack_q8_0": (I32, [P, I32, I32, P, SZ]),
            "q4_unpack_q8_0": (I32, [P, SZ, I32, I32, P]),
            "q4_repack_q4_k": (I32, [P, I32, I32, P, SZ]),
            "q4_unpack_q4_k": (I32, [P, SZ, I32, I32, P]),
            "q4_repack_q1": (I32, [P, I32, I32, P, SZ]),
            "q4_unpack_q1": (I32, [P, SZ, I32, I32, P]),
            "q4_unpack_q4_0": (I32, [P, SZ, I32, I32, P]),
            "q4_unpack_affine": (I32, [P, SZ, I32, I32, P, P, P]),
            "q4_group_sums": (I32, [P, I32, I32, P, P]),
            "q4_gemv": (I32, [W, P, P, I32, P, P]),
            "q4_pack_half": (I32, [P, I32, I32, P, P, P, P]),
            "q4_gemv_half": (I32, [W, P, P, P, I32, P, P]),
            "q4_nrm_gemv": (I32, [W, P, P, F, I32, P, P]),
            "q4_dual_gemv": (I32, [W, W, P, P, F, I32, P, P, P]),
            "q4_gus_nrm": (I32, [W, W, P, P, F, I32, P, P]),
            "q4_res_gemv": (I32, [W, P, P, I32, P, P]),
            "q4_argmax_workspace_bytes": (SZ, [I32, I32]),
            "q4_argmax": (I32, [W, P, P, F, I32, P, P, P, P, SZ, P]),
            "q4_argmax_noalloc": (I32, [W, P, P, F, I32, P, P, P, P]),
            "q4_decode_workspace_bytes": (SZ, [I32]),
            "q4_decode_step": (I32, [P, I32, W, P, F, I32, P, P, P, P, P, P, P, P, P, SZ, P]),
            "q4_decode_attn_workspace_bytes": (SZ, [I32, I32, I32]),
            "q4_decode_step_attn": (I32, [P, I32, P, W, P, F, P, P, P, P, P, P, P, P, P, SZ, P]),
            "q4_decode_check": (I32, [P, P]),
            "q4_device_check": (I32, [P]),
            "q4_debug_wait_limits": (I32, [ctypes.c_int64, I32, ctypes.c_int64, I32]),
            "q4_plan": (I32, [I32, I32, I32, I32, I32, I32, ctypes.POINTER(ctypes.c_int32)]),
            "q4_attn_workspace_bytes": (SZ, [I32, I32, I32]),
            "q4_gemm_workspace_bytes": (SZ, [I32, I32]),
            "q4_gemm": (I32, [W, P, I32, P, I32, P, SZ, P]),
            "q4_attn_decode": (I32, [P, P, P, P, P, I32, I32, I32, I32, I32, I32, F, P, P, P, P, SZ, P]),
            "q4_rope_table": (I32, [I32, I32, ctypes.c_double, P, P]),
            "q4_kv_append": (I32, [KV, P, P, P, I32, P, P, I32, P, P, I32, P, P]),
            "q4_attn_prefill_workspace_bytes": (SZ, [KV, I32, I32]),
            "q4_attn_prefill": (I32, [KV, P, I32, P, P, I32, I32, F, P, P, SZ, P]),
            "q4_attn_paged_workspace_bytes": (SZ, [KV, I32]),
            "q4_attn_paged": (I32, [KV, P, P, P, P, I32, I32, F, P, P, I32, P, P, SZ, P]),
            "q4_logprobs": (I32, [P, I32, I32, P, I32, P, P, P, P, P]),
            "q4_mx_bytes": (SZ, [I32, I32, I32]),
            "q4_mx_quant": (I32, [SRC, MX, P]),
            "q4_mx_dequant": (I32, [MX, I32, P, P]),
            "q4_mx_pack": (I32, [P, P, MX, P]),
            "q4_mx_unpack": (I32, [MX, P, P, P]),
            "q4_mx_gemm": (I32, [MX, MX, P, I32, P, P]),
            "q4_mx_linear": (I32, [MX, SRC, MX, P, I32, P, P]),
            "q4_moe_pack": (I32, [MX, MX, MX, P]),
            "q4_moe_workspace_bytes": (SZ, [MOE, I32]),
            "q4_moe": (I32, [MOE, SRC, P, P, I32, P, P, P, P, SZ, P]),
            "q4_status_str": (ctypes.c_char_p, [I32]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions ``include/q4gemv.h`` declares."""
    src = open(HEADER_PATH).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(q4_[a-z0-9_]+)\s*\(", src)))


def _check(status: int, what: str):
    if status != 0:
        raise Q4Error(status, what)


# ------------------------------------------------------------------ host side

def packed_bytes(fmt: int, n: int, k: int) -> int:
    return int(lib().q4_packed_bytes(fmt, n, k))


def weight_bytes(fmt: int, n: int, k: int) -> int:
    return int(lib().q4_weight_bytes(fmt, n, k))


def repack_q4_0(blocks: np.ndarray, n: int, k: int) -> np.ndarray:
    blocks = np.ascontiguousarray(blocks, dtype=np.uint8)
    if blocks.size != n * (k // 32) * 18:
        raise ValueError("Q4_0 blocks must be uint8[n, k/32, 18]")
    nbytes = packed_bytes(Q4_FMT_Q4_0, n, k)
    if nbytes == 0:
        raise ValueError("bad shape n=%d k=%d" % (n, k))
    out = np.empty(nbytes, dtype=np.uint8)
    _check(lib().q4_repack_q4_0(blocks.ctypes.data, n, k, out.ctypes.data, nbytes), "q4_repack_q4_0")
    return out


def repack_q8_0(blocks: np.ndarray, n: int, k: int) -> np.ndarray:
    blocks = np.ascontiguousarray(blocks, dtype=np.uint8)
    if blocks.size != n * (k // 32) * 34:
        raise ValueError("Q8_0 blocks must be uint8[n, k/32, 34]")
    nbytes = packed_bytes(Q4_FMT_Q8_0, n, k)
    if nbytes == 0:
        raise ValueError("bad shape n=%d k=%d" % (n, k))
    out = np.empty(nbytes, dtype=np.uint8)
    _check(lib().q4_repack_q8_0(blocks.ctypes.data, n, k, out.ctypes.data, nbytes), "q4_repack_q8_0")
    return out


def unpack_q8_0(packed: np.ndarray, n: int, k: int) -> np.ndarray:
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    out = np.zeros((n, k // 32, 34), dtype=np.uint8)
    _check(lib().q4_unpack_q8_0(packed.ctypes.data, packed.size, n, k, out.ctypes.data), "q4_unpack_q8_0")
    return out


def repack_q4_k(blocks: np.ndarray, n: int, k: int) -> np.ndarray:
    blocks = np.ascontiguousarray(blocks, dtype=np.uint8)
    if k % 256 != 0 or blocks.size != n * (k // 256) * 144:
        raise ValueError("Q4_K superblocks must be uint8[n, k/256, 144] with k a multiple of 256")
    nbytes = packed_bytes(Q4_FMT_Q4_K, n, k)
    if nbytes == 0:
        raise ValueError("bad shape n=%d k=%d" % (n, k))
    out = np.empty(nbytes, dtype=np.uint8)
    _check(lib().q4_repack_q4_k(blocks.ctypes.data, n, k, out.ctypes.data, nbytes), "q4_repack_q4_k")
    return out


def unpack_q4_k(packed: np.ndarray, n: int, k: int) -> np.ndarray:
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    out = np.zeros((n, k // 256, 144), dtype=np.uint8)
    _check(lib().q4_unpack_q4_k(packed.ctypes.data, packed.size, n, k, out.ctypes.data), "q4_unpack_q4_k")
    return out


def repack_q1(blocks: np.ndarray, n: int, k: int) -> np.ndarray:
    blocks = np.ascontiguousarray(blocks, dtype=np.uint8)
    if k % 128 != 0 or blocks.size != n * (k // 128) * 18:
        raise ValueError("Q1 superblocks must be uint8[n, k/128, 18] with k a multiple of 128")
    nbytes = packed_bytes(Q4_FMT_Q1, n, k)
    if nbytes == 0:
        raise ValueError("bad shape n=%d k=%d" % (n, k))
    out = np.empty(nbytes, dtype=np.uint8)
    _check(lib().q4_repack_q1(blocks.ctypes.data, n, k, out.ctypes.data, nbytes), "q4_repack_q1")
    return out


def unpack_q1(packed: np.ndarray, n: int, k: int) -> np.ndarray:
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    out = np.zeros((n, k // 128, 18), dtype=np.uint8)
    _check(lib().q4_unpack_q1(packed.ctypes.data, packed.size, n, k, out.ctypes.data), "q4_unpack_q1")
    return out


def repack_affine(nib: np.ndarray, s: np.ndarray, m: np.ndarray, n: int, k: int) -> np.ndarray:
    nib = np.ascontiguousarray(nib, dtype=np.uint8)
    s = np.ascontiguousarray(s, dtype=np.uint16)
    m = np.ascontiguousarray(m, dtype=np.uint16)
    if nib.size != n * k // 2 or s.size != n * k // 32 or m.size != n * k // 32:
        raise ValueError("affine weights must be nib uint8[n, k/2], s/m uint16[n, k/32]")
    nbytes = packed_bytes(Q4_FMT_AFFINE, n, k)
    if nbytes == 0:
        raise ValueError("bad shape n=%d k=%d" % (n, k))
    out = np.empty(nbytes, dtype=np.uint8)
    _check(lib().q4_repack_affine(nib.ctypes.data, s.ctypes.data, m.ctypes.data, n, k,
                                  out.ctypes.data, nbytes), "q4_repack_affine")
    return out


def unpack_q4_0(packed: np.ndarray, n: int, k: int) -> np.ndarray:
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    out = np.zeros((n, k // 32, 18), dtype=np.uint8)
    _check(lib().q4_unpack_q4_0(packed.ctypes.data, packed.size, n, k, out.ctypes.data), "q4_unpack_q4_0")
    return out


def unpack_affine(packed: np.ndarray, n: int, k: int):
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    nib = np.zeros((n, k // 2), dtype=np.uint8)
    s = np.zeros((n, k // 32), dtype=np.uint16)
    m = np.zeros((n, k // 32), dtype=np.uint16)
    _check(lib().q4_unpack_affine(packed.ctypes.data, packed.size, n, k, nib.ctypes.data,
                                  s.ctypes.data, m.ctypes.data), "q4_unpack_affine")
    return nib, s, m


def plan(fmt: int, tiles: int, chunks: int, nb: int, pairs: bool, num_sms: int) -> dict:
    out = (ctypes.c_int32 * 6)()
    _check(lib().q4_plan(fmt, tiles, chunks, nb, int(pairs), num_sms, out), "q4_plan")
    return dict(zip(("TG", "S", "Cs", "groups", "ctas", "smem"), list(out)))


# ---------------------------------------------------------------- device side

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


class Q4Weight:
    """A repacked weight matrix resident in device memory (owns its tensor)."""

    def __init__(self, fmt: int, n: int, k: int, packed: np.ndarray, device="cuda"):
        torch = _torch()
        self.fmt, self.n, self.k = int(fmt), int(n), int(k)
        self.tensor = torch.from_numpy(packed).to(device)
        self.nbytes = int(packed.size)
        self._c = _CWeight(self.fmt, self.n, self.k, self.tensor.data_ptr(), self.nbytes)

    @classmethod
    def from_q4_0(cls, blocks: np.ndarray, n: int, k: int, device="cuda") -> "Q4Weight":
        return cls(Q4_FMT_Q4_0, n, k, repack_q4_0(blocks, n, k), device)

    @classmethod
    def from_q8_0(cls, blocks: np.ndarray, n: int, k: int, device="cuda") -> "Q4Weight":
        return cls(Q4_FMT_Q8_0, n, k, repack_q8_0(blocks, n, k), device)

    @classmethod
    def from_q4_k(cls, blocks: np.ndarray, n: int, k: int, device="cuda") -> "Q4Weight":
        return cls(Q4_FMT_Q4_K, n, k, repack_q4_k(blocks, n, k), device)

    @classmethod
    def from_q1(cls, blocks: np.ndarray, n: int, k: int, device="cuda") -> "Q4Weight":
        return cls(Q4_FMT_Q1, n, k, repack_q1(blocks, n, k), device)

    @classmethod
    def from_affine(cls, nib, s, m, n: int, k: int, device="cuda") -> "Q4Weight":
        return cls(Q4_FMT_AFFINE, n, k, repack_affine(nib, s, m, n, k), device)

    @property
    def weight_bytes(self) -> int:
        """Algorithmic bytes: 18 (Q4_0), 20 (affine) or 34 (Q8_0) per 32
        weights, 144 per 256 (Q4_K), 18 per 128 (Q1)."""
        return weight_bytes(self.fmt, self.n, self.k)

    def cref(self):
        return ctypes.byref(self._c)


def _stream():
    return _torch().cuda.current_stream().cuda_stream


def _dev_f32(t, name, shape=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_cuda:
        raise TypeError("%s must be a CUDA float32 tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    return t


def _dev_buf(t, name, dtype, shape, device, min_numel=None):
    """A caller-supplied output or workspace: a contiguous CUDA tensor of
    `dtype` on `device`, of exactly `shape` (or, for a workspace, at least
    `min_numel` elements).  The C ABI carries no sizes for these buffers, so
    everything is checked here, before any launch."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype:
        raise TypeError("%s must be a CUDA %s tensor" % (name, dtype))
    if t.device != device:
        raise ValueError("%s is on %s, the activations on %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if min_numel is not None:
        if t.numel() < min_numel:
            raise ValueError("%s has %d elements, needs at least %d" % (name, t.numel(), min_numel))
    elif tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    return t


def _argmax_outs(W, x, nb, want_val, want_logits, idx, val, logits):
    torch = _torch()
    if idx is None:
        idx = torch.empty(nb, dtype=torch.int32, device=x.device)
    idx = _dev_buf(idx, "idx", torch.int32, (nb,), x.device)
    if want_val and val is None:
        val = torch.empty(nb, dtype=torch.float32, device=x.device)
    if val is not None:
        val = _dev_buf(val, "val", torch.float32, (nb,), x.device)
    if want_logits and logits is None:
        logits = torch.empty((nb, W.n), dtype=torch.float32, device=x.device)
    if logits is not None:
        logits = _dev_buf(logits, "logits", torch.float32, (nb, W.n), x.device)
    return idx, val, logits


def _rows(x, k):
    x = _dev_f32(x, "x")
    if x.dim() == 1:
        x = x.view(1, -1)
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError("x must be [nb, %d]" % k)
    return x, x.shape[0]


def _out(out, shape, like):
    torch = _torch()
    if out is None:
        return torch.empty(shape, dtype=torch.float32, device=like.device)
    return _dev_f32(out, "out", shape)


def q4_group_sums(x, out=None):
    torch = _torch()
    x = _dev_f32(x, "x")
    if x.dim() == 1:
        x = x.view(1, -1)
    nb, k = x.shape
    out = _out(out, (nb, k // 32), x)
    _check(lib().q4_group_sums(x.data_ptr(), nb, k, out.data_ptr(), _stream()), "q4_group_sums")
    return out


def q4_gemv(W: Q4Weight, x, gsum=None, out=None):
    x, nb = _rows(x, W.k)
    out = _out(out, (nb, W.n), x)
    gp = None
    if gsum is not None:
        gp = _dev_f32(gsum, "gsum", (nb, W.k // 32)).data_ptr()
    _check(lib().q4_gemv(W.cref(), x.data_ptr(), gp, nb, out.data_ptr(), _stream()), "q4_gemv")
    return out


def q4_pack_half(x, with_gsum: bool = True):
    """The HalfSet of fp32 activations ``x [nb, k]``: ``(x_even, x_odd,
    gsum)`` -- float16 ``[nb, k/2]`` streams of the even- and odd-indexed
    elements and the fp32 per-32 group sums of the f16 values (or None)."""
    torch = _torch()
    x = _dev_f32(x, "x")
    if x.dim() == 1:
        x = x.view(1, -1)
    nb, k = x.shape
    xe = torch.empty((nb, k // 2), dtype=torch.float16, device=x.device)
    xo = torch.empty((nb, k // 2), dtype=torch.float16, device=x.device)
    gs = torch.empty((nb, k // 32), dtype=torch.float32, device=x.device) if with_gsum else None
    _check(lib().q4_pack_half(x.data_ptr(), nb, k, xe.data_ptr(), xo.data_ptr(),
                              None if gs is None else gs.data_ptr(), _stream()), "q4_pack_half")
    return xe, xo, gs


def q4_gemv_half(W: Q4Weight, x_even, x_odd, gsum=None, out=None):
    """``y = W x`` for a batch given as a HalfSet (see ``q4_pack_half``)."""
    torch = _torch()
    if x_even.dim() == 1:
        x_even, x_odd = x_even.view(1, -1), x_odd.view(1, -1)
    nb = x_even.shape[0]
    dev = x_even.device
    x_even = _dev_buf(x_even, "x_even", torch.float16, (nb, W.k // 2), dev)
    x_odd = _dev_buf(x_odd, "x_odd", torch.float16, (nb, W.k // 2), dev)
    gp = None
    if gsum is not None:
        gp = _dev_buf(gsum, "gsum", torch.float32, (nb, W.k // 32), dev).data_ptr()
    out = _out(out, (nb, W.n), x_even)
    _check(lib().q4_gemv_half(W.cref(), x_even.data_ptr(), x_odd.data_ptr(), gp, nb, out.data_ptr(), _stream()),
           "q4_gemv_half")
    return out


def q4_nrm_gemv(W: Q4Weight, x, gamma, eps: float, out=None):
    x, nb = _rows(x, W.k)
    gamma = _dev_f32(gamma, "gamma", (W.k,))
    out = _out(out, (nb, W.n), x)
    _check(lib().q4_nrm_gemv(W.cref(), x.data_ptr(), gamma.data_ptr(), float(eps), nb, out.data_ptr(),
                             _stream()), "q4_nrm_gemv")
    return out


def q4_dual_gemv(Wa: Q4Weight, Wb: Q4Weight, x, gamma=None, eps: float = 0.0, out_a=None, out_b=None):
    x, nb = _rows(x, Wa.k)
    gp = None if gamma is None else _dev_f32(gamma, "gamma", (Wa.k,)).data_ptr()
    out_a = _out(out_a, (nb, Wa.n), x)
    out_b = _out(out_b, (nb, Wb.n), x)
    _check(lib().q4_dual_gemv(Wa.cref(), Wb.cref(), x.data_ptr(), gp, float(eps), nb, out_a.data_ptr(),
                              out_b.data_ptr(), _stream()), "q4_dual_gemv")
    return out_a, out_b


def q4_gus_nrm(Wg: Q4Weight, Wu: Q4Weight, x, gamma, eps: float, out=None):
    x, nb = _rows(x, Wg.k)
    gamma = _dev_f32(gamma, "gamma", (Wg.k,))
    out = _out(out, (nb, Wg.n), x)
    _check(lib().q4_gus_nrm(Wg.cref(), Wu.cref(), x.data_ptr(), gamma.data_ptr(), float(eps), nb,
                            out.data_ptr(), _stream()), "q4_gus_nrm")
    return out


def q4_res_gemv(W: Q4Weight, x, r, out=None):
    """``out = W x + r``; pass ``out=r`` for the in-place residual stream."""
    x, nb = _rows(x, W.k)
    r = _dev_f32(r, "r", (nb, W.n)) if _torch().is_tensor(r) and r.dim() == 2 else _dev_f32(r, "r").view(nb, W.n)
    out = _out(out, (nb, W.n), x)
    _check(lib().q4_res_gemv(W.cref(), x.data_ptr(), r.data_ptr(), nb, out.data_ptr(), _stream()),
           "q4_res_gemv")
    return out


def q4_argmax_workspace_bytes(n: int, nb: int) -> int:
    return int(lib().q4_argmax_workspace_bytes(n, nb))


def q4_argmax(W: Q4Weight, x, gamma=None, eps: float = 0.0, want_val=False, want_logits=False,
              workspace=None, idx=None, val=None, logits=None):
    """Greedy argmax of the logits ``W xhat`` per activation row.  Returns
    ``(idx int32[nb], val or None, logits or None)``."""
    torch = _torch()
    x, nb = _rows(x, W.k)
    gp = None if gamma is None else _dev_f32(gamma, "gamma", (W.k,)).data_ptr()
    ws_bytes = q4_argmax_workspace_bytes(W.n, nb)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    workspace = _dev_buf(workspace, "workspace", torch.uint8, None, x.device, min_numel=ws_bytes)
    idx, val, logits = _argmax_outs(W, x, nb, want_val, want_logits, idx, val, logits)
    _check(lib().q4_argmax(W.cref(), x.data_ptr(), gp, float(eps), nb, idx.data_ptr(),
                           None if val is None else val.data_ptr(),
                           None if logits is None else logits.data_ptr(),
                           workspace.data_ptr(), workspace.numel(), _stream()), "q4_argmax")
    return idx, val, logits


def q4_argmax_noalloc(W: Q4Weight, x, gamma=None, eps: float = 0.0, want_val=False, want_logits=False,
                      idx=None, val=None, logits=None):
    """Like ``q4_argmax`` but without a workspace: the pass-1 pairs live in a
    fixed array inside the library (for callers that cannot allocate device
    memory; see ``q4_argmax_noalloc`` in the C header for the size limit and
    the sharing rules).  Returns ``(idx, val or None, logits or None)``."""
    x, nb = _rows(x, W.k)
    gp = None if gamma is None else _dev_f32(gamma, "gamma", (W.k,)).data_ptr()
    idx, val, logits = _argmax_outs(W, x, nb, want_val, want_logits, idx, val, logits)
    _check(lib().q4_argmax_noalloc(W.cref(), x.data_ptr(), gp, float(eps), nb, idx.data_ptr(),
                                   None if val is None else val.data_ptr(),
                                   None if logits is None else logits.data_ptr(), _stream()),
           "q4_argmax_noalloc")
    return idx, val, logits


def q4_decode_workspace_bytes(nb: int) -> int:
    return int(lib().q4_decode_workspace_bytes(nb))


class DecodeLayers:
    """Host array of q4_decode_layer descriptors (keeps the tensors alive)."""

    def __init__(self, layers):
        self.layers = list(layers)
        arr = (_CDecodeLayer * len(self.layers))()
        for i, L in enumerate(self.layers):
            arr[i] = _CDecodeLayer(L.Wq._c, L.Wk._c, L.Wv._c, L.Wo._c, L.Wg._c, L.Wu._c, L.Wd._c,
                                   _dev_f32(L.gamma_in, "gamma_in").data_ptr(),
                                   _dev_f32(L.gamma_post, "gamma_post").data_ptr(),
                                   _dev_f32(L.attn, "attn").data_ptr())
        self.arr = arr

    def __len__(self):
        return len(self.layers)


def q4_decode_attn_workspace_bytes(heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().q4_decode_attn_workspace_bytes(heads, kv_heads, head_dim))


class StepAttention:
    """The decode attention of ``q4_decode_step_attn``: per-layer caches
    (``[kv_heads][max_seq][head_dim]`` float32 CUDA tensors), optional RoPE
    tables, the attention output buffer ``out`` (``[1, heads*head_dim]``)
    and the geometry.  Keeps the tensors and the host pointer arrays alive."""

    def __init__(self, caches, out, position: int, window: int = 0, rope=None, scale: float | None = None):
        torch = _torch()
        self.caches = [(_dev_f32(kc, "k_cache"), _dev_f32(vc, "v_cache")) for kc, vc in caches]
        if not self.caches:
            raise ValueError("no caches")
        kv_heads, max_seq, head_dim = self.caches[0][0].shape
        for kc, vc in self.caches:
            if tuple(kc.shape) != (kv_heads, max_seq, head_dim) or tuple(vc.shape) != (kv_heads, max_seq, head_dim):
                raise ValueError("every cache must be [kv_heads, max_seq, head_dim] like the first")
        self.out = _dev_f32(out, "out")
        heads = self.out.numel() // head_dim
        if heads * head_dim != self.out.numel():
            raise ValueError("out must hold heads * head_dim values")
        self.rope = None
        if rope is not None:
            c, sn = (_dev_f32(t, "rope table") for t in rope)
            if tuple(c.shape) != (max_seq, head_dim // 2) or tuple(sn.shape) != (max_seq, head_dim // 2):
                raise ValueError("rope tables must be [max_seq, head_dim/2]")
            self.rope = (c, sn)
        self._k = (ctypes.c_void_p * len(self.caches))(*[kc.data_ptr() for kc, _ in self.caches])
        self._v = (ctypes.c_void_p * len(self.caches))(*[vc.data_ptr() for _, vc in self.caches])
        self.c = _CStepAttention(ctypes.cast(self._k, ctypes.c_void_p), ctypes.cast(self._v, ctypes.c_void_p),
                                 None if self.rope is None else self.rope[0].data_ptr(),
                                 None if self.rope is None else self.rope[1].data_ptr(), self.out.data_ptr(),
                                 max_seq, int(position), int(window), heads, kv_heads, head_dim,
                                 0.0 if scale is None else float(scale))
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim

    def __len__(self):
        return len(self.caches)


def q4_decode_step_attn(layers: DecodeLayers, att: StepAttention, Wlogits: Q4Weight, gamma_final, eps: float, x_in,
                        hid, q, k, v, h, idx, val, workspace, n_layers: int | None = None):
    """The real decode step (each layer's decode attention between its q/k/v
    and o projections) as a single persistent kernel (``q4_decode_step_attn``
    in the C header); nb = 1.  All buffers are caller-owned CUDA tensors."""
    torch = _torch()
    n = len(layers) if n_layers is None else int(n_layers)
    if n > len(att):
        raise ValueError("fewer caches than layers")
    x_in = _dev_f32(x_in, "x_in")
    if x_in.shape[0] != 1:
        raise ValueError("the attention step takes one activation row")
    idx = _dev_buf(idx, "idx", torch.int32, (1,), x_in.device)
    if val is not None:
        val = _dev_buf(val, "val", torch.float32, (1,), x_in.device)
    workspace = _dev_buf(workspace, "workspace", torch.uint8, None, x_in.device,
                         min_numel=max(1, q4_decode_attn_workspace_bytes(att.heads, att.kv_heads, att.head_dim)))
    L0 = layers.layers[0]
    hidden = L0.Wo.n
    for t, name, width in ((x_in, "x_in", hidden), (hid, "hid", hidden), (q, "q", L0.Wq.n), (k, "k", L0.Wk.n),
                           (v, "v", L0.Wv.n), (h, "h", L0.Wg.n)):
        _dev_buf(t, name, torch.float32, (1, width), x_in.device)
    _check(lib().q4_decode_step_attn(ctypes.cast(layers.arr, ctypes.c_void_p), n, ctypes.byref(att.c),
                                     Wlogits.cref(), _dev_f32(gamma_final, "gamma_final").data_ptr(), float(eps),
                                     x_in.data_ptr(), _dev_f32(hid, "hid").data_ptr(), _dev_f32(q, "q").data_ptr(),
                                     _dev_f32(k, "k").data_ptr(), _dev_f32(v, "v").data_ptr(),
                                     _dev_f32(h, "h").data_ptr(), idx.data_ptr(),
                                     None if val is None else val.data_ptr(), workspace.data_ptr(),
                                     workspace.numel(), _stream()), "q4_decode_step_attn")


def q4_decode_step(layers: DecodeLayers, Wlogits: Q4Weight, gamma_final, eps: float, x_in, hid, q, k, v, h,
                   idx, val, workspace, n_layers: int | None = None):
    """One decode step as a single persistent kernel (see ``q4_decode_step``
    in the C header).  All buffers are caller-owned CUDA tensors."""
    torch = _torch()
    n = len(layers) if n_layers is None else int(n_layers)
    x_in = _dev_f32(x_in, "x_in")
    nb = x_in.shape[0]
    idx = _dev_buf(idx, "idx", torch.int32, (nb,), x_in.device)
    if val is not None:
        val = _dev_buf(val, "val", torch.float32, (nb,), x_in.device)
    workspace = _dev_buf(workspace, "workspace", torch.uint8, None, x_in.device,
                         min_numel=q4_decode_workspace_bytes(nb))
    L0 = layers.layers[0]
    hidden = L0.Wo.n
    for t, name, width in ((x_in, "x_in", hidden), (hid, "hid", hidden), (q, "q", L0.Wq.n), (k, "k", L0.Wk.n),
                           (v, "v", L0.Wv.n), (h, "h", L0.Wg.n)):
        _dev_buf(t, name, torch.float32, (nb, width), x_in.device)
    _check(lib().q4_decode_step(ctypes.cast(layers.arr, ctypes.c_void_p), n, Wlogits.cref(),
                                _dev_f32(gamma_final, "gamma_final").data_ptr(), float(eps), nb,
                                _dev_f32(x_in, "x_in").data_ptr(), _dev_f32(hid, "hid").data_ptr(),
                                _dev_f32(q, "q").data_ptr(), _dev_f32(k, "k").data_ptr(),
                                _dev_f32(v, "v").data_ptr(), _dev_f32(h, "h").data_ptr(), idx.data_ptr(),
                                None if val is None else val.data_ptr(), workspace.data_ptr(),
                                workspace.numel(), _stream()), "q4_decode_step")


def q4_decode_check(workspace):
    workspace = _dev_buf(workspace, "workspace", _torch().uint8, None, workspace.device, min_numel=16)
    _check(lib().q4_decode_check(workspace.data_ptr(), _stream()), "q4_decode_check")


def q4_debug_wait_limits(barrier_polls: int = 0, barrier_extra: int = 0, copy_wait_cycles: int = 0,
                         copy_extra_bytes: int = 0):
    """Testing hook: shorten the kernels' wait bounds and make their waits
    expect arrivals or bytes that never come (see ``q4_debug_wait_limits`` in
    the C header).  ``q4_debug_wait_limits()`` restores the defaults."""
    _check(lib().q4_debug_wait_limits(int(barrier_polls), int(barrier_extra), int(copy_wait_cycles),
                                      int(copy_extra_bytes)), "q4_debug_wait_limits")


def q4_device_check():
    """Synchronise the current stream; raise if a GEMV-family kernel gave up
    waiting for its weight copies since the last check (the flag is cleared)."""
    _check(lib().q4_device_check(_stream()), "q4_device_check")


# ---------------------------------------------------------------- attention

def rope_table(max_seq: int, d: int, rope_theta: float = 10000.0):
    """Host RoPE tables (cos, sin), float32 ``[max_seq, d/2]`` (q4_rope_table)."""
    c = np.empty((max_seq, d // 2), np.float32)
    sn = np.empty((max_seq, d // 2), np.float32)
    _check(lib().q4_rope_table(max_seq, d, float(rope_theta), c.ctypes.data, sn.ctypes.data), "q4_rope_table")
    return c, sn


def q4_attn_decode(q, k_new, v_new, k_cache, v_cache, position: int, window: int = 0, scale=None, rope=None,
                   out=None, workspace=None):
    """Decode attention of one token: q ``[H, D]``, k_new / v_new ``[Hkv, D]``,
    caches ``[Hkv, max_seq, D]`` (row ``position`` is written), ``rope`` an
    optional (cos, sin) pair of ``[max_seq, D/2]`` device tables.  Returns
    out ``[H, D]``; ``scale`` defaults to 1/sqrt(D)."""
    torch = _torch()
    q = _dev_f32(q, "q")
    if q.dim() != 2:
        raise ValueError("q must be [H, D]")
    H, D = q.shape
    dev = q.device
    k_cache = _dev_buf(k_cache, "k_cache", torch.float32, None, dev, min_numel=0)
    if k_cache.dim() != 3 or k_cache.shape[2] != D:
        raise ValueError("k_cache must be [Hkv, max_seq, D]")
    Hkv, max_seq = int(k_cache.shape[0]), int(k_cache.shape[1])
    _dev_buf(v_cache, "v_cache", torch.float32, (Hkv, max_seq, D), dev)
    _dev_buf(k_new, "k_new", torch.float32, (Hkv, D), dev)
    _dev_buf(v_new, "v_new", torch.float32, (Hkv, D), dev)
    cp = sp = None
    if rope is not None:
        cos_t, sin_t = rope
        cp = _dev_buf(cos_t, "rope cos", torch.float32, (max_seq, D // 2), dev).data_ptr()
        sp = _dev_buf(sin_t, "rope sin", torch.float32, (max_seq, D // 2), dev).data_ptr()
    if out is None:
        out = torch.empty((H, D), dtype=torch.float32, device=dev)
    else:
        _dev_buf(out, "out", torch.float32, (H, D), dev)
    wsb = int(lib().q4_attn_workspace_bytes(H, D, max_seq))
    if workspace is None:  # zero-filled: its split counters start at zero
        workspace = torch.zeros(max(16, wsb), dtype=torch.uint8, device=dev)
    else:
        _dev_buf(workspace, "workspace", torch.uint8, None, dev, min_numel=wsb)
    if scale is None:
        scale = 1.0 / float(D) ** 0.5
    _check(lib().q4_attn_decode(q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(),
                                v_cache.data_ptr(), max_seq, int(position), H, Hkv, D, int(window), float(scale),
                                cp, sp, out.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream()),
           "q4_attn_decode")
    return out


# ---------------------------------------------------------------- prefill GEMM

def q4_gemm(W: Q4Weight, x, accumulate: bool = False, out=None, workspace=None):
    """y = x W^T for any batch width (meant for nb > 16): x ``[nb, k]``
    float32 CUDA; with ``accumulate`` the product is added to ``out``."""
    torch = _torch()
    x = _dev_f32(x, "x")
    if x.dim() != 2 or x.shape[1] != W.k:
        raise ValueError("x must be [nb, %d]" % W.k)
    nb = int(x.shape[0])
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((nb, W.n), dtype=torch.float32, device=x.device)
    else:
        _dev_buf(out, "out", torch.float32, (nb, W.n), x.device)
    wsb = int(lib().q4_gemm_workspace_bytes(nb, W.k))
    if workspace is None:
        workspace = torch.empty(max(16, wsb), dtype=torch.uint8, device=x.device)
    else:
        _dev_buf(workspace, "workspace", torch.uint8, None, x.device, min_numel=wsb)
    _check(lib().q4_gemm(W.cref(), x.data_ptr(), nb, out.data_ptr(), int(bool(accumulate)), workspace.data_ptr(),
                         workspace.numel(), _stream()), "q4_gemm")
    return out


# ---------------------------------------------------------------- paged KV cache

def _launch(device, fn, *args):
    """Call `fn` with the raw handle of the current stream of the tensors'
    device appended, that device being current (it need not be the caller's)."""
    torch = _torch()
    index, c = device.index, torch._C
    if c._cuda_getDevice() == index:
        return fn(*args, c._cuda_getCurrentRawStream(index))
    with torch.cuda.device(device):
        return fn(*args, c._cuda_getCurrentRawStream(index))


def _ptr(t, name, dtype, shape, device):
    """Address of a contiguous `dtype` tensor of exactly `shape` on `device`;
    anything else raises (_dev_buf says what is wrong)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _dev_buf(t, name, dtype, shape, device).data_ptr()


class KVPages:
    """A paged KV cache that several sequences share: ``k`` and ``v``
    ``[num_pages, kv_heads, page_size, head_dim]`` CUDA tensors of float32,
    float16 or bfloat16, ``table`` ``[nseq, width]`` int32: position p of
    sequence b lies in page ``table[b, p // page_size]``.  The caller owns the
    tensors and may change the table's values between calls; a contiguous cache
    ``[kv_heads, max_seq, head_dim]`` is ``KVPages(k[None], v[None], table)``
    with ``table = [[0]]``.  Keeps the tensors alive."""

    def __init__(self, k, v, table):
        torch = _torch()
        kinds = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
        if not isinstance(k, torch.Tensor) or not k.is_cuda or k.dtype not in kinds:
            raise TypeError("k pages must be a CUDA float32, float16 or bfloat16 tensor")
        if k.dim() != 4 or 0 in k.shape:
            raise ValueError("k pages must be [num_pages, kv_heads, page_size, head_dim]")
        self.k = _dev_buf(k, "k pages", k.dtype, k.shape, k.device)
        self.v = _dev_buf(v, "v pages", k.dtype, k.shape, k.device)
        if not isinstance(table, torch.Tensor) or table.dim() != 2 or 0 in table.shape:
            raise ValueError("table must be an int32 tensor [nseq, width]")
        self.table = _dev_buf(table, "table", torch.int32, table.shape, k.device)
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = (int(x) for x in k.shape)
        self.nseq, self.width = int(table.shape[0]), int(table.shape[1])
        self.dtype, self.device = k.dtype, k.device
        self._c = _CKvPages(self.k.data_ptr(), self.v.data_ptr(), self.table.data_ptr(), kinds[k.dtype],
                            self.num_pages, self.page_size, self.kv_heads, self.head_dim, self.nseq, self.width)
        self._ref = ctypes.byref(self._c)
        self.itemsize = self.k.element_size()
        self.nbytes = self.k.numel() * self.itemsize  # of the k pages, and of the v pages
        self._paged_ws = {}

    def cref(self):
        return self._ref


    def workspace_bytes(self, call: str, heads: int, rows: int = 0) -> int:
        """Workspace bytes of ``q4_attn_paged`` ("paged") or of
        ``q4_attn_prefill`` ("prefill") with ``heads`` query heads."""
        if call == "paged":
            n = self._paged_ws.get(heads)  # by the shapes alone
            if n is None:
                n = self._paged_ws[heads] = int(lib().q4_attn_paged_workspace_bytes(self._ref, heads))
            return n
        if self._c.dtype != 0 and rows >= 0:
            return 0
        return int(lib().q4_attn_prefill_workspace_bytes(self._ref, rows, heads))


def _pages(pages):
    if not isinstance(pages, KVPages):
        raise TypeError("pages must be a KVPages")
    return pages


def _rope_args(rope, head_dim, device):
    if rope is None:
        return None, None, 0
    cos_t, sin_t = rope
    torch = _torch()
    if not isinstance(cos_t, torch.Tensor) or cos_t.dim() != 2 or cos_t.shape[1] != head_dim // 2:
        raise ValueError("rope tables must be [positions, head_dim/2]")
    shape = cos_t.shape
    return (_ptr(cos_t, "rope cos", torch.float32, shape, device),
            _ptr(sin_t, "rope sin", torch.float32, shape, device), shape[0])


def _heads3(t, name, head_dim):
    """(rows, heads) of a [rows, heads, head_dim] tensor."""
    if not isinstance(t, _torch().Tensor) or t.dim() != 3 or t.shape[2] != head_dim:
        raise ValueError("%s must be [rows, heads, %d]" % (name, head_dim))
    return t.shape[0], t.shape[1]


def _room_ptr(t, nbytes, device):
    """Address of a workspace of at least `nbytes` on `device`."""
    try:
        if t.dtype is _torch().uint8 and t.device == device and t.is_contiguous() and t.numel() >= nbytes:
            return t.data_ptr()
    except AttributeError:
        pass
    return _dev_buf(t, "workspace", _torch().uint8, None, device, min_numel=nbytes).data_ptr()


def _apart(out, nbytes, *others):
    """The output at address `out` must not share memory with the inputs
    (address, bytes): it is written while they are read."""
    end = out + nbytes
    for ptr, n in others:
        if ptr < end and out < ptr + n:
            raise ValueError("out must not overlap the inputs")


def q4_kv_append(k, v, pages: KVPages, cu_rows, start=None, q=None, rope=None, q_out=None):
    """Write packed rows ``k``, ``v`` ``[rows, kv_heads, D]`` (float32) into the
    pages of their sequences: rows ``cu_rows[b] .. cu_rows[b+1]`` belong to
    sequence b, at positions ``start[b] ..`` (``start`` None: zeros); ``rope``
    an optional (cos, sin) pair of ``[positions, D/2]`` tables that rotate k.
    With ``q`` ``[rows, H, D]`` (float32) returns it rotated and in the cache's
    type (``q_out``), the form ``q4_attn_prefill`` takes; else returns None."""
    torch = _torch()
    pages = _pages(pages)
    dev, D, i32, f32 = pages.device, pages.head_dim, torch.int32, torch.float32
    rows, _ = _heads3(k, "k", D)
    kp = _ptr(k, "k", f32, (rows, pages.kv_heads, D), dev)
    vp = _ptr(v, "v", f32, (rows, pages.kv_heads, D), dev)
    cu = _ptr(cu_rows, "cu_rows", i32, (pages.nseq + 1,), dev)
    st = None if start is None else _ptr(start, "start", i32, (pages.nseq,), dev)
    cp, sp, rope_rows = _rope_args(rope, D, dev)
    H, qp, op = 0, None, None
    if q is not None:
        n, H = _heads3(q, "q", D)
        if n != rows:
            raise ValueError("q has %d rows, k %d" % (n, rows))
        shape = (rows, H, D)
        qp = _ptr(q, "q", f32, shape, dev)
        if q_out is None:
            q_out = torch.empty(shape, dtype=pages.dtype, device=dev)
        op = _ptr(q_out, "q_out", pages.dtype, shape, dev)
        if rows:
            nb = 4 * rows * D
            _apart(op, rows * H * D * pages.itemsize, (qp, nb * H), (kp, nb * pages.kv_heads),
                   (vp, nb * pages.kv_heads), (pages._c.k, pages.nbytes), (pages._c.v, pages.nbytes))
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _check(_launch(dev, lib().q4_kv_append, pages._ref, qp, kp, vp, rows, cu, st, H, cp, sp, rope_rows, op),
           "q4_kv_append")
    return q_out


def q4_attn_prefill_workspace(pages: KVPages, rows: int, heads: int):
    """A workspace for ``q4_attn_prefill`` with up to ``rows`` rows (None where
    the call needs none: the 16-bit caches)."""
    n = _pages(pages).workspace_bytes("prefill", int(heads), int(rows))
    return _torch().empty(n, dtype=_torch().uint8, device=pages.device) if n else None


def q4_attn_prefill(q, pages: KVPages, cu_rows, start=None, window: int = 0, scale=None, out=None, workspace=None):
    """Causal attention of packed prompt rows over the pages of their
    sequences: ``q`` ``[rows, H, D]`` of the cache's type (``q4_kv_append``
    returns it), row ``cu_rows[b] + i`` at position ``start[b] + i`` of sequence
    b, whose keys and values are in the pages already.  Returns ``out``
    ``[rows, H, D]`` of the same type; ``scale`` defaults to 1/sqrt(D)."""
    torch = _torch()
    pages = _pages(pages)
    dev, D, i32 = pages.device, pages.head_dim, torch.int32
    rows, H = _heads3(q, "q", D)
    shape = (rows, H, D)
    qp = _ptr(q, "q", pages.dtype, shape, dev)
    cu = _ptr(cu_rows, "cu_rows", i32, (pages.nseq + 1,), dev)
    st = None if start is None else _ptr(start, "start", i32, (pages.nseq,), dev)
    if out is None:
        out = torch.empty(shape, dtype=pages.dtype, device=dev)
    op = _ptr(out, "out", pages.dtype, shape, dev)
    if rows:
        nb = rows * H * D * pages.itemsize
        _apart(op, nb, (qp, nb), (pages._c.k, pages.nbytes), (pages._c.v, pages.nbytes))
    wp, wn = None, 0
    if workspace is None:
        workspace = q4_attn_prefill_workspace(pages, rows, H)
    else:
        _dev_buf(workspace, "workspace", torch.uint8, None, dev, min_numel=pages.workspace_bytes("prefill", H, rows))
    if workspace is not None:
        wp, wn = workspace.data_ptr(), workspace.numel()
    _check(_launch(dev, lib().q4_attn_prefill, pages._ref, qp, rows, cu, st, H, int(window),
                   1.0 / float(D) ** 0.5 if scale is None else float(scale), op, wp, wn), "q4_attn_prefill")
    return out


def q4_attn_paged_workspace(pages: KVPages, heads: int):
    """A (zero-filled) workspace for ``q4_attn_paged``; calls that may run at
    the same time, captured ones too, need one each."""
    n = _pages(pages).workspace_bytes("paged", int(heads))
    return _torch().zeros(max(16, n), dtype=_torch().uint8, device=pages.device)


def q4_attn_paged(q, k_new, v_new, pages: KVPages, positions, window: int = 0, scale=None, rope=None, out=None,
                  workspace=None):
    """Attention of one new token per sequence over its pages: ``q``
    ``[nseq, H, D]``, ``k_new`` / ``v_new`` ``[nseq, kv_heads, D]`` (float32)
    at ``positions`` (int32 ``[nseq]``; negative: an idle row, whose out is
    zero).  RoPE of q and k_new (with ``rope`` tables), append, attention.
    Returns out ``[nseq, H, D]`` float32; ``scale`` defaults to 1/sqrt(D)."""
    torch = _torch()
    pages = _pages(pages)
    dev, D, n, f32 = pages.device, pages.head_dim, pages.nseq, torch.float32
    got, H = _heads3(q, "q", D)
    if got != n:
        raise ValueError("q has %d rows, the table %d sequences" % (got, n))
    shape, kv_shape = (n, H, D), (n, pages.kv_heads, D)
    qp = _ptr(q, "q", f32, shape, dev)
    kp = _ptr(k_new, "k_new", f32, kv_shape, dev)
    vp = _ptr(v_new, "v_new", f32, kv_shape, dev)
    pos = _ptr(positions, "positions", torch.int32, (n,), dev)
    cp, sp, rope_rows = _rope_args(rope, D, dev)
    if out is None:
        out = torch.empty(shape, dtype=f32, device=dev)
    op = _ptr(out, "out", f32, shape, dev)
    nb = 4 * n * D
    _apart(op, nb * H, (qp, nb * H), (kp, nb * pages.kv_heads), (vp, nb * pages.kv_heads),
           (pages._c.k, pages.nbytes), (pages._c.v, pages.nbytes))
    if workspace is None:  # zero-filled: its counters start at zero
        workspace = q4_attn_paged_workspace(pages, H)
    else:
        _dev_buf(workspace, "workspace", torch.uint8, None, dev, min_numel=pages.workspace_bytes("paged", H))
    _check(_launch(dev, lib().q4_attn_paged, pages._ref, qp, kp, vp, pos, H, int(window),
                   1.0 / float(D) ** 0.5 if scale is None else float(scale), cp, sp, rope_rows, op,
                   workspace.data_ptr(), workspace.numel()), "q4_attn_paged")
    return out


# ---------------------------------------------------------------- sampling

def q4_logprobs(logits, tokens=None, top: int = 0, entropy: bool = True):
    """Log probabilities from logit rows ``[rows, n]`` (float32, as
    ``q4_argmax(..., want_logits=True)`` returns them).  Returns ``(logprob of
    tokens int32[rows] or None, entropy [rows] or None, top log probabilities
    [rows, min(top, n)], their indices int32)``; ties go to the lowest index,
    a negative token's log probability is 0 (a row that is not scored)."""
    torch = _torch()
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda:
        raise TypeError("logits must be a CUDA float32 tensor")
    if logits.dim() != 2 or logits.shape[1] == 0:
        raise ValueError("logits must be [rows, n]")
    dev, (rows, n) = logits.device, logits.shape
    x = _ptr(logits, "logits", torch.float32, (rows, n), dev)
    k = min(int(top), n)
    f32, i32 = torch.float32, torch.int32
    lp = tok = ent = lpp = entp = None
    if tokens is not None:
        tok = _ptr(tokens, "tokens", i32, (rows,), dev)
        lp = torch.empty(rows, dtype=f32, device=dev)
        lpp = lp.data_ptr()
    if entropy:
        ent = torch.empty(rows, dtype=f32, device=dev)
        entp = ent.data_ptr()
    val = torch.empty((rows, max(0, k)), dtype=f32, device=dev)
    idx = torch.empty((rows, max(0, k)), dtype=i32, device=dev)
    _check(_launch(dev, lib().q4_logprobs, x, rows, n, tok, k, lpp, entp,
                   val.data_ptr() if k > 0 else None, idx.data_ptr() if k > 0 else None), "q4_logprobs")
    return lp, ent, val, idx


# ---------------------------------------------------------------- microscaled 4-bit

_kinds = {}
_MX_BLOCK = (32, 16)  # columns that share a scale, by format


def _kind(dtype, name):
    if not _kinds:
        torch = _torch()
        _kinds.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
    kind = _kinds.get(dtype)
    if kind is None:
        raise TypeError("%s must be float32, float16 or bfloat16" % name)
    return kind


def _mx_bytes(fmt, rows, k):
    """q4_mx_bytes of a shape that the library takes (else raises)."""
    if fmt not in (0, 1) or not 1 <= rows <= 1 << 24 or not 32 <= k <= 65536 or k % 32:
        raise ValueError("bad format or shape: fmt=%s rows=%s k=%s (k: a multiple of 32, 65536 at most)" % (fmt, rows, k))
    return (rows + 127) // 128 * ((k + 255) // 256) * (17408 + 1024 * fmt)


def _mx_factor(fmt, scale):
    """NVFP4's factor of a whole matrix (2^-60 .. 2^60), or MXFP4's 1; else raises."""
    if not (2.0 ** -60 <= scale <= 2.0 ** 60 if fmt == Q4_MX_NVFP4 else scale == 1.0):
        raise ValueError("scale=%s: NVFP4 takes 2^-60 .. 2^60, MXFP4 1" % scale)
    return scale


class MXMatrix:
    """Matrices of microscaled 4-bit values, ``batch`` of them of ``[rows, k]``, in device memory (owns its
    tensor): E2M1 codes whose blocks of 32 columns share a power of two (``Q4_MX_MXFP4``) or whose blocks of 16
    share an E4M3 factor, with one fp32 factor ``scale`` for all (``Q4_MX_NVFP4``).  ``q4_mx_quant`` and
    ``from_codes`` make one with its contents, which comes back in as many dimensions as it was made from; the
    constructor alone leaves them undefined."""

    def __init__(self, fmt: int, rows: int, k: int, batch: int = 1, scale: float = 1.0, device="cuda", tensor=None):
        torch = _torch()
        if batch < 1:
            raise ValueError("a batch of %s matrices" % batch)
        self.nbytes = n = _mx_bytes(fmt, rows, k) * batch
        self.fmt, self.rows, self.k, self.batch, self.scale = fmt, rows, k, batch, _mx_factor(fmt, scale)
        if tensor is None:
            tensor = torch.empty(n, dtype=torch.uint8, device=device)
        else:
            _dev_buf(tensor, "tensor", torch.uint8, None, tensor.device, min_numel=n)
        self.tensor, self.device = tensor, tensor.device
        self._lead = (batch,) if batch > 1 else ()  # of its plain shapes; a batch of one: from_codes, q4_mx_quant
        self._c = c = _CMx(fmt, rows, k, batch, tensor.data_ptr(), n, scale)
        self._ref = ctypes.byref(c)

    @property
    def block(self) -> int:
        """Columns that share a scale."""
        return _MX_BLOCK[self.fmt]

    @property
    def weight_bytes(self) -> int:
        """Algorithmic bytes: 17 (MXFP4) or 18 (NVFP4) per 32 values."""
        return self.batch * self.rows * (self.k // 2 + self.k // self.block)

    def cref(self):
        return self._ref

    def _plain_shapes(self):
        return self._lead + (self.rows, self.k // 2), self._lead + (self.rows, self.k // self.block)

    @classmethod
    def from_codes(cls, codes, scales, fmt: int, scale: float = 1.0) -> "MXMatrix":
        """From plain rows on the device: ``codes`` uint8 ``[.., rows, k/2]`` (the even column in the low nibble),
        ``scales`` uint8 ``[.., rows, k/32]`` (MXFP4) or ``[.., rows, k/16]`` (NVFP4); three dimensions: a batch."""
        torch = _torch()
        if not isinstance(codes, torch.Tensor) or not codes.is_cuda or codes.dim() not in (2, 3):
            raise TypeError("codes must be a CUDA uint8 tensor [rows, k/2] or [batch, rows, k/2]")
        batch = codes.shape[0] if codes.dim() == 3 else 1
        m = cls(fmt, codes.shape[-2], 2 * codes.shape[-1], batch, scale, codes.device)
        m._lead = tuple(codes.shape[:-2])
        lead = tuple(codes.shape[:-1])
        cp = _ptr(codes, "codes", torch.uint8, lead + (m.k // 2,), m.device)
        sp = _ptr(scales, "scales", torch.uint8, lead + (m.k // m.block,), m.device)
        _check(_launch(m.device, lib().q4_mx_pack, cp, sp, m._ref), "q4_mx_pack")
        return m

    def codes(self):
        """``(codes, scales)`` in plain rows, as ``from_codes`` takes them."""
        torch = _torch()
        c, s = (torch.empty(shape, dtype=torch.uint8, device=self.device) for shape in self._plain_shapes())
        _check(_launch(self.device, lib().q4_mx_unpack, self._ref, c.data_ptr(), s.data_ptr()), "q4_mx_unpack")
        return c, s


def _mx(m, name):
    if not isinstance(m, MXMatrix):
        raise TypeError("%s must be an MXMatrix" % name)
    return m


def _mx_src(x, gamma, eps, up):
    """The q4_mx_src of ``x [.., k]`` (rows at an even distance, values next to each other)."""
    torch = _torch()
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA float32, float16 or bfloat16 tensor")
    kind = _kinds.get(x.dtype)
    if kind is None:
        kind = _kind(x.dtype, "x")
    shape, stride = x.shape, x.stride()
    if len(shape) == 2:
        rows, k = shape
        ld = stride[0] if rows > 1 else k
    elif len(shape) == 3:
        if not x.is_contiguous():
            raise ValueError("a batch x must be contiguous")
        rows, k = shape[0] * shape[1], shape[2]
        ld = k
    else:
        raise ValueError("x must be [rows, k] or [batch, rows, k]")
    if rows == 0 or k == 0:
        raise ValueError("x must have rows and columns")
    if stride[-1] != 1 or ld < k:
        raise ValueError("the values of a row of x must be next to each other")
    up_p = gamma_p = None
    if up is not None:
        if gamma is not None:
            raise ValueError("gamma (a norm) and up (a SwiGLU) exclude each other")
        if not isinstance(up, torch.Tensor) or up.dtype != x.dtype or up.device != x.device or up.shape != shape:
            raise ValueError("up must be like x")
        if up.stride() != stride and (rows > 1 or up.stride(-1) != 1):
            raise ValueError("up must have the strides of x")
        up_p = up.data_ptr()
    if gamma is not None:
        gamma_p = _ptr(gamma, "gamma", torch.float32, (k,), x.device)
    return _CMxSrc(x.data_ptr(), up_p, gamma_p, ld, kind, rows, k, eps)


def q4_mx_quant(x, fmt: int | None = None, gamma=None, eps: float = 0.0, up=None, scale: float | None = None, out=None):
    """``x`` (float32, float16 or bfloat16, ``[rows, k]`` or ``[batch, rows, k]``) as an ``MXMatrix``: as it is,
    behind an RMSNorm (``gamma [k]`` float32, ``eps``), or behind a SwiGLU (silu(x) * ``up``).  Rows may be a view
    (the halves of one projection's output).  ``fmt``: MXFP4 by default; ``scale``: NVFP4's factor of the whole matrix,
    such as amax / (6 * 448), 1 by default.  ``out``: an MXMatrix of the same shape to write into, whose format and scale
    hold (``fmt`` and ``scale``, where given, must be its own), apart from x, up and gamma."""
    src = _mx_src(x, gamma, eps, up)
    batch = x.shape[0] if x.dim() == 3 else 1
    rows, k = src.rows // batch, src.k
    if out is None:
        out = MXMatrix(Q4_MX_MXFP4 if fmt is None else fmt, rows, k, batch, 1.0 if scale is None else scale, x.device)
        if x.dim() == 3:
            out._lead = (batch,)
    else:
        if (_mx(out, "out").rows, out.k, out.batch, out.device) != (rows, k, batch, x.device):
            raise ValueError("out has another shape or device than x")
        if fmt not in (None, out.fmt) or scale not in (None, out.scale):
            raise ValueError("out has another format or scale: fmt=%s scale=%s" % (out.fmt, out.scale))
        span = ((src.rows - 1) * src.ld + k) * x.element_size()
        apart = [(src.x, span)] + ([(src.up, span)] if up is not None else []) + ([(src.gamma, 4 * k)] if gamma is not None else [])
        _apart(out._c.dev, out.nbytes, *apart)
    _check(_launch(out.device, lib().q4_mx_quant, ctypes.byref(src), out._ref), "q4_mx_quant")
    return out


def q4_mx_dequant(m: MXMatrix, dtype=None, out=None):
    """The values of ``m``, ``[rows, k]`` (a batch: ``[batch, rows, k]``) of ``dtype`` (float32 by default); ``out``: a tensor to
    write into, apart from m's."""
    torch = _torch()
    m = _mx(m, "m")
    if dtype is None:
        dtype = torch.float32 if out is None else out.dtype
    kind = _kind(dtype, "dtype")
    shape = m._lead + (m.rows, m.k)
    if out is not None and m.batch == 1 and isinstance(out, torch.Tensor):  # with or without a batch's dimension
        shape = (1,) * (out.dim() - 2) + (m.rows, m.k)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=m.device)
        op = out.data_ptr()
    else:
        op = _ptr(out, "out", dtype, shape, m.device)
        _apart(op, m.batch * m.rows * m.k * out.element_size(), (m._c.dev, m.nbytes))
    _check(_launch(m.device, lib().q4_mx_dequant, m._ref, kind, op), "q4_mx_dequant")
    return out


def q4_mx_gemm_workspace(W: MXMatrix, nb: int):
    """A workspace for ``q4_mx_gemm`` with up to ``nb`` float rows: the room of the quantised rows.  Calls that may
    run at the same time, captured ones too, need one each."""
    return _torch().empty(_mx_bytes(_mx(W, "W").fmt, int(nb), W.k), dtype=_torch().uint8, device=W.device)


def q4_mx_gemm(W: MXMatrix, x, r=None, gamma=None, eps: float = 0.0, up=None, scale: float = 1.0, dtype=None,
               out=None, workspace=None):
    """``y = x W^T (+ r)`` with both sides in microscaled 4-bit: ``W [n, k]``; ``x`` an ``MXMatrix [nb, k]`` of the
    same format, or a float tensor ``[nb, k]`` that is quantised to it first as ``q4_mx_quant`` does (``gamma``,
    ``eps``, ``up``, ``scale``).  ``y`` and ``r`` are ``[nb, n]`` of ``dtype`` (by default x's, float32 for an
    MXMatrix); ``out`` may be ``r``."""
    torch = _torch()
    dev, n, k = _mx(W, "W").device, W.rows, W.k
    given = isinstance(x, MXMatrix)
    if given:
        if gamma is not None or up is not None:
            raise ValueError("x is quantised already: gamma and up are q4_mx_quant's")
        nb, got = x.rows, x.k
    else:
        src = _mx_src(x, gamma, eps, up)
        nb, got = src.rows, src.k
        if x.dim() != 2:
            raise ValueError("x must be [nb, %d]" % k)
    if x.device != dev:
        raise ValueError("x is on %s, W on %s" % (x.device, dev))
    if got != k:
        raise ValueError("x must be [nb, %d]" % k)
    if dtype is None:
        dtype = out.dtype if out is not None else torch.float32 if given else x.dtype
    kind, shape = _kind(dtype, "dtype"), (nb, n)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)  # apart from everything
        op = out.data_ptr()
        rp = None if r is None else _ptr(r, "r", dtype, shape, dev)
    else:
        op = _ptr(out, "out", dtype, shape, dev)
        rp = None if r is None else _ptr(r, "r", dtype, shape, dev)
        nbytes = nb * n * out.element_size()
        apart = [(W._c.dev, W.nbytes)]
        if rp is not None and rp != op:
            apart.append((rp, nbytes))
        if given:
            apart.append((x._c.dev, x.nbytes))
        else:
            span = ((nb - 1) * src.ld + k) * x.element_size()
            apart += [(src.x, span)] + ([(src.up, span)] if up is not None else [])
        _apart(op, nbytes, *apart)
    if given:
        _check(_launch(dev, lib().q4_mx_gemm, W._ref, x._ref, rp, kind, op), "q4_mx_gemm")
        return out
    room = _mx_bytes(W.fmt, nb, k)
    if workspace is None:
        workspace = torch.empty(room, dtype=torch.uint8, device=dev)
    X = _CMx(W.fmt, nb, k, 1, _room_ptr(workspace, room, dev), room, _mx_factor(W.fmt, scale))
    _check(_launch(dev, lib().q4_mx_linear, W._ref, ctypes.byref(src), ctypes.byref(X), rp, kind, op), "q4_mx_linear")
    return out


# ---------------------------------------------------------------- mixture of experts

class MoELayer:
    """The weights of a mixture-of-experts layer (``q4_moe``): ``router`` float32 ``[experts, hidden]``; ``gate`` and
    ``up`` ``MXMatrix`` batches ``[experts, inter, hidden]`` and ``down`` ``[experts, hidden, inter]``, all MXFP4.  Each
    token takes ``top_k`` experts, weighted by the softmax of their logits (``renormalize``) or by their share of the
    softmax over all.  Keeps a copy of gate and up in turns of 32 rows, and router and down themselves."""

    def __init__(self, router, gate: MXMatrix, up: MXMatrix, down: MXMatrix, top_k: int, renormalize: bool = True):
        torch = _torch()
        gate, up, down = _mx(gate, "gate"), _mx(up, "up"), _mx(down, "down")
        E, inter, hidden = gate.batch, gate.rows, gate.k
        if (up.batch, up.rows, up.k) != (E, inter, hidden) or (down.batch, down.rows, down.k) != (E, hidden, inter):
            raise ValueError("gate and up must be [experts, inter, hidden], down [experts, hidden, inter]")
        if any(m.fmt != Q4_MX_MXFP4 for m in (gate, up, down)):
            raise ValueError("the experts' weights must be MXFP4")
        if any(m.device != gate.device for m in (up, down)):
            raise ValueError("the experts' weights are on different devices")
        if not 1 <= int(top_k) <= min(16, E) or E > 1024:
            raise ValueError("top_k must be 1 .. min(16, experts), experts at most 1024")
        self.router = _dev_buf(router, "router", torch.float32, (E, hidden), gate.device)
        self.experts, self.hidden, self.inter, self.top_k = E, hidden, inter, int(top_k)
        self.renormalize, self.down, self.device = bool(renormalize), down, gate.device
        self.gate_up = MXMatrix(Q4_MX_MXFP4, 2 * inter, hidden, E, 1.0, gate.device)
        _check(_launch(self.device, lib().q4_moe_pack, gate._ref, up._ref, self.gate_up._ref), "q4_moe_pack")
        self._c = _CMoELayer(self.gate_up._c, down._c, self.router.data_ptr(), E, hidden, inter, self.top_k,
                             int(self.renormalize))
        self._ref = ctypes.byref(self._c)
        self._ws = {}

    def cref(self):
        return self._ref

    def workspace_bytes(self, rows: int) -> int:
        """Workspace bytes of ``q4_moe`` with ``rows`` tokens, 1 to 16."""
        n = self._ws.get(rows)  # by the shapes alone
        if n is None:
            if not 1 <= rows <= MAX_NB:
                raise ValueError("q4_moe takes 1 to %d tokens, not %s" % (MAX_NB, rows))
            n = self._ws[rows] = int(lib().q4_moe_workspace_bytes(self._ref, rows))
        return n


def _moe(layer):
    if not isinstance(layer, MoELayer):
        raise TypeError("layer must be a MoELayer")
    return layer


def q4_moe_workspace(layer: MoELayer, rows: int):
    """A workspace for ``q4_moe`` with up to ``rows`` tokens; calls that may run at the same time, captured ones too,
    need one each."""
    n = _moe(layer).workspace_bytes(int(rows))
    return _torch().empty(n, dtype=_torch().uint8, device=layer.device)


def q4_moe(x, layer: MoELayer, gamma=None, eps: float = 0.0, r=None, positions=None, dtype=None, out=None,
           workspace=None):
    """A mixture-of-experts layer for 1 to 16 tokens ``x [rows, hidden]`` (float32, float16 or bfloat16): RMSNorm
    (with ``gamma``), router, top-k, the chosen experts' SwiGLU MLPs with MXFP4 activations, their weighted sum, plus
    ``r``.  ``positions`` (int32 ``[rows]``): a negative one marks an idle row, which takes no experts.  Returns
    ``(out [rows, hidden] of dtype (x's by default), experts int32 [rows, top_k], weights float32 [rows, top_k])``;
    ``out`` may be ``r`` or ``x``."""
    torch = _torch()
    layer = _moe(layer)
    dev = layer.device
    src = _mx_src(x, gamma, eps, None)
    rows, hidden = src.rows, layer.hidden
    if x.dim() != 2 or src.k != hidden:
        raise ValueError("x must be [rows, %d]" % hidden)
    if x.device != dev:
        raise ValueError("x is on %s, the layer on %s" % (x.device, dev))
    if rows > MAX_NB:
        raise ValueError("q4_moe takes 1 to %d tokens, not %d" % (MAX_NB, rows))
    if dtype is None:
        dtype = out.dtype if out is not None else x.dtype
    kind, shape = _kind(dtype, "dtype"), (rows, hidden)
    rp = None if r is None else _ptr(r, "r", dtype, shape, dev)
    pos = None if positions is None else _ptr(positions, "positions", torch.int32, (rows,), dev)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)  # apart from everything
        op = out.data_ptr()
    else:
        op = _ptr(out, "out", dtype, shape, dev)
        nbytes = rows * hidden * out.element_size()
        apart = [(layer.gate_up._c.dev, layer.gate_up.nbytes), (layer.down._c.dev, layer.down.nbytes),
                 (layer._c.router, 4 * layer.experts * hidden)]
        if rp is not None and rp != op:
            apart.append((rp, nbytes))
        if src.x != op or x.dtype != dtype or src.ld != hidden:
            apart.append((src.x, ((rows - 1) * src.ld + hidden) * x.element_size()))
        _apart(op, nbytes, *apart)
    idx = torch.empty((rows, layer.top_k), dtype=torch.int32, device=dev)
    weight = torch.empty((rows, layer.top_k), dtype=torch.float32, device=dev)
    need = layer.workspace_bytes(rows)
    if workspace is None:
        workspace = q4_moe_workspace(layer, rows)
    wp = _room_ptr(workspace, need, dev)
    _check(_launch(dev, lib().q4_moe, layer._ref, ctypes.byref(src), pos, rp, kind, op, idx.data_ptr(),
                   weight.data_ptr(), wp, workspace.numel()), "q4_moe")
    return out, idx, weight
