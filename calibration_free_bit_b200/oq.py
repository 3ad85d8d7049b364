"""Thin ctypes binding over liboq.so (C ABI in include/oq.h).

Argument marshalling only: every step of the path runs in liboq's sm_100a kernels.  PyTorch
supplies device memory and the stream.  If liboq.so is missing this module raises at import
of the library (there is no CPU fallback): build it with ``python -m
calibration_free_bit_b200.build`` or ``__graft_entry__.build()``.

Names follow the C ABI: oq_build_rpbh, oq_lloyd_max, oq_quantize_weight, oq_quantize_act,
oq_linear, and for attention beside the quantized layers oq_build_rope, oq_apply_rope,
oq_kv_write, oq_kv_read, oq_kv_attend (plus oq_check and the introspection calls used by the
tests).
"""
from __future__ import annotations

import ctypes as C
import os
import re
from typing import Optional

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liboq.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "oq.h")

OQ_OK, OQ_EINVAL, OQ_EUNSUPPORTED, OQ_ECUDA, OQ_EDEVICE, OQ_ENOMEM = 0, -1, -2, -3, -4, -5
OQ_F32, OQ_BF16, OQ_F16 = 0, 1, 2

_lib = None


class OQError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"liboq error {code}: {msg}")
        self.code = code


def lib():
    """Load liboq.so once and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise OQError(OQ_EUNSUPPORTED, f"{LIB_PATH} is missing: the CUDA extension has not been "
                      "built (run `python -m calibration_free_bit_b200.build`)")
    L = C.CDLL(LIB_PATH)
    vp, i32, u64 = C.c_void_p, C.c_int, C.c_uint64
    L.oq_build_rpbh.argtypes = [i32, i32, u64, C.POINTER(vp)]
    L.oq_build_block_rht.argtypes = [i32, i32, u64, C.POINTER(vp)]
    L.oq_rpbh_tables.argtypes = [vp, vp, vp]
    L.oq_lloyd_max.argtypes = [i32, i32, C.POINTER(vp)]
    L.oq_lloyd_max_marginal.argtypes = [i32, i32, i32, C.POINTER(vp)]
    L.oq_codebook_values.argtypes = [vp, vp, vp]
    L.oq_codebook_grid.argtypes = [vp, C.POINTER(i32), C.POINTER(C.c_double), vp]
    L.oq_quantize_weight.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp]
    L.oq_quantize_act.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp]
    L.oq_quantize_act_gelu.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp]
    L.oq_linear.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, i32, vp]
    L.oq_quantized_linear.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, vp, i32, vp,
                                      i32, vp]
    L.oq_linear_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, i32, vp]
    L.oq_check.argtypes = [vp]
    L.oq_free_rpbh.argtypes = [vp]
    L.oq_free_rpbh.restype = None
    L.oq_free_codebook.argtypes = [vp]
    L.oq_free_codebook.restype = None
    L.oq_debug_arm_wait_timeout.argtypes = [i32, C.c_longlong]
    L.oq_timing_enable.argtypes = [i32]
    L.oq_timing_collect.argtypes = [vp, i32, C.POINTER(i32)]
    L.oq_last_error.restype = C.c_char_p
    L.oq_version.restype = C.c_char_p
    i64, f64 = C.c_longlong, C.c_double
    L.oq_build_rope.argtypes = [i32, i32, f64, i32, f64, i32, C.POINTER(vp)]
    L.oq_rope_values.argtypes = [vp, vp, C.POINTER(f64)]
    L.oq_free_rope.argtypes = [vp]
    L.oq_free_rope.restype = None
    L.oq_apply_rope.argtypes = [vp, vp, i64, vp, i64, i32, vp, i64, vp, i64, i32, i32, i32, i32,
                                vp, i32, vp]
    L.oq_kv_write.argtypes = [vp, vp, vp, vp, i64, vp, i64, i32, i32, vp, vp]
    L.oq_kv_read.argtypes = [vp, vp, vp, vp, i32, vp, i64, vp, i64, i32, vp]
    L.oq_kv_attend.argtypes = [vp, vp, vp, vp, i64, vp, i64, i32, i32, i32, vp, vp, i32, i32, vp,
                               i32, vp, f64, vp]
    for name in ("oq_build_rope", "oq_rope_values", "oq_apply_rope", "oq_kv_write", "oq_kv_read",
                 "oq_kv_attend", "oq_build_rpbh", "oq_build_block_rht", "oq_rpbh_tables", "oq_lloyd_max", "oq_lloyd_max_marginal",
                 "oq_codebook_values",
                 "oq_codebook_grid", "oq_quantize_weight", "oq_quantize_act",
                 "oq_quantize_act_gelu", "oq_linear", "oq_quantized_linear",
                 "oq_linear_noalloc", "oq_check", "oq_timing_enable", "oq_timing_collect",
                 "oq_debug_arm_wait_timeout"):
        getattr(L, name).restype = i32
    _lib = L
    return L


def header_functions() -> list[str]:
    """Names of the functions include/oq.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(oq_[a-z0-9_]+)\s*\(", text)))


def _check(rc: int):
    if rc != OQ_OK:
        raise OQError(rc, lib().oq_last_error().decode())


def _stream(stream) -> Optional[int]:
    if stream is None:
        if torch.cuda.is_initialized():      # the current stream's handle, without its wrapper
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        if torch.cuda.is_available():
            return torch.cuda.current_stream().cuda_stream
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return OQ_F32
    if t.dtype == torch.bfloat16:
        return OQ_BF16
    raise OQError(OQ_EINVAL, f"unsupported dtype {t.dtype} (fp32 or bf16)")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise OQError(OQ_EINVAL, "tensors must be contiguous")
    return t.data_ptr()


class RPBH:
    """Handle of an RPBH rotation (oq_build_rpbh), or of its Block-RHT ablation without the
    leading permutation (oq_build_block_rht, permute=False)."""

    def __init__(self, d: int, h: int, seed: int = 0, permute: bool = True):
        self._h = C.c_void_p()
        build = lib().oq_build_rpbh if permute else lib().oq_build_block_rht
        _check(build(d, h, seed, C.byref(self._h)))
        self.d, self.h, self.seed, self.permute = d, h, seed, permute

    @property
    def handle(self):
        return self._h

    def tables(self):
        perm = np.empty(self.d, dtype=np.int32)
        sign = np.empty(self.d, dtype=np.int8)
        _check(lib().oq_rpbh_tables(self._h, perm.ctypes.data, sign.ctypes.data))
        return perm, sign

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value and _lib is not None:
            _lib.oq_free_rpbh(self._h)
            self._h = C.c_void_p()


MARGINALS = {"gauss": 0, "exact": 1}      # OQ_MARGINAL_GAUSSIAN, OQ_MARGINAL_EXACT


class Codebook:
    """Handle of a Lloyd-Max codebook (oq_lloyd_max_marginal): for N(0, 1/d) ("gauss") or for
    the exact coordinate marginal f_d ("exact")."""

    def __init__(self, d: int, bits: int, marginal: str = "gauss"):
        self._h = C.c_void_p()
        _check(lib().oq_lloyd_max_marginal(d, bits, MARGINALS[marginal], C.byref(self._h)))
        self.d, self.bits, self.marginal = d, bits, marginal

    @property
    def handle(self):
        return self._h

    def values(self):
        L = 1 << self.bits
        c = np.empty(L, dtype=np.float64)
        t = np.empty(L - 1, dtype=np.float64)
        _check(lib().oq_codebook_values(self._h, c.ctypes.data, t.ctypes.data))
        return c, t

    def grid(self):
        G = C.c_int(0)
        delta = C.c_double(0)
        _check(lib().oq_codebook_grid(self._h, C.byref(G), C.byref(delta), None))
        table = np.empty(G.value + 1, dtype=np.uint32)
        _check(lib().oq_codebook_grid(self._h, C.byref(G), C.byref(delta), table.ctypes.data))
        return G.value, delta.value, table

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value and _lib is not None:
            _lib.oq_free_codebook(self._h)
            self._h = C.c_void_p()


def oq_build_rpbh(d: int, h: int, seed: int = 0) -> RPBH:
    return RPBH(d, h, seed)


def oq_build_block_rht(d: int, h: int, seed: int = 0) -> RPBH:
    return RPBH(d, h, seed, permute=False)


def oq_lloyd_max(d: int, bits: int, marginal: str = "gauss") -> Codebook:
    return Codebook(d, bits, marginal)


def _rows_out(x: torch.Tensor, bits: int, codes, norms):
    rows, d = x.shape
    if codes is None:
        codes = torch.empty((rows, d * bits // 8), dtype=torch.uint8, device=x.device)
    if norms is None:
        norms = torch.empty(rows, dtype=torch.float32, device=x.device)
    return codes, norms


def oq_quantize_weight(r: RPBH, cw: Codebook, W: torch.Tensor, W_codes=None, row_norms=None,
                       stream=None):
    """Offline weight step: returns (W_codes uint8 [out, d*bw/8], row_norms fp32 [out])."""
    W_codes, row_norms = _rows_out(W, cw.bits, W_codes, row_norms)
    _check(lib().oq_quantize_weight(r.handle, cw.handle, _ptr(W), _dtype_code(W), W.shape[0],
                                    W.shape[1], _ptr(W_codes), _ptr(row_norms), _stream(stream)))
    return W_codes, row_norms


def oq_quantize_act(r: RPBH, ca: Codebook, x: torch.Tensor, x_codes=None, s=None, stream=None,
                    gelu: bool = False):
    """Online activation step: returns (x_codes uint8 [T, d*ba/8], s fp32 [T]); with
    gelu=True the codes and norms are those of GELU(x) (oq_quantize_act_gelu, bf16 x)."""
    x_codes, s = _rows_out(x, ca.bits, x_codes, s)
    fn = lib().oq_quantize_act_gelu if gelu else lib().oq_quantize_act
    _check(fn(r.handle, ca.handle, _ptr(x), _dtype_code(x), x.shape[0], x.shape[1],
              _ptr(x_codes), _ptr(s), _stream(stream)))
    return x_codes, s


def _out(y, T, N, out_dtype, device):
    if y is None:
        return torch.empty((T, N), dtype=out_dtype, device=device)
    if y.dtype not in (torch.float32, torch.bfloat16) or tuple(y.shape) != (T, N):
        raise ValueError(f"y must be fp32 or bf16 of shape {(T, N)}")
    return y


def oq_linear(ca: Codebook, cw: Codebook, x_codes: torch.Tensor, s: torch.Tensor,
              W_codes: torch.Tensor, row_norms: torch.Tensor, y=None, stream=None,
              out_dtype=torch.float32):
    """Codebook linear layer: y [T, out] = s_t rn_o sum_k ca[xc] cw[wc], fp32 or bf16 (the
    dtype of y when given, else out_dtype)."""
    T, N, d = x_codes.shape[0], W_codes.shape[0], ca.d
    y = _out(y, T, N, out_dtype, x_codes.device)
    _check(lib().oq_linear(ca.handle, cw.handle, _ptr(x_codes), _ptr(s), _ptr(W_codes),
                           _ptr(row_norms), T, d, N, _ptr(y), _dtype_code(y), _stream(stream)))
    return y


OQ_FORWARD_GELU = 1


def oq_quantized_linear(r: RPBH, ca: Codebook, cw: Codebook, x: torch.Tensor,
                        W_codes: torch.Tensor, row_norms: torch.Tensor, y=None, s=None,
                        stream=None, out_dtype=torch.float32, gelu: bool = False):
    """The online path in one call: y = oq_linear(oq_quantize_act(x)) without x_codes in
    memory (with gelu=True: of GELU(x)).  Returns y; the norms go to s when given."""
    T, d, N = x.shape[0], x.shape[1], W_codes.shape[0]
    y = _out(y, T, N, out_dtype, x.device)
    _check(lib().oq_quantized_linear(r.handle, ca.handle, cw.handle, _ptr(x), _dtype_code(x),
                                     _ptr(W_codes), _ptr(row_norms), T, d, N, _ptr(y),
                                     _dtype_code(y), _ptr(s), OQ_FORWARD_GELU if gelu else 0,
                                     _stream(stream)))
    return y


def oq_linear_noalloc(ca: Codebook, cw: Codebook, x_codes: torch.Tensor, s: torch.Tensor,
                      W_codes: torch.Tensor, row_norms: torch.Tensor, y: torch.Tensor,
                      stream=None):
    """oq_linear with the library's fixed workspace: the caller passes y; nothing is
    allocated on the device (see include/oq.h for the size limit and sharing rules)."""
    T, N, d = x_codes.shape[0], W_codes.shape[0], ca.d
    y = _out(y, T, N, None, x_codes.device)
    _check(lib().oq_linear_noalloc(ca.handle, cw.handle, _ptr(x_codes), _ptr(s), _ptr(W_codes),
                                   _ptr(row_norms), T, d, N, _ptr(y), _dtype_code(y),
                                   _stream(stream)))
    return y


# ---- rotary positions and the quantised key/value cache ------------------------------------

OQ_ROPE_HALF, OQ_ROPE_INTERLEAVED = 0, 1
OQ_ROPE_PLAIN, OQ_ROPE_LINEAR, OQ_ROPE_NTK, OQ_ROPE_YARN = 0, 1, 2, 3
ROPE_LAYOUTS = {"half": OQ_ROPE_HALF, "interleaved": OQ_ROPE_INTERLEAVED}
ROPE_SCALINGS = {"plain": OQ_ROPE_PLAIN, "linear": OQ_ROPE_LINEAR, "ntk": OQ_ROPE_NTK,
                 "yarn": OQ_ROPE_YARN}
_ROW_DTYPES = {torch.float32: OQ_F32, torch.bfloat16: OQ_BF16, torch.float16: OQ_F16}


def _bad(msg: str):
    raise OQError(OQ_EINVAL, msg)


def _rows(t: torch.Tensor, what: str, heads=None, d=None, dtype=None):
    """A [tokens, heads, d] tensor whose heads of a token are contiguous; returns its token
    stride in elements."""
    if t.dim() != 3 or t.dtype not in _ROW_DTYPES:
        _bad(f"{what} must be [tokens, heads, d] of fp32, bf16 or fp16")
    if (heads is not None and t.shape[1] != heads) or (d is not None and t.shape[2] != d):
        _bad(f"{what} has shape {tuple(t.shape)}: expected [tokens, {heads}, {d}]")
    if dtype is not None and t.dtype != dtype:
        _bad(f"{what} has dtype {t.dtype}: expected {dtype}")
    n, h, e = t.shape
    sn, sh, se = t.stride()
    if n > 0 and ((e > 1 and se != 1) or (h > 1 and sh != e)):
        _bad(f"{what}: the heads of a token must be contiguous")
    return sn if n > 1 else h * e


def _ints(t: torch.Tensor, what: str, dtype, shape):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        _bad(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}, got {t.dtype} "
             f"{tuple(t.shape)}")
    return t.data_ptr()


def _device(*tensors) -> int:
    """The index of the CUDA device that all of a call's tensors are on."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            _bad(f"tensors on {tensors[0].device} and {t.device}: all must be on one device")
    if dev < 0:
        _bad("tensors on the CPU: a CUDA device is needed")
    return dev


def _run(dev: int, fn, args, stream):
    """fn(*args, stream) with the tensors' device current."""
    if dev == torch._C._cuda_getDevice():
        _check(fn(*args, _stream(stream)))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, _stream(stream)))


def _like(t: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


class Rope:
    """Handle of rotary positions (oq_build_rope)."""

    def __init__(self, rot_dim: int, layout: str = "half", theta: float = 10000.0,
                 scaling: str = "plain", factor: float = 1.0, original_len: int = 1):
        if layout not in ROPE_LAYOUTS or scaling not in ROPE_SCALINGS:
            _bad(f"layout {layout!r} ({', '.join(ROPE_LAYOUTS)}), scaling {scaling!r} "
                 f"({', '.join(ROPE_SCALINGS)})")
        self._h = C.c_void_p()
        _check(lib().oq_build_rope(rot_dim, ROPE_LAYOUTS[layout], theta, ROPE_SCALINGS[scaling],
                                   factor, original_len, C.byref(self._h)))
        self.rot_dim, self.layout, self.scaling = rot_dim, layout, scaling

    @property
    def handle(self):
        return self._h

    def values(self):
        """(freq fp64 [rot_dim/2] in radians a position, amplitude)."""
        freq = np.empty(self.rot_dim // 2, dtype=np.float64)
        amp = C.c_double(0)
        _check(lib().oq_rope_values(self._h, freq.ctypes.data, C.byref(amp)))
        return freq, amp.value

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value and _lib is not None:
            _lib.oq_free_rope(self._h)
            self._h = C.c_void_p()


def oq_build_rope(rot_dim: int, layout: str = "half", theta: float = 10000.0,
                  scaling: str = "plain", factor: float = 1.0, original_len: int = 1) -> Rope:
    return Rope(rot_dim, layout, theta, scaling, factor, original_len)


def oq_apply_rope(rope: Rope, x: torch.Tensor, positions: torch.Tensor, k=None, out=None,
                  k_out=None, inverse: bool = False, stream=None):
    """Rotary positions of x [T, heads, d] and, in the same launch, of k [T, k_heads, d] (fp32,
    bf16 or fp16; token stride free); positions int64 [T].  inverse=True applies the transpose, which
    is also what a gradient goes back through: inputs that require one give outputs that do.  Returns
    out, or (out, k_out); out=x works in place (out and k_out only without gradients)."""
    if torch.is_grad_enabled() and (
            x.requires_grad or (k is not None and k.requires_grad) or
            (out is not None and out.requires_grad) or (k_out is not None and k_out.requires_grad)):
        if out is not None or k_out is not None:
            _bad("oq_apply_rope: out and k_out do not go with tensors that require a gradient")
        return _Turn.apply(rope, x, positions, k, inverse, stream)
    return _turn(rope, x, positions, k, out, k_out, inverse, stream)


class _Turn(torch.autograd.Function):
    """oq_apply_rope with its transpose as the way back (itself differentiable)."""

    @staticmethod
    def forward(ctx, rope, x, positions, k, inverse, stream):
        ctx.rope, ctx.inverse = rope, inverse
        ctx.save_for_backward(positions)
        ctx.set_materialize_grads(False)
        y = _turn(rope, x, positions, k, None, None, inverse, stream)
        if k is not None:
            ctx.mark_non_differentiable(*(t for t, needs in zip(y, (x.requires_grad, k.requires_grad))
                                          if not needs))
        return y

    @staticmethod
    def backward(ctx, gy, gk=None):
        g = [None if t is None else _dense(t) for t in (gy, gk)]
        if g[0] is not None or g[1] is not None:
            back = oq_apply_rope(ctx.rope, g[0] if g[0] is not None else g[1], ctx.saved_tensors[0],
                                 g[1] if g[0] is not None else None, inverse=not ctx.inverse)
            if g[0] is None:
                g[1] = back
            elif g[1] is None:
                g[0] = back
            else:
                g = back
        return None, g[0], None, g[1], None, None


def _dense(t: torch.Tensor) -> torch.Tensor:
    """t as a call takes it: contiguous, at a multiple of 16 bytes."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _turn(rope, x, positions, k, out, k_out, inverse, stream):
    xs = _rows(x, "x")
    T, heads, d = x.shape
    if out is None:
        out, ys = _like(x), heads * d
    else:
        ys = _rows(out, "out", heads, d, x.dtype)
        if out.shape[0] != T:
            _bad(f"out has {out.shape[0]} tokens, x {T}")
    kp, ks, kyp, kys, k_heads = None, 0, None, 0, 0
    if k is not None:
        ks = _rows(k, "k", d=d, dtype=x.dtype)
        kt, k_heads = k.shape[0], k.shape[1]
        if kt != T:
            _bad(f"k has {kt} tokens, x {T}")
        if k_out is None:
            k_out, kys = _like(k), k_heads * d
        else:
            kys = _rows(k_out, "k_out", k_heads, d, x.dtype)
            if k_out.shape[0] != T:
                _bad(f"k_out has {k_out.shape[0]} tokens, x {T}")
        kp, kyp = k.data_ptr(), k_out.data_ptr()
    pos = _ints(positions, "positions", torch.int64, (T,))
    _run(_device(x, positions, out, k, k_out), lib().oq_apply_rope,
         (rope.handle, x.data_ptr(), xs, out.data_ptr(), ys, heads, kp, ks, kyp, kys, k_heads,
          _ROW_DTYPES[x.dtype], T, d, pos, 1 if inverse else 0), stream)
    return out if k is None else (out, k_out)


class _KVCacheStruct(C.Structure):
    _fields_ = [("k_codes", C.c_void_p), ("v_codes", C.c_void_p), ("k_norms", C.c_void_p),
                ("v_norms", C.c_void_p), ("num_pages", C.c_longlong), ("page_size", C.c_int),
                ("kv_heads", C.c_int), ("d", C.c_int), ("bits", C.c_int)]


class KVCache:
    """A paged cache of keys and values as codes (oq_kv_cache): *_codes uint8 [pages, kv_heads,
    page_size, d*bits/8] and *_norms fp32 [pages, kv_heads, page_size], the caller's tensors."""

    def __init__(self, k_codes, v_codes, k_norms, v_norms, bits: int):
        if k_codes.dim() != 4 or bits not in (2, 3, 4, 6, 8):
            _bad("codes must be [pages, kv_heads, page_size, bytes], bits 2, 3, 4, 6 or 8")
        pages, heads, page, nb = k_codes.shape
        if nb * 8 % bits != 0:
            _bad(f"rows of {nb} bytes hold no whole number of {bits}-bit codes")
        for t, what in ((k_codes, "k_codes"), (v_codes, "v_codes")):
            _ints(t, what, torch.uint8, (pages, heads, page, nb))
        for t, what in ((k_norms, "k_norms"), (v_norms, "v_norms")):
            _ints(t, what, torch.float32, (pages, heads, page))
        self.k_codes, self.v_codes, self.k_norms, self.v_norms = k_codes, v_codes, k_norms, v_norms
        self.num_pages, self.kv_heads, self.page_size = pages, heads, page
        self.d, self.bits = nb * 8 // bits, bits
        self._s = _KVCacheStruct(k_codes.data_ptr(), v_codes.data_ptr(), k_norms.data_ptr(),
                                 v_norms.data_ptr(), pages, page, heads, self.d, bits)
        self._at = C.addressof(self._s)
        self._dev = _device(k_codes, v_codes, k_norms, v_norms)

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, page_size: int, d: int, bits: int, device="cuda"):
        """A cache in new (zeroed) device memory."""
        shape = (num_pages, kv_heads, page_size)
        codes = [torch.zeros(*shape, d * bits // 8, dtype=torch.uint8, device=device)
                 for _ in range(2)]
        norms = [torch.zeros(shape, dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*codes, *norms, bits=bits)

    @property
    def handle(self):
        return self._at


def oq_kv_write(r: RPBH, c: Codebook, cache: KVCache, k: torch.Tensor, v: torch.Tensor,
                slots: torch.Tensor, stream=None):
    """Store k, v [T, kv_heads, d] (fp32, bf16 or fp16; token stride free) as codes in the slots
    (int64 [T]; -1: skip; no other slot twice).  No gradient goes through the cache's calls."""
    ks = _rows(k, "k", cache.kv_heads, cache.d)
    vs = _rows(v, "v", cache.kv_heads, cache.d, k.dtype)
    T = k.shape[0]
    if v.shape[0] != T:
        _bad(f"k has {T} tokens, v {v.shape[0]}")
    at = _ints(slots, "slots", torch.int64, (T,))
    _run(_device(cache.k_codes, k, v, slots), lib().oq_kv_write,
         (r.handle, c.handle, cache.handle, k.data_ptr(), ks, v.data_ptr(), vs,
          _ROW_DTYPES[k.dtype], T, at), stream)


def oq_kv_read(r: RPBH, c: Codebook, cache: KVCache, slots: torch.Tensor, k=None, v=None,
               out_dtype=torch.bfloat16, stream=None):
    """The rows that slots (int64 [T]; -1: zeros) stand for: returns (k, v) [T, kv_heads, d]."""
    T = slots.shape[0] if slots.dim() == 1 else -1
    at = _ints(slots, "slots", torch.int64, (T,))
    shape = (T, cache.kv_heads, cache.d)
    ks = vs = cache.kv_heads * cache.d
    if k is None:
        if out_dtype not in _ROW_DTYPES:
            _bad(f"out_dtype {out_dtype}: expected fp32, bf16 or fp16")
        k = slots.new_empty(shape, dtype=out_dtype)
    else:
        ks = _rows(k, "k", cache.kv_heads, cache.d)
    if v is None:
        v = torch.empty_like(k) if ks == vs else slots.new_empty(shape, dtype=k.dtype)
    else:
        vs = _rows(v, "v", cache.kv_heads, cache.d, k.dtype)
    if k.shape[0] != T or v.shape[0] != T:
        _bad(f"k and v must have {T} tokens")
    _run(_device(cache.k_codes, k, v, slots), lib().oq_kv_read,
         (r.handle, c.handle, cache.handle, at, T, k.data_ptr(), ks, v.data_ptr(), vs,
          _ROW_DTYPES[k.dtype]), stream)
    return k, v


def oq_kv_attend(r: RPBH, c: Codebook, cache: KVCache, q: torch.Tensor, q_start: torch.Tensor,
                 prefix: torch.Tensor, page_table: torch.Tensor, max_nodes: int = 1,
                 tree_mask=None, scale=None, out=None, stream=None):
    """Attention of drafted tokens over the cache: q [rows, q_heads, d] (bf16 or fp16), rows
    q_start[b] .. q_start[b+1] - 1 of sequence b behind its prefix[b] cached tokens (q_start int32
    [B+1], prefix int32 [B], page_table int32 [B, width]); tree_mask int64 [rows]: bit j of a
    row's word shows it node j (None: the nodes up to its own).  scale: 1/sqrt(d) unless given.
    Rows of out outside every sequence are left as they were.  Returns out."""
    qs = _rows(q, "q", d=cache.d)
    rows, heads = q.shape[0], q.shape[1]
    if out is None:
        out, os_ = _like(q), heads * cache.d
    else:
        os_ = _rows(out, "out", heads, cache.d, q.dtype)
        if out.shape[0] != rows:
            _bad(f"out has {out.shape[0]} rows, q {rows}")
    B = prefix.shape[0] if prefix.dim() == 1 else -1
    width = page_table.shape[1] if page_table.dim() == 2 else 0
    start_p = _ints(q_start, "q_start", torch.int32, (B + 1,))
    prefix_p = _ints(prefix, "prefix", torch.int32, (B,))
    table_p = _ints(page_table, "page_table", torch.int32, (B, width))
    mask_p = None if tree_mask is None else _ints(tree_mask, "tree_mask", torch.int64, (rows,))
    if scale is None:
        scale = cache.d ** -0.5
    _run(_device(cache.k_codes, q, out, q_start, prefix, page_table, tree_mask),
         lib().oq_kv_attend,
         (r.handle, c.handle, cache.handle, q.data_ptr(), qs, out.data_ptr(), os_,
          _ROW_DTYPES[q.dtype], rows, heads, start_p, prefix_p, B, max_nodes, table_p, width,
          mask_p, scale), stream)
    return out


def oq_check(stream=None):
    _check(lib().oq_check(_stream(stream)))


KERNEL_NAMES = {1: "quantize", 2: "decode", 3: "gemm", 4: "fused", 5: "aux", 6: "rope",
                7: "kv_write", 8: "kv_read", 9: "kv_attend"}
OQ_KERNEL_QUANTIZE, OQ_KERNEL_DECODE, OQ_KERNEL_GEMM, OQ_KERNEL_FUSED = 1, 2, 3, 4
OQ_KERNEL_AUX = 5
OQ_KERNEL_ROPE, OQ_KERNEL_KV_WRITE, OQ_KERNEL_KV_READ, OQ_KERNEL_KV_ATTEND = 6, 7, 8, 9


def oq_debug_arm_wait_timeout(kernel: int, limit_cycles: int):
    """Arm the one-shot test of the bounded waits for this thread's next launch of `kernel`
    (OQ_KERNEL_QUANTIZE or OQ_KERNEL_GEMM; 0 disarms); see include/oq.h."""
    _check(lib().oq_debug_arm_wait_timeout(kernel, limit_cycles))


class _TimingRecord(C.Structure):
    _fields_ = [("kernel", C.c_int), ("ms", C.c_float)]


def oq_timing_enable(on: bool = True):
    """Bracket every kernel this thread launches through liboq with CUDA events."""
    _check(lib().oq_timing_enable(1 if on else 0))


def oq_timing_collect(capacity: int = 1 << 20):
    """Wait for the pending timing events; returns [(kernel name, ms), ...] in launch order."""
    buf = (_TimingRecord * capacity)()
    n = C.c_int(0)
    _check(lib().oq_timing_collect(buf, capacity, C.byref(n)))
    return [(KERNEL_NAMES.get(buf[i].kernel, str(buf[i].kernel)), buf[i].ms)
            for i in range(n.value)]


def version() -> str:
    return lib().oq_version().decode()
