"""MI355X (gfx950) mHC site library: Python binding of libmhc.so.

The two calls mirror the C ABI in ``include/mhc.h``:

* :func:`site_pre`  -> ``mhc_site_pre``  (mixes GEMV, RMS rescale, gates, Sinkhorn, collapse)
* :func:`site_post` -> ``mhc_site_post`` (post mix)

This module only marshals arguments: it checks that the operands are contiguous
float32 CUDA (HIP) tensors of matching shapes, allocates outputs with
``torch.empty`` when none are given, and passes raw device pointers and the
current HIP stream to the library.  Every step of the computation runs in the
library's kernels.  There is no fallback: if ``libmhc.so`` is missing the calls
raise.
"""
from __future__ import annotations

import ctypes
import math
import os

__all__ = ["site_pre", "site_post", "site_pre_zq8", "site_pre_check", "site_post_check",
           "site_pre_zq8_check", "site_post_pre", "site_post_pre_check", "expand", "mean",
           "head", "head_check", "bandwidth_probe", "packed_weight_bytes", "pack_weight",
           "site_pre_scratch_bytes",
           "Workspace",
           "f8_encode", "f8_repack", "f8_decode", "f8_matmul", "f8_encode_check",
           "f8_matmul_check", "site_post_bwd", "site_post_bwd_check", "site_pre_bwd",
           "site_pre_bwd_check", "site_pre_bwd_work_bytes",
           "workspace_bytes", "load_library", "MhcError", "LIB_PATH", "EXPORTED_SYMBOLS",
           "STATUS"]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmhc.so")

EXPORTED_SYMBOLS = ("mhc_site_pre", "mhc_site_post", "mhc_site_pre_exact", "mhc_site_pre_zq8",
                    "mhc_site_pre_check", "mhc_site_post_check", "mhc_site_pre_zq8_check",
                    "mhc_workspace_bytes", "mhc_workspace_struct_bytes", "mhc_workspace_init",
                    "mhc_ws_site_pre", "mhc_ws_site_pre_zq8", "mhc_ws_site_post",
                    "mhc_expand", "mhc_mean", "mhc_head", "mhc_head_check",
                    "mhc_site_post_pre", "mhc_site_post_pre_zq8", "mhc_site_post_pre_check",
                    "mhc_status_string", "mhc_probe_sink_floats", "mhc_bandwidth_probe",
                    "mhc_packed_weight_bytes", "mhc_pack_weight", "mhc_site_pre_packed",
                    "mhc_site_post_pre_packed", "mhc_site_pre_scratch_bytes",
                    "mhc_site_pre_static",
                    "mhc_f8_encode", "mhc_f8_repack", "mhc_f8_decode", "mhc_f8_matmul",
                    "mhc_f8_encode_check", "mhc_f8_matmul_check", "mhc_site_post_bwd",
                    "mhc_site_post_bwd_check", "mhc_site_pre_bwd", "mhc_site_pre_bwd_check",
                    "mhc_site_pre_bwd_work_bytes")

STATUS = {0: "MHC_OK", 1: "MHC_EINVAL", 2: "MHC_EALIGN", 3: "MHC_EUNSUPPORTED",
          4: "MHC_EHIP", 5: "MHC_EOVERLAP", 6: "MHC_ECAPTURE"}

_lib = None


class MhcError(RuntimeError):
    def __init__(self, call: str, status: int, text: str):
        super().__init__(f"{call} failed: {STATUS.get(status, status)} ({text})")
        self.status = status


def load_library() -> ctypes.CDLL:
    """Load libmhc.so from this package directory (built by __graft_entry__.build())."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first "
                           "(there is no non-HIP fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, fl, i = ctypes.c_void_p, ctypes.c_float, ctypes.c_int
    lib.mhc_site_pre.argtypes = [vp, vp, vp, vp, i, i, i, i, fl, vp, vp, vp, vp, vp]
    lib.mhc_site_pre.restype = i
    lib.mhc_site_pre_exact.argtypes = [vp, vp, vp, vp, i, i, i, i, fl, vp, vp, vp, vp, vp]
    lib.mhc_site_pre_exact.restype = i
    lib.mhc_site_post.argtypes = [vp, vp, vp, vp, i, i, i, vp, vp]
    lib.mhc_site_post.restype = i
    lib.mhc_site_pre_check.argtypes = [vp, vp, vp, vp, i, i, i, i, fl, vp, vp, vp, vp]
    lib.mhc_site_pre_check.restype = i
    lib.mhc_site_post_check.argtypes = [vp, vp, vp, vp, i, i, i, vp]
    lib.mhc_site_post_check.restype = i
    lib.mhc_site_pre_zq8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, fl, fl, vp, vp, vp, vp,
                                     vp, vp, vp, vp]
    lib.mhc_site_pre_zq8.restype = i
    lib.mhc_site_pre_zq8_check.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, fl, fl, vp, vp, vp,
                                           vp, vp, vp, vp]
    lib.mhc_site_pre_zq8_check.restype = i
    lib.mhc_status_string.argtypes = [i]
    lib.mhc_status_string.restype = ctypes.c_char_p
    sz, wsp = ctypes.c_size_t, ctypes.POINTER(_WsStruct)
    lib.mhc_workspace_bytes.argtypes = [i, i, i]
    lib.mhc_workspace_bytes.restype = sz
    lib.mhc_workspace_struct_bytes.argtypes = []
    lib.mhc_workspace_struct_bytes.restype = sz
    lib.mhc_workspace_init.argtypes = [wsp, vp, sz, i, i, i]
    lib.mhc_workspace_init.restype = i
    lib.mhc_ws_site_pre.argtypes = [wsp, vp, vp, vp, i, i, fl, vp]
    lib.mhc_ws_site_pre.restype = i
    lib.mhc_ws_site_pre_zq8.argtypes = [wsp, vp, vp, vp, vp, i, i, fl, fl, vp]
    lib.mhc_ws_site_pre_zq8.restype = i
    lib.mhc_ws_site_post.argtypes = [wsp, vp, i, vp]
    lib.mhc_ws_site_post.restype = i
    lib.mhc_site_post_pre.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, fl, vp, vp, vp,
                                      vp, vp, vp]
    lib.mhc_site_post_pre.restype = i
    lib.mhc_site_post_pre_zq8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, fl, fl,
                                          vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.mhc_site_post_pre_zq8.restype = i
    lib.mhc_site_post_pre_check.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, fl, vp, vp,
                                            vp, vp, vp]
    lib.mhc_site_post_pre_check.restype = i
    lib.mhc_expand.argtypes = [vp, i, i, i, vp, vp]
    lib.mhc_expand.restype = i
    lib.mhc_mean.argtypes = [vp, i, i, i, vp, vp]
    lib.mhc_mean.restype = i
    lib.mhc_head.argtypes = [vp, vp, vp, vp, i, i, i, fl, vp, vp, vp]
    lib.mhc_head.restype = i
    lib.mhc_head_check.argtypes = [vp, vp, vp, vp, i, i, i, fl, vp, vp]
    lib.mhc_head_check.restype = i
    lib.mhc_packed_weight_bytes.argtypes = [i, i]
    lib.mhc_packed_weight_bytes.restype = sz
    lib.mhc_pack_weight.argtypes = [vp, i, i, vp, vp]
    lib.mhc_pack_weight.restype = i
    lib.mhc_site_pre_packed.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, fl, vp, vp, vp, vp, vp]
    lib.mhc_site_pre_packed.restype = i
    lib.mhc_site_post_pre_packed.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, fl, vp,
                                             vp, vp, vp, vp, vp]
    lib.mhc_site_post_pre_packed.restype = i
    lib.mhc_site_pre_static.argtypes = [vp, vp, vp, vp, i, i, i, i, fl, vp, vp, vp, vp, vp]
    lib.mhc_site_pre_static.restype = i
    lib.mhc_site_pre_scratch_bytes.argtypes = [i, i, i]
    lib.mhc_site_pre_scratch_bytes.restype = sz
    lib.mhc_probe_sink_floats.argtypes = [sz]
    lib.mhc_probe_sink_floats.restype = sz
    lib.mhc_bandwidth_probe.argtypes = [vp, vp, sz, i, vp]
    lib.mhc_bandwidth_probe.restype = i
    lib.mhc_f8_encode.argtypes = [vp, i, i, i, i, vp, vp, vp, vp, vp]
    lib.mhc_f8_encode.restype = i
    lib.mhc_f8_encode_check.argtypes = [vp, i, i, i, i, vp, vp, vp, vp]
    lib.mhc_f8_encode_check.restype = i
    lib.mhc_f8_repack.argtypes = [vp, vp, i, i, vp, vp, vp]
    lib.mhc_f8_repack.restype = i
    lib.mhc_f8_decode.argtypes = [vp, vp, i, i, vp, vp]
    lib.mhc_f8_decode.restype = i
    lib.mhc_f8_matmul.argtypes = [vp, vp, vp, vp, i, i, i, i, vp, i, vp]
    lib.mhc_f8_matmul.restype = i
    lib.mhc_f8_matmul_check.argtypes = [vp, vp, vp, vp, i, i, i, i, vp, i]
    lib.mhc_f8_matmul_check.restype = i
    lib.mhc_site_post_bwd.argtypes = [vp] * 7 + [i, i, i] + [vp] * 5
    lib.mhc_site_post_bwd.restype = i
    lib.mhc_site_post_bwd_check.argtypes = [vp] * 7 + [i, i, i] + [vp] * 4
    lib.mhc_site_post_bwd_check.restype = i
    lib.mhc_site_pre_bwd.argtypes = [vp] * 5 + [i, i, i, i, fl] + [vp] * 10 + [sz, vp]
    lib.mhc_site_pre_bwd.restype = i
    lib.mhc_site_pre_bwd_check.argtypes = [vp] * 5 + [i, i, i, i, fl] + [vp] * 10 + [sz]
    lib.mhc_site_pre_bwd_check.restype = i
    lib.mhc_site_pre_bwd_work_bytes.argtypes = [i, i, i]
    lib.mhc_site_pre_bwd_work_bytes.restype = sz
    if lib.mhc_workspace_struct_bytes() != ctypes.sizeof(_WsStruct):
        raise RuntimeError("mhc_workspace layout of the library and the binding differ")
    _lib = lib
    return lib


class _WsStruct(ctypes.Structure):
    """Mirror of struct mhc_workspace (include/mhc.h)."""
    _fields_ = [("max_tokens", ctypes.c_int), ("streams", ctypes.c_int),
                ("hidden", ctypes.c_int), ("cur", ctypes.c_int),
                ("state", ctypes.c_void_p * 2), ("pre", ctypes.c_void_p),
                ("post", ctypes.c_void_p), ("comb", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("z", ctypes.c_void_p), ("q", ctypes.c_void_p), ("d", ctypes.c_void_p),
                ("scratch", ctypes.c_void_p), ("scratch_bytes", ctypes.c_size_t)]


def _status_text(lib, rc: int) -> str:
    return lib.mhc_status_string(rc).decode()


def _dev(t, name, shape=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 GPU tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def site_pre(x, fn_w, scale, base, iters: int, eps: float, *, out=None, stream=None,
             exact: bool = False, packed=None, static_scratch: bool = False):
    """Pre half of a site.  x: [T,S,H]; fn_w: [(2+S)*S, S*H]; scale: [3]; base: [(2+S)*S].
    Returns (pre [T,S], post [T,S], comb [T,S,S], y [T,H]); `out` may supply that tuple.
    exact=True calls mhc_site_pre_exact (every row bit-identical to a solo T=1 call);
    packed (from pack_weight) calls mhc_site_pre_packed (same results, no per-call pack);
    static_scratch=True calls mhc_site_pre_static (the library's fixed scratch array,
    no device allocation by the library; pass `out` to allocate nothing at all)."""
    if (exact, packed is not None, static_scratch).count(True) > 1:
        raise ValueError("exact, packed and static_scratch are separate calls")
    import torch
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be [T, S, H]")
    T, S, H = x.shape
    R = (2 + S) * S
    px = _dev(x, "x")
    pw = _dev(fn_w, "fn_w", (R, S * H))
    ps = _dev(scale, "scale", (3,))
    pb = _dev(base, "base", (R,))
    if out is None:
        out = (torch.empty((T, S), device=x.device, dtype=torch.float32),
               torch.empty((T, S), device=x.device, dtype=torch.float32),
               torch.empty((T, S, S), device=x.device, dtype=torch.float32),
               torch.empty((T, H), device=x.device, dtype=torch.float32))
    pre, post, comb, y = out
    ptrs = (_dev(pre, "pre", (T, S)), _dev(post, "post", (T, S)),
            _dev(comb, "comb", (T, S, S)), _dev(y, "y", (T, H)))
    if packed is not None:
        nbytes = int(lib.mhc_packed_weight_bytes(S, H))
        pk = _dev(packed, "packed", (nbytes // 4,)) if nbytes else None
        rc = lib.mhc_site_pre_packed(px, pw, pk, ps, pb, T, S, H, int(iters), float(eps), *ptrs,
                                     _stream_handle(stream))
        if rc != 0:
            raise MhcError("mhc_site_pre_packed", rc, _status_text(lib, rc))
        return out
    if exact:
        fn, name = lib.mhc_site_pre_exact, "mhc_site_pre_exact"
    elif static_scratch:
        fn, name = lib.mhc_site_pre_static, "mhc_site_pre_static"
    else:
        fn, name = lib.mhc_site_pre, "mhc_site_pre"
    rc = fn(px, pw, ps, pb, T, S, H, int(iters), float(eps), *ptrs, _stream_handle(stream))
    if rc != 0:
        raise MhcError(name, rc, _status_text(lib, rc))
    return out


def site_pre_scratch_bytes(T: int, streams: int, hidden: int) -> int:
    """Bytes of library scratch a site_pre call of this shape needs (0: rejected shape)."""
    return int(load_library().mhc_site_pre_scratch_bytes(T, streams, hidden))


def packed_weight_bytes(streams: int, hidden: int) -> int:
    """Bytes of a site weight's packed form (0: the shape has none)."""
    return int(load_library().mhc_packed_weight_bytes(streams, hidden))


def pack_weight(fn_w, streams: int, hidden: int, *, out=None, stream=None):
    """Pack a site weight fn_w [(2+S)*S, S*H] once for site_pre(..., packed=...).
    Returns a float32 GPU tensor of packed_weight_bytes(S, H) / 4 floats."""
    import torch
    lib = load_library()
    S, H = int(streams), int(hidden)
    R = (2 + S) * S
    nbytes = int(lib.mhc_packed_weight_bytes(S, H))
    if nbytes == 0:
        raise MhcError("mhc_pack_weight", 3, _status_text(lib, 3))
    pw = _dev(fn_w, "fn_w", (R, S * H))
    if out is None:
        out = torch.empty(nbytes // 4, device=fn_w.device, dtype=torch.float32)
    rc = lib.mhc_pack_weight(pw, S, H, _dev(out, "packed", (nbytes // 4,)), _stream_handle(stream))
    if rc != 0:
        raise MhcError("mhc_pack_weight", rc, _status_text(lib, rc))
    return out


def site_pre_zq8(x, fn_w, scale, base, nw, iters: int, eps: float, norm_eps: float = 1e-5, *,
                 out=None, stream=None):
    """Pre half of a site plus the branch-input epilogue (RMS norm of y with weight nw,
    then q8 codes).  Returns (pre, post, comb, y, z [T,H] f32, q [T,H] int8, d [T,H/32] f32);
    `out` may supply that tuple."""
    import torch
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be [T, S, H]")
    T, S, H = x.shape
    R = (2 + S) * S
    px = _dev(x, "x")
    pw = _dev(fn_w, "fn_w", (R, S * H))
    ps = _dev(scale, "scale", (3,))
    pb = _dev(base, "base", (R,))
    pn = _dev(nw, "nw", (H,))
    if out is None:
        e = lambda s, dt=torch.float32: torch.empty(s, device=x.device, dtype=dt)  # noqa: E731
        out = (e((T, S)), e((T, S)), e((T, S, S)), e((T, H)), e((T, H)), e((T, H), torch.int8),
               e((T, H // 32)))
    pre, post, comb, y, z, q, d = out
    if q.dtype != torch.int8 or not q.is_cuda or not q.is_contiguous() or tuple(q.shape) != (T, H):
        raise ValueError("q must be a contiguous int8 GPU tensor of shape [T, H]")
    ptrs = (_dev(pre, "pre", (T, S)), _dev(post, "post", (T, S)), _dev(comb, "comb", (T, S, S)),
            _dev(y, "y", (T, H)), _dev(z, "z", (T, H)), q.data_ptr(), _dev(d, "d", (T, H // 32)))
    rc = lib.mhc_site_pre_zq8(px, pw, ps, pb, pn, T, S, H, int(iters), float(eps),
                              float(norm_eps), *ptrs, _stream_handle(stream))
    if rc != 0:
        raise MhcError("mhc_site_pre_zq8", rc, _status_text(lib, rc))
    return out


def site_post(x, f, post, comb, *, out=None, stream=None):
    """Post half of a site: x' [T,S,H] from x [T,S,H], f [T,H], post [T,S], comb [T,S,S]."""
    import torch
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be [T, S, H]")
    T, S, H = x.shape
    px = _dev(x, "x")
    pf = _dev(f, "f", (T, H))
    pp = _dev(post, "post", (T, S))
    pc = _dev(comb, "comb", (T, S, S))
    if out is None:
        out = torch.empty((T, S, H), device=x.device, dtype=torch.float32)
    po = _dev(out, "out", (T, S, H))
    rc = lib.mhc_site_post(px, pf, pp, pc, T, S, H, po, _stream_handle(stream))
    if rc != 0:
        raise MhcError("mhc_site_post", rc, _status_text(lib, rc))
    return out


def site_pre_check(x_ptr, fn_w_ptr, scale_ptr, base_ptr, T, S, H, iters, eps,
                   pre_ptr, post_ptr, comb_ptr, y_ptr) -> int:
    """The library's host-side argument check on raw addresses (no HIP call)."""
    lib = load_library()
    return lib.mhc_site_pre_check(x_ptr, fn_w_ptr, scale_ptr, base_ptr, T, S, H, iters,
                                  float(eps), pre_ptr, post_ptr, comb_ptr, y_ptr)


def site_post_check(x_ptr, f_ptr, post_ptr, comb_ptr, T, S, H, out_ptr) -> int:
    lib = load_library()
    return lib.mhc_site_post_check(x_ptr, f_ptr, post_ptr, comb_ptr, T, S, H, out_ptr)


def site_pre_zq8_check(x_ptr, fn_w_ptr, scale_ptr, base_ptr, nw_ptr, T, S, H, iters, eps,
                       norm_eps, pre_ptr, post_ptr, comb_ptr, y_ptr, z_ptr, q_ptr, d_ptr) -> int:
    lib = load_library()
    return lib.mhc_site_pre_zq8_check(x_ptr, fn_w_ptr, scale_ptr, base_ptr, nw_ptr, T, S, H,
                                      iters, float(eps), float(norm_eps), pre_ptr, post_ptr,
                                      comb_ptr, y_ptr, z_ptr, q_ptr, d_ptr)


def site_post_pre(x, f, post, comb, fn_w, scale, base, iters: int, eps: float, *, nw=None,
                  norm_eps: float = 1e-5, out=None, stream=None, packed=None):
    """The post half of a site (x, f, post, comb) followed by the pre half of the
    next site (fn_w, scale, base) on its output.  Returns (x_out, pre, post, comb, y),
    plus (z, q, d) when the norm weight nw of the next site's epilogue is given;
    `out` may supply that tuple.  packed (from pack_weight, without nw) calls
    mhc_site_post_pre_packed."""
    if packed is not None and nw is not None:
        raise ValueError("the packed call has no epilogue")
    import torch
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be [T, S, H]")
    T, S, H = x.shape
    R = (2 + S) * S
    px = _dev(x, "x")
    pf = _dev(f, "f", (T, H))
    ppi = _dev(post, "post", (T, S))
    pci = _dev(comb, "comb", (T, S, S))
    pw = _dev(fn_w, "fn_w", (R, S * H))
    ps = _dev(scale, "scale", (3,))
    pb = _dev(base, "base", (R,))
    if out is None:
        e = lambda s, dt=torch.float32: torch.empty(s, device=x.device, dtype=dt)  # noqa: E731
        out = (e((T, S, H)), e((T, S)), e((T, S)), e((T, S, S)), e((T, H)))
        if nw is not None:
            out = out + (e((T, H)), e((T, H), torch.int8), e((T, H // 32)))
    ptrs = [_dev(out[0], "x_out", (T, S, H)), _dev(out[1], "pre", (T, S)),
            _dev(out[2], "post", (T, S)), _dev(out[3], "comb", (T, S, S)),
            _dev(out[4], "y", (T, H))]
    st = _stream_handle(stream)
    if packed is not None:
        nbytes = int(lib.mhc_packed_weight_bytes(S, H))
        pk = _dev(packed, "packed", (nbytes // 4,)) if nbytes else None
        rc = lib.mhc_site_post_pre_packed(px, pf, ppi, pci, pw, pk, ps, pb, T, S, H, int(iters),
                                          float(eps), *ptrs, st)
        name = "mhc_site_post_pre_packed"
    elif nw is None:
        rc = lib.mhc_site_post_pre(px, pf, ppi, pci, pw, ps, pb, T, S, H, int(iters),
                                   float(eps), *ptrs, st)
        name = "mhc_site_post_pre"
    else:
        z, q, d = out[5], out[6], out[7]
        if q.dtype != torch.int8 or not q.is_cuda or not q.is_contiguous():
            raise ValueError("q must be a contiguous int8 GPU tensor")
        rc = lib.mhc_site_post_pre_zq8(px, pf, ppi, pci, pw, ps, pb, _dev(nw, "nw", (H,)), T, S,
                                       H, int(iters), float(eps), float(norm_eps), *ptrs,
                                       _dev(z, "z", (T, H)), q.data_ptr(),
                                       _dev(d, "d", (T, H // 32)), st)
        name = "mhc_site_post_pre_zq8"
    if rc != 0:
        raise MhcError(name, rc, _status_text(lib, rc))
    return out


def site_post_pre_check(x_ptr, f_ptr, post_ptr, comb_ptr, fn_w_ptr, scale_ptr, base_ptr, T, S,
                        H, iters, eps, x_out_ptr, pre2_ptr, post2_ptr, comb2_ptr, y2_ptr) -> int:
    """The library's host-side argument check of mhc_site_post_pre on raw addresses."""
    lib = load_library()
    return lib.mhc_site_post_pre_check(x_ptr, f_ptr, post_ptr, comb_ptr, fn_w_ptr, scale_ptr,
                                       base_ptr, T, S, H, iters, float(eps), x_out_ptr, pre2_ptr,
                                       post2_ptr, comb2_ptr, y2_ptr)


def expand(e, streams: int, *, out=None, stream=None):
    """Trunk entry: e [T, H] -> x [T, S, H] (a copy of e in every stream)."""
    import torch
    lib = load_library()
    if e.dim() != 2:
        raise ValueError("e must be [T, H]")
    T, H = e.shape
    pe = _dev(e, "e")
    if out is None:
        out = torch.empty((T, streams, H), device=e.device, dtype=torch.float32)
    po = _dev(out, "out", (T, streams, H))
    rc = lib.mhc_expand(pe, T, streams, H, po, _stream_handle(stream))
    if rc != 0:
        raise MhcError("mhc_expand", rc, _status_text(lib, rc))
    return out


def mean(x, *, out=None, stream=None):
    """Trunk exit (unweighted): x [T, S, H] -> y [T, H], the mean over the streams."""
    import torch
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be [T, S, H]")
    T, S, H = x.shape
    px = _dev(x, "x")
    if out is None:
        out = torch.empty((T, H), device=x.device, dtype=torch.float32)
    po = _dev(out, "out", (T, H))
    rc = lib.mhc_mean(px, T, S, H, po, _stream_handle(stream))
    if rc != 0:
        raise MhcError("mhc_mean", rc, _status_text(lib, rc))
    return out


def head(x, fn_w, scale, base, eps: float, *, out=None, stream=None):
    """Trunk exit (gated head): x [T, S, H], fn_w [S, S*H], scale [1], base [S] ->
    (gates [T, S], y [T, H]); `out` may supply that pair."""
    import torch
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be [T, S, H]")
    T, S, H = x.shape
    px = _dev(x, "x")
    pw = _dev(fn_w, "fn_w", (S, S * H))
    ps = _dev(scale, "scale", (1,))
    pb = _dev(base, "base", (S,))
    if out is None:
        out = (torch.empty((T, S), device=x.device, dtype=torch.float32),
               torch.empty((T, H), device=x.device, dtype=torch.float32))
    g, y = out
    rc = lib.mhc_head(px, pw, ps, pb, T, S, H, float(eps), _dev(g, "gates", (T, S)),
                      _dev(y, "y", (T, H)), _stream_handle(stream))
    if rc != 0:
        raise MhcError("mhc_head", rc, _status_text(lib, rc))
    return out


F8_BLOCK = 128


def _blocks(n: int) -> int:
    return (n + F8_BLOCK - 1) // F8_BLOCK


def _gpu(t, name, dtype, shape=None):
    """Device address of a contiguous GPU tensor of this dtype (and shape, a tuple)."""
    try:
        if t.is_cuda and t.dtype == dtype and t.is_contiguous() and (
                shape is None or t.shape == shape):
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    raise ValueError(f"{name} must be a contiguous {dtype} GPU tensor")


_entry = {}  # name -> function, so that a small call does not look it up twice
_gpus = None


def _on(stream, device, fn, *args, **kw):
    """fn with `stream` (torch's, or a handle) as the current one, so that what the call
    allocates belongs to that stream and is not memory that work on another one still uses."""
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the operands on {device}")
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _call(name, device, args, others):
    """One library call on `device` (an index; the operands' own, made current where it
    is not), on that device's current stream."""
    import torch
    global _gpus
    fn = _entry.get(name)
    if fn is None:
        _gpus = torch.cuda.device_count()  # before the entry, which says that it is there
        fn = _entry[name] = getattr(load_library(), name)
    stream = torch._C._cuda_getCurrentRawStream(device)
    if _gpus > 1:
        for t in others:
            if t is not None and t.get_device() != device:
                raise ValueError(f"operands are on GPUs {device} and {t.get_device()}")
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    else:
        rc = fn(*args, stream)
    if rc != 0:
        raise MhcError(name, rc, _status_text(_lib, rc))


def _outputs(out, names, shapes, dtypes, device):
    """The outputs of a call, new or as given (checked), and their addresses."""
    if out is None:
        import torch
        out = tuple([torch.empty(s, device=device, dtype=d) for s, d in zip(shapes, dtypes)])
        return out, [o.data_ptr() for o in out]
    if len(out) != len(shapes):
        raise ValueError(f"out must hold {len(shapes)} tensors")
    return out, [_gpu(o, n, d, s) for o, n, s, d in zip(out, names, shapes, dtypes)]


def _kept(x, name, rows, H):
    """Addresses (data, scales or None) and tensors of an activation [..., H] that is
    a float32 tensor or the (codes, scales) pair of its 8-bit checkpoint."""
    import torch
    if isinstance(x, (tuple, list)):
        codes, scales = x
        kb = _blocks(H)
        pc = _gpu(codes, f"{name} codes", torch.float8_e4m3fn, (*rows, kb * F8_BLOCK))
        return pc, _gpu(scales, f"{name} scales", torch.uint8, (*rows, kb)), (codes, scales)
    return _gpu(x, name, torch.float32, (*rows, H)), None, (x,)


def f8_encode(x, *, transposed=False, square: bool = False, out=None, stream=None):
    """8-bit blocks of x [..., cols] (float32 or bfloat16; include/mhc.h, "8-bit blocks").
    Returns (codes [..., P] float8_e4m3fn, scales [..., P/128] uint8), P = cols rounded up
    to 128.  transposed=True adds (codes_t [cols, Pt], scales_t), the encoded transpose of
    the matrix x (leading dimensions together its rows), from the same pass;
    transposed="only" returns that pair alone.  square=True (x [rows, cols]) uses one scale
    per 128 x 128 square, for weights: scales [ceil(rows/128), P/128].
    `out` may supply the tuple that the call returns."""
    import torch
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dtype = x.dtype
    bf16 = dtype == torch.bfloat16
    if not bf16 and dtype != torch.float32:
        raise ValueError("x must be float32 or bfloat16")
    *lead, cols = x.shape
    if not lead or (square and len(lead) != 1):
        raise ValueError("x must be [rows, cols]" if square else "x must be [..., rows, cols]")
    if transposed not in (False, True, "only"):
        raise ValueError('transposed must be False, True or "only"')
    px = _gpu(x, "x", dtype)
    if stream is not None:
        return _on(stream, x.device, f8_encode, x, transposed=transposed, square=square, out=out)
    rows = math.prod(lead)
    kb = _blocks(cols)
    f8, u8 = torch.float8_e4m3fn, torch.uint8
    if not transposed:
        shapes = ((*lead, kb * F8_BLOCK), (_blocks(rows), kb) if square else (*lead, kb))
    else:
        rb = _blocks(rows)
        shapes = ((cols, rb * F8_BLOCK), (kb, rb) if square else (cols, rb))
        if transposed != "only":
            shapes = ((*lead, kb * F8_BLOCK), (rb, kb) if square else (*lead, kb)) + shapes
    out, ptrs = _outputs(out, ("out[0]", "out[1]", "out[2]", "out[3]"), shapes,
                         (f8, u8, f8, u8), x.device)
    if not transposed:
        ptrs += [None, None]
    elif transposed == "only":
        ptrs = [None, None] + ptrs
    _call("mhc_f8_encode", x.get_device(),
          (px, int(bf16), rows, cols, int(square), *ptrs), out)
    return out


def f8_repack(codes, scales, cols: int, *, out=None, stream=None):
    """The encoded transpose (codes_t [cols, Pt], scales_t [cols, Pt/128]) of an encoded
    matrix codes [rows, P], scales [rows, P/128] of `cols` columns: a kept activation in the
    form a weight gradient's product needs.  `out` may supply that pair."""
    import torch
    if stream is not None:
        return _on(stream, codes.device, f8_repack, codes, scales, cols, out=out)
    kb = _blocks(cols)
    if codes.dim() != 2:
        raise ValueError("codes must be [rows, P]")
    rows = codes.shape[0]
    rb = _blocks(rows)
    pc = _gpu(codes, "codes", torch.float8_e4m3fn, (rows, kb * F8_BLOCK))
    ps = _gpu(scales, "scales", torch.uint8, (rows, kb))
    out, ptrs = _outputs(out, ("out[0]", "out[1]"), ((cols, rb * F8_BLOCK), (cols, rb)),
                         (torch.float8_e4m3fn, torch.uint8), codes.device)
    _call("mhc_f8_repack", codes.get_device(), (pc, ps, rows, cols, *ptrs), (scales, *out))
    return out


def f8_decode(codes, scales, cols: int, *, out=None, stream=None):
    """The float32 values [..., cols] of 8-bit blocks codes [..., P], scales [..., P/128]."""
    import torch
    if stream is not None:
        return _on(stream, codes.device, f8_decode, codes, scales, cols, out=out)
    kb = _blocks(cols)
    lead = tuple(codes.shape[:-1])
    pc = _gpu(codes, "codes", torch.float8_e4m3fn, (*lead, kb * F8_BLOCK))
    ps = _gpu(scales, "scales", torch.uint8, (*lead, kb))
    if out is None:
        out = torch.empty((*lead, cols), device=codes.device, dtype=torch.float32)
    rows = 1
    for d in lead:
        rows *= d
    _call("mhc_f8_decode", codes.get_device(),
          (pc, ps, rows, cols, _gpu(out, "out", torch.float32, (*lead, cols))), (scales, out))
    return out


def f8_matmul(a, a_scales, b, b_scales, *, dtype=None, out=None, stream=None):
    """a [M, K] times b [N, K] transposed, both 8-bit blocks: [M, N] float32 (default) or
    bfloat16.  K is the padded width of both (a multiple of 128).  b_scales is [N, K/128],
    or [ceil(N/128), K/128] for the square form of a weight.  `out` may supply the result;
    its dtype is then the product's."""
    import torch
    if stream is not None:
        return _on(stream, a.device, f8_matmul, a, a_scales, b, b_scales, dtype=dtype, out=out)
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[1]:
        raise ValueError("a must be [M, K] and b [N, K]")
    (M, K), N = a.shape, b.shape[0]
    kb = K // F8_BLOCK
    dtype = out.dtype if out is not None else dtype if dtype is not None else torch.float32
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("the product is float32 or bfloat16")
    square = b_scales.dim() == 2 and b_scales.shape[0] != N
    pa = _gpu(a, "a", torch.float8_e4m3fn)
    pb = _gpu(b, "b", torch.float8_e4m3fn)
    pas = _gpu(a_scales, "a_scales", torch.uint8, (M, kb))
    pbs = _gpu(b_scales, "b_scales", torch.uint8, (_blocks(N) if square else N, kb))
    if out is None:
        out = torch.empty((M, N), device=a.device, dtype=dtype)
        po = out.data_ptr()
    else:
        po = _gpu(out, "out", dtype, (M, N))
    _call("mhc_f8_matmul", a.get_device(),
          (pa, pas, pb, pbs, int(square), M, N, K, po, int(dtype == torch.bfloat16)),
          (a_scales, b, b_scales, out))
    return out


def f8_encode_check(x_ptr, x_type, rows, cols, square, codes_ptr, scales_ptr, codes_t_ptr,
                    scales_t_ptr) -> int:
    """The library's host-side argument check of mhc_f8_encode on raw addresses."""
    return load_library().mhc_f8_encode_check(x_ptr, x_type, rows, cols, square, codes_ptr,
                                              scales_ptr, codes_t_ptr, scales_t_ptr)


def f8_matmul_check(a_ptr, a_scales_ptr, b_ptr, b_scales_ptr, b_square, M, N, K, out_ptr,
                    out_type) -> int:
    """The library's host-side argument check of mhc_f8_matmul on raw addresses."""
    return load_library().mhc_f8_matmul_check(a_ptr, a_scales_ptr, b_ptr, b_scales_ptr, b_square,
                                              M, N, K, out_ptr, out_type)


def site_post_bwd(g, x, f, post, comb, *, out=None, stream=None):
    """Gradient of site_post: from g [T,S,H] = dL/dx', the forward's x [T,S,H], f [T,H],
    post [T,S] and comb [T,S,S].  x and f are float32 tensors or the (codes, scales) pairs
    that f8_encode(x), f8_encode(f) returned.  Returns (dx [T,S,H], df [T,H], dpost [T,S],
    dcomb [T,S,S]); `out` may supply that tuple."""
    import torch
    if stream is not None:
        return _on(stream, g.device, site_post_bwd, g, x, f, post, comb, out=out)
    if g.dim() != 3:
        raise ValueError("g must be [T, S, H]")
    T, S, H = g.shape
    f32 = torch.float32
    pg = _gpu(g, "g", f32)
    px, pxs, tx = _kept(x, "x", (T, S), H)
    pf, pfs, tf = _kept(f, "f", (T,), H)
    out, po = _outputs(out, ("dx", "df", "dpost", "dcomb"),
                       ((T, S, H), (T, H), (T, S), (T, S, S)), (f32, f32, f32, f32), g.device)
    _call("mhc_site_post_bwd", g.get_device(),
          (pg, px, pxs, pf, pfs, _gpu(post, "post", f32, (T, S)),
           _gpu(comb, "comb", f32, (T, S, S)), T, S, H, *po),
          (*tx, *tf, post, comb, *out))
    return out


def site_post_bwd_check(g_ptr, x_ptr, x_scales_ptr, f_ptr, f_scales_ptr, post_ptr, comb_ptr, T,
                        S, H, dx_ptr, df_ptr, dpost_ptr, dcomb_ptr) -> int:
    """The library's host-side argument check of mhc_site_post_bwd on raw addresses."""
    return load_library().mhc_site_post_bwd_check(g_ptr, x_ptr, x_scales_ptr, f_ptr, f_scales_ptr,
                                                  post_ptr, comb_ptr, T, S, H, dx_ptr, df_ptr,
                                                  dpost_ptr, dcomb_ptr)


def site_pre_bwd_work_bytes(T: int, streams: int, hidden: int) -> int:
    """Bytes of device scratch a site_pre_bwd call of this shape needs."""
    return int(load_library().mhc_site_pre_bwd_work_bytes(T, streams, hidden))


def site_pre_bwd(x, fn_w, scale, base, iters: int, eps: float, dy, dpost, dcomb, *, dpre=None,
                 dx_in=None, out=None, work=None, stream=None):
    """Gradient of site_pre, recomputed from its input x [T,S,H] (a float32 tensor or the
    (codes, scales) pair that f8_encode(x) returned): dy [T,H], dpost [T,S], dcomb [T,S,S]
    are the gradients of its outputs, dpre [T,S] a further one of pre, and dx_in [T,S,H]
    is added to dx (site_post_bwd's dx; it may be out's dx itself).  Returns (dx [T,S,H],
    dfn_w, dscale, dbase); `out` may supply that tuple.  `work` is a uint8 tensor of at
    least site_pre_bwd_work_bytes bytes (allocated per call when not given)."""
    import torch
    if stream is not None:
        return _on(stream, dy.device, site_pre_bwd, x, fn_w, scale, base, iters, eps, dy, dpost,
                   dcomb, dpre=dpre, dx_in=dx_in, out=out, work=work)
    if dy.dim() != 2 or dcomb.dim() != 3:
        raise ValueError("dy must be [T, H] and dcomb [T, S, S]")
    (T, H), S = dy.shape, dcomb.shape[1]
    R = (2 + S) * S
    f32 = torch.float32
    px, pxs, tx = _kept(x, "x", (T, S), H)
    out, po = _outputs(out, ("dx", "dfn_w", "dscale", "dbase"),
                       ((T, S, H), (R, S * H), (3,), (R,)), (f32, f32, f32, f32), dy.device)
    if work is None:
        work = torch.empty(site_pre_bwd_work_bytes(T, S, H), device=dy.device, dtype=torch.uint8)
    _call("mhc_site_pre_bwd", dy.get_device(),
          (px, pxs, _gpu(fn_w, "fn_w", f32, (R, S * H)), _gpu(scale, "scale", f32, (3,)),
           _gpu(base, "base", f32, (R,)), T, S, H, int(iters), float(eps),
           _gpu(dy, "dy", f32), None if dpre is None else _gpu(dpre, "dpre", f32, (T, S)),
           _gpu(dpost, "dpost", f32, (T, S)), _gpu(dcomb, "dcomb", f32, (T, S, S)),
           None if dx_in is None else _gpu(dx_in, "dx_in", f32, (T, S, H)), *po,
           _gpu(work, "work", torch.uint8), work.numel()),
          (*tx, fn_w, scale, base, dpre, dpost, dcomb, dx_in, *out, work))
    return out


def site_pre_bwd_check(x_ptr, x_scales_ptr, fn_w_ptr, scale_ptr, base_ptr, T, S, H, iters, eps,
                       dy_ptr, dpre_ptr, dpost_ptr, dcomb_ptr, dx_in_ptr, dx_ptr, dfn_w_ptr,
                       dscale_ptr, dbase_ptr, work_ptr, work_bytes) -> int:
    """The library's host-side argument check of mhc_site_pre_bwd on raw addresses."""
    return load_library().mhc_site_pre_bwd_check(
        x_ptr, x_scales_ptr, fn_w_ptr, scale_ptr, base_ptr, T, S, H, iters, float(eps), dy_ptr,
        dpre_ptr, dpost_ptr, dcomb_ptr, dx_in_ptr, dx_ptr, dfn_w_ptr, dscale_ptr, dbase_ptr,
        work_ptr, work_bytes)


def bandwidth_probe(src, dst, copy: bool, *, stream=None):
    """Pure-stream probe (mhc_bandwidth_probe): copy src into dst (same size), or
    read src and write block sums into dst (probe_sink_floats(src) floats)."""
    lib = load_library()
    ps = _dev(src, "src")
    want = src.numel() if copy else int(lib.mhc_probe_sink_floats(src.numel() * 4))
    if dst.numel() != want:
        raise ValueError(f"dst must hold {want} floats")
    pd = _dev(dst, "dst")
    rc = lib.mhc_bandwidth_probe(ps, pd, src.numel() * 4, int(bool(copy)), _stream_handle(stream))
    if rc != 0:
        raise MhcError("mhc_bandwidth_probe", rc, _status_text(lib, rc))
    return dst


def head_check(x_ptr, fn_w_ptr, scale_ptr, base_ptr, T, S, H, eps, gates_ptr, y_ptr) -> int:
    """The library's host-side argument check of mhc_head on raw addresses."""
    lib = load_library()
    return lib.mhc_head_check(x_ptr, fn_w_ptr, scale_ptr, base_ptr, T, S, H, float(eps),
                              gates_ptr, y_ptr)


def workspace_bytes(max_tokens: int, streams: int, hidden: int) -> int:
    """Device bytes a workspace of this shape needs (0 for an invalid shape)."""
    return int(load_library().mhc_workspace_bytes(max_tokens, streams, hidden))


class Workspace:
    """A persistent site workspace (mhc_workspace_init and the mhc_ws_* calls).

    The device memory is one torch uint8 buffer owned by this object; the library
    carves it and never allocates on the workspace path.  Tensor views of the
    regions: ``state`` (the current stream state, [max_tokens, S, H], writable),
    ``pre``, ``post``, ``comb``, ``y``, ``z``, ``q``, ``d`` (max_tokens rows; a call
    with T tokens writes the first T)."""

    def __init__(self, max_tokens: int, streams: int, hidden: int, device=None):
        import torch
        lib = load_library()
        nbytes = int(lib.mhc_workspace_bytes(max_tokens, streams, hidden))
        if nbytes == 0:
            raise ValueError(f"invalid workspace shape ({max_tokens}, {streams}, {hidden})")
        self._mem = torch.empty(nbytes + 256, dtype=torch.uint8,
                                device=device if device is not None else "cuda")
        base = self._mem.data_ptr()
        self._base = base
        off = (-base) % 256
        self._ws = _WsStruct()
        rc = lib.mhc_workspace_init(ctypes.byref(self._ws), base + off, nbytes, max_tokens,
                                    streams, hidden)
        if rc != 0:
            raise MhcError("mhc_workspace_init", rc, _status_text(lib, rc))
        self.max_tokens, self.streams, self.hidden = max_tokens, streams, hidden
        T, S, H = max_tokens, streams, hidden
        f32, i8 = torch.float32, torch.int8
        w = self._ws
        self._states = (self._view(w.state[0], (T, S, H), f32),
                        self._view(w.state[1], (T, S, H), f32))
        self.pre = self._view(w.pre, (T, S), f32)
        self.post = self._view(w.post, (T, S), f32)
        self.comb = self._view(w.comb, (T, S, S), f32)
        self.y = self._view(w.y, (T, H), f32)
        self.z = self._view(w.z, (T, H), f32)
        self.q = self._view(w.q, (T, H), i8)
        self.d = self._view(w.d, (T, (H + 31) // 32), f32)

    def _view(self, ptr, shape, dtype):
        import torch
        itemsize = torch.empty((), dtype=dtype).element_size()
        count = 1
        for s in shape:
            count *= s
        o = ptr - self._base
        return self._mem[o:o + count * itemsize].view(dtype).view(shape)

    @property
    def cur(self) -> int:
        return int(self._ws.cur)

    @property
    def state(self):
        """The current stream state [max_tokens, S, H] (state[cur])."""
        return self._states[self._ws.cur]

    def site_pre(self, fn_w, scale, base, iters: int, eps: float, T: int = None, stream=None):
        lib = load_library()
        T = self.max_tokens if T is None else T
        S, H = self.streams, self.hidden
        R = (2 + S) * S
        rc = lib.mhc_ws_site_pre(ctypes.byref(self._ws), _dev(fn_w, "fn_w", (R, S * H)),
                                 _dev(scale, "scale", (3,)), _dev(base, "base", (R,)), T,
                                 int(iters), float(eps), _stream_handle(stream))
        if rc != 0:
            raise MhcError("mhc_ws_site_pre", rc, _status_text(lib, rc))

    def site_pre_zq8(self, fn_w, scale, base, nw, iters: int, eps: float,
                     norm_eps: float = 1e-5, T: int = None, stream=None):
        lib = load_library()
        T = self.max_tokens if T is None else T
        S, H = self.streams, self.hidden
        R = (2 + S) * S
        rc = lib.mhc_ws_site_pre_zq8(ctypes.byref(self._ws), _dev(fn_w, "fn_w", (R, S * H)),
                                     _dev(scale, "scale", (3,)), _dev(base, "base", (R,)),
                                     _dev(nw, "nw", (H,)), T, int(iters), float(eps),
                                     float(norm_eps), _stream_handle(stream))
        if rc != 0:
            raise MhcError("mhc_ws_site_pre_zq8", rc, _status_text(lib, rc))

    def site_post(self, f, T: int = None, stream=None):
        lib = load_library()
        T = self.max_tokens if T is None else T
        if not (f.is_cuda and f.dtype.is_floating_point and f.is_contiguous()):
            raise ValueError("f must be a contiguous float32 GPU tensor")
        if f.dim() != 2 or f.shape[0] < T or f.shape[1] != self.hidden:
            raise ValueError(f"f must be [>= {T}, {self.hidden}]")
        rc = lib.mhc_ws_site_post(ctypes.byref(self._ws), _dev(f, "f"), T,
                                  _stream_handle(stream))
        if rc != 0:
            raise MhcError("mhc_ws_site_post", rc, _status_text(lib, rc))
