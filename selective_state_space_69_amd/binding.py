"""Thin ctypes binding of libssscan.so (C ABI declared in include/ss_scan.h,
include/ss_conv.h, include/ss_ssd.h, include/ss_norm.h, include/ss_linear.h and
include/ss_ckpt.h).

The functions named like the C entry points (ss_scan_fwd, ss_scan_fwd_noalloc, ss_scan_fwd_dir,
ss_scan_fwd_complex, ss_scan_fwd_complex_ws, ss_scan_bwd, ss_scan_step, ss_scan_step_complex, ss_scan_workspace_bytes, ss_scan_strerror, ss_scan_version,
ss_conv1d_fwd, ss_conv1d_bwd, ss_conv1d_step, ss_conv1d_workspace_bytes, ss_ssd_fwd,
ss_ssd_fwd_state, ss_ssd_step, ss_layernorm_fwd, ss_layernorm_bwd, ss_layernorm_workspace_bytes,
ss_linear_fwd, ss_linear_bwd, ss_linear_bwd_ckpt, ss_linear_workspace_bytes, ss_ckpt_pack,
ss_ckpt_unpack) only
marshal arguments: torch tensors become device pointers, None becomes NULL and
the stream defaults to torch's current HIP stream.  Every step runs in the HIP
kernels; there is no fallback.  The convenience wrappers scan_fwd, scan_bwd,
scan_bidir, scan_fwd_complex, scan_step, scan_step_complex, conv1d_fwd, conv1d_bwd, conv1d_step, ssd_fwd, ssd_step, layernorm_fwd, layernorm_bwd, linear_fwd, linear_bwd, ckpt_pack
and ckpt_unpack additionally allocate outputs and workspace with torch.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libssscan.so")

SS_OK, SS_ERR_INVALID_ARG, SS_ERR_UNSUPPORTED, SS_ERR_WORKSPACE, SS_ERR_HIP = 0, -1, -2, -3, -4
SS_ERR_SCRATCH_LIMIT = -5
SS_SCAN_STATIC_SCRATCH_BYTES = 32 << 20
SS_F32, SS_BF16 = 0, 1
SS_ZOH, SS_EULER = 0, 1
SS_OP_FWD, SS_OP_BWD, SS_OP_FWD_COMPLEX = 0, 1, 2
SS_DIR_FORWARD, SS_DIR_REVERSE = 0, 1

_DTYPE = {torch.float32: SS_F32, torch.bfloat16: SS_BF16}
SS_ACT_NONE, SS_ACT_SILU, SS_ACT_GELU, SS_ACT_SOFTPLUS = 0, 1, 2, 3
SS_LINEAR_FWD, SS_LINEAR_BWD, SS_LINEAR_BWD_CKPT = 0, 1, 2
SS_CKPT_BLOCK = 32
_ACT = {"none": SS_ACT_NONE, "silu": SS_ACT_SILU, "gelu": SS_ACT_GELU,
        "softplus": SS_ACT_SOFTPLUS}
_DISC = {"zoh": SS_ZOH, "euler": SS_EULER}


class ss_desc_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("in_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("disc", ctypes.c_int32),
                ("delta_softplus", ctypes.c_int32), ("bc_stride", ctypes.c_int64)]


class ss_conv_desc_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("width", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("silu", ctypes.c_int32)]


class ss_ssd_desc_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64),
                ("ngroups", ctypes.c_int64), ("in_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("dt_softplus", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class ss_norm_desc_t(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("in_dtype", ctypes.c_int32), ("res_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class ss_ckpt_desc_t(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ss_linear_desc_t(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("in_dim", ctypes.c_int64), ("out_dim", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("in_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("res_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class ScanError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__("%s failed: %d (%s)" % (where, status, ss_scan_strerror(status)))
        self.status = status


_lib = None


def load_library():
    """Load libssscan.so from the package directory; raise if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libssscan.so is not built (%s); run "
                              "`python -m selective_state_space_69_amd.build`" % LIB_PATH)
        lib = ctypes.CDLL(LIB_PATH)
        P, SZ, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        D = ctypes.POINTER(ss_desc_t)
        lib.ss_scan_workspace_bytes.argtypes = [D, I]
        lib.ss_scan_workspace_bytes.restype = SZ
        lib.ss_scan_fwd.argtypes = [D] + [P] * 11 + [P, SZ, P]
        lib.ss_scan_fwd.restype = I
        lib.ss_scan_fwd_noalloc.argtypes = [D] + [P] * 11 + [P]
        lib.ss_scan_fwd_noalloc.restype = I
        lib.ss_scan_fwd_dir.argtypes = [D, I, I] + [P] * 11 + [P, SZ, P]
        lib.ss_scan_fwd_dir.restype = I
        lib.ss_scan_fwd_complex.argtypes = [D] + [P] * 11 + [P]
        lib.ss_scan_fwd_complex.restype = I
        lib.ss_scan_fwd_complex_ws.argtypes = [D] + [P] * 11 + [P, SZ, P]
        lib.ss_scan_fwd_complex_ws.restype = I
        lib.ss_scan_bwd.argtypes = [D] + [P] * 19 + [P, SZ, P]
        lib.ss_scan_bwd.restype = I
        lib.ss_scan_step.argtypes = [D] + [P] * 10 + [P]
        lib.ss_scan_step.restype = I
        lib.ss_scan_step_complex.argtypes = [D] + [P] * 10 + [P]
        lib.ss_scan_step_complex.restype = I
        C = ctypes.POINTER(ss_conv_desc_t)
        lib.ss_conv1d_workspace_bytes.argtypes = [C]
        lib.ss_conv1d_workspace_bytes.restype = SZ
        lib.ss_conv1d_fwd.argtypes = [C] + [P] * 4 + [P]
        lib.ss_conv1d_fwd.restype = I
        lib.ss_conv1d_bwd.argtypes = [C] + [P] * 7 + [P, SZ, P]
        lib.ss_conv1d_bwd.restype = I
        lib.ss_conv1d_step.argtypes = [C] + [P] * 5 + [P]
        lib.ss_conv1d_step.restype = I
        lib.ss_ssd_fwd.argtypes = [ctypes.POINTER(ss_ssd_desc_t)] + [P] * 8 + [P]
        lib.ss_ssd_fwd.restype = I
        lib.ss_ssd_fwd_state.argtypes = [ctypes.POINTER(ss_ssd_desc_t)] + [P] * 10 + [P]
        lib.ss_ssd_fwd_state.restype = I
        lib.ss_ssd_step.argtypes = [ctypes.POINTER(ss_ssd_desc_t)] + [P] * 9 + [P]
        lib.ss_ssd_step.restype = I
        NM = ctypes.POINTER(ss_norm_desc_t)
        lib.ss_layernorm_fwd.argtypes = [NM] + [P] * 8 + [P]
        lib.ss_layernorm_fwd.restype = I
        lib.ss_layernorm_workspace_bytes.argtypes = [NM]
        lib.ss_layernorm_workspace_bytes.restype = SZ
        lib.ss_layernorm_bwd.argtypes = [NM] + [P] * 9 + [P, SZ, P]
        lib.ss_layernorm_bwd.restype = I
        LN = ctypes.POINTER(ss_linear_desc_t)
        lib.ss_linear_workspace_bytes.argtypes = [LN, I]
        lib.ss_linear_workspace_bytes.restype = SZ
        lib.ss_linear_fwd.argtypes = [LN] + [P] * 6 + [P, SZ, P]
        lib.ss_linear_fwd.restype = I
        lib.ss_linear_bwd.argtypes = [LN] + [P] * 7 + [P, SZ, P]
        lib.ss_linear_bwd.restype = I
        lib.ss_linear_bwd_ckpt.argtypes = [LN] + [P] * 8 + [P, SZ, P]
        lib.ss_linear_bwd_ckpt.restype = I
        CK = ctypes.POINTER(ss_ckpt_desc_t)
        lib.ss_ckpt_pack.argtypes = [CK] + [P] * 3 + [P]
        lib.ss_ckpt_pack.restype = I
        lib.ss_ckpt_unpack.argtypes = [CK] + [P] * 3 + [P]
        lib.ss_ckpt_unpack.restype = I
        lib.ss_scan_strerror.argtypes = [I]
        lib.ss_scan_strerror.restype = ctypes.c_char_p
        lib.ss_scan_version.argtypes = []
        lib.ss_scan_version.restype = I
        lib.ss_scan_arch_supported.argtypes = [ctypes.c_char_p]
        lib.ss_scan_arch_supported.restype = I
        _lib = lib
    return _lib


def make_desc(batch, seqlen, dim, dstate, in_dtype=SS_BF16, out_dtype=SS_F32, disc=SS_ZOH,
              delta_softplus=True, bc_stride=0) -> ss_desc_t:
    return ss_desc_t(int(batch), int(seqlen), int(dim), int(dstate), int(in_dtype),
                     int(out_dtype), int(disc), int(bool(delta_softplus)), int(bc_stride))


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


# ---------------------------------------------------------------- C-named entry points
def ss_scan_version() -> int:
    return load_library().ss_scan_version()


def ss_scan_arch_supported(arch_name) -> int:
    return load_library().ss_scan_arch_supported(
        None if arch_name is None else arch_name.encode())


def ss_scan_strerror(status: int) -> str:
    return load_library().ss_scan_strerror(int(status)).decode()


def ss_scan_workspace_bytes(desc: ss_desc_t, op: int) -> int:
    return int(load_library().ss_scan_workspace_bytes(ctypes.byref(desc), int(op)))


def ss_scan_fwd(desc, u, delta, A, Bm, Cm, D_skip, delta_bias, z, h0, y, h_last,
                workspace, ws_bytes, stream=None) -> int:
    return load_library().ss_scan_fwd(ctypes.byref(desc), _p(u), _p(delta), _p(A), _p(Bm), _p(Cm),
                                      _p(D_skip), _p(delta_bias), _p(z), _p(h0), _p(y), _p(h_last),
                                      _p(workspace), int(ws_bytes), _stream(stream))


def ss_scan_fwd_noalloc(desc, u, delta, A, Bm, Cm, D_skip, delta_bias, z, h0, y, h_last,
                        stream=None) -> int:
    return load_library().ss_scan_fwd_noalloc(ctypes.byref(desc), _p(u), _p(delta), _p(A), _p(Bm),
                                              _p(Cm), _p(D_skip), _p(delta_bias), _p(z), _p(h0),
                                              _p(y), _p(h_last), _stream(stream))


def ss_scan_fwd_dir(desc, direction, accumulate, u, delta, A, Bm, Cm, D_skip, delta_bias, z, h0,
                    y, h_last, workspace, ws_bytes, stream=None) -> int:
    return load_library().ss_scan_fwd_dir(ctypes.byref(desc), int(direction), int(accumulate),
                                          _p(u), _p(delta), _p(A), _p(Bm), _p(Cm), _p(D_skip),
                                          _p(delta_bias), _p(z), _p(h0), _p(y), _p(h_last),
                                          _p(workspace), int(ws_bytes), _stream(stream))


def ss_scan_fwd_complex(desc, u, delta, A, Bm, Cm, D_skip, delta_bias, z, h0, y, h_last,
                        stream=None) -> int:
    return load_library().ss_scan_fwd_complex(ctypes.byref(desc), _p(u), _p(delta), _p(A), _p(Bm),
                                              _p(Cm), _p(D_skip), _p(delta_bias), _p(z), _p(h0),
                                              _p(y), _p(h_last), _stream(stream))


def ss_scan_fwd_complex_ws(desc, u, delta, A, Bm, Cm, D_skip, delta_bias, z, h0, y, h_last,
                           workspace, ws_bytes, stream=None) -> int:
    return load_library().ss_scan_fwd_complex_ws(ctypes.byref(desc), _p(u), _p(delta), _p(A),
                                                 _p(Bm), _p(Cm), _p(D_skip), _p(delta_bias), _p(z),
                                                 _p(h0), _p(y), _p(h_last), _p(workspace),
                                                 int(ws_bytes), _stream(stream))


def ss_scan_bwd(desc, u, delta, A, Bm, Cm, D_skip, delta_bias, z, h0, dy, du, ddelta, dA, dB, dC,
                dD_skip, ddelta_bias, dz, dh0, workspace, ws_bytes, stream=None) -> int:
    return load_library().ss_scan_bwd(ctypes.byref(desc), _p(u), _p(delta), _p(A), _p(Bm), _p(Cm),
                                      _p(D_skip), _p(delta_bias), _p(z), _p(h0), _p(dy), _p(du),
                                      _p(ddelta), _p(dA), _p(dB), _p(dC), _p(dD_skip),
                                      _p(ddelta_bias), _p(dz), _p(dh0), _p(workspace),
                                      int(ws_bytes), _stream(stream))


def ss_scan_step(desc, h, u, delta, A, Bm, Cm, D_skip, delta_bias, z, y, stream=None) -> int:
    return load_library().ss_scan_step(ctypes.byref(desc), _p(h), _p(u), _p(delta), _p(A), _p(Bm),
                                       _p(Cm), _p(D_skip), _p(delta_bias), _p(z), _p(y),
                                       _stream(stream))


def ss_scan_step_complex(desc, h, u, delta, A, Bm, Cm, D_skip, delta_bias, z, y,
                         stream=None) -> int:
    return load_library().ss_scan_step_complex(ctypes.byref(desc), _p(h), _p(u), _p(delta),
                                               _p(A), _p(Bm), _p(Cm), _p(D_skip),
                                               _p(delta_bias), _p(z), _p(y), _stream(stream))


def make_conv_desc(batch, seqlen, dim, width, in_dtype=SS_F32, out_dtype=SS_F32, silu=True):
    return ss_conv_desc_t(int(batch), int(seqlen), int(dim), int(width), int(in_dtype),
                          int(out_dtype), int(bool(silu)))


def ss_conv1d_workspace_bytes(desc: ss_conv_desc_t) -> int:
    return int(load_library().ss_conv1d_workspace_bytes(ctypes.byref(desc)))


def ss_conv1d_fwd(desc, x, w, bias, u, stream=None) -> int:
    return load_library().ss_conv1d_fwd(ctypes.byref(desc), _p(x), _p(w), _p(bias), _p(u),
                                        _stream(stream))


def ss_conv1d_bwd(desc, x, w, bias, du, dx, dw, dbias, workspace, ws_bytes, stream=None) -> int:
    return load_library().ss_conv1d_bwd(ctypes.byref(desc), _p(x), _p(w), _p(bias), _p(du),
                                        _p(dx), _p(dw), _p(dbias), _p(workspace), int(ws_bytes),
                                        _stream(stream))


def ss_conv1d_step(desc, state, x, w, bias, u, stream=None) -> int:
    return load_library().ss_conv1d_step(ctypes.byref(desc), _p(state), _p(x), _p(w), _p(bias),
                                         _p(u), _stream(stream))


# ---------------------------------------------------------------- allocating wrappers
def make_ssd_desc(batch, seqlen, nheads, headdim, dstate, ngroups=1, in_dtype=SS_BF16,
                  out_dtype=SS_F32, dt_softplus=True) -> ss_ssd_desc_t:
    return ss_ssd_desc_t(int(batch), int(seqlen), int(nheads), int(headdim), int(dstate),
                         int(ngroups), int(in_dtype), int(out_dtype), int(bool(dt_softplus)), 0)


def ss_ssd_fwd(desc, x, dt, A, Bm, Cm, D, dt_bias, y, stream=None) -> int:
    return load_library().ss_ssd_fwd(ctypes.byref(desc), _p(x), _p(dt), _p(A), _p(Bm), _p(Cm),
                                      _p(D), _p(dt_bias), _p(y), _stream(stream))


def ss_ssd_fwd_state(desc, x, dt, A, Bm, Cm, D, dt_bias, h0, y, h_last, stream=None) -> int:
    return load_library().ss_ssd_fwd_state(ctypes.byref(desc), _p(x), _p(dt), _p(A), _p(Bm),
                                            _p(Cm), _p(D), _p(dt_bias), _p(h0), _p(y),
                                            _p(h_last), _stream(stream))


def ss_ssd_step(desc, h, x, dt, A, Bm, Cm, D, dt_bias, y, stream=None) -> int:
    return load_library().ss_ssd_step(ctypes.byref(desc), _p(h), _p(x), _p(dt), _p(A), _p(Bm),
                                       _p(Cm), _p(D), _p(dt_bias), _p(y), _stream(stream))


def make_norm_desc(rows, dim, x_stride=0, in_dtype=SS_BF16, res_dtype=SS_F32, out_dtype=SS_BF16,
                   eps=1e-5) -> ss_norm_desc_t:
    return ss_norm_desc_t(int(rows), int(dim), int(x_stride), int(in_dtype), int(res_dtype),
                          int(out_dtype), float(eps))


def ss_layernorm_fwd(desc, x, residual, weight, bias, y, sum, mean, rstd, stream=None) -> int:
    return load_library().ss_layernorm_fwd(ctypes.byref(desc), _p(x), _p(residual), _p(weight),
                                           _p(bias), _p(y), _p(sum), _p(mean), _p(rstd),
                                           _stream(stream))


def ss_layernorm_workspace_bytes(desc: ss_norm_desc_t) -> int:
    return int(load_library().ss_layernorm_workspace_bytes(ctypes.byref(desc)))


def ss_layernorm_bwd(desc, s, weight, mean, rstd, dy, dsum, dx, dweight, dbias, workspace,
                     ws_bytes, stream=None) -> int:
    return load_library().ss_layernorm_bwd(ctypes.byref(desc), _p(s), _p(weight), _p(mean),
                                           _p(rstd), _p(dy), _p(dsum), _p(dx), _p(dweight),
                                           _p(dbias), _p(workspace), int(ws_bytes),
                                           _stream(stream))


def make_linear_desc(rows, in_dim, out_dim, x_stride=0, in_dtype=SS_BF16, out_dtype=SS_BF16,
                     res_dtype=SS_BF16, grad_dtype=SS_BF16, act=SS_ACT_NONE) -> ss_linear_desc_t:
    return ss_linear_desc_t(int(rows), int(in_dim), int(out_dim), int(x_stride), int(in_dtype),
                            int(out_dtype), int(res_dtype), int(grad_dtype), int(act), 0)


def ss_linear_workspace_bytes(desc: ss_linear_desc_t, op: int) -> int:
    return int(load_library().ss_linear_workspace_bytes(ctypes.byref(desc), int(op)))


def ss_linear_fwd(desc, x, w, bias, residual, y, pre, workspace, ws_bytes, stream=None) -> int:
    return load_library().ss_linear_fwd(ctypes.byref(desc), _p(x), _p(w), _p(bias), _p(residual),
                                        _p(y), _p(pre), _p(workspace), int(ws_bytes),
                                        _stream(stream))


def ss_linear_bwd(desc, x, w, pre, dy, dx, dw, dbias, workspace, ws_bytes, stream=None) -> int:
    return load_library().ss_linear_bwd(ctypes.byref(desc), _p(x), _p(w), _p(pre), _p(dy), _p(dx),
                                        _p(dw), _p(dbias), _p(workspace), int(ws_bytes),
                                        _stream(stream))


def ss_linear_bwd_ckpt(desc, q, e, w, pre, dy, dx, dw, dbias, workspace, ws_bytes,
                       stream=None) -> int:
    return load_library().ss_linear_bwd_ckpt(ctypes.byref(desc), _p(q), _p(e), _p(w), _p(pre),
                                             _p(dy), _p(dx), _p(dw), _p(dbias), _p(workspace),
                                             int(ws_bytes), _stream(stream))


def make_ckpt_desc(rows, dim, x_stride=0, dtype=SS_BF16) -> ss_ckpt_desc_t:
    return ss_ckpt_desc_t(int(rows), int(dim), int(x_stride), int(dtype), 0)


def ss_ckpt_pack(desc, x, q, e, stream=None) -> int:
    return load_library().ss_ckpt_pack(ctypes.byref(desc), _p(x), _p(q), _p(e), _stream(stream))


def ss_ckpt_unpack(desc, q, e, x, stream=None) -> int:
    return load_library().ss_ckpt_unpack(ctypes.byref(desc), _p(q), _p(e), _p(x), _stream(stream))


def _check(rc, where):
    if rc != SS_OK:
        raise ScanError(rc, where)


def _row_stride(t, name):
    """Elements from one row of t to the next, over every leading axis flattened
    ((B, L, N) -> B*L rows of N, (B, N) -> B rows); the last axis must be unit
    stride."""
    shape, stride = t.shape, t.stride()
    if shape[-1] > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: the last axis must have unit stride")
    S = None
    step = None
    for n, st in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if S is None:
            S, step = st, st * n
        elif st != step:
            raise ValueError(f"{name}: rows must be evenly spaced (one stride over all rows)")
        else:
            step = st * n
    return shape[-1] if S is None else S


def _bc_stride(B, C, N):
    """ss_desc_t.bc_stride for B and C read in place: 0 for dense rows, else the
    common row stride (e.g. B, C sliced from the input projection's output)."""
    sb, sc = _row_stride(B, "B"), _row_stride(C, "C")
    if sb != sc:
        raise ValueError("B and C must share one row stride")
    if sb < N:
        raise ValueError("B, C rows overlap (row stride below dstate)")
    # dense rows are read in place with 16-byte loads; a dense view at another
    # offset goes through the strided path, which needs element alignment only
    dense_ok = B.data_ptr() % 16 == 0 and C.data_ptr() % 16 == 0
    return 0 if sb == N and dense_ok else sb


def _dense(**tensors):
    """The library reads every tensor but strided B, C as dense rows: refuse
    views with other strides instead of reading the wrong elements."""
    for name, t in tensors.items():
        if t is not None and not t.is_contiguous():
            raise ValueError("%s must be contiguous (got strides %s)" % (name, tuple(t.stride())))


def _desc_from(u, A, B, C, disc, softplus, out_dtype):
    Bt, L, D = u.shape
    N = A.shape[1]
    return make_desc(Bt, L, D, N, _DTYPE[u.dtype], _DTYPE[out_dtype], _DISC[disc], softplus,
                     _bc_stride(B, C, N))


def workspace(nbytes: int, device) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def scan_fwd(u, delta, A, B, C, D=None, delta_bias=None, z=None, h0=None, disc="zoh",
             softplus=True, out_dtype=torch.float32, return_last_state=False, stream=None,
             ws=None, reverse=False, y=None):
    """Forward scan on device tensors; returns y (and h_last).  reverse=True runs
    the system from the last step to the first; passing y adds the result to it
    (in place) instead of allocating a new output.  B and C may be views with a
    row stride (column ranges of one projection output); the other tensors are
    dense."""
    _dense(u=u, delta=delta, A=A, D=D, delta_bias=delta_bias, z=z, h0=h0, y=y)
    desc = _desc_from(u, A, B, C, disc, softplus, out_dtype if y is None else y.dtype)
    acc = y is not None
    if y is None:
        y = torch.empty(u.shape, dtype=out_dtype, device=u.device)
    h_last = (torch.empty((u.shape[0], u.shape[2], A.shape[1]), dtype=torch.float32,
                          device=u.device) if return_last_state else None)
    nb = ss_scan_workspace_bytes(desc, SS_OP_FWD)
    if ws is None or ws.numel() < nb:
        ws = workspace(nb, u.device)
    _check(ss_scan_fwd_dir(desc, SS_DIR_REVERSE if reverse else SS_DIR_FORWARD, int(acc), u, delta,
                           A, B, C, D, delta_bias, z, h0, y, h_last, ws, nb, stream),
           "ss_scan_fwd_dir")
    return (y, h_last) if return_last_state else y


def scan_fwd_complex(u, delta, A, B, C, D=None, delta_bias=None, z=None, h0=None, disc="zoh",
                     softplus=True, out_dtype=torch.float32, return_last_state=False,
                     stream=None):
    """Complex-A forward: A (D, N, 2) float32, B and C (B, L, N, 2) in u's dtype,
    h0 (B, D, N, 2) float32 ((re, im) pairs).  Returns y (and h_last (B, D, N, 2)).
    Uses ss_scan_fwd_complex_ws with a torch workspace (time chunks where the
    plan wants them)."""
    _dense(u=u, delta=delta, A=A, B=B, C=C, D=D, delta_bias=delta_bias, z=z, h0=h0)
    Bt, L, Dd = u.shape
    N = A.shape[1]
    desc = make_desc(Bt, L, Dd, N, _DTYPE[u.dtype], _DTYPE[out_dtype], _DISC[disc], softplus)
    y = torch.empty(u.shape, dtype=out_dtype, device=u.device)
    h_last = (torch.empty((Bt, Dd, N, 2), dtype=torch.float32, device=u.device)
              if return_last_state else None)
    nb = ss_scan_workspace_bytes(desc, SS_OP_FWD_COMPLEX)
    ws = workspace(nb, u.device)
    _check(ss_scan_fwd_complex_ws(desc, u, delta, A, B, C, D, delta_bias, z, h0, y, h_last, ws,
                                  nb, stream), "ss_scan_fwd_complex_ws")
    return (y, h_last) if return_last_state else y


def scan_bidir(u, delta, A, B, C, D=None, delta_bias=None, z=None, disc="zoh", softplus=True,
               A_rev=None, D_rev=None, delta_bias_rev=None, out_dtype=torch.float32, stream=None):
    """Bidirectional scan: the forward scan plus the reverse-time scan (with its
    own A, D, delta_bias when given), summed inside the second kernel."""
    y = scan_fwd(u, delta, A, B, C, D=D, delta_bias=delta_bias, z=z, disc=disc,
                 softplus=softplus, out_dtype=out_dtype, stream=stream)
    scan_fwd(u, delta, A if A_rev is None else A_rev, B, C,
             D=D if D_rev is None else D_rev,
             delta_bias=delta_bias if delta_bias_rev is None else delta_bias_rev, z=z, disc=disc,
             softplus=softplus, stream=stream, reverse=True, y=y)
    return y


def scan_bwd(u, delta, A, B, C, dy, D=None, delta_bias=None, z=None, h0=None, disc="zoh",
             softplus=True, want_dh0=False, stream=None):
    """Backward scan; returns a dict of fp32 gradients (dB, dC dense even when B
    and C are strided views)."""
    _dense(u=u, delta=delta, A=A, D=D, delta_bias=delta_bias, z=z, h0=h0, dy=dy)
    desc = _desc_from(u, A, B, C, disc, softplus, torch.float32)
    dev = u.device
    f32 = dict(dtype=torch.float32, device=dev)
    g = {"du": torch.empty(u.shape, **f32), "ddelta": torch.empty(u.shape, **f32),
         "dA": torch.empty(A.shape, **f32), "dB": torch.empty(B.shape, **f32),
         "dC": torch.empty(C.shape, **f32),
         "dD": torch.empty(D.shape, **f32) if D is not None else None,
         "ddelta_bias": torch.empty(delta_bias.shape, **f32) if delta_bias is not None else None,
         "dz": torch.empty(u.shape, **f32) if z is not None else None,
         "dh0": torch.empty((u.shape[0], u.shape[2], A.shape[1]), **f32) if want_dh0 else None}
    nb = ss_scan_workspace_bytes(desc, SS_OP_BWD)
    ws = workspace(nb, dev)
    _check(ss_scan_bwd(desc, u, delta, A, B, C, D, delta_bias, z, h0, dy, g["du"], g["ddelta"],
                       g["dA"], g["dB"], g["dC"], g["dD"], g["ddelta_bias"], g["dz"], g["dh0"],
                       ws, nb, stream), "ss_scan_bwd")
    return g


def scan_step(h, u, delta, A, B, C, D=None, delta_bias=None, z=None, disc="zoh", softplus=True,
              out_dtype=torch.float32, stream=None):
    """One recurrent step; h (B,D,N) fp32 is updated in place; returns y (B,D).
    B and C (B,N) may be strided views, as in scan_fwd."""
    _dense(h=h, u=u, delta=delta, A=A, D=D, delta_bias=delta_bias, z=z)
    Bt, Dd = u.shape
    desc = make_desc(Bt, 1, Dd, A.shape[1], _DTYPE[u.dtype], _DTYPE[out_dtype], _DISC[disc],
                     softplus, _bc_stride(B, C, A.shape[1]))
    y = torch.empty(u.shape, dtype=out_dtype, device=u.device)
    _check(ss_scan_step(desc, h, u, delta, A, B, C, D, delta_bias, z, y, stream), "ss_scan_step")
    return y


def scan_step_complex(h, u, delta, A, B, C, D=None, delta_bias=None, z=None, disc="zoh",
                      softplus=True, out_dtype=torch.float32, stream=None):
    """One step with complex A: h (B,D,N,2) fp32 updated in place, A (D,N,2),
    B and C (B,N,2); returns y (B,D)."""
    _dense(h=h, u=u, delta=delta, A=A, B=B, C=C, D=D, delta_bias=delta_bias, z=z)
    Bt, Dd = u.shape
    desc = make_desc(Bt, 1, Dd, A.shape[1], _DTYPE[u.dtype], _DTYPE[out_dtype], _DISC[disc],
                     softplus)
    y = torch.empty(u.shape, dtype=out_dtype, device=u.device)
    _check(ss_scan_step_complex(desc, h, u, delta, A, B, C, D, delta_bias, z, y, stream),
           "ss_scan_step_complex")
    return y


def conv1d_fwd(x, w, bias=None, silu=True, out_dtype=None, stream=None):
    """Causal depthwise conv of width w.shape[1] (+ SiLU) over x (B, L, D);
    returns u (B, L, D) in out_dtype (default: x's dtype)."""
    _dense(x=x, w=w, bias=bias)
    Bt, L, Dd = x.shape
    out_dtype = x.dtype if out_dtype is None else out_dtype
    desc = make_conv_desc(Bt, L, Dd, w.shape[1], _DTYPE[x.dtype], _DTYPE[out_dtype], silu)
    u = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    _check(ss_conv1d_fwd(desc, x, w, bias, u, stream), "ss_conv1d_fwd")
    return u


def conv1d_bwd(x, w, du, bias=None, silu=True, stream=None):
    """Backward of conv1d_fwd given du (fp32); returns dict dx, dw, dbias (fp32)."""
    _dense(x=x, w=w, du=du, bias=bias)
    Bt, L, Dd = x.shape
    desc = make_conv_desc(Bt, L, Dd, w.shape[1], _DTYPE[x.dtype], SS_F32, silu)
    f32 = dict(dtype=torch.float32, device=x.device)
    g = {"dx": torch.empty(x.shape, **f32), "dw": torch.empty(w.shape, **f32),
         "dbias": torch.empty(bias.shape, **f32) if bias is not None else None}
    nb = ss_conv1d_workspace_bytes(desc)
    ws = workspace(nb, x.device)
    _check(ss_conv1d_bwd(desc, x, w, bias, du, g["dx"], g["dw"], g["dbias"], ws, nb, stream),
           "ss_conv1d_bwd")
    return g


def conv1d_step(state, x, w, bias=None, silu=True, out_dtype=torch.float32, stream=None):
    """One decode step: state (B, D, K-1) fp32 updated in place, x (B, D); returns u."""
    _dense(state=state, x=x, w=w, bias=bias)
    Bt, Dd = x.shape
    desc = make_conv_desc(Bt, 1, Dd, w.shape[1], _DTYPE[x.dtype], _DTYPE[out_dtype], silu)
    u = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    _check(ss_conv1d_step(desc, state, x, w, bias, u, stream), "ss_conv1d_step")
    return u


def ssd_fwd(x, dt, A, B, C, D=None, dt_bias=None, softplus=True, out_dtype=torch.float32,
            stream=None, h0=None, return_last=False):
    """SSD (Mamba-2) layer forward: x (Bt, L, H, P), dt (Bt, L, H), B and C
    (Bt, L, G, N) in bf16; A, D, dt_bias (H,) fp32; optional start state h0
    (Bt, H, N, P) fp32.  Returns y (Bt, L, H, P), and with return_last the
    state after the last step as well."""
    _dense(x=x, dt=dt, A=A, B=B, C=C, D=D, dt_bias=dt_bias, h0=h0)
    Bt, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    desc = make_ssd_desc(Bt, L, H, P, N, G, _DTYPE[x.dtype], _DTYPE[out_dtype], softplus)
    y = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    if h0 is None and not return_last:
        _check(ss_ssd_fwd(desc, x, dt, A, B, C, D, dt_bias, y, stream), "ss_ssd_fwd")
        return y
    h_last = (torch.empty((Bt, H, N, P), dtype=torch.float32, device=x.device)
              if return_last else None)
    _check(ss_ssd_fwd_state(desc, x, dt, A, B, C, D, dt_bias, h0, y, h_last, stream),
           "ss_ssd_fwd_state")
    return (y, h_last) if return_last else y


def ssd_step(h, x, dt, A, B, C, D=None, dt_bias=None, softplus=True, out_dtype=torch.float32,
             stream=None):
    """One SSD decode step: h (Bt, H, N, P) fp32 updated in place; x (Bt, H, P),
    dt (Bt, H), B and C (Bt, G, N) bf16.  Returns y (Bt, H, P)."""
    _dense(h=h, x=x, dt=dt, A=A, B=B, C=C, D=D, dt_bias=dt_bias)
    Bt, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    desc = make_ssd_desc(Bt, 1, H, P, N, G, _DTYPE[x.dtype], _DTYPE[out_dtype], softplus)
    y = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    _check(ss_ssd_step(desc, h, x, dt, A, B, C, D, dt_bias, y, stream), "ss_ssd_step")
    return y


# ------------------------------------------- the operators around the scan in a block
# Decode calls of these take a few microseconds on the GPU, so their wrappers keep
# to plain integers (devices, streams, pointers) on the way to the library.
def _dt(t, name):
    d = _DTYPE.get(t)
    if d is None:
        raise ValueError("%s must be float32 or bfloat16 (got %s)" % (name, t))
    return d


def _f32(t, name):
    if t is not None and t.dtype is not torch.float32:
        raise ValueError("%s must be float32 (got %s)" % (name, t.dtype))


def _arg(t, name, shape):
    """Device pointer of a dense tensor of this shape (None: no tensor)."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous (got strides %s)" % (name, tuple(t.stride())))
    return t.data_ptr()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _like(t, dtype):
    """A dense tensor of t's shape (empty_like costs half of what empty does)."""
    if t.dtype is dtype and t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty(t.shape, dtype=dtype, device=t.device)


def _x_stride(x, name):
    """x_stride of rows read in place: 0 for dense rows at a 16-byte aligned
    address, else the elements from one row to the next.  Rows that overlap (an
    expanded axis) are refused."""
    dim = x.shape[-1]
    if x.is_contiguous():
        return 0 if x.data_ptr() % 16 == 0 else dim
    s = _row_stride(x, name)
    if s < dim:
        raise ValueError("%s: rows overlap (row stride below the row's length)" % name)
    return s


def _on_device(fn, stream, tensors, *args):
    """fn(raw stream, *args) with the tensors' GPU and the stream current, so that
    its outputs and workspace are allocated for the stream the kernels run on.
    stream: None (the device's current one), a torch stream or a raw hipStream_t;
    memory of the tensors is kept from reuse until a stream other than their own
    is done."""
    dev = -1
    for t in tensors:
        if t is None:
            continue
        d = t.get_device()
        if d < 0:
            raise ValueError("all tensors must be on the GPU")
        if dev < 0:
            dev = d
        elif d != dev:
            raise ValueError("all tensors must be on one GPU")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
        if dev == torch._C._cuda_getDevice():
            return fn(raw, *args)
        with torch.cuda.device(dev):
            return fn(raw, *args)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    if stream.device.index != dev:
        raise ValueError("the stream belongs to another GPU than the tensors")
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return fn(stream.cuda_stream, *args)


def layernorm_fwd(x, weight=None, bias=None, residual=None, eps=1e-5, out_dtype=None,
                  save_stats=False, stream=None):
    """Layer norm over the last axis of s = x + residual.  x may have a row
    stride (a column range of a wider tensor); weight and bias are float32.
    Returns a dict: y (out_dtype, default x's), sum (s in residual's dtype, the
    new residual stream; None without a residual), mean and rstd (float32, None
    unless save_stats)."""
    return _on_device(_layernorm_fwd, stream, (x, weight, bias, residual), x, weight, bias,
                      residual, eps, x.dtype if out_dtype is None else out_dtype, save_stats)


def _layernorm_fwd(raw, x, weight, bias, residual, eps, odt, save_stats):
    shape = x.shape
    dim = shape[-1]
    _f32(weight, "weight")
    _f32(bias, "bias")
    dt = _dt(x.dtype, "x")
    desc = ss_norm_desc_t(x.numel() // dim if dim else 0, dim, _x_stride(x, "x"), dt,
                          dt if residual is None else _dt(residual.dtype, "residual"),
                          _dt(odt, "out_dtype"), eps)
    wp, bp = _arg(weight, "weight", (dim,)), _arg(bias, "bias", (dim,))
    rp = _arg(residual, "residual", shape)
    y = _like(x, odt)
    s = None if residual is None else torch.empty_like(residual)
    mean = rstd = None
    if save_stats:
        mean = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    _check(load_library().ss_layernorm_fwd(ctypes.byref(desc), x.data_ptr(), rp, wp, bp,
                                           y.data_ptr(), _ptr(s), _ptr(mean), _ptr(rstd), raw),
           "ss_layernorm_fwd")
    return {"y": y, "sum": s, "mean": mean, "rstd": rstd}


def layernorm_bwd(s, dy, mean, rstd, weight=None, dsum=None, dx_dtype=None, stream=None):
    """Backward of layernorm_fwd: s is what was normalised (x, or the returned
    sum; a row stride is taken), dsum the gradient that reaches s from elsewhere.
    Returns a dict: dx (dx_dtype, default dsum's dtype or float32; the gradient
    of x and of the residual alike), dweight and dbias (float32)."""
    if dx_dtype is None:
        dx_dtype = torch.float32 if dsum is None else dsum.dtype
    return _on_device(_layernorm_bwd, stream, (s, dy, mean, rstd, weight, dsum), s, dy, mean, rstd,
                      weight, dsum, dx_dtype)


def _layernorm_bwd(raw, s, dy, mean, rstd, weight, dsum, rdt):
    shape = s.shape
    dim = shape[-1]
    _f32(weight, "weight")
    _f32(mean, "mean")
    _f32(rstd, "rstd")
    if dsum is not None and dsum.dtype != rdt:
        raise ValueError("dx_dtype must be dsum's dtype")
    desc = ss_norm_desc_t(s.numel() // dim if dim else 0, dim, _x_stride(s, "s"),
                          _dt(s.dtype, "s"), _dt(rdt, "dx_dtype"), _dt(dy.dtype, "dy"), 1.0)
    wp, mp = _arg(weight, "weight", (dim,)), _arg(mean, "mean", shape[:-1])
    rp, dyp = _arg(rstd, "rstd", shape[:-1]), _arg(dy, "dy", shape)
    dsp = _arg(dsum, "dsum", shape)
    dx = _like(s, rdt)
    dw = torch.empty(dim, dtype=torch.float32, device=s.device)
    db = torch.empty_like(dw)
    lib = load_library()
    nb = lib.ss_layernorm_workspace_bytes(ctypes.byref(desc))
    ws = workspace(nb, s.device)
    _check(lib.ss_layernorm_bwd(ctypes.byref(desc), s.data_ptr(), wp, mp, rp, dyp, dsp,
                                dx.data_ptr(), dw.data_ptr(), db.data_ptr(), _ptr(ws), nb, raw),
           "ss_layernorm_bwd")
    return {"dx": dx, "dweight": dw, "dbias": db}


def linear_fwd(x, w, bias=None, residual=None, act="none", out_dtype=None, save_pre=False,
               stream=None):
    """act(x w^T + bias) + residual for x (..., K) and w (N, K) of one dtype; x
    may have a row stride.  bias is float32, residual (..., N) float32 or
    bfloat16, act one of "none", "silu", "gelu", "softplus".  Returns y (..., N)
    in out_dtype (default x's), and with save_pre the pre-activation values in
    x's dtype as well."""
    return _on_device(_linear_fwd, stream, (x, w, bias, residual), x, w, bias, residual, _ACT[act],
                      x.dtype if out_dtype is None else out_dtype, save_pre)


def _linear_fwd(raw, x, w, bias, residual, act, odt, save_pre):
    n, k = w.shape
    oshape = (*x.shape[:-1], n)
    if x.shape[-1] != k:
        raise ValueError("x must have %d columns (got %d)" % (k, x.shape[-1]))
    if x.dtype != w.dtype:
        raise ValueError("x and w must have one dtype")
    _f32(bias, "bias")
    od = _dt(odt, "out_dtype")
    desc = ss_linear_desc_t(x.numel() // k if k else 0, k, n, _x_stride(x, "x"),
                            _dt(x.dtype, "x"), od,
                            od if residual is None else _dt(residual.dtype, "residual"), SS_F32,
                            act, 0)
    wp, bp, rp = _arg(w, "w", (n, k)), _arg(bias, "bias", (n,)), _arg(residual, "residual", oshape)
    y = torch.empty(oshape, dtype=odt, device=x.device)
    pre = _like(y, x.dtype) if save_pre else None
    lib = load_library()
    nb = lib.ss_linear_workspace_bytes(ctypes.byref(desc), SS_LINEAR_FWD)
    ws = workspace(nb, x.device)
    _check(lib.ss_linear_fwd(ctypes.byref(desc), x.data_ptr(), wp, bp, rp, y.data_ptr(), _ptr(pre),
                             _ptr(ws), nb, raw), "ss_linear_fwd")
    return (y, pre) if save_pre else y


def linear_bwd(x, w, dy, pre=None, act="none", bias=False, grad_dtype=None, need_dx=True,
               need_dw=True, stream=None):
    """Backward of linear_fwd given dy (..., N).  x: the forward's input, or its
    8-bit checkpoint (q, e) from ckpt_pack (None when need_dw is false).  pre:
    the forward's pre-activation values, with an activation.  Returns a dict: dx
    (..., K) and dw (N, K) in grad_dtype (default w's), dbias (N) float32 when
    bias is true; what is not asked for is None.  With bf16 operands and a dy that
    is float32 or passes an activation, float32 gradients keep it to 2^-16 (twice
    the matrix work), bf16 ones round it to bf16."""
    q, e = x if isinstance(x, tuple) else (None, None)
    x = None if isinstance(x, tuple) else x
    return _on_device(_linear_bwd, stream, (w, dy, x, q, e, pre), x, q, e, w, dy, pre, _ACT[act],
                      bias, w.dtype if grad_dtype is None else grad_dtype, need_dx, need_dw)


def _linear_bwd(raw, x, q, e, w, dy, pre, act, bias, gdt, need_dx, need_dw):
    n, k = w.shape
    lead = dy.shape[:-1]
    if pre is not None and pre.dtype != w.dtype:
        raise ValueError("pre must have w's dtype")
    if need_dw and x is None and q is None:
        raise ValueError("dw needs x")
    dyp, prep, wp = _arg(dy, "dy", (*lead, n)), _arg(pre, "pre", (*lead, n)), _arg(w, "w", (n, k))
    xs = 0
    if q is not None:
        qp, ep = _ckpt_args(q, e, (*lead, k))
    elif x is not None:
        if x.shape != (*lead, k):
            raise ValueError("x must have shape %s (got %s)" % ((*lead, k), tuple(x.shape)))
        if x.dtype != w.dtype:
            raise ValueError("x and w must have one dtype")
        xs = _x_stride(x, "x")
    desc = ss_linear_desc_t(dy.numel() // n if n else 0, k, n, xs, _dt(w.dtype, "w"),
                            _dt(dy.dtype, "dy"), SS_F32, _dt(gdt, "grad_dtype"), act, 0)
    dx = torch.empty((*lead, k), dtype=gdt, device=w.device) if need_dx else None
    dw = _like(w, gdt) if need_dw else None
    db = torch.empty(n, dtype=torch.float32, device=w.device) if bias else None
    lib = load_library()
    nb = lib.ss_linear_workspace_bytes(ctypes.byref(desc),
                                       SS_LINEAR_BWD if q is None else SS_LINEAR_BWD_CKPT)
    ws = workspace(nb, w.device)
    rest = (wp, prep, dyp, _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws), nb, raw)
    if q is None:
        _check(lib.ss_linear_bwd(ctypes.byref(desc), _ptr(x), *rest), "ss_linear_bwd")
    else:
        _check(lib.ss_linear_bwd_ckpt(ctypes.byref(desc), qp, ep, *rest), "ss_linear_bwd_ckpt")
    return {"dx": dx, "dw": dw, "dbias": db}


def _ckpt_args(q, e, shape):
    if q.dtype != torch.int8 or e.dtype != torch.uint8:
        raise ValueError("a checkpoint is int8 values and uint8 exponents")
    return _arg(q, "q", shape), _arg(e, "e", (*shape[:-1], -(-shape[-1] // SS_CKPT_BLOCK)))


def ckpt_pack(x, stream=None):
    """8-bit checkpoint of x (..., D): (q, e), int8 values and one uint8 exponent
    per 32 channels.  x may have a row stride."""
    return _on_device(_ckpt_pack, stream, (x,), x)


def _ckpt_pack(raw, x):
    dim = x.shape[-1]
    desc = ss_ckpt_desc_t(x.numel() // dim if dim else 0, dim, _x_stride(x, "x"),
                          _dt(x.dtype, "x"), 0)
    q = _like(x, torch.int8)
    e = torch.empty((*x.shape[:-1], -(-dim // SS_CKPT_BLOCK)), dtype=torch.uint8, device=x.device)
    _check(load_library().ss_ckpt_pack(ctypes.byref(desc), x.data_ptr(), q.data_ptr(),
                                       e.data_ptr(), raw), "ss_ckpt_pack")
    return q, e


def ckpt_unpack(q, e, dtype=torch.bfloat16, stream=None):
    """The values of a checkpoint (q, e), in dtype."""
    return _on_device(_ckpt_unpack, stream, (q, e), q, e, dtype)


def _ckpt_unpack(raw, q, e, dtype):
    dim = q.shape[-1]
    qp, ep = _ckpt_args(q, e, q.shape)
    desc = ss_ckpt_desc_t(q.numel() // dim if dim else 0, dim, 0, _dt(dtype, "dtype"), 0)
    x = _like(q, dtype)
    _check(load_library().ss_ckpt_unpack(ctypes.byref(desc), qp, ep, x.data_ptr(), raw),
           "ss_ckpt_unpack")
    return x
