"""Thin ctypes binding of libgla.so (C ABI in include/gla.h).

Argument marshalling only: every step runs in the HIP kernels of libgla.so.  torch provides
device memory (tensors) and the stream (torch's current stream on the tensors' device).
There is no CPU fallback: without the built library every call raises.

Low-level calls carry the C names (gla_chunk_fwd, gla_segment_scan, gla_segment_correct,
gla_chunk_bwd, and for the other order gla_chunk_state, gla_chunk_fwd_from, gla_chunk_dstate,
gla_chunk_bwd_from).  ``zeco_forward`` / ``zeco_backward`` chain them in the order of the method:
local pass -> segment scan -> correction, and the same for the backward.
``states_first_forward`` / ``states_first_backward`` chain the same decomposition with the
segments' incoming states first: state pass -> segment scan -> local pass from the true incoming
state, with no correction pass (cheaper where the decay is weak and the corrections would reach
every chunk).  All four take a join (gla_join_fwd / gla_join_bwd): the block's output norm, gate,
residual and the next block's norm.

The other operators of a recurrent block: gla_recur_fwd, gla_recur_bwd (elementwise gated linear
recurrence), gla_step and gla_recur_step (single tokens on a pool of states), gla_delta_fwd,
gla_delta_bwd and gla_delta_step (gated delta rule), gla_layernorm_fwd and gla_layernorm_bwd.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import threading

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgla.so")
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gla.h")

GLA_OK, GLA_ERR_INVALID_ARG, GLA_ERR_UNSUPPORTED, GLA_ERR_HIP = 0, 1, 2, 3
GLA_F32, GLA_BF16 = 0, 1
GLA_FWD, GLA_BWD = 0, 1
RECUR_MODES = {"plain": 0, "lerp": 1, "norm": 2}
RECUR_CHUNK = 128
ACTS = {"silu": 0, "sigmoid": 1}

_lib = None
_lock = threading.Lock()


class GLAError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def load_library(path: str = LIB_PATH):
    """Open libgla.so and declare the C signatures.  Raises if the library is not built."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    with _lock:
        if _lib is not None and path == LIB_PATH:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError("libgla.so is not built (%s); run `python -m sequence_state_scan_amd.build`" % path)
        lib = ctypes.CDLL(path)
        vp, fp, i = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
        lib.gla_supported.argtypes = [i, i, i, i]
        lib.gla_supported.restype = i
        lib.gla_status_string.argtypes = [i]
        lib.gla_status_string.restype = ctypes.c_char_p
        lib.gla_last_error.argtypes = []
        lib.gla_last_error.restype = ctypes.c_char_p
        sz = ctypes.c_size_t
        lib.gla_workspace_size.argtypes = [i] * 9
        lib.gla_workspace_size.restype = sz
        lib.gla_chunk_fwd.argtypes = [vp, vp, vp, fp, vp, vp, fp, fp] + [i] * 8 + [vp, sz, vp]
        lib.gla_chunk_fwd.restype = i
        lib.gla_chunk_fwd_noalloc.argtypes = [vp, vp, vp, fp, vp, vp, fp, fp] + [i] * 8 + [vp]
        lib.gla_chunk_fwd_noalloc.restype = i
        lib.gla_segment_scan.argtypes = [fp, fp, fp, fp, fp] + [i] * 7 + [vp]
        lib.gla_segment_scan.restype = i
        lib.gla_segment_scan_allgather.argtypes = [fp, fp, fp, fp, fp] + [i] * 6 + [vp]
        lib.gla_segment_scan_allgather.restype = i
        lib.gla_segment_correct.argtypes = [i, vp, vp, vp, fp, fp, fp, vp, vp, vp, vp, fp] + [i] * 8 + [vp]
        lib.gla_segment_correct.restype = i
        lib.gla_chunk_bwd.argtypes = [vp, vp, vp, fp, vp, vp, fp, vp, vp, vp, fp, fp] + [i] * 8 + [vp, sz, vp]
        lib.gla_chunk_bwd.restype = i
        lib.gla_chunk_state.argtypes = [vp, vp, fp, fp, fp] + [i] * 8 + [vp, sz, vp]
        lib.gla_chunk_state.restype = i
        lib.gla_chunk_fwd_from.argtypes = [vp, vp, vp, fp, fp, vp, vp] + [i] * 8 + [vp, sz, vp]
        lib.gla_chunk_fwd_from.restype = i
        lib.gla_chunk_dstate.argtypes = [vp, fp, vp, fp] + [i] * 8 + [vp, sz, vp]
        lib.gla_chunk_dstate.restype = i
        lib.gla_chunk_bwd_from.argtypes = [vp, vp, vp, fp, vp, vp, fp, fp, vp, vp, vp, fp] + [i] * 8 + [vp, sz, vp]
        lib.gla_chunk_bwd_from.restype = i
        fl = ctypes.c_float
        lib.gla_recur_workspace_size.argtypes = [i] * 3
        lib.gla_recur_workspace_size.restype = sz
        lib.gla_recur_fwd.argtypes = [vp] * 9 + [i] * 5 + [vp, sz, vp]
        lib.gla_recur_fwd.restype = i
        lib.gla_recur_bwd.argtypes = [vp] * 12 + [i] * 5 + [vp, sz, vp]
        lib.gla_recur_bwd.restype = i
        lib.gla_recur_step.argtypes = [vp] * 7 + [i] * 5 + [vp]
        lib.gla_recur_step.restype = i
        lib.gla_step.argtypes = [vp] * 11 + [i] * 7 + [vp]
        lib.gla_step.restype = i
        lib.gla_join_workspace_size.argtypes = [i] * 4
        lib.gla_join_workspace_size.restype = sz
        lib.gla_join_fwd.argtypes = [vp] * 13 + [i] * 5 + [fl, i, i, vp]
        lib.gla_join_fwd.restype = i
        lib.gla_join_bwd.argtypes = [vp] * 21 + [i] * 7 + [vp, sz, vp]
        lib.gla_join_bwd.restype = i
        lib.gla_delta_workspace_size.argtypes = [i] * 8
        lib.gla_delta_workspace_size.restype = sz
        lib.gla_delta_saved_size.argtypes = [i] * 7
        lib.gla_delta_saved_size.restype = sz
        lib.gla_delta_fwd.argtypes = [vp] * 15 + [sz] + [i] * 7 + [vp, sz, vp]
        lib.gla_delta_fwd.restype = i
        lib.gla_delta_bwd.argtypes = [vp] * 14 + [sz] + [vp] * 8 + [i] * 7 + [vp, sz, vp]
        lib.gla_delta_bwd.restype = i
        lib.gla_delta_step.argtypes = [vp] * 13 + [i] * 8 + [vp]
        lib.gla_delta_step.restype = i
        lib.gla_layernorm_workspace_size.argtypes = [i] * 3
        lib.gla_layernorm_workspace_size.restype = sz
        lib.gla_layernorm_fwd.argtypes = [vp] * 10 + [i] * 3 + [fl, i, i, vp]
        lib.gla_layernorm_fwd.restype = i
        lib.gla_layernorm_bwd.argtypes = [vp] * 15 + [i] * 5 + [vp, sz, vp]
        lib.gla_layernorm_bwd.restype = i
        if path == LIB_PATH:
            _lib = lib
        return lib


def declared_functions(header: str = HEADER):
    """Names of the functions include/gla.h declares."""
    text = open(header).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][\w\s\*]*?\b(gla_\w+)\s*\(", text, re.M)))


def supported(dtype: torch.dtype, dk: int, dv: int, chunk: int) -> bool:
    return bool(load_library().gla_supported(_dtype_code(dtype), dk, dv, chunk))


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return GLA_BF16
    if dt == torch.float32:
        return GLA_F32
    raise TypeError("q, k, v must be torch.bfloat16 or torch.float32, got %s" % dt)


def _check(status: int):
    if status != GLA_OK:
        lib = load_library()
        raise GLAError(status, "%s: %s" % (lib.gla_status_string(status).decode(), lib.gla_last_error().decode()))


def _p(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libgla works on device tensors only (got a %s tensor)" % t.device)
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _f32(t, name):
    if t is not None and t.dtype != torch.float32:
        raise TypeError("%s must be float32" % name)
    return _p(t)


def _expect(t, name, shape, dtype, device, optional=False):
    """Check one tensor argument against the shape, dtype and device the call implies.  The
    kernels index every buffer from (B, H, T, dk, dv, P, chunk) alone, so a mismatch here would
    read or write outside the buffer: it is rejected before anything reaches the library."""
    if t is None:
        if optional:
            return
        raise ValueError("%s is required" % name)
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _stream(t):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _dims(q, v):
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q and v must be [B, H, T, d] tensors")
    B, H, T, dk = q.shape
    return B, H, T, dk, v.shape[-1]


def _head_args(q, k, v, g, extra=()):
    """(B, H, T, dk, dv) from q and v, after checking q, k, v, g and the (name, tensor, last dim)
    triples of ``extra`` that share their [B, H, T] layout."""
    B, H, T, dk, dv = _dims(q, v)
    if not q.is_cuda:
        raise ValueError("libgla works on device tensors only (got a %s tensor)" % q.device)
    _dtype_code(q.dtype)
    _expect(q, "q", (B, H, T, dk), q.dtype, q.device)
    _expect(k, "k", (B, H, T, dk), q.dtype, q.device)
    _expect(v, "v", (B, H, T, dv), q.dtype, q.device)
    _expect(g, "g", (B, H, T, dk), torch.float32, q.device)
    for name, t, d, dt in extra:
        _expect(t, name, (B, H, T, d), dt, q.device)
    return B, H, T, dk, dv


def workspace_size(which: int, B: int, H: int, T: int, dk: int, dv: int, chunk: int, P: int, dtype) -> int:
    """Bytes of workspace gla_chunk_fwd (which=GLA_FWD) or gla_chunk_bwd (GLA_BWD) needs."""
    lib = load_library()
    n = lib.gla_workspace_size(which, B, H, T, dk, dv, chunk, P, _dtype_code(dtype))
    if n == 0:
        raise GLAError(GLA_ERR_INVALID_ARG, "gla_workspace_size: %s" % lib.gla_last_error().decode())
    return int(n)


def flags_workspace_size(B: int, H: int, P: int) -> int:
    """The smallest workspace gla_chunk_fwd / gla_chunk_bwd accept (include/gla.h,
    gla_workspace_size): one int per unit (b, h, segment), rounded up to 256 bytes.  With it a call
    cuts no segment into sub-segments and runs the units it flags whole (no re-split)."""
    return (B * H * P * 4 + 255) // 256 * 256


def _workspace(ws, which, B, H, T, dk, dv, chunk, P, dtype, device):
    """The caller's workspace, or one of the size for the fastest schedule.  A smaller one is the
    library's to accept (no re-split, fewer sub-segments) or reject, before any HIP call."""
    if ws is None:
        ws = torch.empty(workspace_size(which, B, H, T, dk, dv, chunk, P, dtype), dtype=torch.uint8, device=device)
    if not isinstance(ws, torch.Tensor) or ws.device != device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % device)
    return ws, ws.numel() * ws.element_size()


# ------------------------------------------------------------------------------------ C calls

def chunk_states_dense(cs):
    """View of chunk states in the tiled layout of include/gla.h as ordinary row-major [dk][dv]
    states (a copy; for inspection and tests, not used by any entry point)."""
    *lead, dk, dv = cs.shape
    L = len(lead)
    if (dv // 16) % 2 == 1:
        t = cs.reshape(*lead, dk // 16, dv // 16, 4, 16, 4)  # tile row, tile column, j / 4, c, j % 4
        return t.permute(*range(L), L, L + 3, L + 1, L + 2, L + 4).reshape(*lead, dk, dv)
    # tile row, pair of tile columns, j / 4 within the tile, c, tile of the pair, j % 4
    t = cs.reshape(*lead, dk // 16, dv // 32, 4, 16, 2, 4)
    return t.permute(*range(L), L, L + 3, L + 1, L + 4, L + 2, L + 5).reshape(*lead, dk, dv)


def _seg_shapes(B, H, T, dk, dv, chunk, P):
    if P < 1 or chunk < 1 or T % P != 0 or (T // P) % chunk != 0:
        raise ValueError("T=%d must split into P=%d segments of whole chunks of %d tokens" % (T, P, chunk))
    return (B, H, T // chunk, dk, dv), (B, H, P, dk, dv), (B, H, P, dk)


def gla_chunk_fwd(q, k, v, g, chunk: int, P: int, o=None, chunk_states=None, seg_state=None, seg_logdecay=None,
                  workspace=None, keep_chunk_states: bool = True):
    """Local pass.  Returns (o_local, chunk_states [B,H,T/chunk,dk,dv] (local, q's dtype, each
    state in the tiled layout: chunk_states_dense gives the row-major view),
    seg_state [B,H,P,dk,dv], seg_logdecay [B,H,P,dk]).  ``workspace`` (a device tensor of at
    least workspace_size(GLA_FWD, ...) bytes) is allocated when not given.
    keep_chunk_states=False (a forward-only caller: no backward follows) keeps no per-chunk states
    and returns None in their place; the other results are the same bit for bit."""
    B, H, T, dk, dv = _head_args(q, k, v, g)
    cs_shape, st_shape, ld_shape = _seg_shapes(B, H, T, dk, dv, chunk, P)
    dev, f32 = q.device, torch.float32
    o = torch.empty_like(v) if o is None else o
    if not keep_chunk_states:
        if chunk_states is not None:
            raise ValueError("chunk_states given with keep_chunk_states=False")
    elif chunk_states is None:
        chunk_states = torch.empty(cs_shape, device=dev, dtype=q.dtype)
    if seg_state is None:
        seg_state = torch.empty(st_shape, device=dev, dtype=f32)
    if seg_logdecay is None:
        seg_logdecay = torch.empty(ld_shape, device=dev, dtype=f32)
    _expect(o, "o", (B, H, T, dv), q.dtype, dev)
    _expect(chunk_states, "chunk_states", cs_shape, q.dtype, dev, optional=not keep_chunk_states)
    _expect(seg_state, "seg_state", st_shape, f32, dev)
    _expect(seg_logdecay, "seg_logdecay", ld_shape, f32, dev)
    ws, nbytes = _workspace(workspace, GLA_FWD, B, H, T, dk, dv, chunk, P, q.dtype, dev)
    _check(load_library().gla_chunk_fwd(_p(q), _p(k), _p(v), _p(g), _p(o), _p(chunk_states), _p(seg_state),
                                        _p(seg_logdecay), B, H, T, dk, dv, chunk, P, _dtype_code(q.dtype),
                                        _p(ws), nbytes, _stream(q)))
    return o, chunk_states, seg_state, seg_logdecay


def gla_chunk_fwd_noalloc(q, k, v, g, chunk: int, P: int, o, chunk_states, seg_state, seg_logdecay):
    """gla_chunk_fwd without a workspace (the library's static one): every output is the caller's
    and must be given (chunk_states may be None: no per-chunk states kept); nothing is allocated."""
    B, H, T, dk, dv = _head_args(q, k, v, g)
    cs_shape, st_shape, ld_shape = _seg_shapes(B, H, T, dk, dv, chunk, P)
    dev, f32 = q.device, torch.float32
    _expect(o, "o", (B, H, T, dv), q.dtype, dev)
    _expect(chunk_states, "chunk_states", cs_shape, q.dtype, dev, optional=True)
    _expect(seg_state, "seg_state", st_shape, f32, dev)
    _expect(seg_logdecay, "seg_logdecay", ld_shape, f32, dev)
    _check(load_library().gla_chunk_fwd_noalloc(_p(q), _p(k), _p(v), _p(g), _p(o), _p(chunk_states), _p(seg_state),
                                                _p(seg_logdecay), B, H, T, dk, dv, chunk, P, _dtype_code(q.dtype),
                                                _stream(q)))
    return o, chunk_states, seg_state, seg_logdecay


def _scan_args(seg_state, seg_logdecay, h_boundary, seg_carry, h_out, want_h_out):
    if not isinstance(seg_state, torch.Tensor) or seg_state.dim() != 5:
        raise ValueError("seg_state must be a [B, H, P, dk, dv] tensor")
    B, H, P, dk, dv = seg_state.shape
    dev, f32 = seg_state.device, torch.float32
    _expect(seg_state, "seg_state", (B, H, P, dk, dv), f32, dev)
    _expect(seg_logdecay, "seg_logdecay", (B, H, P, dk), f32, dev)
    _expect(h_boundary, "h_boundary", (B, H, dk, dv), f32, dev, optional=True)
    seg_carry = torch.empty_like(seg_state) if seg_carry is None else seg_carry
    _expect(seg_carry, "seg_carry", (B, H, P, dk, dv), f32, dev)
    if h_out is None and want_h_out:
        h_out = torch.empty((B, H, dk, dv), device=dev, dtype=f32)
    _expect(h_out, "h_out", (B, H, dk, dv), f32, dev, optional=True)
    return B, H, P, dk, dv, seg_carry, h_out


def gla_segment_scan(seg_state, seg_logdecay, K: int, h_boundary=None, reverse: bool = False,
                     seg_carry=None, h_out=None, want_h_out: bool = True):
    """Decay-and-add scan over segments.  Returns (seg_carry, h_out)."""
    B, H, P, dk, dv, seg_carry, h_out = _scan_args(seg_state, seg_logdecay, h_boundary, seg_carry, h_out, want_h_out)
    _check(load_library().gla_segment_scan(_f32(seg_state, "seg_state"), _f32(seg_logdecay, "seg_logdecay"),
                                           _f32(h_boundary, "h_boundary"), _f32(seg_carry, "seg_carry"),
                                           _f32(h_out, "h_out"), B, H, P, dk, dv, K, int(bool(reverse)),
                                           _stream(seg_state)))
    return seg_carry, h_out


def gla_segment_scan_allgather(seg_state, seg_logdecay, h_boundary=None, reverse: bool = False,
                               seg_carry=None, h_out=None, want_h_out: bool = True):
    """The same scan in the all-gather order (every carry combined directly from all the local
    states it depends on).  Returns (seg_carry, h_out)."""
    B, H, P, dk, dv, seg_carry, h_out = _scan_args(seg_state, seg_logdecay, h_boundary, seg_carry, h_out, want_h_out)
    _check(load_library().gla_segment_scan_allgather(_f32(seg_state, "seg_state"), _f32(seg_logdecay, "seg_logdecay"),
                                                     _f32(h_boundary, "h_boundary"), _f32(seg_carry, "seg_carry"),
                                                     _f32(h_out, "h_out"), B, H, P, dk, dv, int(bool(reverse)),
                                                     _stream(seg_state)))
    return seg_carry, h_out


def _scan(method: str, seg_state, seg_logdecay, K: int, h_boundary, reverse: bool):
    if method == "chain":
        return gla_segment_scan(seg_state, seg_logdecay, K, h_boundary=h_boundary, reverse=reverse)
    if method == "allgather":
        return gla_segment_scan_allgather(seg_state, seg_logdecay, h_boundary=h_boundary, reverse=reverse)
    raise ValueError("unknown scan method %r" % method)


def gla_segment_correct(mode: int, chunk: int, P: int, q=None, k=None, v=None, g=None, seg_in=None,
                        seg_grad=None, o=None, chunk_states=None, dk=None, dv=None, dg=None):
    """Cumulative-decay correction, in place: o and chunk_states for GLA_FWD; dk, dv, dg for
    GLA_BWD (which reads the global chunk_states)."""
    if mode not in (GLA_FWD, GLA_BWD):
        raise ValueError("mode must be GLA_FWD or GLA_BWD")
    ref_k = q if mode == GLA_FWD else k
    ref_v = o if mode == GLA_FWD else dv
    if ref_k is None or ref_v is None:
        raise ValueError("GLA_FWD needs q and o, GLA_BWD needs k and dv")
    B, H, T, d_k, d_v = _dims(ref_k, ref_v)
    dt, dev, f32 = ref_k.dtype, ref_k.device, torch.float32
    cs_shape, st_shape, _ = _seg_shapes(B, H, T, d_k, d_v, chunk, P)
    _expect(g, "g", (B, H, T, d_k), f32, dev)
    _expect(seg_in, "seg_in", st_shape, f32, dev)
    # GLA_FWD may go without chunk states (a forward-only caller kept none)
    _expect(chunk_states, "chunk_states", cs_shape, dt, dev, optional=mode == GLA_FWD)
    if mode == GLA_FWD:
        _expect(q, "q", (B, H, T, d_k), dt, dev)
        _expect(o, "o", (B, H, T, d_v), dt, dev)
    else:
        for name, t, d in (("k", k, d_k), ("v", v, d_v), ("dk", dk, d_k), ("dv", dv, d_v)):
            _expect(t, name, (B, H, T, d), dt, dev)
        _expect(dg, "dg", (B, H, T, d_k), f32, dev)
        _expect(seg_grad, "seg_grad", st_shape, f32, dev)
    _check(load_library().gla_segment_correct(mode, _p(q), _p(k), _p(v), _f32(g, "g"), _f32(seg_in, "seg_in"),
                                              _f32(seg_grad, "seg_grad"), _p(o), _p(chunk_states), _p(dk), _p(dv),
                                              _f32(dg, "dg"), B, H, T, d_k, d_v, chunk, P,
                                              _dtype_code(ref_k.dtype), _stream(ref_k)))


def gla_chunk_bwd(q, k, v, g, do, chunk_states, seg_in, chunk: int, P: int, dq=None, dk=None, dv=None,
                  dg=None, seg_dstate=None, workspace=None):
    """Backward of every segment given the global chunk states and incoming segment states.

    Returns (dq global, dk local, dv local, dg local, seg_dstate [B,H,P,dk,dv]).  ``workspace`` as
    in gla_chunk_fwd (GLA_BWD size)."""
    B, H, T, d_k, d_v = _head_args(q, k, v, g, (("do", do, v.shape[-1], q.dtype),))
    cs_shape, st_shape, _ = _seg_shapes(B, H, T, d_k, d_v, chunk, P)
    dev, f32 = q.device, torch.float32
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    dg = torch.empty_like(g) if dg is None else dg
    if seg_dstate is None:
        seg_dstate = torch.empty(st_shape, device=dev, dtype=f32)
    _expect(chunk_states, "chunk_states", cs_shape, q.dtype, dev)
    _expect(seg_in, "seg_in", st_shape, f32, dev)
    for name, t, d in (("dq", dq, d_k), ("dk", dk, d_k), ("dv", dv, d_v)):
        _expect(t, name, (B, H, T, d), q.dtype, dev)
    _expect(dg, "dg", (B, H, T, d_k), f32, dev)
    _expect(seg_dstate, "seg_dstate", st_shape, f32, dev)
    ws, nbytes = _workspace(workspace, GLA_BWD, B, H, T, d_k, d_v, chunk, P, q.dtype, dev)
    _check(load_library().gla_chunk_bwd(_p(q), _p(k), _p(v), _p(g), _p(do), _p(chunk_states), _p(seg_in),
                                        _p(dq), _p(dk), _p(dv), _p(dg), _p(seg_dstate), B, H, T, d_k, d_v, chunk,
                                        P, _dtype_code(q.dtype), _p(ws), nbytes, _stream(q)))
    return dq, dk, dv, dg, seg_dstate


def _seg_args(name_a, a, v, g, extra=()):
    """(B, H, T, dk, dv) for the state passes, whose inputs are a ([B,H,T,dk]: k or q), v or do
    ([B,H,T,dv]) and g, after checking them and ``extra``'s (name, tensor, last dim, dtype)."""
    if not isinstance(a, torch.Tensor) or not isinstance(v, torch.Tensor) or a.dim() != 4 or v.dim() != 4:
        raise ValueError("%s and the value-side input must be [B, H, T, d] tensors" % name_a)
    B, H, T, dk = a.shape
    dv = v.shape[-1]
    if not a.is_cuda:
        raise ValueError("libgla works on device tensors only (got a %s tensor)" % a.device)
    _dtype_code(a.dtype)
    _expect(a, name_a, (B, H, T, dk), a.dtype, a.device)
    _expect(g, "g", (B, H, T, dk), torch.float32, a.device)
    for name, t, d, dt in extra:
        _expect(t, name, (B, H, T, d), dt, a.device)
    return B, H, T, dk, dv


def gla_chunk_state(k, v, g, chunk: int, P: int, seg_state=None, seg_logdecay=None, workspace=None):
    """State pass: each segment's local end state and summed log-gates from a zero start (reads k,
    v, g only).  Returns (seg_state [B,H,P,dk,dv], seg_logdecay [B,H,P,dk]), the same quantities as
    gla_chunk_fwd's.  ``workspace`` (GLA_FWD size) lets it cut segments into sub-segments."""
    B, H, T, dk, dv = _seg_args("k", k, v, g, (("v", v, v.shape[-1], k.dtype),))
    _, st_shape, ld_shape = _seg_shapes(B, H, T, dk, dv, chunk, P)
    dev, f32 = k.device, torch.float32
    seg_state = torch.empty(st_shape, device=dev, dtype=f32) if seg_state is None else seg_state
    seg_logdecay = torch.empty(ld_shape, device=dev, dtype=f32) if seg_logdecay is None else seg_logdecay
    _expect(seg_state, "seg_state", st_shape, f32, dev)
    _expect(seg_logdecay, "seg_logdecay", ld_shape, f32, dev)
    ws, nbytes = _workspace(workspace, GLA_FWD, B, H, T, dk, dv, chunk, P, k.dtype, dev)
    _check(load_library().gla_chunk_state(_p(k), _p(v), _p(g), _p(seg_state), _p(seg_logdecay), B, H, T, dk, dv,
                                          chunk, P, _dtype_code(k.dtype), _p(ws), nbytes, _stream(k)))
    return seg_state, seg_logdecay


def gla_chunk_fwd_from(q, k, v, g, seg_in, chunk: int, P: int, o=None, chunk_states=None, workspace=None,
                       keep_chunk_states: bool = True):
    """Local pass with every segment starting from its true incoming state seg_in [B,H,P,dk,dv]
    (the forward scan's carry): returns (o, chunk_states), both GLOBAL; no correction follows.
    chunk_states (tiled layout) is None with keep_chunk_states=False."""
    B, H, T, dk, dv = _head_args(q, k, v, g)
    cs_shape, st_shape, _ = _seg_shapes(B, H, T, dk, dv, chunk, P)
    dev = q.device
    o = torch.empty_like(v) if o is None else o
    if not keep_chunk_states:
        if chunk_states is not None:
            raise ValueError("chunk_states given with keep_chunk_states=False")
    elif chunk_states is None:
        chunk_states = torch.empty(cs_shape, device=dev, dtype=q.dtype)
    _expect(seg_in, "seg_in", st_shape, torch.float32, dev)
    _expect(o, "o", (B, H, T, dv), q.dtype, dev)
    _expect(chunk_states, "chunk_states", cs_shape, q.dtype, dev, optional=not keep_chunk_states)
    ws, nbytes = _workspace(workspace, GLA_FWD, B, H, T, dk, dv, chunk, P, q.dtype, dev)
    _check(load_library().gla_chunk_fwd_from(_p(q), _p(k), _p(v), _p(g), _p(seg_in), _p(o), _p(chunk_states), B, H,
                                             T, dk, dv, chunk, P, _dtype_code(q.dtype), _p(ws), nbytes, _stream(q)))
    return o, chunk_states


def gla_chunk_dstate(q, g, do, chunk: int, P: int, seg_dstate=None, workspace=None):
    """State-gradient pass: each segment's gradient w.r.t. its incoming state from its own outputs
    (reads q, g, do only).  Returns seg_dstate [B,H,P,dk,dv], the same quantity as gla_chunk_bwd's.
    ``workspace`` (GLA_BWD size) lets it cut segments into sub-segments."""
    B, H, T, dk, dv = _seg_args("q", q, do, g, (("do", do, do.shape[-1], q.dtype),))
    _, st_shape, _ = _seg_shapes(B, H, T, dk, dv, chunk, P)
    dev = q.device
    seg_dstate = torch.empty(st_shape, device=dev, dtype=torch.float32) if seg_dstate is None else seg_dstate
    _expect(seg_dstate, "seg_dstate", st_shape, torch.float32, dev)
    ws, nbytes = _workspace(workspace, GLA_BWD, B, H, T, dk, dv, chunk, P, q.dtype, dev)
    _check(load_library().gla_chunk_dstate(_p(q), _p(g), _p(do), _p(seg_dstate), B, H, T, dk, dv, chunk, P,
                                           _dtype_code(q.dtype), _p(ws), nbytes, _stream(q)))
    return seg_dstate


def gla_chunk_bwd_from(q, k, v, g, do, chunk_states, seg_in, seg_grad, chunk: int, P: int, dq=None, dk=None,
                       dv=None, dg=None, workspace=None):
    """Backward of every segment starting from seg_grad [B,H,P,dk,dv] (the reverse scan's carry)
    at its end, given the global chunk states and incoming states: returns (dq, dk, dv, dg), all
    GLOBAL; no correction follows."""
    B, H, T, d_k, d_v = _head_args(q, k, v, g, (("do", do, v.shape[-1], q.dtype),))
    cs_shape, st_shape, _ = _seg_shapes(B, H, T, d_k, d_v, chunk, P)
    dev, f32 = q.device, torch.float32
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    dg = torch.empty_like(g) if dg is None else dg
    _expect(chunk_states, "chunk_states", cs_shape, q.dtype, dev)
    _expect(seg_in, "seg_in", st_shape, f32, dev)
    _expect(seg_grad, "seg_grad", st_shape, f32, dev)
    for name, t, d in (("dq", dq, d_k), ("dk", dk, d_k), ("dv", dv, d_v)):
        _expect(t, name, (B, H, T, d), q.dtype, dev)
    _expect(dg, "dg", (B, H, T, d_k), f32, dev)
    ws, nbytes = _workspace(workspace, GLA_BWD, B, H, T, d_k, d_v, chunk, P, q.dtype, dev)
    _check(load_library().gla_chunk_bwd_from(_p(q), _p(k), _p(v), _p(g), _p(do), _p(chunk_states), _p(seg_in),
                                             _p(seg_grad), _p(dq), _p(dk), _p(dv), _p(dg), B, H, T, d_k, d_v, chunk,
                                             P, _dtype_code(q.dtype), _p(ws), nbytes, _stream(q)))
    return dq, dk, dv, dg


# --------------------------------------------------------------- a recurrent block's other operators

def _view(t, name, shape, dtype, device):
    """(pointer, strides) of an input that may be a view with a contiguous last dimension, after
    checking it as _expect does; strides are None for a contiguous tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _expect(t, name, shape, dtype, device)
    if t.is_contiguous():
        return t.data_ptr(), None
    st = t.stride()
    if st[-1] != 1 and shape[-1] != 1:
        raise ValueError("%s must be contiguous in its last dimension (strides %s)" % (name, st))
    if len(st) == 4:
        return t.data_ptr(), (ctypes.c_longlong * 3)(st[0], st[1], st[2])
    return t.data_ptr(), (ctypes.c_longlong * 3)(st[0], 0, st[1] if len(st) == 3 else 0)


def _out(t, name, shape, dtype, device, optional=False):
    """Pointer of a contiguous tensor (None for an optional one that is not given), checked."""
    if t is None and optional:
        return None
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != dtype or t.device != device or \
            not t.is_contiguous():
        _expect(t, name, shape, dtype, device)  # says which
    return t.data_ptr()


def _new(t, name, shape, dtype, device, like=None):
    """(tensor, pointer) of an output: the caller's, checked, or a new one (made like a tensor of its
    shape where there is one: the quickest way to an empty tensor)."""
    if t is None:
        if like is None:
            t = torch.empty(shape, dtype=dtype, device=device)
        else:
            t = torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
        return t, t.data_ptr()
    return t, _out(t, name, shape, dtype, device)


def _on_gpu(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("libgla works on device tensors only (got a %s tensor)" % t.device)


def _code(table, key, name):
    if key not in table:
        raise ValueError("unknown %s %r (one of %s)" % (name, key, ", ".join(sorted(table))))
    return table[key]


def _raw_stream(index):
    """hipStream_t of torch's current stream on device ``index``."""
    return torch.cuda.current_stream(index).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):  # the same number without the Stream object around it
    _raw_stream = torch._C._cuda_getCurrentRawStream


def _launch(fn, device, *args):
    """The C call on torch's current stream of ``device``, with that device current (a kernel is
    launched on the current one)."""
    stream = _raw_stream(device.index)
    if torch.cuda.current_device() == device.index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status != GLA_OK:
        _check(status)


@functools.lru_cache(maxsize=4096)
def recur_workspace_size(B: int, T: int, D: int) -> int:
    """Bytes of workspace gla_recur_fwd and gla_recur_bwd need (0: none)."""
    lib = load_library()
    n = lib.gla_recur_workspace_size(B, T, D)
    if n == 0 and lib.gla_last_error():
        raise GLAError(GLA_ERR_INVALID_ARG, lib.gla_last_error().decode())
    return int(n)


@functools.lru_cache(maxsize=4096)
def join_workspace_size(B: int, H: int, T: int, d: int) -> int:
    """Bytes of workspace gla_join_bwd needs for the weights' gradients."""
    lib = load_library()
    n = lib.gla_join_workspace_size(B, H, T, d)
    if n == 0:
        raise GLAError(GLA_ERR_INVALID_ARG, lib.gla_last_error().decode())
    return int(n)


def _scratch(ws, need, device):
    """(tensor to keep alive, pointer, bytes) of a workspace: the caller's, or one of ``need`` bytes."""
    if ws is None:
        if need == 0:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    if not isinstance(ws, torch.Tensor) or ws.device != device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % device)
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _recur_dims(x):
    _on_gpu(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be a [B, T, D] tensor")
    return x.shape


def gla_recur_fwd(x, g, h0=None, lens=None, mode: str = "plain", h=None, chunk_in=None, h_final=None, workspace=None,
                  keep_chunk_states: bool = True):
    """Elementwise gated linear recurrence h_t = exp(g_t) h_{t-1} + beta(g_t) x_t over x [B, T, D]
    (bf16 or float32) and log-gates g [B, T, D] (float32, <= 0, or -inf for a reset), from h0
    [B, D] (float32, default zero).  mode: the input's factor beta, "plain" (1), "lerp" (1 - a) or
    "norm" (sqrt(1 - a^2)).  lens: int32 [B], the sequences' lengths in a padded batch (h is zero
    behind them).  x and g may be views whose last dimension is contiguous.
    Returns (h [B, T, D] in x's dtype, chunk_in [B, ceil(T/128), D], h_final [B, D], float32).
    chunk_in is what gla_recur_bwd rebuilds the states from; None with keep_chunk_states=False."""
    B, T, D = _recur_dims(x)
    dev, f32 = x.device, torch.float32
    m, dt = _code(RECUR_MODES, mode, "mode"), _dtype_code(x.dtype)
    xp, xs = _view(x, "x", (B, T, D), x.dtype, dev)
    gp, gs = _view(g, "g", (B, T, D), f32, dev)
    h0p = _out(h0, "h0", (B, D), f32, dev, optional=True)
    lp = _out(lens, "lens", (B,), torch.int32, dev, optional=True)
    h, hp = _new(h, "h", (B, T, D), x.dtype, dev, x)
    h_final, fp = _new(h_final, "h_final", (B, D), f32, dev, h0)
    cp = None
    if keep_chunk_states:
        chunk_in, cp = _new(chunk_in, "chunk_in", (B, (T + RECUR_CHUNK - 1) // RECUR_CHUNK, D), f32, dev)
    elif chunk_in is not None:
        raise ValueError("chunk_in given with keep_chunk_states=False")
    workspace, wp, wn = _scratch(workspace, recur_workspace_size(B, T, D), dev)
    _launch(load_library().gla_recur_fwd, dev, xp, xs, gp, gs, h0p, lp, hp, cp, fp, B, T, D, m, dt, wp, wn)
    return h, chunk_in, h_final


def gla_recur_bwd(x, g, dh, chunk_in, lens=None, dhT=None, mode: str = "plain", dx=None, dg=None, dh0=None,
                  workspace=None):
    """Gradients of gla_recur_fwd for dh [B, T, D] (the gradient of h, x's dtype) and dhT [B, D]
    (of h_final, float32, default zero), over the forward's x, g, lens, mode and the chunk_in it
    returned.  Returns (dx [B, T, D] in x's dtype, dg [B, T, D], dh0 [B, D], float32)."""
    B, T, D = _recur_dims(x)
    dev, f32 = x.device, torch.float32
    m, dt = _code(RECUR_MODES, mode, "mode"), _dtype_code(x.dtype)
    xp, xs = _view(x, "x", (B, T, D), x.dtype, dev)
    gp, gs = _view(g, "g", (B, T, D), f32, dev)
    dp, ds = _view(dh, "dh", (B, T, D), x.dtype, dev)
    cp = _out(chunk_in, "chunk_in", (B, (T + RECUR_CHUNK - 1) // RECUR_CHUNK, D), f32, dev)
    lp = _out(lens, "lens", (B,), torch.int32, dev, optional=True)
    tp = _out(dhT, "dhT", (B, D), f32, dev, optional=True)
    dx, dxp = _new(dx, "dx", (B, T, D), x.dtype, dev, x)
    dg, dgp = _new(dg, "dg", (B, T, D), f32, dev, g)
    dh0, d0p = _new(dh0, "dh0", (B, D), f32, dev, dhT)
    workspace, wp, wn = _scratch(workspace, recur_workspace_size(B, T, D), dev)
    _launch(load_library().gla_recur_bwd, dev, xp, xs, gp, gs, dp, ds, cp, lp, tp, dxp, dgp, d0p, B, T, D, m, dt, wp, wn)
    return dx, dg, dh0


def _pool(state, slots, B, shape, dev):
    """(pointer of the pool, pointer of the slots, states in the pool), checked."""
    if not isinstance(state, torch.Tensor) or state.dim() != len(shape) + 1:
        raise ValueError("state must be a [slots%s] tensor" % "".join(", %d" % n for n in shape))
    n = state.shape[0]
    sp = _out(state, "state", (n,) + shape, torch.float32, dev)
    if slots is None and n < B:
        raise ValueError("state holds %d states, the batch has %d rows" % (n, B))
    return sp, _out(slots, "slots", (B,), torch.int32, dev, optional=True), n


def gla_recur_step(x, g, state, slots=None, mode: str = "plain", h=None):
    """One token of gla_recur_fwd for every row of x [B, D], in place on the pool ``state``
    [n_slots, D] (float32): row b's state is state[slots[b]] (slots int32; default state[b]).  A
    negative slot leaves its row out (h is zero there); a slot outside the pool, or one that an
    earlier row names, gives NaN and touches no state.  Returns h [B, D] in x's dtype."""
    _on_gpu(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be a [B, D] tensor")
    B, D = x.shape
    dev = x.device
    m, dt = _code(RECUR_MODES, mode, "mode"), _dtype_code(x.dtype)
    xp, xs = _view(x, "x", (B, D), x.dtype, dev)
    gp, gs = _view(g, "g", (B, D), torch.float32, dev)
    sp, ip, n = _pool(state, slots, B, (D,), dev)
    h, hp = _new(h, "h", (B, D), x.dtype, dev, x)
    _launch(load_library().gla_recur_step, dev, xp, xs, gp, gs, sp, ip, hp, B, D, n, m, dt)
    return h


def gla_step(q, k, v, g, state, slots=None, o=None):
    """The next n tokens of gated linear attention for every row of a batch (n = 1: decoding), in
    place on the pool ``state`` [n_slots, H, dk, dv] (float32; a forward chain's h_final is B such
    states): q, k [B, H, n, dk], v [B, H, n, dv] (bf16 or float32), g [B, H, n, dk] (float32).
    Row b's state is state[slots[b]], with the rules of gla_recur_step.  q, k, v and g may be views
    whose last dimension is contiguous.  dk <= 256.  Returns o [B, H, n, dv]."""
    _on_gpu(q, "q")
    if q.dim() != 4 or not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("q and v must be [B, H, n, d] tensors")
    B, H, n, dk = q.shape
    dv, dev, dt = v.shape[3], q.device, _dtype_code(q.dtype)
    qp, qs = _view(q, "q", (B, H, n, dk), q.dtype, dev)
    kp, ks = _view(k, "k", (B, H, n, dk), q.dtype, dev)
    vp, vs = _view(v, "v", (B, H, n, dv), q.dtype, dev)
    gp, gs = _view(g, "g", (B, H, n, dk), torch.float32, dev)
    sp, ip, n_slots = _pool(state, slots, B, (H, dk, dv), dev)
    o, op = _new(o, "o", (B, H, n, dv), q.dtype, dev, v)
    _launch(load_library().gla_step, dev, qp, qs, kp, ks, vp, vs, gp, gs, sp, ip, op, B, H, n, dk, dv, n_slots, dt)
    return o


def _join_args(y, z, w_post, residual, scale, w_pre):
    _on_gpu(y, "y")
    if y.dim() != 4:
        raise ValueError("y must be a [B, H, T, d] tensor")
    B, H, T, d = y.shape
    dev, D, f32 = y.device, H * d, torch.float32
    dt = _dtype_code(y.dtype)
    yp, ys = _view(y, "y", (B, H, T, d), y.dtype, dev)
    zp, zs = (None, None) if z is None else _view(z, "z", (B, T, D), y.dtype, dev)
    wp = _out(w_post, "w_post", (d,), f32, dev, optional=True)
    st = y.dtype
    rp = rs = None
    if residual is not None:
        if not isinstance(residual, torch.Tensor):
            raise TypeError("residual must be a torch.Tensor")
        st = residual.dtype
        rp, rs = _view(residual, "residual", (B, T, D), st, dev)
    sp = _out(scale, "scale", (D,), f32, dev, optional=True)
    np_ = _out(w_pre, "w_pre", (D,), f32, dev, optional=True)
    return (B, H, T, d), st, dt, (yp, ys, zp, zs, wp, rp, rs, sp, np_)


def gla_join_fwd(y, z=None, w_post=None, residual=None, scale=None, w_pre=None, act: str = "silu", eps: float = 1e-6,
                 out=None, normed=None, keep_rstd: bool = True):
    """A block's output y [B, H, T, d] (the layout of o; H = 1 for a [B, T, D] output, y[:, None])
    joins the residual stream, in one pass: per-head RMS norm with w_post [d], gate act(z) with z
    [B, T, H d] ("silu" or "sigmoid"), out = residual + scale * that, and the next block's input
    normed = RMS norm of out with w_pre [H d].  Each of z, w_post, residual, scale and w_pre may be
    None (that step is then left out).  The weights are float32; residual and out have one dtype
    (float32 or y's), without a residual out has y's.  out may be the residual tensor itself.
    H d <= 8192 and H <= 2048.
    Returns a dict: out, normed (None without w_pre), and rstd_post [B, T, H], rstd_pre [B, T] for
    gla_join_bwd (None with keep_rstd=False)."""
    (B, H, T, d), st, dt, ptrs = _join_args(y, z, w_post, residual, scale, w_pre)
    dev, D, f32 = y.device, H * d, torch.float32
    out, op = _new(out, "out", (B, T, D), st, dev, z if residual is None else residual)
    np_ = None
    if w_pre is not None:
        normed, np_ = _new(normed, "normed", (B, T, D), y.dtype, dev, out)
    elif normed is not None:
        raise ValueError("normed given without w_pre")
    r_post = torch.empty((B, T, H), dtype=f32, device=dev) if keep_rstd and w_post is not None else None
    r_pre = torch.empty((B, T), dtype=f32, device=dev) if keep_rstd and w_pre is not None else None
    _launch(load_library().gla_join_fwd, dev, *ptrs, op, np_, None if r_post is None else r_post.data_ptr(),
            None if r_pre is None else r_pre.data_ptr(), B, H, T, d, _code(ACTS, act, "act"), eps, dt, _dtype_code(st))
    return {"out": out, "normed": normed, "rstd_post": r_post, "rstd_pre": r_pre}


def gla_join_bwd(y, fwd: dict, d_out=None, d_normed=None, z=None, w_post=None, residual=None, scale=None, w_pre=None,
                 act: str = "silu", workspace=None):
    """Gradients of gla_join_fwd for d_out (the gradient of out, out's dtype) and d_normed (of
    normed, y's dtype), at least one of them given, over the forward's inputs and the dict it
    returned.  Returns a dict: dy [B, H, T, d], dz, d_residual, dw_post [d], dscale [H d], dw_pre
    [H d] (weights' gradients float32; None for the inputs that were not given)."""
    (B, H, T, d), st, dt, ptrs = _join_args(y, z, w_post, residual, scale, w_pre)
    dev, D, f32 = y.device, H * d, torch.float32
    if d_out is None and d_normed is None:
        raise ValueError("one of d_out and d_normed is required")
    if d_normed is not None and w_pre is None:
        raise ValueError("d_normed given without w_pre")
    if residual is not None and fwd["out"].data_ptr() == residual.data_ptr():
        raise ValueError("the forward wrote out in the residual's place: its inputs are gone")
    rpost = None if w_post is None else _out(fwd["rstd_post"], "fwd['rstd_post']", (B, T, H), f32, dev)
    rpre = None if d_normed is None else _out(fwd["rstd_pre"], "fwd['rstd_pre']", (B, T), f32, dev)
    dop, dos = (None, None) if d_out is None else _view(d_out, "d_out", (B, T, D), st, dev)
    dnp, dns = (None, None) if d_normed is None else _view(d_normed, "d_normed", (B, T, D), y.dtype, dev)
    grads = [None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format)
             for t in (y, z, residual, w_post, scale, w_pre)]
    sums = not (w_post is None and scale is None and w_pre is None)
    workspace, wp, wn = _scratch(workspace, join_workspace_size(B, H, T, d) if sums else 0, dev)
    _launch(load_library().gla_join_bwd, dev, *ptrs, rpost, rpre, dop, dos, dnp, dns,
            *[None if t is None else t.data_ptr() for t in grads], B, H, T, d, _code(ACTS, act, "act"), dt,
            _dtype_code(st), wp, wn)
    return dict(zip(("dy", "dz", "d_residual", "dw_post", "dscale", "dw_pre"), grads))


# -------------------------------------------------------------------------------- gated delta rule

@functools.lru_cache(maxsize=4096)
def delta_workspace_size(which: int, B: int, H: int, Hk: int, T: int, dk: int, dv: int, dtype) -> int:
    """Bytes of workspace gla_delta_fwd (which=GLA_FWD) or gla_delta_bwd (GLA_BWD) needs."""
    return _size(load_library().gla_delta_workspace_size, which, B, H, Hk, T, dk, dv, _dtype_code(dtype))


@functools.lru_cache(maxsize=4096)
def delta_saved_size(B: int, H: int, Hk: int, T: int, dk: int, dv: int, dtype) -> int:
    """Bytes of the buffer that a training forward keeps for gla_delta_bwd."""
    return _size(load_library().gla_delta_saved_size, B, H, Hk, T, dk, dv, _dtype_code(dtype))


def _size(fn, *args):
    n = fn(*args)
    if n == 0:
        raise GLAError(GLA_ERR_INVALID_ARG, load_library().gla_last_error().decode())
    return int(n)


def _gates(t, name, shape, device):
    """(pointer, strides) of a [B, H, T] tensor of one value a token, at any strides."""
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != torch.float32 or t.device != device:
        if isinstance(t, torch.Tensor):
            t = t.contiguous()
        _expect(t, name, shape, torch.float32, device)  # says which
    st = t.stride()
    return t.data_ptr(), (ctypes.c_longlong * 3)(st[0], st[1], st[2])


def _delta_args(q, k, v, g, beta):
    """((B, H, Hk, T, dk, dv, dtype code), the inputs' pointers and strides), checked."""
    _on_gpu(q, "q")
    if q.dim() != 4 or not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("q and v must be [B, heads, T, d] tensors")
    B, Hk, T, dk = q.shape
    H, dv, dev = v.shape[1], v.shape[3], q.device
    return ((B, H, Hk, T, dk, dv, _dtype_code(q.dtype)),
            _view(q, "q", (B, Hk, T, dk), q.dtype, dev) + _view(k, "k", (B, Hk, T, dk), q.dtype, dev) +
            _view(v, "v", (B, H, T, dv), q.dtype, dev) + _gates(g, "g", (B, H, T), dev) +
            _gates(beta, "beta", (B, H, T), dev))


def gla_delta_fwd(q, k, v, g, beta, h0=None, lens=None, o=None, h_final=None, saved=None, workspace=None,
                  keep_saved: bool = True):
    """The gated delta rule: S <- exp(g_t) S, then S <- S + beta_t k_t (v_t - S^T k_t)^T and o_t = S^T q_t, over q, k
    [B, Hk, T, dk], v [B, H, T, dv] (bf16 or float32; value head h reads key head h // (H // Hk)) and g (log-gates <= 0,
    or -inf for a reset), beta [B, H, T] (float32), from h0 [B, H, dk, dv] (float32, default zero; a reset at the first token
    drops it whatever it holds).  lens: int32 [B], the sequences' lengths in a padded batch (o is zero behind them).  q, k and
    v may be views whose last dimension is contiguous, g and beta any views.  dk <= 128.
    Returns (o [B, H, T, dv], h_final [B, H, dk, dv], saved): saved is what gla_delta_bwd needs besides, a buffer of
    delta_saved_size bytes, None with keep_saved=False (a forward-only call)."""
    dims, ptrs = _delta_args(q, k, v, g, beta)
    B, H, Hk, T, dk, dv, dt = dims
    dev, f32 = q.device, torch.float32
    h0p = _out(h0, "h0", (B, H, dk, dv), f32, dev, optional=True)
    lp = _out(lens, "lens", (B,), torch.int32, dev, optional=True)
    ws, wp, wn = _scratch(workspace, delta_workspace_size(GLA_FWD, *dims[:6], q.dtype), dev)
    svp, svn = None, 0
    if keep_saved:
        saved, svp, svn = _scratch(saved, delta_saved_size(*dims[:6], q.dtype), dev)
    elif saved is not None:
        raise ValueError("saved given with keep_saved=False")
    o, op = _new(o, "o", (B, H, T, dv), q.dtype, dev, v)
    h_final, fp = _new(h_final, "h_final", (B, H, dk, dv), f32, dev, h0)
    _launch(load_library().gla_delta_fwd, dev, *ptrs, h0p, lp, op, fp, svp, svn, *dims, wp, wn)
    return o, h_final, saved


def gla_delta_bwd(q, k, v, g, beta, o, do, saved, lens=None, dhT=None, dq=None, dk=None, dv=None, dg=None, dbeta=None,
                  dh0=None, workspace=None):
    """Gradients of gla_delta_fwd for do [B, H, T, dv] (the gradient of o) and dhT [B, H, dk, dv] (of h_final, float32,
    default zero), over the forward's inputs, the o and the saved it returned.  Returns (dq, dk [B, Hk, T, dk], dv
    [B, H, T, dv] in q's dtype, dg, dbeta [B, H, T], dh0 [B, H, dk, dv], float32)."""
    dims, ptrs = _delta_args(q, k, v, g, beta)
    B, H, Hk, T, d_k, d_v, dt = dims
    dev, f32 = q.device, torch.float32
    op = _out(o, "o", (B, H, T, d_v), q.dtype, dev)
    dop, dos = _view(do, "do", (B, H, T, d_v), q.dtype, dev)
    lp = _out(lens, "lens", (B,), torch.int32, dev, optional=True)
    tp = _out(dhT, "dhT", (B, H, d_k, d_v), f32, dev, optional=True)
    if saved is None:
        raise ValueError("saved is required (a forward with keep_saved=True returns it)")
    _, svp, svn = _scratch(saved, 0, dev)
    ws, wp, wn = _scratch(workspace, delta_workspace_size(GLA_BWD, *dims[:6], q.dtype), dev)
    dq, dqp = _new(dq, "dq", (B, Hk, T, d_k), q.dtype, dev, q)
    dk, dkp = _new(dk, "dk", (B, Hk, T, d_k), q.dtype, dev, k)
    dv, dvp = _new(dv, "dv", (B, H, T, d_v), q.dtype, dev, v)
    dg, dgp = _new(dg, "dg", (B, H, T), f32, dev, g)
    dbeta, dbp = _new(dbeta, "dbeta", (B, H, T), f32, dev, beta)
    dh0, dhp = _new(dh0, "dh0", (B, H, d_k, d_v), f32, dev, dhT)
    _launch(load_library().gla_delta_bwd, dev, *ptrs, op, dop, dos, svp, svn, lp, tp, dqp, dkp, dvp, dgp, dbp, dhp, *dims,
            wp, wn)
    return dq, dk, dv, dg, dbeta, dh0


def gla_delta_step(q, k, v, g, beta, state, slots=None, o=None):
    """The next n tokens of the gated delta rule for every row of a batch (n = 1: decoding), in place on the pool
    ``state`` [n_slots, H, dk, dv] (float32; gla_delta_fwd's h_final is B such states): q, k [B, Hk, n, dk], v
    [B, H, n, dv], g, beta [B, H, n].  Row b's state is state[slots[b]], with the rules of gla_recur_step.  Views as in
    gla_delta_fwd.  dk <= 256.  Returns o [B, H, n, dv]."""
    dims, ptrs = _delta_args(q, k, v, g, beta)
    B, H, Hk, n, dk, dv, dt = dims
    dev = q.device
    sp, ip, n_slots = _pool(state, slots, B, (H, dk, dv), dev)
    o, op = _new(o, "o", (B, H, n, dv), q.dtype, dev, v)
    _launch(load_library().gla_delta_step, dev, *ptrs, sp, ip, op, B, H, Hk, n, dk, dv, n_slots, dt)
    return o


# ------------------------------------------------------------------------------------- layer norm

@functools.lru_cache(maxsize=4096)
def layernorm_workspace_size(B: int, T: int, D: int) -> int:
    """Bytes of workspace gla_layernorm_bwd needs for the weights' gradients."""
    return _size(load_library().gla_layernorm_workspace_size, B, T, D)


def _norm_args(x, w, residual):
    _on_gpu(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be a [B, T, D] tensor")
    (B, T, D), dev, st = x.shape, x.device, x.dtype
    dt = _dtype_code(x.dtype)
    xp, xs = _view(x, "x", (B, T, D), x.dtype, dev)
    rp = rs = None
    if residual is not None:
        if not isinstance(residual, torch.Tensor):
            raise TypeError("residual must be a torch.Tensor")
        st = residual.dtype
        rp, rs = _view(residual, "residual", (B, T, D), st, dev)
    return (B, T, D), st, dt, (xp, xs, rp, rs, _out(w, "w", (D,), torch.float32, dev, optional=True))


def gla_layernorm_fwd(x, w=None, b=None, residual=None, eps: float = 1e-5, out=None, normed=None,
                      keep_stats: bool = True):
    """The residual add and layer norm before a block, in one pass over x [B, T, D] (bf16 or float32): out = residual + x,
    normed = (out - mean) / sqrt(var + eps) * w + b.  residual [B, T, D] and out have one dtype (float32 or x's); without a
    residual it is the norm of x alone.  w and b [D] (float32) may be None (1 and 0).  out may be the residual tensor
    itself.  D <= 16384.
    Returns a dict: out (None without a residual), normed, and mean, rstd [B, T] for gla_layernorm_bwd (None with
    keep_stats=False)."""
    (B, T, D), st, dt, ptrs = _norm_args(x, w, residual)
    dev, f32 = x.device, torch.float32
    bp = _out(b, "b", (D,), f32, dev, optional=True)
    op = None
    if residual is not None:
        out, op = _new(out, "out", (B, T, D), st, dev, residual)
    elif out is not None:
        raise ValueError("out given without a residual")
    normed, np_ = _new(normed, "normed", (B, T, D), x.dtype, dev, x)
    mean = rstd = mp = rp = None
    if keep_stats:
        mean, mp = _new(None, "mean", (B, T), f32, dev)
        rstd, rp = _new(None, "rstd", (B, T), f32, dev)
    _launch(load_library().gla_layernorm_fwd, dev, *ptrs, bp, op, np_, mp, rp, B, T, D, eps, dt, _dtype_code(st))
    return {"out": out, "normed": normed, "mean": mean, "rstd": rstd}


def gla_layernorm_bwd(x, fwd: dict, d_normed, w=None, d_out=None, residual=None, bias: bool = True, workspace=None):
    """Gradients of gla_layernorm_fwd for d_normed (the gradient of normed, x's dtype) and d_out (of out, out's dtype,
    default zero), over the forward's inputs and the dict it returned.  Returns a dict: dx; d_residual (None without a
    residual; dx itself where the dtypes are the same, as the values are); dw [D] (None without w) and db [D] (None with
    bias=False), float32."""
    (B, T, D), st, dt, ptrs = _norm_args(x, w, residual)
    dev, f32 = x.device, torch.float32
    if residual is not None and fwd["out"] is not None and fwd["out"].data_ptr() == residual.data_ptr():
        raise ValueError("the forward wrote out in the residual's place: its inputs are gone")
    mp = _out(fwd["mean"], "fwd['mean']", (B, T), f32, dev)
    rp = _out(fwd["rstd"], "fwd['rstd']", (B, T), f32, dev)
    dnp, dns = _view(d_normed, "d_normed", (B, T, D), x.dtype, dev)
    dop, dos = (None, None) if d_out is None else _view(d_out, "d_out", (B, T, D), st, dev)
    dx, dxp = _new(None, "dx", (B, T, D), x.dtype, dev, x)
    d_residual, drp = None, None
    if residual is not None and st == x.dtype:
        d_residual = dx
    elif residual is not None:
        d_residual, drp = _new(None, "d_residual", (B, T, D), st, dev, residual)
    dw, dwp = (None, None) if w is None else _new(None, "dw", (D,), f32, dev, w)
    db, dbp = _new(None, "db", (D,), f32, dev, w) if bias else (None, None)
    sums = dw is not None or db is not None
    ws, wp, wn = _scratch(workspace, layernorm_workspace_size(B, T, D) if sums else 0, dev)
    _launch(load_library().gla_layernorm_bwd, dev, *ptrs, mp, rp, dop, dos, dnp, dns, dxp, drp, dwp, dbp, B, T, D, dt,
            _dtype_code(st), wp, wn)
    return {"dx": dx, "d_residual": d_residual, "dw": dw, "db": db}


# ------------------------------------------------------------------------------ method chains

def _join_backward(do, fwd, join, d_out, d_normed):
    """(do, gla_join_bwd's dict) of a backward chain: the gradient of o, through the join where the
    forward had one."""
    if join is None:
        if d_out is not None or d_normed is not None:
            raise ValueError("d_out and d_normed go with join")
        return do, None
    if do is not None:
        raise ValueError("with join the gradients come in as d_out and d_normed, not as do")
    args = {n: t for n, t in join.items() if n in ("z", "w_post", "residual", "scale", "w_pre", "act")}
    b = gla_join_bwd(fwd["o"], fwd["join"], d_out=d_out, d_normed=d_normed, **args)
    return b["dy"], b


def zeco_forward(q, k, v, g, chunk: int, P: int, K: int, h0=None, scan: str = "chain",
                 keep_chunk_states: bool = True, join: dict | None = None):
    """Local pass -> forward segment scan -> correction.  Returns a dict of tensors:
    o (global output), chunk_states (global state after every chunk; None with
    keep_chunk_states=False, for a forward-only caller), seg_in (state entering each segment),
    h_final (state after the last token), seg_state / seg_logdecay (local pass).
    scan: "chain" (gla_segment_scan) or "allgather" (gla_segment_scan_allgather).
    join: gla_join_fwd's arguments besides y (z, w_post, residual, scale, w_pre, act, eps): o then
    joins the residual stream, and the dict holds gla_join_fwd's under "join"."""
    o, chunk_states, seg_state, seg_logdecay = gla_chunk_fwd(q, k, v, g, chunk, P,
                                                             keep_chunk_states=keep_chunk_states)
    seg_in, h_final = _scan(scan, seg_state, seg_logdecay, K, h0, False)
    gla_segment_correct(GLA_FWD, chunk, P, q=q, g=g, seg_in=seg_in, o=o, chunk_states=chunk_states)
    res = {"o": o, "chunk_states": chunk_states, "seg_in": seg_in, "h_final": h_final, "seg_state": seg_state,
           "seg_logdecay": seg_logdecay}
    if join is not None:
        res["join"] = gla_join_fwd(o, **join)
    return res


def zeco_backward(q, k, v, g, do, fwd: dict, chunk: int, P: int, K: int, dhT=None, scan: str = "chain",
                  join: dict | None = None, d_out=None, d_normed=None):
    """Local backward -> reverse segment scan -> gradient correction.  ``fwd`` is the dict
    zeco_forward returned.  Returns dq, dk, dv, dg, dh0 (and the intermediates).
    join: the forward's; the gradients then come in as d_out and d_normed (of the join's out and
    normed) with do None, and the dict holds gla_join_bwd's under "join"."""
    do, joined = _join_backward(do, fwd, join, d_out, d_normed)
    dq, dk, dv, dg, seg_dstate = gla_chunk_bwd(q, k, v, g, do, fwd["chunk_states"], fwd["seg_in"], chunk, P)
    seg_grad, dh0 = _scan(scan, seg_dstate, fwd["seg_logdecay"], K, dhT, True)
    gla_segment_correct(GLA_BWD, chunk, P, k=k, v=v, g=g, seg_in=fwd["seg_in"], seg_grad=seg_grad,
                        chunk_states=fwd["chunk_states"], dk=dk, dv=dv, dg=dg)
    res = {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dh0": dh0, "seg_dstate": seg_dstate, "seg_grad": seg_grad}
    return res if joined is None else dict(res, join=joined)


def states_first_segments(B: int, H: int, T: int, chunk: int, P: int) -> int:
    """The segment count the order with the incoming states first runs at: P, each segment cut in
    two while the B*H*P' units leave CUs idle (fewer than 256) and the halves keep at least 2
    chunks.  In this order nothing depends on the segmentation beyond rounding (there is no
    correction whose work grows with it), and with P' segments no call cuts sub-segments of its
    own, whose state pass would repeat gla_chunk_state's."""
    if P < 1 or chunk < 1 or T % P or (T // P) % chunk:
        raise ValueError("T=%d must split into P=%d segments of whole chunks of %d tokens" % (T, P, chunk))
    n = T // P // chunk
    while B * H * P < 256 and n % 2 == 0 and n // 2 >= 2:
        P, n = 2 * P, n // 2
    return P


def states_first_forward(q, k, v, g, chunk: int, P: int, K: int, h0=None, scan: str = "chain",
                         keep_chunk_states: bool = True, fill: bool = True, join: dict | None = None):
    """The same forward with the incoming states first: state pass -> forward segment scan ->
    local pass from each segment's true incoming state (no correction).  With fill, the segments
    are first cut to fill the chip (states_first_segments); the per-segment results then count
    those segments, whose number the dict holds as "P".  Returns the dict zeco_forward returns
    (o, chunk_states, seg_in, h_final, seg_state, seg_logdecay) plus "P".  join as in zeco_forward."""
    if fill:
        P = states_first_segments(q.shape[0], q.shape[1], q.shape[2], chunk, P)
    seg_state, seg_logdecay = gla_chunk_state(k, v, g, chunk, P)
    seg_in, h_final = _scan(scan, seg_state, seg_logdecay, K, h0, False)
    o, chunk_states = gla_chunk_fwd_from(q, k, v, g, seg_in, chunk, P, keep_chunk_states=keep_chunk_states)
    res = {"o": o, "chunk_states": chunk_states, "seg_in": seg_in, "h_final": h_final, "seg_state": seg_state,
           "seg_logdecay": seg_logdecay, "P": P}
    if join is not None:
        res["join"] = gla_join_fwd(o, **join)
    return res


def states_first_backward(q, k, v, g, do, fwd: dict, chunk: int, K: int, dhT=None, scan: str = "chain",
                          join: dict | None = None, d_out=None, d_normed=None):
    """The same backward with the incoming gradients first: state-gradient pass -> reverse segment
    scan -> local backward from each segment's true outgoing gradient (no correction), over the
    segments of ``fwd``, the dict states_first_forward returned.  Returns the dict zeco_backward
    returns; join, d_out and d_normed as there."""
    do, joined = _join_backward(do, fwd, join, d_out, d_normed)
    P = fwd["P"]
    seg_dstate = gla_chunk_dstate(q, g, do, chunk, P)
    seg_grad, dh0 = _scan(scan, seg_dstate, fwd["seg_logdecay"], K, dhT, True)
    dq, dk, dv, dg = gla_chunk_bwd_from(q, k, v, g, do, fwd["chunk_states"], fwd["seg_in"], seg_grad, chunk, P)
    res = {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dh0": dh0, "seg_dstate": seg_dstate, "seg_grad": seg_grad}
    return res if joined is None else dict(res, join=joined)


# ------------------------------------------------------------------------ several streams at once

_streams = {}


def _side_streams(device, n):
    """n streams of default priority on ``device``, created once and reused."""
    key = (device.index, n)
    if key not in _streams:
        _streams[key] = [torch.cuda.Stream(device=device) for _ in range(n)]
    return _streams[key]


def _rows(t, lo, hi):
    """Sequences lo..hi-1 of a [B, H, ...] tensor, as a contiguous [hi-lo, 1, ...] view."""
    if t is None:
        return None
    flat = t.view(t.shape[0] * t.shape[1], 1, *t.shape[2:])
    return flat[lo:hi]


def zeco_step_streams(q, k, v, g, do, chunk: int, P: int, K: int, n_streams: int = 2, h0=None, dhT=None,
                      out=None, stagger: bool = False):
    """The whole fwd+bwd path with the B*H sequences cut into ``n_streams`` groups, each group's six
    calls (local pass, scan, correction; local backward, reverse scan, correction) in order on a
    stream of its own.  The streams fork from torch's current stream and join back into it, so
    the result is ordered like any other call on the current stream.  While one group runs its
    scans and corrections, another group's local passes can use the CUs they leave free.  The
    groups' calls get flag-only workspaces, so none cuts its segments into sub-segments: every unit
    is computed exactly as in the one-stream chain run with such workspaces, bit for bit.

    ``out``: optional dict of preallocated buffers (as returned by a previous call) to reuse.
    ``stagger``: each group's chain waits for the previous group's local pass, so that a group's
    scan and correction run while the next group's local pass does (the overlap the ZeCO pages
    measure; on one GPU it serialises the local passes of the groups, which costs more than the
    scans it hides).
    Returns a dict: o, h_final, dq, dk, dv, dg, dh0 and the intermediates."""
    B, H, T, dk_, dv_ = _head_args(q, k, v, g, (("do", do, v.shape[-1], q.dtype),))
    cs_shape, st_shape, ld_shape = _seg_shapes(B, H, T, dk_, dv_, chunk, P)
    dev, f32, edt = q.device, torch.float32, q.dtype
    if out is None:
        out = {
            "o": torch.empty_like(v), "chunk_states": torch.empty(cs_shape, device=dev, dtype=edt),
            "seg_state": torch.empty(st_shape, device=dev, dtype=f32),
            "seg_logdecay": torch.empty(ld_shape, device=dev, dtype=f32),
            "seg_in": torch.empty(st_shape, device=dev, dtype=f32),
            "h_final": torch.empty((B, H, dk_, dv_), device=dev, dtype=f32),
            "dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
            "dg": torch.empty_like(g), "seg_dstate": torch.empty(st_shape, device=dev, dtype=f32),
            "seg_grad": torch.empty(st_shape, device=dev, dtype=f32),
            "dh0": torch.empty((B, H, dk_, dv_), device=dev, dtype=f32),
        }
    BH = B * H
    n = max(1, min(n_streams, BH))
    bounds = [BH * i // n for i in range(n + 1)]
    if "workspaces" not in out or len(out["workspaces"]) != n:
        # flags only: a group's calls cut no segment into sub-segments, because the groups share the
        # chip; each call on its own would cut its fewer units to fill it
        out["workspaces"] = [torch.empty(flags_workspace_size(bounds[i + 1] - bounds[i], 1, P), device=dev,
                                         dtype=torch.uint8) for i in range(n)]
    main = torch.cuda.current_stream(dev)
    streams = _side_streams(dev, n)
    local_done = None
    for i, st in enumerate(streams):
        lo, hi = bounds[i], bounds[i + 1]
        r = {name: _rows(t, lo, hi) for name, t in out.items() if isinstance(t, torch.Tensor)}
        x = {name: _rows(t, lo, hi) for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("do", do),
                                                     ("h0", h0), ("dhT", dhT))}
        ws = out["workspaces"][i]
        st.wait_stream(main)
        if stagger and local_done is not None:
            st.wait_event(local_done)
        with torch.cuda.stream(st):
            gla_chunk_fwd(x["q"], x["k"], x["v"], x["g"], chunk, P, o=r["o"], chunk_states=r["chunk_states"],
                          seg_state=r["seg_state"], seg_logdecay=r["seg_logdecay"], workspace=ws)
            if stagger:
                local_done = torch.cuda.Event()
                local_done.record(st)
            gla_segment_scan(r["seg_state"], r["seg_logdecay"], K, h_boundary=x["h0"], seg_carry=r["seg_in"],
                             h_out=r["h_final"])
            gla_segment_correct(GLA_FWD, chunk, P, q=x["q"], g=x["g"], seg_in=r["seg_in"], o=r["o"],
                                chunk_states=r["chunk_states"])
            gla_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], r["chunk_states"], r["seg_in"], chunk, P,
                          dq=r["dq"], dk=r["dk"], dv=r["dv"], dg=r["dg"], seg_dstate=r["seg_dstate"], workspace=ws)
            gla_segment_scan(r["seg_dstate"], r["seg_logdecay"], K, h_boundary=x["dhT"], reverse=True,
                             seg_carry=r["seg_grad"], h_out=r["dh0"])
            gla_segment_correct(GLA_BWD, chunk, P, k=x["k"], v=x["v"], g=x["g"], seg_in=r["seg_in"],
                                seg_grad=r["seg_grad"], chunk_states=r["chunk_states"], dk=r["dk"], dv=r["dv"],
                                dg=r["dg"])
    for st in streams:
        main.wait_stream(st)
    return out

