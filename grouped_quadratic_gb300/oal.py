"""ctypes binding of liboal.so (include/oal.h), same entry-point names.

Argument marshalling only: every step of OAL runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  If the
library is missing or fails to load, every call raises ``OALError`` -- there
is no CPU fallback.

Tensor layouts (row-major, contiguous, CUDA):
  Q [B,Hq,T,64], K/V [B,Hkv,T,64] (float32 or bfloat16)
  L [Hq,G+1,G+1] float32 (lower triangle), group [Hq,64] int32 in 1..G
  state [B,Hkv,F,65] float32 (F = 4161 FULL, 2145 PACKED)
  gated recurrence: g [B,Hkv,T] float32 (log decays), state [B,Hkv,64,64] float32
  paged cache: Kp/Vp [n_pages,Hkv,page_size,64] (pages may lie apart), table [B,max_pages] int32
  rotations: Q, K, V of oal_rope and oal_page_append may be views whose rows are contiguous

A call given a `stream` waits there for the tensors that it makes itself (on the
current stream); tensors given to it have to be ready on `stream`.
"""
import ctypes
import functools
import os
import struct

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liboal.so")

OAL_OK, OAL_ERR_INVALID_ARG, OAL_ERR_UNSUPPORTED, OAL_ERR_CUDA, OAL_ERR_TIMEOUT = range(5)
OAL_F32, OAL_BF16 = 0, 1
OAL_STATE_FULL, OAL_STATE_PACKED = 0, 1
OAL_ROPE_HALVES, OAL_ROPE_PAIRS = 0, 1
_STATUS_NAMES = {0: "OAL_OK", 1: "OAL_ERR_INVALID_ARG", 2: "OAL_ERR_UNSUPPORTED",
                 3: "OAL_ERR_CUDA", 4: "OAL_ERR_TIMEOUT"}


class OALError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("%s: %s" % (_STATUS_NAMES.get(status, status), msg))
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH):
    """Load liboal.so (raises OALError if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OALError(OAL_ERR_CUDA, "liboal.so not found at %s; run "
                       "`python -m grouped_quadratic_gb300.build`" % path)
    lib = ctypes.CDLL(path)
    vp, sz, ci, cf = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    lib.oal_state_rows.argtypes = [ci, ci]
    lib.oal_state_rows.restype = sz
    lib.oal_state_elems.argtypes = [ci, ci, ci]
    lib.oal_state_elems.restype = sz
    lib.oal_coeff_table_elems.argtypes = [ci, ci]
    lib.oal_coeff_table_elems.restype = sz
    lib.oal_expand_coeffs.argtypes = [vp, vp, ci, ci, ci, cf, ci, vp, vp, vp, vp]
    lib.oal_expand_coeffs.restype = ci
    lib.oal_prefill_workspace_bytes.argtypes = [ci] * 6 + [ci, ci, ci]
    lib.oal_prefill_workspace_bytes.restype = sz
    lib.oal_prefill.argtypes = ([vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, vp, vp, ci, cf,
                                 vp, vp, vp, ci, vp, ci, vp, ci, vp, sz, vp])
    lib.oal_prefill.restype = ci
    lib.oal_prefill_noalloc.argtypes = ([vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, vp, vp, ci,
                                         cf, vp, vp, vp, ci, vp, ci, vp, ci, vp])
    lib.oal_prefill_noalloc.restype = ci
    lib.oal_prefill_backward_workspace_bytes.argtypes = [ci] * 6
    lib.oal_prefill_backward_workspace_bytes.restype = sz
    lib.oal_prefill_backward.argtypes = ([vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, vp, vp, ci,
                                          cf, vp, vp, vp, vp, vp, sz, vp])
    lib.oal_prefill_backward.restype = ci
    lib.oal_decode_workspace_bytes.argtypes = [ci] * 5 + [ci]
    lib.oal_decode_workspace_bytes.restype = sz
    lib.oal_decode_step.argtypes = [vp, vp, vp, ci, ci, ci, ci, ci, ci, vp, vp, vp, ci,
                                    vp, vp, vp, sz, vp]
    lib.oal_decode_step.restype = ci
    lib.oal_contribution_workspace_bytes.argtypes = [ci] * 5
    lib.oal_contribution_workspace_bytes.restype = sz
    lib.oal_contribution_scores.argtypes = [vp, vp, ci, ci, ci, ci, ci, ci, vp, vp, vp, sz, vp]
    lib.oal_contribution_scores.restype = ci
    lib.oal_gated_prefill_workspace_bytes.argtypes = [ci] * 7
    lib.oal_gated_prefill_workspace_bytes.restype = sz
    lib.oal_gated_prefill.argtypes = [vp, vp, vp, ci, vp, ci, ci, ci, ci, ci, ci, cf, vp, vp, ci,
                                      vp, vp, sz, vp]
    lib.oal_gated_prefill.restype = ci
    lib.oal_gated_backward_workspace_bytes.argtypes = [ci] * 7
    lib.oal_gated_backward_workspace_bytes.restype = sz
    lib.oal_gated_backward.argtypes = [vp, vp, vp, ci, vp, vp, ci, ci, ci, ci, ci, ci, cf, vp, vp,
                                       vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.oal_gated_backward.restype = ci
    lib.oal_gated_decode_step.argtypes = [vp, vp, vp, ci, vp, ci, ci, ci, ci, ci, cf, vp, ci, vp,
                                          vp, vp]
    lib.oal_gated_decode_step.restype = ci
    lib.oal_state_remap.argtypes = [vp, sz, ci, vp, vp]
    lib.oal_state_remap.restype = ci
    lib.oal_rope_plan.argtypes = [vp, vp, vp]
    lib.oal_rope_plan.restype = ci
    i64 = ctypes.c_int64
    lib.oal_rope.argtypes = [vp, vp, ci, vp, ci, ci, ci, ci, ci, vp, ci, vp, ci, vp, vp, ci, vp, vp, vp]
    lib.oal_rope.restype = ci
    lib.oal_page_append.argtypes = [vp, vp, vp, ci, vp, ci, ci, ci, ci, ci, ci, vp, ci, vp, ci, vp, vp,
                                    vp, vp, ci, ci, i64, vp, ci, vp, vp]
    lib.oal_page_append.restype = ci
    lib.oal_paged_attention_workspace_bytes.argtypes = [ci] * 9
    lib.oal_paged_attention_workspace_bytes.restype = sz
    lib.oal_paged_attention.argtypes = [vp, ci, ci, ci, ci, ci, ci, ci, vp, vp, ci, ci, i64, vp, ci, vp,
                                        vp, cf, cf, ci, vp, vp, vp, vp, vp, sz, vp]
    lib.oal_paged_attention.restype = ci
    cd = ctypes.c_double
    lib.oal_group_dims.argtypes = [vp, ci, ci, vp, ci, cd, cd, cd, ci, cd, vp, vp]
    lib.oal_group_dims.restype = ci
    lib.oal_sync_status.argtypes = [vp]
    lib.oal_sync_status.restype = ci
    lib.oal_debug_wait_test.argtypes = [ctypes.c_uint64, ci]
    lib.oal_debug_wait_test.restype = ci
    lib.oal_debug_intra_heads.argtypes = [ci]
    lib.oal_debug_intra_heads.restype = ci
    lib.oal_prefill_noalloc_scratch_bytes.argtypes = []
    lib.oal_prefill_noalloc_scratch_bytes.restype = sz
    lib.oal_last_error.argtypes = []
    lib.oal_last_error.restype = ctypes.c_char_p
    lib.oal_version.argtypes = []
    lib.oal_version.restype = ctypes.c_char_p
    lib.oal_launch_counter.argtypes = []
    lib.oal_launch_counter.restype = ctypes.c_uint64
    lib.oal_set_launch_events.argtypes = [vp, ci]
    lib.oal_set_launch_events.restype = ci
    lib.oal_last_call_launches.argtypes = []
    lib.oal_last_call_launches.restype = ci
    lib.oal_last_call_launch_name.argtypes = [ci]
    lib.oal_last_call_launch_name.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(status):
    if status != OAL_OK:
        raise OALError(status, _lib.oal_last_error().decode())


def _order(stream, made):
    """Orders the tensors a call made, from the current stream's pool, with the
    stream it launches on.  Work queued on the current stream may still use
    their memory, and some are being zeroed there, so `stream` waits for it;
    and the memory must not be handed out again before `stream` is done with
    it.  Tensors the caller gives are the caller's to order."""
    if made:
        current = torch.cuda.current_stream(stream.device)
        if stream != current:
            stream.wait_stream(current)
            for t in made:
                t.record_stream(stream)


def _stream(stream, made=()):
    """The handle to launch on; `made`: tensors the call allocated."""
    if stream is None:
        stream = torch.cuda.current_stream()
    else:
        _order(stream, made)
    return ctypes.c_void_p(stream.cuda_stream)


def _make(made, t, shape, dtype, dev):
    """t, or a new tensor, which joins `made`."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=dev)
        made.append(t)
    return t


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _dtype_code(t):
    if t.dtype == torch.float32:
        return OAL_F32
    if t.dtype == torch.bfloat16:
        return OAL_BF16
    raise OALError(OAL_ERR_INVALID_ARG, "unsupported dtype %s" % t.dtype)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise OALError(OAL_ERR_INVALID_ARG, "tensors must be contiguous CUDA tensors")


def oal_version():
    return load_library().oal_version().decode()


def oal_state_rows(d=64, layout=OAL_STATE_FULL):
    return int(load_library().oal_state_rows(d, layout))


def oal_state_elems(d=64, dv=64, layout=OAL_STATE_FULL):
    return int(load_library().oal_state_elems(d, dv, layout))


def oal_coeff_table_elems(d=64, layout=OAL_STATE_FULL):
    return int(load_library().oal_coeff_table_elems(d, layout))


def oal_expand_coeffs(L, group, eps, layout=OAL_STATE_FULL, a=None, b=None, C=None,
                      stream=None):
    """Coefficient tables (a [Hq], b [Hq,64], C [Hq, 4096 or 2080]) on the device."""
    lib = load_library()
    Hq, G1, _ = L.shape
    d = group.shape[1]
    dev, f32, made = L.device, torch.float32, []
    a = _make(made, a, (Hq,), f32, dev)
    b = _make(made, b, (Hq, d), f32, dev)
    C = _make(made, C, (Hq, lib.oal_coeff_table_elems(d, layout)), f32, dev)
    _need_cuda(L, group, a, b, C)
    _check(lib.oal_expand_coeffs(_ptr(L), _ptr(group), Hq, G1 - 1, d, float(eps), layout,
                                 _ptr(a), _ptr(b), _ptr(C), _stream(stream, made)))
    return a, b, C


def oal_prefill_workspace_bytes(B, Hq, Hkv, T, d=64, dv=64, dtype=OAL_BF16,
                                layout=OAL_STATE_FULL, chunk=0):
    return int(load_library().oal_prefill_workspace_bytes(B, Hq, Hkv, T, d, dv, dtype,
                                                          layout, chunk))


def oal_prefill(Q, K, V, L, group, eps, a, b, C, layout=OAL_STATE_FULL, state=None,
                continue_from_state=False, Y=None, chunk=0, workspace=None, stream=None):
    """Causal OAL prefill.  Returns (Y, state)."""
    lib = load_library()
    B, Hq, T, d = Q.shape
    Hkv, dv = K.shape[1], V.shape[3]
    G = L.shape[1] - 1
    dt = _dtype_code(Q)
    dev, made = Q.device, []
    state = _make(made, state, (B, Hkv, lib.oal_state_rows(d, layout), dv + 1), torch.float32, dev)
    Y = _make(made, Y, (B, Hq, T, dv), Q.dtype, dev)
    need = lib.oal_prefill_workspace_bytes(B, Hq, Hkv, T, d, dv, dt, layout, chunk)
    workspace = _make(made, workspace, (max(int(need), 256),), torch.uint8, dev)
    _need_cuda(Q, K, V, L, group, a, b, C, state, Y, workspace)
    _check(lib.oal_prefill(_ptr(Q), _ptr(K), _ptr(V), dt, B, Hq, Hkv, T, d, dv, _ptr(L),
                           _ptr(group), G, float(eps), _ptr(a), _ptr(b), _ptr(C), layout,
                           _ptr(state), int(bool(continue_from_state)), _ptr(Y), chunk,
                           _ptr(workspace), workspace.numel() * workspace.element_size(),
                           _stream(stream, made)))
    return Y, state


def oal_prefill_noalloc_scratch_bytes():
    """Size of the library's fixed prefill scratch array, read from the library."""
    return int(load_library().oal_prefill_noalloc_scratch_bytes())


def oal_prefill_noalloc(Q, K, V, L, group, eps, a, b, C, state, Y, layout=OAL_STATE_FULL,
                        continue_from_state=False, chunk=0, stream=None):
    """oal_prefill with the library's fixed scratch instead of a workspace.

    For callers that cannot allocate device memory: `state` and `Y` must be
    passed in, and this wrapper allocates nothing either.  Problems whose
    workspace would exceed oal_prefill_noalloc_scratch_bytes() are rejected.
    """
    lib = load_library()
    B, Hq, T, d = Q.shape
    Hkv, dv = K.shape[1], V.shape[3]
    G = L.shape[1] - 1
    _need_cuda(Q, K, V, L, group, a, b, C, state, Y)
    _check(lib.oal_prefill_noalloc(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(Q), B, Hq, Hkv, T,
                                   d, dv, _ptr(L), _ptr(group), G, float(eps), _ptr(a),
                                   _ptr(b), _ptr(C), layout, _ptr(state),
                                   int(bool(continue_from_state)), _ptr(Y), chunk,
                                   _stream(stream)))
    return Y, state


def oal_prefill_backward_workspace_bytes(B, Hq, Hkv, T, d=64, dv=64):
    return int(load_library().oal_prefill_backward_workspace_bytes(B, Hq, Hkv, T, d, dv))


def oal_prefill_backward(Q, K, V, dY, L, group, eps, dQ=None, dK=None, dV=None, dL=None,
                         workspace=None, stream=None):
    """Gradients of <dY, Y> for Y = oal_prefill(Q, K, V, L, group, eps).
    Returns (dQ, dK, dV, dL), fp32."""
    lib = load_library()
    B, Hq, T, d = Q.shape
    Hkv, dv = K.shape[1], V.shape[3]
    G = L.shape[1] - 1
    dev, f32, made = Q.device, torch.float32, []
    dQ = _make(made, dQ, (B, Hq, T, d), f32, dev)
    dK = _make(made, dK, (B, Hkv, T, d), f32, dev)
    dV = _make(made, dV, (B, Hkv, T, dv), f32, dev)
    dL = _make(made, dL, (Hq, G + 1, G + 1), f32, dev)
    need = lib.oal_prefill_backward_workspace_bytes(B, Hq, Hkv, T, d, dv)
    workspace = _make(made, workspace, (max(int(need), 256),), torch.uint8, dev)
    if dY.dtype != Q.dtype:
        raise OALError(OAL_ERR_INVALID_ARG, "dY must have the dtype of Q")
    _need_cuda(Q, K, V, dY, L, group, dQ, dK, dV, dL, workspace)
    _check(lib.oal_prefill_backward(_ptr(Q), _ptr(K), _ptr(V), _ptr(dY), _dtype_code(Q), B, Hq,
                                    Hkv, T, d, dv, _ptr(L), _ptr(group), G, float(eps), _ptr(dQ),
                                    _ptr(dK), _ptr(dV), _ptr(dL), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _stream(stream, made)))
    return dQ, dK, dV, dL


def oal_decode_workspace_bytes(B, Hq, Hkv, d=64, dv=64, layout=OAL_STATE_FULL):
    return int(load_library().oal_decode_workspace_bytes(B, Hq, Hkv, d, dv, layout))


def oal_decode_step(q, k, v, a, b, C, state, layout=OAL_STATE_FULL, y=None,
                    workspace=None, stream=None):
    """One decode token for all sequences: q [B,Hq,64], k/v [B,Hkv,64]. Returns y."""
    lib = load_library()
    B, Hq, d = q.shape
    Hkv, dv = k.shape[1], v.shape[2]
    dt, made = _dtype_code(q), []
    y = _make(made, y, (B, Hq, dv), q.dtype, q.device)
    if workspace is None:
        need = lib.oal_decode_workspace_bytes(B, Hq, Hkv, d, dv, layout)
        workspace = _make(made, None, (max(int(need), 256),), torch.uint8, q.device)
    _need_cuda(q, k, v, a, b, C, state, y, workspace)
    _check(lib.oal_decode_step(_ptr(q), _ptr(k), _ptr(v), dt, B, Hq, Hkv, d, dv, _ptr(a),
                               _ptr(b), _ptr(C), layout, _ptr(state), _ptr(y),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream, made)))
    return y


def oal_contribution_workspace_bytes(P, Hq, Hkv, T, d=64):
    return int(load_library().oal_contribution_workspace_bytes(P, Hq, Hkv, T, d))


def oal_contribution_scores(Q, K, lengths=None, chi=None, workspace=None, stream=None):
    """Per-prompt contribution scores: Q [P,Hq,T,64], K [P,Hkv,T,64], lengths
    [P] int32 (CUDA) or None for T tokens each.  Returns chi [P,Hq,64] float32."""
    lib = load_library()
    P, Hq, T, d = Q.shape
    Hkv, made = K.shape[1], []
    chi = _make(made, chi, (P, Hq, d), torch.float32, Q.device)
    need = lib.oal_contribution_workspace_bytes(P, Hq, Hkv, T, d)
    workspace = _make(made, workspace, (max(int(need), 256),), torch.uint8, Q.device)
    _need_cuda(Q, K, lengths, chi, workspace)
    _check(lib.oal_contribution_scores(_ptr(Q), _ptr(K), _dtype_code(Q), P, Hq, Hkv, T, d,
                                       _ptr(lengths), _ptr(chi), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(),
                                       _stream(stream, made)))
    return chi


def oal_group_dims(chi_p, boot_idx, alpha, tau, gamma, g_min, eps=1e-12):
    """Dimension groups of one query head (host arrays, no GPU): chi_p [P, d]
    per-prompt scores, boot_idx [nboot, P] bootstrap prompt indices.
    Returns (group [d] int32 in 1..G, G)."""
    import numpy as np
    lib = load_library()
    chi_p = np.ascontiguousarray(np.asarray(chi_p, dtype=np.float32))
    boot_idx = np.ascontiguousarray(np.asarray(boot_idx, dtype=np.int32))
    if chi_p.ndim != 2 or boot_idx.ndim != 2 or boot_idx.shape[1] != chi_p.shape[0]:
        raise OALError(OAL_ERR_INVALID_ARG, "chi_p must be [P, d] and boot_idx [nboot, P]")
    P, d = chi_p.shape
    group = np.zeros(d, np.int32)
    G = ctypes.c_int(0)
    _check(lib.oal_group_dims(chi_p.ctypes.data, P, d, boot_idx.ctypes.data, boot_idx.shape[0],
                              float(alpha), float(tau), float(gamma), int(g_min), float(eps),
                              group.ctypes.data, ctypes.byref(G)))
    return group, G.value


def _need(ok, what):
    if not ok:
        raise OALError(OAL_ERR_INVALID_ARG, what)


def _need_tensor(t, name, dtype, shape, dev):
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == dev:
        return
    if t.dtype != dtype or t.shape != shape:
        raise OALError(OAL_ERR_INVALID_ARG, "%s must be %s %s (got %s %s)"
                       % (name, dtype, tuple(shape), t.dtype, tuple(t.shape)))
    raise OALError(OAL_ERR_INVALID_ARG, "%s must be contiguous on %s" % (name, dev))


def _elsewhere(dev):
    """Whether dev is a CUDA device other than the current one (the call then
    repeats itself with dev current)."""
    if dev.type != "cuda":
        raise OALError(OAL_ERR_INVALID_ARG, "tensors must be contiguous CUDA tensors")
    return dev.index != torch.cuda.current_device()


def _stream_on(dev, stream, made):
    """The handle to launch on: that of `stream`, or of the current stream of
    dev.  `made`: tensors this call allocated."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev.index)
    if stream.device != dev:
        raise OALError(OAL_ERR_INVALID_ARG, "the stream is on %s, the tensors on %s"
                       % (stream.device, dev))
    _order(stream, made)
    return stream.cuda_stream


def _ptr_or_null(t):
    return None if t is None else t.data_ptr()


def _gated_shapes(Q, K, V, g):
    _need(Q.dim() == 4 and K.dim() == 4 and V.dim() == 4, "Q, K and V must have 4 dimensions")
    B, Hq, T, d = Q.shape
    Hkv, dv = K.shape[1], V.shape[3]
    dev = Q.device
    _need_tensor(Q, "Q", Q.dtype, (B, Hq, T, d), dev)
    _need_tensor(K, "K", Q.dtype, (B, Hkv, T, d), dev)
    _need_tensor(V, "V", Q.dtype, (B, Hkv, T, dv), dev)
    _need_tensor(g, "g", torch.float32, (B, Hkv, T), dev)
    return B, Hq, Hkv, T, d, dv, dev


def _need_lengths(lengths, B, dev):
    if lengths is not None:
        _need_tensor(lengths, "lengths", torch.int32, (B,), dev)


def _workspace(given, size, made, sizes, dev):
    if given is None:
        given = torch.empty(max(size(*sizes), 256), dtype=torch.uint8, device=dev)
        made.append(given)
    _need_tensor(given, "workspace", given.dtype, given.shape, dev)
    return given


def oal_gated_prefill_workspace_bytes(B, Hq, Hkv, T, d=64, dv=64, dtype=OAL_BF16):
    return int(load_library().oal_gated_prefill_workspace_bytes(B, Hq, Hkv, T, d, dv, dtype))


def oal_gated_prefill(Q, K, V, g, scale=0.125, lengths=None, state=None,
                      continue_from_state=False, Y=None, workspace=None, stream=None):
    """Gated linear recurrence over T tokens: Q [B,Hq,T,64], K/V [B,Hkv,T,64],
    g [B,Hkv,T] float32 log decays, lengths [B] int32 (CUDA) or None.  `state`
    [B,Hkv,64,64] float32 is updated in place (from zeros unless
    continue_from_state).  Returns (Y, state).  Rows of Y behind a sequence's
    length stay as given; a Y made here has zeros there."""
    lib = load_library()
    B, Hq, Hkv, T, d, dv, dev = _gated_shapes(Q, K, V, g)
    dt = _dtype_code(Q)
    _need_lengths(lengths, B, dev)
    _need(state is not None or not continue_from_state, "continue_from_state needs a state")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return oal_gated_prefill(Q, K, V, g, scale, lengths, state, continue_from_state, Y,
                                     workspace, stream)
    made = []
    if state is None:
        state = torch.empty(B, Hkv, d, dv, dtype=torch.float32, device=dev)
        made.append(state)
    if Y is None:
        make = torch.empty if lengths is None else torch.zeros
        Y = make(B, Hq, T, dv, dtype=Q.dtype, device=dev)
        made.append(Y)
    workspace = _workspace(workspace, lib.oal_gated_prefill_workspace_bytes, made,
                           (B, Hq, Hkv, T, d, dv, dt), dev)
    _need_tensor(state, "state", torch.float32, (B, Hkv, d, dv), dev)
    _need_tensor(Y, "Y", Q.dtype, (B, Hq, T, dv), dev)
    _check(lib.oal_gated_prefill(Q.data_ptr(), K.data_ptr(), V.data_ptr(), dt, g.data_ptr(), B, Hq,
                                 Hkv, T, d, dv, scale, _ptr_or_null(lengths), state.data_ptr(),
                                 bool(continue_from_state), Y.data_ptr(), workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(),
                                 _stream_on(dev, stream, made)))
    return Y, state


def oal_gated_backward_workspace_bytes(B, Hq, Hkv, T, d=64, dv=64, dtype=OAL_BF16):
    return int(load_library().oal_gated_backward_workspace_bytes(B, Hq, Hkv, T, d, dv, dtype))


def oal_gated_backward(Q, K, V, g, dY, scale=0.125, lengths=None, state0=None, dstate=None,
                       dQ=None, dK=None, dV=None, dg=None, dstate0=None, workspace=None,
                       stream=None):
    """Gradients of <dY, Y> + <dstate, S_T> for oal_gated_prefill from state0
    (None: zeros).  Returns (dQ, dK, dV, dg, dstate0): the first three in the
    dtype of Q, dg and dstate0 float32.  Rows behind a sequence's length stay
    as given; gradients made here have zeros there."""
    lib = load_library()
    B, Hq, Hkv, T, d, dv, dev = _gated_shapes(Q, K, V, g)
    dt = _dtype_code(Q)
    _need_lengths(lengths, B, dev)
    _need_tensor(dY, "dY", Q.dtype, (B, Hq, T, dv), dev)
    for name, t in (("state0", state0), ("dstate", dstate)):
        if t is not None:
            _need_tensor(t, name, torch.float32, (B, Hkv, d, dv), dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return oal_gated_backward(Q, K, V, g, dY, scale, lengths, state0, dstate, dQ, dK, dV,
                                      dg, dstate0, workspace, stream)
    made, out = [], []
    make = torch.empty if lengths is None else torch.zeros
    for name, t, like in (("dQ", dQ, Q), ("dK", dK, K), ("dV", dV, V), ("dg", dg, g)):
        if t is None:
            t = make(like.shape, dtype=like.dtype, device=dev)
            made.append(t)
        _need_tensor(t, name, like.dtype, like.shape, dev)
        out.append(t)
    if dstate0 is None:
        dstate0 = torch.empty(B, Hkv, d, dv, dtype=torch.float32, device=dev)
        made.append(dstate0)
    _need_tensor(dstate0, "dstate0", torch.float32, (B, Hkv, d, dv), dev)
    out.append(dstate0)
    workspace = _workspace(workspace, lib.oal_gated_backward_workspace_bytes, made,
                           (B, Hq, Hkv, T, d, dv, dt), dev)
    _check(lib.oal_gated_backward(Q.data_ptr(), K.data_ptr(), V.data_ptr(), dt, g.data_ptr(),
                                  dY.data_ptr(), B, Hq, Hkv, T, d, dv, scale,
                                  _ptr_or_null(lengths), _ptr_or_null(state0),
                                  _ptr_or_null(dstate), *(t.data_ptr() for t in out),
                                  workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(),
                                  _stream_on(dev, stream, made)))
    return tuple(out)


def oal_gated_decode_step(q, k, v, g, state, scale=0.125, slots=None, y=None, stream=None):
    """One token of the gated recurrence: q [B,Hq,64], k/v [B,Hkv,64], g [B,Hkv]
    float32.  `state` is a pool [n,Hkv,64,64] float32, updated in place;
    sequence b has slot slots[b] (int32 CUDA; -1: no sequence, y is 0), or slot
    b without slots.  Returns y."""
    lib = load_library()
    _need(q.dim() == 3 and k.dim() == 3 and v.dim() == 3 and state.dim() == 4,
          "q, k and v must have 3 dimensions, state 4")
    B, Hq, d = q.shape
    Hkv, dv = k.shape[1], v.shape[2]
    dt, dev, n, t = _dtype_code(q), q.device, state.shape[0], q.dtype
    at = q.get_device()
    # (one expression: a token's call is worth a few microseconds)
    if not (k.dtype is t and v.dtype is t and g.dtype is torch.float32
            and state.dtype is torch.float32 and k.shape == (B, Hkv, d) and v.shape == (B, Hkv, dv)
            and g.shape == (B, Hkv) and state.shape == (n, Hkv, d, dv)
            and k.get_device() == at and v.get_device() == at and g.get_device() == at
            and state.get_device() == at and q.is_contiguous() and k.is_contiguous()
            and v.is_contiguous() and g.is_contiguous() and state.is_contiguous()):
        _need_tensor(q, "q", t, (B, Hq, d), dev)
        _need_tensor(k, "k", t, (B, Hkv, d), dev)
        _need_tensor(v, "v", t, (B, Hkv, dv), dev)
        _need_tensor(g, "g", torch.float32, (B, Hkv), dev)
        _need_tensor(state, "state", torch.float32, (n, Hkv, d, dv), dev)
    if slots is not None:
        _need_tensor(slots, "slots", torch.int32, (B,), dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return oal_gated_decode_step(q, k, v, g, state, scale, slots, y, stream)
    made = ()
    if y is None:
        y = torch.empty_like(q) if d == dv else q.new_empty(B, Hq, dv)
        made = (y,)
    else:
        _need_tensor(y, "y", q.dtype, (B, Hq, dv), dev)
    _check(lib.oal_gated_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, g.data_ptr(), B,
                                     Hq, Hkv, d, dv, scale, _ptr_or_null(slots), n,
                                     state.data_ptr(), y.data_ptr(),
                                     _stream_on(dev, stream, made)))
    return y


def oal_state_remap(pool, map, stream=None):
    """Moves the slots of `pool` (first dimension: slots) in place:
    new[i] = old[map[i]], zeros where map[i] is -1; map [n] int32 (CUDA).
    Copies, forks, compacts and frees states of any kind.  Returns pool."""
    lib = load_library()
    _need(pool.dim() >= 1, "pool must have a dimension of slots")
    n, dev = pool.shape[0], pool.device
    _need_tensor(pool, "pool", pool.dtype, pool.shape, dev)
    _need_tensor(map, "map", torch.int32, (n,), dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return oal_state_remap(pool, map, stream)
    _check(lib.oal_state_remap(pool.data_ptr(), pool.numel() // n * pool.element_size() if n else 0,
                               n, map.data_ptr(), _stream_on(dev, stream, ())))
    return pool


def oal_rope_plan(freq, axes=None, device="cuda"):
    """What the rotations need of their angles: freq [32] radians per position of
    each pair (host, float64), axes [32] the axis of each pair's positions (None:
    axis 0).  Returns an int64 tensor [2,32] on `device`, to be kept."""
    import numpy as np
    lib = load_library()
    freq = np.ascontiguousarray(np.asarray(freq, dtype=np.float64))
    _need(freq.shape == (32,), "freq must have 32 entries")
    if axes is not None:
        axes = np.ascontiguousarray(np.asarray(axes, dtype=np.int32))
        _need(axes.shape == (32,), "axes must have 32 entries")
    plan = np.empty((2, 32), np.int64)
    _check(lib.oal_rope_plan(freq.ctypes.data, None if axes is None else axes.ctypes.data,
                             plan.ctypes.data))
    return torch.from_numpy(plan).to(device)


def _rows(t, name, dtype, shape, at):
    """The strides of a tensor whose rows of 64 are contiguous."""
    s = t.stride()
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == at and s[3] == 1):
        raise OALError(OAL_ERR_INVALID_ARG, "%s must be %s %s on CUDA device %d, its rows contiguous (got %s %s on %s)"
                       % (name, dtype, tuple(shape), at, t.dtype, tuple(t.shape), t.device))
    # (the stride of a dimension of one says nothing)
    return s[:3] if min(shape) > 1 else tuple([x if n > 1 else 0 for x, n in zip(s, shape[:3])])


_strides6, _strides9 = struct.Struct("6q").pack, struct.Struct("9q").pack


# The calls below check their arguments in one expression each, of the cheapest
# questions that settle them (a token's call is worth a few microseconds); where
# that fails, the slow checks say why.
_I32, _I64, _F32, _BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16


def _vector(t, n, at, dtype=_I32):
    """Whether t is None or n contiguous numbers on device `at`."""
    return t is None or (t.dtype is dtype and t.dim() == 1 and t.numel() == n
                         and t.is_contiguous() and t.get_device() == at)


def _positions(positions, B, T, past, lengths, plan, at, x):
    """Number of axes of the positions; checks them, past, lengths and plan.  x: a tensor on device `at`."""
    if not ((plan is None or (plan.dtype is _I64 and plan.shape == (2, 32) and plan.is_contiguous()
                              and plan.get_device() == at))
            and _vector(past, B, at) and _vector(lengths, B, at)):
        if plan is not None:
            _need_tensor(plan, "plan", _I64, (2, 32), x.device)
        if past is not None:
            _need_tensor(past, "past", _I32, (B,), x.device)
        _need_lengths(lengths, B, x.device)
    if positions is None:
        return 0
    _need(positions.dim() == 3, "positions must have 3 dimensions")
    n = positions.shape[0]
    _need_tensor(positions, "positions", _I32, (n, B, T), x.device)
    return n


def _given(t, name, dtype, shape, at, x):
    """An output that the caller gives."""
    if not (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == at):
        _need_tensor(t, name, dtype, shape, x.device)


def _handle(at, x, stream, made):
    return torch._C._cuda_getCurrentRawStream(at) if stream is None else _stream_on(x.device, stream, made)


def oal_rope(Q, K, plan, positions=None, past=None, lengths=None, form=OAL_ROPE_HALVES,
             inverse=False, Yq=None, Yk=None, stream=None):
    """Rotary positions: Q [B,Hq,T,64] and K [B,Hkv,T,64] (or None), views whose
    rows are contiguous; plan of oal_rope_plan; positions [n_axes,B,T] int32, or
    past[b] + t (past [B] int32 or None) on every axis; lengths [B] int32 or None.
    inverse: by the opposite angles, for gradients.  Returns (Yq, Yk), contiguous;
    they may be given, also as Q and K themselves.  Rows behind a sequence's
    length stay as given; outputs made here have zeros there."""
    lib = load_library()
    _need(Q.dim() == 4 and (K is None or K.dim() == 4), "Q and K must have 4 dimensions")
    _need(plan is not None, "plan is needed")
    q = Q.shape
    B, Hq, T, d = q
    at, t = Q.get_device(), Q.dtype
    dt = _dtype_code(Q)
    _need(at >= 0, "tensors must be CUDA tensors")
    sq = _rows(Q, "Q", t, q, at)
    if K is None:
        Hkv, k, sk = 0, None, sq
    else:
        Hkv = K.size(1)
        k = (B, Hkv, T, d)
        sk = _rows(K, "K", t, k, at)
    n_axes = _positions(positions, B, T, past, lengths, plan, at, Q)
    if at != torch._C._cuda_getDevice():
        with torch.cuda.device(at):
            return oal_rope(Q, K, plan, positions, past, lengths, form, inverse, Yq, Yk, stream)
    made = []
    make = torch.empty if lengths is None else torch.zeros
    if Yq is None:
        Yq = make(q, dtype=t, device=Q.device)
        made.append(Yq)
    else:
        _given(Yq, "Yq", t, q, at, Q)
    if K is None:
        _need(Yk is None, "Yk without K")
    elif Yk is None:
        Yk = make(k, dtype=t, device=Q.device)
        made.append(Yk)
    else:
        _given(Yk, "Yk", t, k, at, Q)
    _check(lib.oal_rope(Q.data_ptr(), _ptr_or_null(K), dt, _strides6(*sq, *sk), B, Hq, Hkv, T, d,
                        plan.data_ptr(), form, _ptr_or_null(positions), n_axes, _ptr_or_null(past),
                        _ptr_or_null(lengths), bool(inverse), Yq.data_ptr(), _ptr_or_null(Yk),
                        _handle(at, Q, stream, made)))
    return Yq, Yk


def _pages(Kp, Vp, pages, Hkv, d, table, B, dtype, at):
    """Elements from page to page, entries of the table; checks the cache."""
    n, h, P, dk = pages
    if not (Kp.dtype is dtype and Vp.dtype is dtype and h == Hkv and dk == d and Vp.shape == pages
            and Kp.get_device() == at and Vp.get_device() == at):
        raise OALError(OAL_ERR_INVALID_ARG, "Kp and Vp must be %s [n_pages,%d,page_size,%d] on CUDA device %d"
                       % (dtype, Hkv, d, at))
    if not (table.dtype is _I32 and table.dim() == 2 and table.size(0) == B and table.is_contiguous()
            and table.get_device() == at):
        raise OALError(OAL_ERR_INVALID_ARG, "table must be contiguous int32 [%d,max_pages] on CUDA device %d" % (B, at))
    if Kp.is_contiguous() and Vp.is_contiguous():
        return h * P * d, table.size(1)
    sk, sv = Kp.stride(), Vp.stride()
    _need((n < 2 or sk[0] == sv[0]) and (h < 2 or sk[1] == sv[1] == P * d)
          and sk[2] == sv[2] == d and sk[3] == sv[3] == 1,
          "the pages of Kp and Vp must be contiguous and equally far apart")
    # (one page: how far the next would be is anyone's guess)
    return sk[0] if n > 1 else h * P * d, table.size(1)


def oal_page_append(Q, K, V, plan, Kp, Vp, table, past, positions=None, lengths=None,
                    form=OAL_ROPE_HALVES, Yq=None, stream=None):
    """T new tokens behind the past[b] of each sequence enter the paged cache: K
    [B,Hkv,T,64], turned as by oal_rope, and V as it is go to Kp and Vp
    [n_pages,Hkv,page_size,64] by table [B,max_pages] int32; past [B] int32.  Q
    [B,Hq,T,64] is turned along into Yq (both may be None); plan None: nothing
    is turned.  Q, K, V may be views whose rows are contiguous.  Returns Yq."""
    lib = load_library()
    _need(K.dim() == 4 and V.dim() == 4 and Kp.dim() == 4 and (Q is None or Q.dim() == 4),
          "Q, K, V, Kp and Vp must have 4 dimensions")
    _need(past is not None, "past is needed")
    k, pages = K.shape, Kp.shape
    B, Hkv, T, d = k
    at, t = K.get_device(), K.dtype
    dt = _dtype_code(K)
    _need(at >= 0, "tensors must be CUDA tensors")
    sk = _rows(K, "K", t, k, at)
    sv = _rows(V, "V", t, k, at)
    if Q is None:
        Hq, q, sq = 0, None, sk
    else:
        Hq = Q.size(1)
        q = (B, Hq, T, d)
        sq = _rows(Q, "Q", t, q, at)
    n_axes = _positions(positions, B, T, past, lengths, plan, at, K)
    apart, most = _pages(Kp, Vp, pages, Hkv, d, table, B, t, at)
    if at != torch._C._cuda_getDevice():
        with torch.cuda.device(at):
            return oal_page_append(Q, K, V, plan, Kp, Vp, table, past, positions, lengths, form, Yq,
                                   stream)
    made = []
    if Q is None:
        _need(Yq is None, "Yq without Q")
    elif Yq is None:
        Yq = (torch.empty if lengths is None else torch.zeros)(q, dtype=t, device=K.device)
        made.append(Yq)
    else:
        _given(Yq, "Yq", t, q, at, K)
    _check(lib.oal_page_append(_ptr_or_null(Q), K.data_ptr(), V.data_ptr(), dt,
                               _strides9(*sq, *sk, *sv), B, Hq, Hkv, T, d, d, _ptr_or_null(plan),
                               form, _ptr_or_null(positions), n_axes, past.data_ptr(),
                               _ptr_or_null(lengths), Kp.data_ptr(), Vp.data_ptr(), pages[0],
                               pages[2], apart, table.data_ptr(), most, _ptr_or_null(Yq),
                               _handle(at, K, stream, made)))
    return Yq


@functools.lru_cache(maxsize=4096)
def _paged_attention_bytes(*sizes):
    return max(int(load_library().oal_paged_attention_workspace_bytes(*sizes)), 256)


def oal_paged_attention_workspace_bytes(B, Hq, Hkv, T, page_size, max_pages, d=64, dv=64,
                                        dtype=OAL_BF16):
    return int(load_library().oal_paged_attention_workspace_bytes(B, Hq, Hkv, T, d, dv, dtype,
                                                                  page_size, max_pages))


def oal_paged_attention(Q, Kp, Vp, table, past, lengths=None, scale=0.125, cap=0.0, window=0,
                        slopes=None, prefix=None, first=None, Y=None, workspace=None, stream=None):
    """Softmax attention of T >= 1 new tokens, already appended, over the paged
    cache: Q [B,Hq,T,64]; Kp, Vp, table, past, lengths as for oal_page_append.
    Token t at i = past[b] + t sees key j if first[b,t] <= j, i - window < j
    (window 0: no such limit), and j <= i or j < prefix[b].  Scores scale q.k are
    capped by cap tanh(s / cap) (cap 0: not) and take -slopes[h] |i - j|.
    slopes [Hq] float32, prefix [B] int32, first [B,T] int32, or None.  Returns
    Y; rows behind a sequence's length stay as given (a Y made here has zeros
    there), tokens that see nothing get zeros."""
    lib = load_library()
    _need(0 <= window < 1 << 31, "window must be 0 .. 2^31 - 1")   # (a C int would take it modulo 2^32)
    _need(Q.dim() == 4 and Kp.dim() == 4, "Q, Kp and Vp must have 4 dimensions")
    q, pages = Q.shape, Kp.shape
    B, Hq, T, d = q
    n, Hkv, P, _ = pages
    at, t = Q.get_device(), Q.dtype
    dt = _dtype_code(Q)
    _need(at >= 0 and Q.is_contiguous(), "Q must be a contiguous CUDA tensor")
    apart, most = _pages(Kp, Vp, pages, Hkv, d, table, B, t, at)
    if not (past is not None and _vector(past, B, at) and _vector(lengths, B, at)
            and _vector(slopes, Hq, at, _F32) and _vector(prefix, B, at)):
        dev = Q.device
        _need(past is not None, "past is needed")
        _need_tensor(past, "past", _I32, (B,), dev)
        _need_lengths(lengths, B, dev)
        if slopes is not None:
            _need_tensor(slopes, "slopes", _F32, (Hq,), dev)
        if prefix is not None:
            _need_tensor(prefix, "prefix", _I32, (B,), dev)
    if first is not None:
        _need_tensor(first, "first", _I32, (B, T), Q.device)
    if at != torch._C._cuda_getDevice():
        with torch.cuda.device(at):
            return oal_paged_attention(Q, Kp, Vp, table, past, lengths, scale, cap, window, slopes,
                                       prefix, first, Y, workspace, stream)
    made = []
    if Y is None:
        Y = (torch.empty if lengths is None else torch.zeros)(q, dtype=t, device=Q.device)
        made.append(Y)
    else:
        _given(Y, "Y", t, q, at, Q)
    handle = _handle(at, Q, stream, made)
    # A workspace of the call's own comes from the allocator as memory of the stream
    # that it launches on, and goes back in that stream's order.
    room, own = _paged_attention_bytes(B, Hq, Hkv, T, d, d, dt, P, most), None
    if workspace is not None:
        _need_tensor(workspace, "workspace", workspace.dtype, workspace.shape, Q.device)
        room, where = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    elif room > 256:
        where = own = torch._C._cuda_cudaCachingAllocator_raw_alloc(room, handle)
    else:
        where = None
    try:
        status = lib.oal_paged_attention(
            Q.data_ptr(), dt, B, Hq, Hkv, T, d, d, Kp.data_ptr(), Vp.data_ptr(), n, P, apart,
            table.data_ptr(), most, past.data_ptr(), None if lengths is None else lengths.data_ptr(),
            scale, cap, window, None if slopes is None else slopes.data_ptr(),
            None if prefix is None else prefix.data_ptr(), None if first is None else first.data_ptr(),
            Y.data_ptr(), where, room, handle)
    finally:
        if own is not None:
            torch._C._cuda_cudaCachingAllocator_raw_delete(own)
    _check(status)
    return Y


def oal_sync_status(stream=None):
    lib = load_library()
    _check(lib.oal_sync_status(_stream(stream)))


def oal_debug_wait_test(wait_limit_cycles=0, starve=0):
    """Test-only: the limit of the kernels' bounded waits in SM cycles (0: the
    built-in limit) and the prefill kernel whose UMMA issuer waits on a barrier
    nothing arrives on (0 none, 1 readout, 2 state, 3 intra-chunk), for kernels
    launched afterwards on the current device.  (0, 0) restores normal operation."""
    _check(load_library().oal_debug_wait_test(int(wait_limit_cycles), int(starve)))


def oal_debug_intra_heads(heads=0):
    """Test-only: query heads per block of the bf16 prefill's intra-chunk kernel
    at chunk sizes 64 and 128 (1 or 2; 0 restores the automatic choice)."""
    _check(load_library().oal_debug_intra_heads(int(heads)))


def oal_last_error():
    return load_library().oal_last_error().decode()
