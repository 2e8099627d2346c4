"""Thin ctypes binding over libgdn.so (the headers in include/).

Argument marshalling only: tensors are checked for device, dtype, layout and
alignment, outputs and workspaces are allocated with PyTorch when the caller
does not pass them, and the raw device pointers plus the current CUDA stream
go to the C entry points, which run every step of the computation in the
library's own kernels.  There is no fallback: if the library is missing or a
call fails, a RuntimeError is raised.
"""
import ctypes
import functools
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgdn.so")
_lib = None

GDN_OK = 0
GDN_F32, GDN_BF16 = 0, 1
OP_FWD, OP_DECODE, OP_BWD = 0, 1, 2
DEVERR_CU_SEQLENS, DEVERR_TIMEOUT, DEVERR_SMEM_ALIGN = 1, 2, 4

_P = ctypes.c_void_p

SYMBOLS = ("gdn_workspace_size", "gdn_recurrent_fwd", "gdn_decode_step", "gdn_chunk_bwd",
           "gdn_read_device_error", "gdn_status_string", "gdn_recurrent_fwd_noalloc",
           "gdn_recurrent_fwd_snapshots", "gdn_gates", "gdn_gated_rmsnorm", "gdn_causal_conv1d_fwd",
           "gdn_causal_conv1d_update", "gdn_replay_block_floats", "gdn_replay_workspace_size",
           "gdn_replay_prefill", "gdn_replay_decode", "gdn_causal_conv1d_bwd",
           "gdn_causal_conv1d_bwd_workspace_size", "gdn_qk_norm_rope", "gdn_qk_norm_rope_bwd",
           "gdn_qk_norm_rope_bwd_workspace_size", "gdn_selective_scan_fwd", "gdn_selective_scan_update",
           "gdn_selective_scan_bwd", "gdn_selective_scan_bwd_workspace_size")


class GdnShape(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("T_total", ctypes.c_int), ("HK", ctypes.c_int),
                ("HV", ctypes.c_int), ("dk", ctypes.c_int), ("dv", ctypes.c_int),
                ("dtype", ctypes.c_int), ("use_qk_l2norm", ctypes.c_int), ("dv_slice", ctypes.c_int)]


class ConvShape(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("T_total", ctypes.c_int), ("C", ctypes.c_int), ("W", ctypes.c_int),
                ("dtype", ctypes.c_int), ("activation", ctypes.c_int)]


class QkShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("HQ", ctypes.c_int), ("HK", ctypes.c_int), ("d", ctypes.c_int),
                ("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("norm", ctypes.c_int),
                ("max_positions", ctypes.c_int), ("eps", ctypes.c_float), ("dtype", ctypes.c_int),
                ("ldq", ctypes.c_int64), ("ldk", ctypes.c_int64)]


class ScanShape(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("T_total", ctypes.c_int), ("C", ctypes.c_int), ("G", ctypes.c_int),
                ("S", ctypes.c_int), ("dtype", ctypes.c_int), ("dt_softplus", ctypes.c_int),
                ("ldx", ctypes.c_int64), ("lddt", ctypes.c_int64), ("ldz", ctypes.c_int64),
                ("ldB", ctypes.c_int64), ("ldC", ctypes.c_int64)]


class GdnError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} ({code})")


def lib():
    """Load libgdn.so once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with invariant_linear_attention_gb300."
                               "build_lib.build() (or __graft_entry__.build())")
        L = ctypes.CDLL(_LIB_PATH)
        L.gdn_workspace_size.argtypes = [ctypes.POINTER(GdnShape), ctypes.c_int]
        L.gdn_workspace_size.restype = ctypes.c_size_t
        L.gdn_recurrent_fwd.argtypes = [ctypes.POINTER(GdnShape)] + [_P] * 10 + [ctypes.c_size_t, _P]
        L.gdn_recurrent_fwd.restype = ctypes.c_int
        L.gdn_recurrent_fwd_noalloc.argtypes = [ctypes.POINTER(GdnShape)] + [_P] * 10
        L.gdn_recurrent_fwd_noalloc.restype = ctypes.c_int
        L.gdn_recurrent_fwd_snapshots.argtypes = ([ctypes.POINTER(GdnShape)] + [_P] * 9 +
                                                  [ctypes.c_int, _P, ctypes.c_int, _P, _P, ctypes.c_size_t, _P])
        L.gdn_recurrent_fwd_snapshots.restype = ctypes.c_int
        L.gdn_decode_step.argtypes = [ctypes.POINTER(GdnShape)] + [_P] * 7 + [ctypes.c_int, _P, _P]
        L.gdn_decode_step.restype = ctypes.c_int
        L.gdn_chunk_bwd.argtypes = [ctypes.POINTER(GdnShape)] + [_P] * 16 + [ctypes.c_size_t, _P]
        L.gdn_chunk_bwd.restype = ctypes.c_int
        L.gdn_read_device_error.argtypes = [_P, ctypes.POINTER(ctypes.c_uint), _P]
        L.gdn_read_device_error.restype = ctypes.c_int
        L.gdn_gates.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int] + [_P] * 7
        L.gdn_gates.restype = ctypes.c_int
        L.gdn_gated_rmsnorm.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, _P, _P, _P, ctypes.c_float,
                                        _P, _P]
        L.gdn_gated_rmsnorm.restype = ctypes.c_int
        L.gdn_causal_conv1d_fwd.argtypes = [ctypes.POINTER(ConvShape)] + [_P] * 6 + [ctypes.c_int, _P, _P, _P]
        L.gdn_causal_conv1d_fwd.restype = ctypes.c_int
        L.gdn_causal_conv1d_update.argtypes = [ctypes.POINTER(ConvShape)] + [_P] * 5 + [ctypes.c_int, _P, _P]
        L.gdn_causal_conv1d_update.restype = ctypes.c_int
        L.gdn_replay_block_floats.argtypes = [ctypes.c_int, ctypes.c_int]
        L.gdn_replay_block_floats.restype = ctypes.c_size_t
        L.gdn_replay_workspace_size.argtypes = [ctypes.POINTER(GdnShape)]
        L.gdn_replay_workspace_size.restype = ctypes.c_size_t
        L.gdn_replay_prefill.argtypes = [ctypes.POINTER(GdnShape)] + [_P] * 9 + [ctypes.c_int, _P, _P,
                                                                                ctypes.c_size_t, _P]
        L.gdn_replay_prefill.restype = ctypes.c_int
        L.gdn_replay_decode.argtypes = [ctypes.POINTER(GdnShape)] + [_P] * 8 + [ctypes.c_int, _P, _P]
        L.gdn_replay_decode.restype = ctypes.c_int
        i, n, z = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        conv, qk, scan = (ctypes.POINTER(c) for c in (ConvShape, QkShape, ScanShape))
        for name, args, res in (
                ("gdn_causal_conv1d_bwd_workspace_size", [conv], z),
                ("gdn_causal_conv1d_bwd", [conv] + [_P] * 12 + [z, _P], i),
                ("gdn_qk_norm_rope", [qk] + [_P] * 10, i),
                ("gdn_qk_norm_rope_bwd_workspace_size", [qk], z),
                ("gdn_qk_norm_rope_bwd", [qk] + [_P] * 11 + [n, n] + [_P] * 3 + [z, _P], i),
                ("gdn_selective_scan_fwd", [scan] + [_P] * 11 + [i, _P, _P, _P], i),
                ("gdn_selective_scan_update", [scan] + [_P] * 10 + [i, _P, _P], i),
                ("gdn_selective_scan_bwd_workspace_size", [scan], z),
                ("gdn_selective_scan_bwd", [scan] + [_P] * 22 + [z, _P], i)):
            getattr(L, name).argtypes, getattr(L, name).restype = args, res
        L.gdn_status_string.argtypes = [ctypes.c_int]
        L.gdn_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().gdn_status_string(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _need(t, name, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def make_shape(q, v, N, use_qk_l2norm=True, dv_slice=0, T_total=None):
    T, HK, dk = q.shape
    HV, dv = v.shape[1], v.shape[2]
    return GdnShape(int(N), int(T if T_total is None else T_total), int(HK), int(HV), int(dk), int(dv),
                    _dtype_code(q), int(bool(use_qk_l2norm)), int(dv_slice))


def gdn_workspace_size(shape: GdnShape, op: int) -> int:
    return int(lib().gdn_workspace_size(ctypes.byref(shape), int(op)))


def _check(rc, what):
    if rc != GDN_OK:
        raise GdnError(rc, what)


def gdn_recurrent_fwd(q, k, v, g, beta, cu_seqlens, init_state=None, out=None, final_state=None,
                      workspace=None, use_qk_l2norm=True, dv_slice=0, output_final_state=True,
                      stream=None):
    """Batch-invariant recurrent forward over a packed varlen batch.

    q, k [T, HK, dk] and v [T, HV, dv] (bf16 or fp32, same dtype), g, beta
    [T, HV] fp32, cu_seqlens int32 [N+1] on the device, init_state
    [N, HV, dv, dk] fp32 or None.  Returns (out [T, HV, dv], final_state
    [N, HV, dv, dk] fp32 or None).  final_state may be init_state (in place).
    """
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, dev)
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    N = cu_seqlens.numel() - 1
    T, HK, dk = q.shape
    HV, dv = v.shape[1], v.shape[2]
    if k.shape != q.shape or v.shape[0] != T or g.shape != (T, HV) or beta.shape != (T, HV):
        raise ValueError("inconsistent shapes")
    if init_state is not None:
        _need(init_state, "init_state", torch.float32, dev)
        if init_state.shape != (N, HV, dv, dk):
            raise ValueError("init_state must be [N, HV, dv, dk]")
    shape = make_shape(q, v, N, use_qk_l2norm, dv_slice)
    if out is None:
        out = torch.empty_like(v)
    _need(out, "out", q.dtype, dev)
    if final_state is None and output_final_state:
        final_state = torch.empty(N, HV, dv, dk, dtype=torch.float32, device=dev)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32, dev)
    need = gdn_workspace_size(shape, OP_FWD)
    if workspace is None:
        workspace = torch.zeros(max(need, 256), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    with torch.cuda.device(dev):
        rc = lib().gdn_recurrent_fwd(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                     _ptr(init_state), _ptr(cu_seqlens), _ptr(out), _ptr(final_state),
                                     _ptr(workspace), ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check(rc, "gdn_recurrent_fwd")
    return out, final_state


def gdn_recurrent_fwd_noalloc(q, k, v, g, beta, cu_seqlens, init_state=None, out=None, final_state=None,
                              use_qk_l2norm=True, dv_slice=0, output_final_state=True, stream=None):
    """gdn_recurrent_fwd through the entry point that needs no workspace (its
    scratch is a fixed array inside the library; calls must not overlap on the
    GPU).  Same arguments and results as gdn_recurrent_fwd minus `workspace`;
    out / final_state are allocated here only when the caller passes none."""
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, dev)
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    N = cu_seqlens.numel() - 1
    T, HK, dk = q.shape
    HV, dv = v.shape[1], v.shape[2]
    if init_state is not None:
        _need(init_state, "init_state", torch.float32, dev)
    shape = make_shape(q, v, N, use_qk_l2norm, dv_slice)
    if out is None:
        out = torch.empty_like(v)
    if final_state is None and output_final_state:
        final_state = torch.empty(N, HV, dv, dk, dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        rc = lib().gdn_recurrent_fwd_noalloc(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                             _ptr(beta), _ptr(init_state), _ptr(cu_seqlens), _ptr(out),
                                             _ptr(final_state), _stream(stream))
    _check(rc, "gdn_recurrent_fwd_noalloc")
    return out, final_state


def snapshot_offsets(lengths, snap_every):
    """int32 [N+1] slot offsets giving each sequence floor(len / snap_every) snapshot slots."""
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + int(n) // int(snap_every))
    return torch.tensor(cu, dtype=torch.int32)


def gdn_recurrent_fwd_snapshots(q, k, v, g, beta, cu_seqlens, snap_every, snap_cu=None, snap_states=None,
                                init_state=None, out=None, final_state=None, workspace=None,
                                use_qk_l2norm=True, dv_slice=0, stream=None):
    """gdn_recurrent_fwd plus fp32 state snapshots after every snap_every-th token of
    each sequence (prefix caching).  snap_cu: int32 [N+1] device slot offsets (built
    from cu_seqlens with a host copy when None).  Returns (out, final_state,
    snap_states [slots, HV, dv, dk], snap_cu)."""
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, dev)
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    N = cu_seqlens.numel() - 1
    T, HK, dk = q.shape
    HV, dv = v.shape[1], v.shape[2]
    if init_state is not None:
        _need(init_state, "init_state", torch.float32, dev)
    if snap_cu is None:
        cuh = cu_seqlens.cpu().tolist()
        snap_cu = snapshot_offsets([cuh[i + 1] - cuh[i] for i in range(N)], snap_every).to(dev)
    _need(snap_cu, "snap_cu", torch.int32, dev)
    slots = int(snap_cu[-1].item()) if snap_states is None else int(snap_states.shape[0])
    if snap_states is None:
        snap_states = torch.empty(max(slots, 0), HV, dv, dk, dtype=torch.float32, device=dev)
    _need(snap_states, "snap_states", torch.float32, dev)
    shape = make_shape(q, v, N, use_qk_l2norm, dv_slice)
    if out is None:
        out = torch.empty_like(v)
    if final_state is None:
        final_state = torch.empty(N, HV, dv, dk, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.zeros(max(gdn_workspace_size(shape, OP_FWD), 256), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        rc = lib().gdn_recurrent_fwd_snapshots(
            ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(init_state),
            _ptr(cu_seqlens), _ptr(out), _ptr(final_state), int(snap_every), _ptr(snap_cu), slots,
            _ptr(snap_states) if slots > 0 else None, _ptr(workspace), ctypes.c_size_t(workspace.numel()),
            _stream(stream))
    _check(rc, "gdn_recurrent_fwd_snapshots")
    return out, final_state, snap_states, snap_cu


def gdn_decode_step(q, k, v, g, beta, state, state_indices=None, out=None, use_qk_l2norm=True,
                    dv_slice=0, stream=None):
    """One token per sequence on the cached fp32 state pool, updated in place.

    q, k [B, HK, dk], v [B, HV, dv], g, beta [B, HV]; state [slots, HV, dv, dk]
    fp32; state_indices int32 [B] or None (slot b).  Returns out [B, HV, dv].
    """
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, dev)
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    _need(state, "state", torch.float32, dev)
    B = q.shape[0]
    if state_indices is not None:
        _need(state_indices, "state_indices", torch.int32, dev)
    shape = make_shape(q, v, B, use_qk_l2norm, dv_slice)
    if out is None:
        out = torch.empty_like(v)
    _need(out, "out", q.dtype, dev)
    with torch.cuda.device(dev):
        rc = lib().gdn_decode_step(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                   _ptr(state), _ptr(state_indices), int(state.shape[0]), _ptr(out),
                                   _stream(stream))
    _check(rc, "gdn_decode_step")
    return out


def gdn_chunk_bwd(q, k, v, g, beta, cu_seqlens, d_out, init_state=None, d_final_state=None,
                  workspace=None, use_qk_l2norm=True, need_d_init_state=True, stream=None):
    """Chunked (WY) backward.  Returns dict dq, dk, dv (dtype of q), dg, dbeta, d_init_state (fp32)."""
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (d_out, "d_out")):
        _need(t, n, q.dtype, dev)
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    N = cu_seqlens.numel() - 1
    T, HK, dk = q.shape
    HV, dv = v.shape[1], v.shape[2]
    for t, n in ((init_state, "init_state"), (d_final_state, "d_final_state")):
        if t is not None:
            _need(t, n, torch.float32, dev)
    shape = make_shape(q, v, N, use_qk_l2norm, 0)
    res = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               dg=torch.empty(T, HV, dtype=torch.float32, device=dev),
               dbeta=torch.empty(T, HV, dtype=torch.float32, device=dev),
               d_init_state=torch.empty(N, HV, dv, dk, dtype=torch.float32, device=dev)
               if need_d_init_state else None)
    need = gdn_workspace_size(shape, OP_BWD)
    if workspace is None:
        workspace = torch.zeros(max(need, 256), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    with torch.cuda.device(dev):
        rc = lib().gdn_chunk_bwd(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                 _ptr(init_state), _ptr(cu_seqlens), _ptr(d_out), _ptr(d_final_state),
                                 _ptr(res["dq"]), _ptr(res["dk"]), _ptr(res["dv"]), _ptr(res["dg"]),
                                 _ptr(res["dbeta"]), _ptr(res["d_init_state"]), _ptr(workspace),
                                 ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check(rc, "gdn_chunk_bwd")
    return res


def read_device_error(workspace, stream=None) -> int:
    """Device error bits left in a FWD/BWD workspace (synchronises the stream)."""
    bits = ctypes.c_uint(0)
    rc = lib().gdn_read_device_error(_ptr(workspace), ctypes.byref(bits), _stream(stream))
    _check(rc, "gdn_read_device_error")
    return int(bits.value)


# ---------------------------------------------------------------- layer ops (include/gdn_layer.h)

def gdn_gates(a, b, A_log, dt_bias=None, g=None, beta=None, stream=None):
    """(g, beta) [T, HV] fp32 from the raw projections a, b [T, HV] (bf16 or fp32):
    g = -exp(A_log) * softplus(a + dt_bias), beta = sigmoid(b)."""
    dev = a.device
    _need(a, "a", None, dev)
    _need(b, "b", a.dtype, dev)
    _need(A_log, "A_log", torch.float32, dev)
    if dt_bias is not None:
        _need(dt_bias, "dt_bias", torch.float32, dev)
    if a.dim() != 2 or b.shape != a.shape or A_log.shape != (a.shape[1],):
        raise ValueError("a, b must be [T, HV] and A_log [HV]")
    T, HV = a.shape
    g = torch.empty(T, HV, dtype=torch.float32, device=dev) if g is None else g
    beta = torch.empty(T, HV, dtype=torch.float32, device=dev) if beta is None else beta
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    with torch.cuda.device(dev):
        rc = lib().gdn_gates(int(T), int(HV), _dtype_code(a), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias),
                             _ptr(g), _ptr(beta), _stream(stream))
    _check(rc, "gdn_gates")
    return g, beta


def gdn_gated_rmsnorm(o, z, weight, eps=1e-6, out=None, stream=None):
    """y = o / sqrt(mean(o^2, -1) + eps) * weight * silu(z) over the last axis of
    o [..., d] (bf16 or fp32); z like o or None; weight [d] fp32.  out may be o."""
    dev = o.device
    _need(o, "o", None, dev)
    if z is not None:
        _need(z, "z", o.dtype, dev)
        if z.shape != o.shape:
            raise ValueError("z must have o's shape")
    _need(weight, "weight", torch.float32, dev)
    d = o.shape[-1]
    if weight.shape != (d,):
        raise ValueError("weight must be [d]")
    out = torch.empty_like(o) if out is None else out
    _need(out, "out", o.dtype, dev)
    with torch.cuda.device(dev):
        rc = lib().gdn_gated_rmsnorm(int(o.numel() // d), int(d), _dtype_code(o), _ptr(o), _ptr(z), _ptr(weight),
                                     float(eps), _ptr(out), _stream(stream))
    _check(rc, "gdn_gated_rmsnorm")
    return out


def _conv_shape(x, weight, N, activation):
    T, C = x.shape
    if weight.dim() != 2 or weight.shape[0] != C:
        raise ValueError("weight must be [C, W]")
    return ConvShape(int(N), int(T), int(C), int(weight.shape[1]), _dtype_code(x), int(bool(activation)))


def gdn_causal_conv1d_fwd(x, weight, cu_seqlens, bias=None, conv_state=None, state_indices=None,
                          has_initial_state=None, activation=True, out=None, stream=None):
    """Causal depthwise conv over packed varlen x [T, C] with taps weight [C, W]
    fp32.  conv_state [slots, W-1, C] (dtype of x) is read as the initial state
    and overwritten with the final state of each sequence's slot (in place).
    Returns y [T, C]."""
    dev = x.device
    _need(x, "x", None, dev)
    _need(weight, "weight", torch.float32, dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    for t, n, dt in ((bias, "bias", torch.float32), (conv_state, "conv_state", x.dtype),
                     (state_indices, "state_indices", torch.int32),
                     (has_initial_state, "has_initial_state", torch.int32)):
        if t is not None:
            _need(t, n, dt, dev)
    N = cu_seqlens.numel() - 1
    shape = _conv_shape(x, weight, N, activation)
    if conv_state is not None and tuple(conv_state.shape[1:]) != (shape.W - 1, shape.C):
        raise ValueError("conv_state must be [slots, W-1, C]")
    out = torch.empty_like(x) if out is None else out
    _need(out, "out", x.dtype, dev)
    slots = 0 if conv_state is None else int(conv_state.shape[0])
    with torch.cuda.device(dev):
        rc = lib().gdn_causal_conv1d_fwd(ctypes.byref(shape), _ptr(x), _ptr(weight), _ptr(bias), _ptr(cu_seqlens),
                                         _ptr(conv_state), _ptr(state_indices), slots, _ptr(has_initial_state),
                                         _ptr(out), _stream(stream))
    _check(rc, "gdn_causal_conv1d_fwd")
    return out


def gdn_causal_conv1d_update(x, weight, conv_state, state_indices=None, bias=None, activation=True, out=None,
                             stream=None):
    """One decode token per sequence: x [B, C]; conv_state [slots, W-1, C]
    updated in place.  Returns y [B, C] (rows of skipped sequences untouched)."""
    dev = x.device
    _need(x, "x", None, dev)
    _need(weight, "weight", torch.float32, dev)
    _need(conv_state, "conv_state", x.dtype, dev)
    for t, n, dt in ((bias, "bias", torch.float32), (state_indices, "state_indices", torch.int32)):
        if t is not None:
            _need(t, n, dt, dev)
    shape = _conv_shape(x, weight, x.shape[0], activation)
    if tuple(conv_state.shape[1:]) != (shape.W - 1, shape.C):
        raise ValueError("conv_state must be [slots, W-1, C]")
    out = torch.empty_like(x) if out is None else out
    _need(out, "out", x.dtype, dev)
    with torch.cuda.device(dev):
        rc = lib().gdn_causal_conv1d_update(ctypes.byref(shape), _ptr(x), _ptr(weight), _ptr(bias),
                                            _ptr(conv_state), _ptr(state_indices), int(conv_state.shape[0]),
                                            _ptr(out), _stream(stream))
    _check(rc, "gdn_causal_conv1d_update")
    return out


# ---------------------------------------------------------------- gradients, q/k norm with rotation, selective scan
#
# A decode step calls these once per layer with little to compute: the checks read each attribute
# once, in one expression that holds for a good argument, and look for what is wrong only after it
# does not; shape structs and workspace sizes are kept by their values.

def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _on(call, args):
    """call(**args) on the stream that args name: its outputs and workspace belong to that stream, and
    the tensors it is given are recorded on it, so that memory freed right after the call is not
    reused while the stream still reads it."""
    stream = args.pop("stream")
    tensors = [t for t in args.values() if isinstance(t, torch.Tensor) and t.is_cuda]
    for t in tensors:
        if t.device != stream.device:
            raise ValueError(f"stream is on {stream.device}, a tensor on {t.device}")
    if stream != torch.cuda.current_stream(stream.device):
        for t in tensors:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return call(**args)


def _invoke(name, index, *args):
    """The C entry point on the current stream of device `index`."""
    entry = getattr(lib(), name)
    if torch.cuda.current_device() == index:
        rc = entry(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = entry(*args, _raw_stream(index))
    if rc != GDN_OK:
        raise GdnError(rc, name)


def _wrong(t, name, shape, dtype, index):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def _is(t, name, shape, dtype, index):
    """Address of t, a dense tensor of this shape (None: null)."""
    if t is None:
        return None
    try:
        if t.get_device() == index and t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _wrong(t, name, shape, dtype, index)
    raise ValueError(f"{name} must be contiguous")


def _rows(t, name, shape, dtype, index):
    """Address of t, a tensor of this shape with dense rows t[i], and the elements from one row to the next."""
    try:
        if t.get_device() == index and t.dtype is dtype and t.shape == shape:
            dense = shape[1] if len(shape) == 2 else shape[1] * shape[2]
            if t.is_contiguous():
                return t.data_ptr(), dense
            step = t.stride()
            inner = step[-1] == 1 or shape[-1] == 1
            if len(step) == 3:
                inner = inner and (step[1] == shape[2] or shape[1] == 1)
            if inner and (step[0] >= dense or shape[0] == 1):
                return t.data_ptr(), dense if shape[0] == 1 else step[0]
    except AttributeError:
        pass
    _wrong(t, name, shape, dtype, index)
    raise ValueError(f"the rows of {name} must be contiguous and must not overlap")


def _first(t, name, dims):
    """Shape, dtype and device index of the tensor that the others are checked against."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    return t.shape, t.dtype, t.get_device()


def _dims(t, name, n):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got {t.dim()}")
    return t.shape


def _sequences(cu_seqlens, index):
    """Number of sequences and address of cu_seqlens."""
    n = _dims(cu_seqlens, "cu_seqlens", 1)[0]
    if n < 1:
        raise ValueError("cu_seqlens must have at least one entry")
    return n - 1, _is(cu_seqlens, "cu_seqlens", (n,), torch.int32, index)


def _like(t):
    """A dense tensor like t to write to (t's rows may be slices); t None: None."""
    return None if t is None else torch.empty_like(t)


def _space(workspace, need, device):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    _need(workspace, "workspace", torch.uint8, device)
    return workspace


@functools.lru_cache(4096)
def _struct(kind, *values):
    shape = kind(*values)
    for (name, ty), value in zip(kind._fields_, values):  # ctypes would cut a larger number to its low bits
        if ty is not ctypes.c_float and getattr(shape, name) != value:
            raise ValueError(f"{name} is too large: {value}")
    return ctypes.byref(shape)


@functools.lru_cache(4096)
def _space_of(entry, kind, *values):
    return max(int(getattr(lib(), entry)(_struct(kind, *values))), 16)


def gdn_causal_conv1d_bwd(x, weight, cu_seqlens, d_out, bias=None, init_state=None, d_final_state=None,
                          activation=True, workspace=None, need_d_init_state=True, stream=None):
    """Gradient of gdn_causal_conv1d_fwd.  x, d_out [T, C]; weight [C, W], bias [C]
    fp32; init_state, d_final_state [N, W-1, C] (dtype of x) or None (zero), in
    the order of the sequences.  Returns dict dx (dtype of x), dweight, dbias
    (fp32, dbias None without a bias), d_init_state (dtype of x or None).  Rows
    of dx behind cu_seqlens[N] are not written."""
    if stream is not None:
        return _on(gdn_causal_conv1d_bwd, locals())
    shape, ty, index = _first(x, "x", 2)
    (T, C), W, f32 = shape, _dims(weight, "weight", 2)[1], torch.float32
    N, cu = _sequences(cu_seqlens, index)
    state = (N, W - 1, C)
    ptrs = (_is(x, "x", shape, ty, index), _is(weight, "weight", (C, W), f32, index), _is(bias, "bias", (C,), f32, index),
            cu, _is(init_state, "init_state", state, ty, index), _is(d_out, "d_out", shape, ty, index),
            _is(d_final_state, "d_final_state", state, ty, index))
    sizes = (ConvShape, N, T, C, W, _dtype_code(x), int(bool(activation)))
    dx, dw, db = _like(x), _like(weight), _like(bias)
    dh = torch.empty(state, dtype=ty, device=x.device) if need_d_init_state else None
    ws = _space(workspace, _space_of("gdn_causal_conv1d_bwd_workspace_size", *sizes), x.device)
    _invoke("gdn_causal_conv1d_bwd", index, _struct(*sizes), *ptrs, dx.data_ptr(), dw.data_ptr(), _at(db), _at(dh),
            ws.data_ptr(), ws.numel())
    return dict(dx=dx, dweight=dw, dbias=db, d_init_state=dh)


def _at(t):
    return None if t is None else t.data_ptr()


_NORMS = {"rms": 0, "l2": 1}


def _qk(q, k, cos, sin, positions, q_weight, k_weight, norm, eps, interleaved):
    """Sizes for the struct, the inputs' addresses, the device index."""
    qs, ty, index = _first(q, "q", 3)
    ks, angles = _dims(k, "k", 3), _dims(cos, "cos", 2)
    (T, HQ, d), HK, f32 = qs, ks[1], torch.float32
    if norm not in _NORMS:
        raise ValueError(f"norm must be one of {sorted(_NORMS)}, got {norm!r}")
    (qp, ldq), (kp, ldk) = _rows(q, "q", qs, ty, index), _rows(k, "k", (T, HK, d), ty, index)
    ptrs = (qp, kp, _is(q_weight, "q_weight", (d,), f32, index), _is(k_weight, "k_weight", (d,), f32, index),
            _is(cos, "cos", angles, f32, index), _is(sin, "sin", angles, f32, index),
            _is(positions, "positions", (T,), torch.int32, index))
    return (QkShape, T, HQ, HK, d, 2 * angles[1], int(bool(interleaved)), _NORMS[norm], angles[0], float(eps),
            _dtype_code(q), ldq, ldk), ptrs, index


def gdn_qk_norm_rope(q, k, cos, sin, positions=None, q_weight=None, k_weight=None, norm="rms", eps=1e-6,
                     interleaved=False, q_out=None, k_out=None, stream=None):
    """Norm of each head of q [T, HQ, d] and k [T, HK, d] (norm "rms":
    x / sqrt(mean(x^2) + eps), "l2": x / sqrt(sum(x^2) + eps), times a weight [d]
    fp32 or None) and rotation of its first 2 * cos.shape[1] values by row
    positions[t] (int32, None: row t) of cos, sin [max_positions, rotary_dim / 2]
    fp32: pairs (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved.  q and k
    may be column slices of wider rows.  Returns dense (q_out, k_out).  A token
    whose position is outside the tables is skipped (its rows untouched)."""
    if stream is not None:
        return _on(gdn_qk_norm_rope, locals())
    sizes, ptrs, index = _qk(q, k, cos, sin, positions, q_weight, k_weight, norm, eps, interleaved)
    q_out = _like(q) if q_out is None else q_out
    k_out = _like(k) if k_out is None else k_out
    _invoke("gdn_qk_norm_rope", index, _struct(*sizes), *ptrs, _is(q_out, "q_out", q.shape, q.dtype, index),
            _is(k_out, "k_out", k.shape, q.dtype, index))
    return q_out, k_out


def gdn_qk_norm_rope_bwd(q, k, cos, sin, d_q_out, d_k_out, positions=None, q_weight=None, k_weight=None, norm="rms",
                         eps=1e-6, interleaved=False, dq=None, dk=None, workspace=None, stream=None):
    """Gradient of gdn_qk_norm_rope at its inputs q, k.  dq, dk: written in place
    when given (they may be column slices of wider rows), else dense.  Returns
    dict dq, dk, dq_weight, dk_weight (fp32, None without the weight)."""
    if stream is not None:
        return _on(gdn_qk_norm_rope_bwd, locals())
    sizes, ptrs, index = _qk(q, k, cos, sin, positions, q_weight, k_weight, norm, eps, interleaved)
    qs, ks, ty = q.shape, k.shape, q.dtype
    grads = (_is(d_q_out, "d_q_out", qs, ty, index), _is(d_k_out, "d_k_out", ks, ty, index))
    dq = _like(q) if dq is None else dq
    dk = _like(k) if dk is None else dk
    (dqp, lddq), (dkp, lddk) = _rows(dq, "dq", qs, ty, index), _rows(dk, "dk", ks, ty, index)
    dqw, dkw = _like(q_weight), _like(k_weight) if ks[1] else None
    ws = None
    if dqw is not None or dkw is not None:
        ws = _space(workspace, _space_of("gdn_qk_norm_rope_bwd_workspace_size", *sizes), q.device)
    _invoke("gdn_qk_norm_rope_bwd", index, _struct(*sizes), *ptrs, *grads, dqp, dkp, lddq, lddk, _at(dqw), _at(dkw),
            _at(ws), 0 if ws is None else ws.numel())
    return dict(dq=dq, dk=dk, dq_weight=dqw, dk_weight=dkw)


def _scan(shape, ty, index, x, dt, A_log, B, C, N, D, z, dt_bias, dt_softplus):
    """Sizes for the struct and the inputs' addresses, x to dt_bias."""
    (T, ch), S, G = shape, _dims(A_log, "A_log", 2)[1], _dims(B, "B", 3)[1]
    f32, bc = torch.float32, (T, G, S)
    (xp, ldx), (dtp, lddt) = _rows(x, "x", shape, ty, index), _rows(dt, "dt", shape, ty, index)
    zp, ldz = (None, 0) if z is None else _rows(z, "z", shape, ty, index)
    (Bp, ldB), (Cp, ldC) = _rows(B, "B", bc, ty, index), _rows(C, "C", bc, ty, index)
    ptrs = (xp, dtp, _is(A_log, "A_log", (ch, S), f32, index), Bp, Cp, _is(D, "D", (ch,), f32, index), zp,
            _is(dt_bias, "dt_bias", (ch,), f32, index))
    return (ScanShape, N, T, ch, G, S, _dtype_code(x), int(bool(dt_softplus)), ldx, lddt, ldz, ldB, ldC), ptrs


def gdn_selective_scan_fwd(x, dt, A_log, B, C, cu_seqlens, D=None, z=None, dt_bias=None, state=None,
                           state_indices=None, has_initial_state=None, dt_softplus=True, out=None, stream=None):
    """Selective state space scan over a packed varlen batch.

    x, dt, z [T, channels], B, C [T, G, S] (bf16 or fp32, one dtype, rows may be
    slices of wider ones); A_log [channels, S], D, dt_bias [channels] fp32;
    cu_seqlens int32 [N+1] on the device.  state [slots, channels, S] fp32 is read
    as the initial state and overwritten with the final state of each sequence's
    slot (in place; int32 state_indices, has_initial_state as in
    gdn_causal_conv1d_fwd).  Returns y [T, channels] (rows behind cu_seqlens[N]
    not written)."""
    if stream is not None:
        return _on(gdn_selective_scan_fwd, locals())
    shape, ty, index = _first(x, "x", 2)
    N, cu = _sequences(cu_seqlens, index)
    sizes, ptrs = _scan(shape, ty, index, x, dt, A_log, B, C, N, D, z, dt_bias, dt_softplus)
    slots = 0 if state is None else _dims(state, "state", 3)[0]
    state_ptrs = (_is(state, "state", (slots, sizes[3], sizes[5]), torch.float32, index),
                  _is(state_indices, "state_indices", (N,), torch.int32, index), slots,
                  _is(has_initial_state, "has_initial_state", (N,), torch.int32, index))
    out = _like(x) if out is None else out
    _invoke("gdn_selective_scan_fwd", index, _struct(*sizes), *ptrs, cu, *state_ptrs, _is(out, "out", shape, ty, index))
    return out


def gdn_selective_scan_update(x, dt, A_log, B, C, state, state_indices=None, D=None, z=None, dt_bias=None,
                              dt_softplus=True, out=None, stream=None):
    """One token per sequence: x, dt, z [N, channels], B, C [N, G, S]; state
    [slots, channels, S] fp32 updated in place.  Returns y [N, channels] (rows of
    skipped slots untouched)."""
    if stream is not None:
        return _on(gdn_selective_scan_update, locals())
    shape, ty, index = _first(x, "x", 2)
    sizes, ptrs = _scan(shape, ty, index, x, dt, A_log, B, C, shape[0], D, z, dt_bias, dt_softplus)
    slots = _dims(state, "state", 3)[0]
    state_ptrs = (_is(state, "state", (slots, sizes[3], sizes[5]), torch.float32, index),
                  _is(state_indices, "state_indices", (shape[0],), torch.int32, index), slots)
    out = _like(x) if out is None else out
    _invoke("gdn_selective_scan_update", index, _struct(*sizes), *ptrs, *state_ptrs, _is(out, "out", shape, ty, index))
    return out


def gdn_selective_scan_bwd(x, dt, A_log, B, C, cu_seqlens, d_out, D=None, z=None, dt_bias=None, init_state=None,
                           d_final_state=None, dt_softplus=True, workspace=None, need_d_init_state=True, stream=None):
    """Gradient of gdn_selective_scan_fwd.  d_out [T, channels]; init_state,
    d_final_state [N, channels, S] fp32 or None (zero), in the order of the
    sequences.  Returns dict dx, ddt, dz, dB, dC (dtype of x), dA_log, dD,
    ddt_bias, d_init_state (fp32); None where the input is None.  Rows behind
    cu_seqlens[N] are not written."""
    if stream is not None:
        return _on(gdn_selective_scan_bwd, locals())
    shape, ty, index = _first(x, "x", 2)
    N, cu = _sequences(cu_seqlens, index)
    sizes, ptrs = _scan(shape, ty, index, x, dt, A_log, B, C, N, D, z, dt_bias, dt_softplus)
    state = (N, sizes[3], sizes[5])
    more = (cu, _is(init_state, "init_state", state, torch.float32, index), _is(d_out, "d_out", shape, ty, index),
            _is(d_final_state, "d_final_state", state, torch.float32, index))
    res = dict(dx=_like(x), ddt=_like(dt), dA_log=_like(A_log), dB=_like(B), dC=_like(C), dD=_like(D), dz=_like(z),
               ddt_bias=_like(dt_bias),
               d_init_state=torch.empty(state, dtype=torch.float32, device=x.device) if need_d_init_state else None)
    ws = _space(workspace, _space_of("gdn_selective_scan_bwd_workspace_size", *sizes), x.device)
    _invoke("gdn_selective_scan_bwd", index, _struct(*sizes), *ptrs, *more, *map(_at, res.values()), ws.data_ptr(),
            ws.numel())
    return res


# ---------------------------------------------------------------- chunk-replay variant (include/gdn_replay.h)

REPLAY_CHUNK = 64


def replay_block_floats(dk, dv):
    """Floats per (slot, head) in a replay-state pool."""
    return int(lib().gdn_replay_block_floats(int(dk), int(dv)))


def replay_state_new(slots, HV, dk, dv, init_state=None, device="cuda"):
    """A zeroed replay-state pool [slots, HV, B] fp32 whose chunk-start states are
    init_state [slots, HV, dv, dk] (zeros when None)."""
    rs = torch.zeros(slots, HV, replay_block_floats(dk, dv), dtype=torch.float32, device=device)
    if init_state is not None:
        replay_views(rs, dk, dv)["S0"].copy_(init_state)
    return rs


def replay_views(rs, dk, dv):
    """Views of a replay-state pool: S0 [slots, HV, dv, dk], K [.., C, dk], D [.., C, dv], gam [.., C]."""
    C = REPLAY_CHUNK
    a, b, c = dv * dk, dv * dk + C * dk, dv * dk + C * (dk + dv)
    sl, HV = rs.shape[0], rs.shape[1]
    return dict(S0=rs[..., :a].unflatten(-1, (dv, dk)), K=rs[..., a:b].unflatten(-1, (C, dk)),
                D=rs[..., b:c].unflatten(-1, (C, dv)), gam=rs[..., c:c + C])


def gdn_replay_prefill(q, k, v, g, beta, cu_seqlens, replay_state, seq_pos=None, state_indices=None, out=None,
                       workspace=None, use_qk_l2norm=True, stream=None):
    """Chunked prefill that continues every sequence from its replay state (at
    position seq_pos[n], int32 on the device; None: 0) and leaves the state
    after its last token.  Returns out [T, HV, dv]."""
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, dev)
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    _need(replay_state, "replay_state", torch.float32, dev)
    for t, n in ((seq_pos, "seq_pos"), (state_indices, "state_indices")):
        if t is not None:
            _need(t, n, torch.int32, dev)
    N = cu_seqlens.numel() - 1
    shape = make_shape(q, v, N, use_qk_l2norm, 0)
    if replay_state.shape[1:] != (shape.HV, replay_block_floats(shape.dk, shape.dv)):
        raise ValueError("replay_state must be [slots, HV, replay_block_floats(dk, dv)]")
    out = torch.empty_like(v) if out is None else out
    _need(out, "out", q.dtype, dev)
    if workspace is None:
        workspace = torch.zeros(max(int(lib().gdn_replay_workspace_size(ctypes.byref(shape))), 256),
                                dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        rc = lib().gdn_replay_prefill(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                      _ptr(cu_seqlens), _ptr(seq_pos), _ptr(replay_state), _ptr(state_indices),
                                      int(replay_state.shape[0]), _ptr(out), _ptr(workspace),
                                      ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check(rc, "gdn_replay_prefill")
    return out


def gdn_replay_decode(q, k, v, g, beta, replay_state, seq_pos, state_indices=None, out=None, use_qk_l2norm=True,
                      stream=None):
    """One token per sequence replaying the chunked order; seq_pos [B] int32 (tokens
    already processed).  Returns out [B, HV, dv] (rows of skipped slots untouched)."""
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, dev)
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    _need(replay_state, "replay_state", torch.float32, dev)
    _need(seq_pos, "seq_pos", torch.int32, dev)
    if state_indices is not None:
        _need(state_indices, "state_indices", torch.int32, dev)
    shape = make_shape(q, v, q.shape[0], use_qk_l2norm, 0)
    out = torch.empty_like(v) if out is None else out
    _need(out, "out", q.dtype, dev)
    with torch.cuda.device(dev):
        rc = lib().gdn_replay_decode(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                     _ptr(seq_pos), _ptr(replay_state), _ptr(state_indices),
                                     int(replay_state.shape[0]), _ptr(out), _stream(stream))
    _check(rc, "gdn_replay_decode")
    return out
