"""Python binding of the verifier hot-path library (libvgv.so, include/vgv.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libvgv.so. The functions carry the C names and take torch tensors
(device memory, any stream) or ``None``; they return nothing and raise
``VgError`` on a non-OK status. There is no CPU fallback: if the library is not
built, the first call raises.

    import greedy_speculative_verify_b200 as vgv
    ws = torch.empty(vgv.vg_moe_workspace_bytes(vgv.MOE_DIMS, T), dtype=torch.uint8, device="cuda")
    vgv.vg_moe_ffn(vgv.MOE_DIMS, T, x, router_w, None, expert_w, shared_w, 1, out, None, ws)
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libvgv.so")

VG_OK = 0
STATUS_NAMES = {0: "VG_OK", 1: "VG_ERR_INVALID_ARG", 2: "VG_ERR_UNSUPPORTED", 3: "VG_ERR_WORKSPACE",
                4: "VG_ERR_CUDA", 5: "VG_ERR_TIMEOUT", 6: "VG_ERR_DEVICE_BOUNDS"}

# every symbol include/vgv.h declares
EXPORTS = (
    "vg_status_string", "vg_abi_version", "vg_moe_workspace_bytes", "vg_moe_ffn",
    "vg_moe_stack_workspace_bytes", "vg_moe_ffn_stack", "vg_verify_workspace_bytes",
    "vg_verify_greedy", "vg_get_device_status", "vg_set_wait_timeout_ns", "vg_debug_wait_flag", "vg_debug_wait_site",
    "vg_profile_set_events", "vg_profile_count", "vg_verify_greedy_noalloc",
    "vg_embed_rows", "vg_spec_rows", "vg_spec_commit", "vg_spec_rows_given",
    "vg_mtp_workspace_bytes", "vg_mtp_draft", "vg_attn_workspace_bytes", "vg_attn_verify",
    "vg_verify_step_small_workspace_bytes", "vg_verify_step_small",
    "vg_kv8_append", "vg_kv8_read", "vg_kv8_attn_workspace_bytes", "vg_kv8_attn",
    "vg_attn_verify_kv8_workspace_bytes", "vg_attn_verify_kv8",
    "vg_token_logprobs_workspace_bytes", "vg_token_logprobs",
)

# vg_kv8 formats and output element types
VG_KV8_INT8, VG_KV8_E4M3 = 0, 1
VG_BF16, VG_F32 = 0, 1

# vg_kernel
VG_KERNEL_ROUTER, VG_KERNEL_GROUPING, VG_KERNEL_EXPERTS = 0, 1, 2
VG_KERNEL_COMBINE, VG_KERNEL_LM_HEAD, VG_KERNEL_ACCEPT = 3, 4, 5
VG_KERNEL_ATTENTION = 6


class VgError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class vg_moe_dims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("intermediate", ctypes.c_int32), ("n_routed", ctypes.c_int32),
                ("n_shared", ctypes.c_int32), ("top_k", ctypes.c_int32)]


class vg_moe_taps(ctypes.Structure):
    _fields_ = [("topk_idx", ctypes.c_void_p), ("topk_weight", ctypes.c_void_p),
                ("expert_offsets", ctypes.c_void_p), ("perm", ctypes.c_void_p), ("inv_perm", ctypes.c_void_p),
                ("act", ctypes.c_void_p), ("expert_out", ctypes.c_void_p)]


class vg_spec_state(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32),
                ("last", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("committed", ctypes.c_void_p),
                ("cap", ctypes.c_int32), ("ref", ctypes.c_void_p), ("ref_len", ctypes.c_int32),
                ("p", ctypes.c_float), ("seed", ctypes.c_uint64), ("step", ctypes.c_void_p),
                ("tokens", ctypes.c_void_p), ("drafts", ctypes.c_void_p)]


class vg_mtp_weights(ctypes.Structure):
    _fields_ = [("proj", ctypes.c_void_p), ("ffn", ctypes.c_void_p), ("gamma_h", ctypes.c_void_p),
                ("gamma_e", ctypes.c_void_p), ("gamma_f", ctypes.c_void_p), ("emb", ctypes.c_void_p),
                ("lm_head", ctypes.c_void_p), ("V", ctypes.c_int32)]


class vg_kv8(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("B", ctypes.c_int32), ("L_max", ctypes.c_int32), ("n_kv", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("block", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_amax", ctypes.c_void_p), ("v_amax", ctypes.c_void_p)]


MOE_DIMS = vg_moe_dims(1280, 896, 64, 2, 6)

_lib = None


def load():
    """Loads libvgv.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with greedy_speculative_verify_b200.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, u64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64, ctypes.c_size_t
    dims_p = ctypes.POINTER(vg_moe_dims)
    kv8_p, i64 = ctypes.POINTER(vg_kv8), ctypes.c_int64
    sig = {
        "vg_status_string": (ctypes.c_char_p, [i32]),
        "vg_abi_version": (i32, []),
        "vg_moe_workspace_bytes": (sz, [dims_p, i32]),
        "vg_moe_ffn": (i32, [dims_p, i32, vp, vp, vp, vp, vp, i32, vp, ctypes.POINTER(vg_moe_taps), vp, sz, vp]),
        "vg_moe_stack_workspace_bytes": (sz, [dims_p, i32]),
        "vg_moe_ffn_stack": (i32, [dims_p, i32, i32, vp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp),
                                   ctypes.POINTER(vp), vp, vp, sz, vp]),
        "vg_verify_workspace_bytes": (sz, [i32, i32, i32, i32]),
        "vg_verify_greedy": (i32, [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "vg_get_device_status": (i32, [vp, ctypes.POINTER(i32)]),
        "vg_set_wait_timeout_ns": (i32, [u64]),
        "vg_debug_wait_flag": (i32, [vp, i32, u64, vp]),
        "vg_debug_wait_site": (i32, [i32, vp, u64, vp]),
        "vg_profile_set_events": (i32, [i32, ctypes.POINTER(vp), ctypes.POINTER(vp), i32]),
        "vg_profile_count": (ctypes.c_int64, [i32]),
        "vg_verify_greedy_noalloc": (i32, [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]),
        "vg_embed_rows": (i32, [vp, i32, vp, i32, i32, vp, vp]),
        "vg_spec_rows": (i32, [ctypes.POINTER(vg_spec_state), vp]),
        "vg_spec_commit": (i32, [ctypes.POINTER(vg_spec_state), vp, vp, vp]),
        "vg_spec_rows_given": (i32, [ctypes.POINTER(vg_spec_state), vp]),
        "vg_mtp_workspace_bytes": (sz, [i32, i32]),
        "vg_mtp_draft": (i32, [i32, i32, ctypes.POINTER(vg_mtp_weights), vp, i32, vp, vp, vp, vp, vp, sz, vp]),
        "vg_attn_workspace_bytes": (sz, [i32, i32, i32]),
        "vg_attn_verify": (i32, [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "vg_verify_step_small_workspace_bytes": (sz, []),
        "vg_verify_step_small": (i32, [dims_p, i32, i32, i32, vp, ctypes.POINTER(vp), ctypes.POINTER(vp),
                                       ctypes.POINTER(vp), ctypes.POINTER(vp), vp, i32, vp, vp, vp, vp, vp, vp,
                                       vp, sz, vp]),
        "vg_kv8_append": (i32, [kv8_p, i32, vp, i64, vp, i64, vp, vp, vp]),
        "vg_kv8_read": (i32, [kv8_p, i32, vp, vp, i32, vp, i64, vp, i64, vp]),
        "vg_kv8_attn_workspace_bytes": (sz, [kv8_p, i32, i32]),
        "vg_kv8_attn": (i32, [kv8_p, i32, i32, vp, i64, vp, vp, vp, ctypes.c_float, vp, i64, vp, sz, vp]),
        "vg_attn_verify_kv8_workspace_bytes": (sz, [kv8_p, i32]),
        "vg_attn_verify_kv8": (i32, [kv8_p, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "vg_token_logprobs_workspace_bytes": (sz, [i32, i32, i32, i32]),
        "vg_token_logprobs": (i32, [i32, i32, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_torch = None


def _t():
    """torch, imported on first use."""
    global _torch
    if _torch is None:
        import torch

        _torch = torch
    return _torch


_raw_stream = _device = None


def _stream(stream):
    if stream is None:
        global _raw_stream, _device
        if _raw_stream is None:
            torch = _t()
            _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
            # the same handle, without the 3 us that a Stream object takes
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
            torch.cuda.current_device()  # (brings CUDA up, which the calls above do not)
        return _raw_stream(_device())
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(st: int, where: str):
    if st != VG_OK:
        raise VgError(st, where)


def vg_abi_version() -> int:
    return load().vg_abi_version()


def vg_status_string(s: int) -> str:
    return load().vg_status_string(s).decode()


def vg_moe_workspace_bytes(dims: vg_moe_dims, T_max: int) -> int:
    return load().vg_moe_workspace_bytes(ctypes.byref(dims), T_max)


def vg_moe_stack_workspace_bytes(dims: vg_moe_dims, T_max: int) -> int:
    return load().vg_moe_stack_workspace_bytes(ctypes.byref(dims), T_max)


def vg_verify_workspace_bytes(B: int, K: int, H: int, V: int) -> int:
    return load().vg_verify_workspace_bytes(B, K, H, V)


def make_taps(topk_idx=None, topk_weight=None, expert_offsets=None, perm=None, inv_perm=None, act=None,
              expert_out=None) -> vg_moe_taps:
    return vg_moe_taps(*(None if t is None else t.data_ptr()
                         for t in (topk_idx, topk_weight, expert_offsets, perm, inv_perm, act, expert_out)))


def vg_moe_ffn(dims, T, x, router_w, router_bias, expert_w, shared_w, add_residual, out, taps, workspace,
               stream=None):
    st = load().vg_moe_ffn(ctypes.byref(dims), T, _ptr(x), _ptr(router_w), _ptr(router_bias), _ptr(expert_w),
                           _ptr(shared_w), int(add_residual), _ptr(out),
                           None if taps is None else ctypes.byref(taps), _ptr(workspace),
                           0 if workspace is None else workspace.numel() * workspace.element_size(),
                           _stream(stream))
    _check(st, "vg_moe_ffn")


def vg_moe_ffn_stack(dims, n_layers, T, x, router_w, router_bias, expert_w, shared_w, out, workspace, stream=None):
    """router_w, expert_w, shared_w: sequences of n_layers tensors; router_bias:
    None or a sequence of tensors/None."""
    arr = ctypes.c_void_p * n_layers
    rw = arr(*(t.data_ptr() for t in router_w))
    ew = arr(*(t.data_ptr() for t in expert_w))
    sw = arr(*(t.data_ptr() for t in shared_w))
    rb = None if router_bias is None else arr(*(None if t is None else t.data_ptr() for t in router_bias))
    st = load().vg_moe_ffn_stack(ctypes.byref(dims), n_layers, T, _ptr(x), rw, rb, ew, sw, _ptr(out),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "vg_moe_ffn_stack")


def vg_verify_greedy(B, K, H, V, h, lm_head, drafts, argmax, accepted, out_tokens, workspace, stream=None):
    st = load().vg_verify_greedy(B, K, H, V, _ptr(h), _ptr(lm_head), _ptr(drafts), _ptr(argmax), _ptr(accepted),
                                 _ptr(out_tokens), _ptr(workspace),
                                 0 if workspace is None else workspace.numel() * workspace.element_size(),
                                 _stream(stream))
    _check(st, "vg_verify_greedy")


def vg_verify_step_small_workspace_bytes() -> int:
    return load().vg_verify_step_small_workspace_bytes()


def vg_verify_step_small(dims, n_layers, B, K, x, router_w, router_bias, expert_w, shared_w, lm_head, V, drafts,
                         argmax, accepted, out_tokens, workspace, states_out=None, topk_idx_out=None, stream=None):
    """The whole verify step (n_layers MoE layers, LM-head argmax, accept) for
    B (K+1) <= 16 rows in one launch. Sequences of n_layers tensors as in
    vg_moe_ffn_stack."""
    arr = ctypes.c_void_p * n_layers
    rw = arr(*(t.data_ptr() for t in router_w))
    ew = arr(*(t.data_ptr() for t in expert_w))
    sw = arr(*(t.data_ptr() for t in shared_w))
    rb = None if router_bias is None else arr(*(None if t is None else t.data_ptr() for t in router_bias))
    st = load().vg_verify_step_small(ctypes.byref(dims), n_layers, B, K, _ptr(x), rw, rb, ew, sw, _ptr(lm_head), V,
                                     _ptr(drafts), _ptr(argmax), _ptr(accepted), _ptr(out_tokens),
                                     _ptr(states_out), _ptr(topk_idx_out), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "vg_verify_step_small")


def vg_get_device_status(stream=None) -> tuple[int, int]:
    """(status code, site) of the first fault recorded on the current device; clears it."""
    info = ctypes.c_int32(0)
    st = load().vg_get_device_status(_stream(stream), ctypes.byref(info))
    return st, info.value


def vg_set_wait_timeout_ns(ns: int):
    _check(load().vg_set_wait_timeout_ns(ns), "vg_set_wait_timeout_ns")


def vg_debug_wait_flag(flag, expect: int, max_ns: int, stream=None):
    _check(load().vg_debug_wait_flag(_ptr(flag), expect, max_ns, _stream(stream)), "vg_debug_wait_flag")


VG_WAIT_MBARRIER, VG_WAIT_GRID_BARRIER = 1, 2


def vg_debug_wait_site(which: int, ctr, max_ns: int, stream=None):
    _check(load().vg_debug_wait_site(which, _ptr(ctr), max_ns, _stream(stream)), "vg_debug_wait_site")


def vg_profile_set_events(kind: int, starts, stops):
    """starts/stops: sequences of torch.cuda.Event (enable_timing=True); empty clears."""
    n = len(starts)
    arr = ctypes.c_void_p * max(n, 1)
    a = arr(*(e.cuda_event for e in starts))
    b = arr(*(e.cuda_event for e in stops))
    _check(load().vg_profile_set_events(kind, a, b, n), "vg_profile_set_events")


def vg_profile_count(kind: int) -> int:
    return load().vg_profile_count(kind)


NOALLOC_SCRATCH_KEYS = (2 << 20) // 8


def vg_verify_greedy_noalloc(B, K, H, V, h, lm_head, drafts, argmax, accepted, out_tokens, stream=None):
    """vg_verify_greedy without a workspace, for callers that cannot allocate
    device memory; see include/vgv.h for the scratch limit and its sharing."""
    st = load().vg_verify_greedy_noalloc(B, K, H, V, _ptr(h), _ptr(lm_head), _ptr(drafts), _ptr(argmax),
                                         _ptr(accepted), _ptr(out_tokens), _stream(stream))
    _check(st, "vg_verify_greedy_noalloc")


# ------------------------------------------------------------ decode loop
def vg_embed_rows(tokens, emb, out, stream=None):
    """out[i] = emb[tokens[i]] (bf16 rows)."""
    _check(load().vg_embed_rows(_ptr(tokens), tokens.numel(), _ptr(emb), emb.shape[0], emb.shape[1], _ptr(out),
                                _stream(stream)), "vg_embed_rows")


def make_spec_state(B, K, V, last, pos, committed, ref, p, seed, step, tokens, drafts):
    """vg_spec_state over caller-owned device tensors (ref may be None); every
    tensor is read as dense rows, so each must be contiguous."""
    for t in (last, pos, committed, ref, step, tokens, drafts):
        if t is not None and not t.is_contiguous():
            raise ValueError("vg_spec_state tensors must be contiguous")
    return vg_spec_state(B, K, V, last.data_ptr(), pos.data_ptr(), committed.data_ptr(), committed.shape[1],
                         None if ref is None else ref.data_ptr(), 0 if ref is None else ref.shape[1],
                         float(p), int(seed), step.data_ptr(), tokens.data_ptr(),
                         None if drafts is None else drafts.data_ptr())


def vg_spec_rows(state, stream=None):
    _check(load().vg_spec_rows(ctypes.byref(state), _stream(stream)), "vg_spec_rows")


def vg_spec_commit(state, accepted, out_tokens, stream=None):
    _check(load().vg_spec_commit(ctypes.byref(state), _ptr(accepted), _ptr(out_tokens), _stream(stream)),
           "vg_spec_commit")


def vg_spec_rows_given(state, stream=None):
    _check(load().vg_spec_rows_given(ctypes.byref(state), _stream(stream)), "vg_spec_rows_given")


# ------------------------------------------------------------ draft block
def make_mtp_weights(proj, ffn, gamma_h, gamma_e, gamma_f, emb, lm_head):
    """vg_mtp_weights over caller-owned device tensors (fp32 gammas, bf16 rest)."""
    for t in (proj, ffn, gamma_h, gamma_e, gamma_f, emb, lm_head):
        if not t.is_contiguous():
            raise ValueError("vg_mtp_weights tensors must be contiguous")
    return vg_mtp_weights(proj.data_ptr(), ffn.data_ptr(), gamma_h.data_ptr(), gamma_e.data_ptr(),
                          gamma_f.data_ptr(), emb.data_ptr(), lm_head.data_ptr(), lm_head.shape[0])


def vg_mtp_workspace_bytes(B, V):
    return load().vg_mtp_workspace_bytes(B, V)


def vg_mtp_draft(B, K, weights, h, rows_per_seq, accepted, y0, drafts, workspace, hidden_out=None, stream=None):
    _check(load().vg_mtp_draft(B, K, ctypes.byref(weights), _ptr(h), rows_per_seq, _ptr(accepted), _ptr(y0),
                               _ptr(drafts), _ptr(hidden_out), _ptr(workspace), workspace.numel(), _stream(stream)),
           "vg_mtp_draft")


# ------------------------------------------------------------ verifier attention
def vg_attn_workspace_bytes(B, K, L_max):
    return load().vg_attn_workspace_bytes(B, K, L_max)


def vg_attn_verify(B, K, x, w_qkv, w_o, kv_cache, lens, out, workspace, o_out=None, stream=None):
    """One attention layer of a verify step; kv_cache [B, 2, L_max, H] (its
    third dimension is passed as L_max, so it must be that dense shape)."""
    if kv_cache.dim() != 4 or kv_cache.shape[0] != B or kv_cache.shape[1] != 2 or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be a contiguous [B, 2, L_max, H] tensor")
    _check(load().vg_attn_verify(B, K, kv_cache.shape[2], _ptr(x), _ptr(w_qkv), _ptr(w_o), _ptr(kv_cache), _ptr(lens),
                                 _ptr(out), _ptr(o_out), _ptr(workspace), workspace.numel(), _stream(stream)),
           "vg_attn_verify")


# ------------------------------------------------------------ 8-bit KV cache
# A call of these costs a few microseconds on the GPU at its smallest, so the
# checks below are kept to a comparison each.
def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _same_device(device, *tensors):
    """Every tensor lies on `device`, a CUDA device and the current one: the
    library launches there, and its kernels take the addresses as they are."""
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"a tensor is on {t.device}, not on {device}")
    index = device.index
    if index is None:  # host memory
        raise ValueError(f"tensors are on {device}, not on a CUDA device")
    if index != (_device or _t().cuda.current_device)():
        raise ValueError(f"tensors are on {device}, which is not the current device")


def _rows(name, t, n, width, dtypes):
    """Row stride of a [n, width] matrix with dense rows."""
    if t is None:
        return 0
    if t.shape != (n, width) or t.dtype not in dtypes:
        raise ValueError(f"{name} must be [{n}, {width}] of {dtypes}, got {tuple(t.shape)} of {t.dtype}")
    step, one = t.stride()
    if one != 1 and width > 1:
        raise ValueError(f"{name} must have dense rows")
    return step if n > 1 else width  # (of a single row it says nothing)


def _dense(name, t, shape, dtype):
    if t is not None and (t.shape != shape or t.dtype is not dtype or not t.is_contiguous()):
        raise ValueError(f"{name} must be dense {tuple(shape)} of {dtype}, got {tuple(t.shape)} of {t.dtype}")


def _at(t):
    return None if t is None else t.data_ptr()


def _bytes_of(workspace):
    if workspace is None:
        return 0
    _need(workspace.is_contiguous(), "workspace must be contiguous")
    return workspace.nbytes


def make_kv8(k, v, k_amax, v_amax):
    """vg_kv8 over caller-owned device tensors: k and v [B, n_kv, L_max, dim] of
    codes (torch.int8 or torch.float8_e4m3fn; inside a (sequence, head) they lie
    in the order include/vgv.h documents), k_amax and v_amax fp32
    [B, n_kv, L_max / block]. The handle keeps the tensors alive."""
    torch = _t()
    formats = {torch.int8: VG_KV8_INT8, torch.float8_e4m3fn: VG_KV8_E4M3}
    _need(k.dim() == 4 and k.dtype in formats, "k must be [B, n_kv, L_max, dim] of int8 or float8_e4m3fn")
    B, n_kv, L_max, dim = k.shape
    _dense("k", k, k.shape, k.dtype)
    _dense("v", v, k.shape, k.dtype)
    _need(k_amax.dim() == 3 and k_amax.shape[2] > 0 and L_max % k_amax.shape[2] == 0,
          "k_amax must be [B, n_kv, L_max / block]")
    for name, t in (("k_amax", k_amax), ("v_amax", v_amax)):
        _dense(name, t, (B, n_kv, k_amax.shape[2]), torch.float32)
    for name, t in (("v", v), ("k_amax", k_amax), ("v_amax", v_amax)):
        _need(t.device == k.device, f"{name} is on {t.device}, not on {k.device}")
    c = vg_kv8(formats[k.dtype], B, L_max, n_kv, dim, L_max // k_amax.shape[2], k.data_ptr(), v.data_ptr(),
               k_amax.data_ptr(), v_amax.data_ptr())
    c.tensors = (k, v, k_amax, v_amax)
    c.device = k.device
    return c


def vg_kv8_append(cache, rows, k, v, pos, n_new=None, stream=None):
    """Quantises `rows` new rows per sequence (k, v: bf16 [B * rows, n_kv * dim],
    rows a multiple of 8 elements apart) into the cache at positions pos[b] .. (the first n_new[b])."""
    torch = _t()
    B, width, bf16 = cache.B, cache.n_kv * cache.dim, (torch.bfloat16,)
    ks, vs = _rows("k", k, B * rows, width, bf16), _rows("v", v, B * rows, width, bf16)
    _dense("pos", pos, (B,), torch.int32)
    _dense("n_new", n_new, (B,), torch.int32)
    _same_device(cache.device, k, v, pos, n_new)
    _check(load().vg_kv8_append(cache, rows, _at(k), ks, _at(v), vs, _at(pos), _at(n_new), _stream(stream)),
           "vg_kv8_append")


def vg_kv8_read(cache, rows, pos, k_out, v_out, n_rows=None, stream=None):
    """Positions pos[b] .. pos[b] + n_rows[b] - 1 of every sequence as values, into
    rows b * rows .. of k_out and v_out ([B * rows, n_kv * dim], bf16 or fp32
    alike; either may be None)."""
    torch = _t()
    B, width, types = cache.B, cache.n_kv * cache.dim, (torch.bfloat16, torch.float32)
    ks, vs = _rows("k_out", k_out, B * rows, width, types), _rows("v_out", v_out, B * rows, width, types)
    out = k_out if k_out is not None else v_out
    _need(v_out is None or out.dtype is v_out.dtype, "k_out and v_out must have one type")
    _dense("pos", pos, (B,), torch.int32)
    _dense("n_rows", n_rows, (B,), torch.int32)
    _same_device(cache.device, k_out, v_out, pos, n_rows)
    kind = VG_F32 if out is not None and out.dtype is torch.float32 else VG_BF16
    _check(load().vg_kv8_read(cache, rows, _at(pos), _at(n_rows), kind, _at(k_out), ks, _at(v_out), vs,
                              _stream(stream)), "vg_kv8_read")


def vg_kv8_attn_workspace_bytes(cache, rows, n_heads):
    return load().vg_kv8_attn_workspace_bytes(cache, rows, n_heads)


def vg_kv8_attn(cache, rows, n_heads, q, lens, scale, o, workspace, first=None, n_new=None, stream=None):
    """Attention of `rows` query rows per sequence (q, o: bf16 [B * rows,
    n_heads * dim], rows a multiple of 8 elements apart) over the cache."""
    torch = _t()
    B, width, bf16 = cache.B, n_heads * cache.dim, (torch.bfloat16,)
    qs, os_ = _rows("q", q, B * rows, width, bf16), _rows("o", o, B * rows, width, bf16)
    _dense("lens", lens, (B,), torch.int32)
    _dense("first", first, (B,), torch.int32)
    _dense("n_new", n_new, (B,), torch.int32)
    _same_device(cache.device, q, o, lens, first, n_new, workspace)
    _check(load().vg_kv8_attn(cache, rows, n_heads, _at(q), qs, _at(lens), _at(first), _at(n_new), scale, _at(o), os_,
                              _at(workspace), _bytes_of(workspace), _stream(stream)), "vg_kv8_attn")


def vg_attn_verify_kv8_workspace_bytes(cache, K):
    return load().vg_attn_verify_kv8_workspace_bytes(cache, K)


def vg_attn_verify_kv8(cache, K, x, w_qkv, w_o, lens, out, workspace, o_out=None, stream=None):
    """One attention layer of a verify step on an 8-bit cache (vg_attn_verify's
    arguments; the batch is the cache's)."""
    torch = _t()
    R, H, bf16 = cache.B * (K + 1), cache.n_kv * cache.dim, torch.bfloat16
    for name, t, shape in (("x", x, (R, H)), ("w_qkv", w_qkv, (3 * H, H)), ("w_o", w_o, (H, H)), ("out", out, (R, H)),
                           ("o_out", o_out, (R, H))):
        _dense(name, t, shape, bf16)
    _dense("lens", lens, (cache.B,), torch.int32)
    _same_device(cache.device, x, w_qkv, w_o, lens, out, o_out, workspace)
    _check(load().vg_attn_verify_kv8(cache, K, _at(x), _at(w_qkv), _at(w_o), _at(lens), _at(out), _at(o_out),
                                     _at(workspace), _bytes_of(workspace), _stream(stream)), "vg_attn_verify_kv8")


# ------------------------------------------------------------ log probabilities
def vg_token_logprobs_workspace_bytes(R, H, V, n_top):
    return load().vg_token_logprobs_workspace_bytes(R, H, V, n_top)


def vg_token_logprobs(h, lm_head, tokens, logprob, entropy, top_ids, top_logprobs, workspace, stream=None):
    """Log probabilities of tokens[r] after hidden row h[r], the entropy and the
    top_ids.shape[1] most likely tokens of each row; tokens with logprob, entropy,
    and top_ids with top_logprobs may be None."""
    torch = _t()
    _need(h.dim() == 2 and lm_head.dim() == 2, "h must be [R, H], lm_head [V, H]")
    (R, H), V = h.shape, lm_head.shape[0]
    n_top = 0 if top_ids is None else top_ids.shape[-1]
    _dense("h", h, (R, H), torch.bfloat16)
    _dense("lm_head", lm_head, (V, H), torch.bfloat16)
    _dense("tokens", tokens, (R,), torch.int32)
    _dense("logprob", logprob, (R,), torch.float32)
    _dense("entropy", entropy, (R,), torch.float32)
    _dense("top_ids", top_ids, (R, n_top), torch.int32)
    _dense("top_logprobs", top_logprobs, (R, n_top), torch.float32)
    _same_device(h.device, lm_head, tokens, logprob, entropy, top_ids, top_logprobs, workspace)
    _check(load().vg_token_logprobs(R, H, V, _at(h), _at(lm_head), _at(tokens), n_top, _at(logprob), _at(entropy),
                                    _at(top_ids), _at(top_logprobs), _at(workspace), _bytes_of(workspace),
                                    _stream(stream)), "vg_token_logprobs")
