"""Python binding of the GB300 Gated DeltaNet verify library (C ABI in
``include/gdn_verify.h``).

Argument marshalling only: every step runs in the CUDA kernels of
``libgdn_verify.so``.  Buffers are passed as torch tensors (their
``data_ptr()``) or raw integer device addresses; the stream defaults to
torch's current stream.  If the library has not been built the import of
``lib()`` raises -- there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn_verify.so")

GDN_OK = 0
GDN_ERR_ARG = 1
GDN_ERR_SHAPE = 2
GDN_ERR_ALIGN = 3
GDN_ERR_DTYPE = 4
GDN_ERR_TRIM_RANGE = 5
GDN_ERR_NO_CAPTURE = 6
GDN_ERR_LAUNCH = 7
GDN_ERR_TIMEOUT = 8
GDN_ERR_WORKSPACE = 9
GDN_ERR_TREE = 10
GDN_ERR_BOUNDS = 11
GDN_ERR_SAMPLE = 12
GDN_ERR_LENGTH = 13
GDN_ERR_ADAPTER = 14
GDN_ERR_PAGE = 15
STATUS_NAMES = {0: "GDN_OK", 1: "GDN_ERR_ARG", 2: "GDN_ERR_SHAPE", 3: "GDN_ERR_ALIGN", 4: "GDN_ERR_DTYPE",
                5: "GDN_ERR_TRIM_RANGE", 6: "GDN_ERR_NO_CAPTURE", 7: "GDN_ERR_LAUNCH", 8: "GDN_ERR_TIMEOUT",
                9: "GDN_ERR_WORKSPACE", 10: "GDN_ERR_TREE",
                11: "GDN_ERR_BOUNDS", 12: "GDN_ERR_SAMPLE", 13: "GDN_ERR_LENGTH", 14: "GDN_ERR_ADAPTER",
                15: "GDN_ERR_PAGE"}

GDN_F32 = 0
GDN_BF16 = 1

EXPORTED_SYMBOLS = ("gdn_verify_forward", "gdn_verify_tree", "gdn_rollback", "gdn_rollback_tree",
                    "gdn_rollback_layers", "gdn_rollback_tree_layers", "gdn_verify_after_rollback", "gdn_verify_lazy", "gdn_commit_lazy", "gdn_step_io_layout",
                    "gdn_verify_step_host", "gdn_proj_in_ld", "gdn_layer_workspace_bytes",
                    "gdn_project_in", "gdn_project_out", "gdn_layer_verify", "gdn_lora_workspace_bytes",
                    "gdn_project_in_lora", "gdn_project_out_lora", "gdn_layer_lora_workspace_bytes",
                    "gdn_layer_verify_lora", "gdn_sample", "gdn_accept", "gdn_accept_tree",
                    "gdn_kv_append", "gdn_attend_workspace_bytes", "gdn_attend",
                    "gdn_prefill_workspace_bytes",
                    "gdn_prefill_chunked", "gdn_prefill_chunked_static", "gdn_prefill_static_scratch_bytes",
                    "gdn_last_error", "gdn_version")


class GdnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("n_slots", ctypes.c_int), ("n_qk_heads", ctypes.c_int), ("n_v_heads", ctypes.c_int),
                ("d_k", ctypes.c_int), ("d_v", ctypes.c_int), ("conv_width", ctypes.c_int),
                ("n_tokens", ctypes.c_int), ("act_dtype", ctypes.c_int), ("rms_eps", ctypes.c_float),
                ("l2_eps", ctypes.c_float), ("q_scale", ctypes.c_float)]


class LayerParams(ctypes.Structure):
    _fields_ = [("conv_w", ctypes.c_void_p), ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("norm_w", ctypes.c_void_p)]


class StepIO(ctypes.Structure):
    _fields_ = [("qkv", ctypes.c_size_t), ("z", ctypes.c_size_t), ("alpha", ctypes.c_size_t),
                ("beta_raw", ctypes.c_size_t), ("trim", ctypes.c_size_t), ("in_bytes", ctypes.c_size_t),
                ("out_bytes", ctypes.c_size_t)]


class ProjWeights(ctypes.Structure):
    _fields_ = [("n_embd", ctypes.c_int), ("w_in", ctypes.c_void_p), ("w_out", ctypes.c_void_p)]


class Lora(ctypes.Structure):
    _fields_ = [("n_adapters", ctypes.c_int), ("rank", ctypes.c_int), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("scale", ctypes.c_void_p)]


class SampleDims(ctypes.Structure):
    _fields_ = [("n_slots", ctypes.c_int), ("n_tokens", ctypes.c_int), ("vocab", ctypes.c_int),
                ("dtype", ctypes.c_int), ("ld", ctypes.c_longlong)]


class SampleParams(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p),
                ("min_p", ctypes.c_void_p)]


class AttnDims(ctypes.Structure):
    _fields_ = [("n_slots", ctypes.c_int), ("n_tokens", ctypes.c_int), ("n_heads", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("d_head", ctypes.c_int), ("page_tokens", ctypes.c_int),
                ("n_pages", ctypes.c_int), ("max_pages", ctypes.c_int), ("page_stride", ctypes.c_longlong),
                ("dtype", ctypes.c_int)]


class KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("past", ctypes.c_void_p)]


class QkParams(ctypes.Structure):
    _fields_ = [("rope_dims", ctypes.c_int), ("adjacent", ctypes.c_int), ("freq", ctypes.c_void_p),
                ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p), ("norm_eps", ctypes.c_float)]


class AttnParams(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("window", ctypes.c_int), ("n_sink", ctypes.c_int)]


def make_dims(n_slots: int, n_qk_heads: int, n_v_heads: int, d_k: int, d_v: int, n_tokens: int,
              act_dtype: int = GDN_BF16, conv_width: int = 4, rms_eps: float = 1e-6,
              l2_eps: float = 1e-6, q_scale: float = 1.0) -> Dims:
    return Dims(n_slots, n_qk_heads, n_v_heads, d_k, d_v, conv_width, n_tokens, act_dtype,
                rms_eps, l2_eps, q_scale)


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it was not built (no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        vp, ip = ctypes.c_void_p, ctypes.c_int
        L.gdn_verify_forward.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(LayerParams)] + [vp] * 11
        L.gdn_verify_forward.restype = ip
        L.gdn_rollback.argtypes = [ctypes.POINTER(Dims)] + [vp] * 7
        L.gdn_rollback.restype = ip
        L.gdn_verify_tree.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(LayerParams)] + [vp] * 12
        L.gdn_verify_tree.restype = ip
        L.gdn_rollback_tree.argtypes = [ctypes.POINTER(Dims)] + [vp] * 7
        L.gdn_rollback_tree.restype = ip
        L.gdn_rollback_layers.argtypes = [ctypes.POINTER(Dims), ctypes.c_int] + [vp] * 7
        L.gdn_rollback_layers.restype = ip
        L.gdn_rollback_tree_layers.argtypes = [ctypes.POINTER(Dims), ctypes.c_int] + [vp] * 7
        L.gdn_rollback_tree_layers.restype = ip
        L.gdn_verify_after_rollback.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(LayerParams)] + [vp] * 12
        L.gdn_verify_after_rollback.restype = ip
        L.gdn_step_io_layout.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(StepIO)]
        L.gdn_step_io_layout.restype = ip
        L.gdn_verify_step_host.argtypes = ([ctypes.POINTER(Dims), ctypes.POINTER(LayerParams), ip] + [vp] * 3 +
                                           [ctypes.c_size_t] + [vp] * 6)
        L.gdn_verify_step_host.restype = ip
        L.gdn_verify_lazy.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(LayerParams)] + [vp] * 13
        L.gdn_verify_lazy.restype = ip
        L.gdn_commit_lazy.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(LayerParams)] + [vp] * 8
        L.gdn_commit_lazy.restype = ip
        L.gdn_proj_in_ld.argtypes = [ctypes.POINTER(Dims)]
        L.gdn_proj_in_ld.restype = ctypes.c_longlong
        L.gdn_layer_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ip]
        L.gdn_layer_workspace_bytes.restype = ctypes.c_size_t
        for fn in (L.gdn_project_in, L.gdn_project_out):
            fn.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(ProjWeights), vp, vp, vp, ctypes.c_size_t, vp]
            fn.restype = ip
        L.gdn_layer_verify.argtypes = ([ctypes.POINTER(Dims), ctypes.POINTER(LayerParams),
                                        ctypes.POINTER(ProjWeights)] + [vp] * 7 + [ctypes.c_size_t, vp, vp])
        L.gdn_layer_verify.restype = ip
        L.gdn_lora_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ip]
        L.gdn_lora_workspace_bytes.restype = ctypes.c_size_t
        L.gdn_layer_lora_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ip, ip]
        L.gdn_layer_lora_workspace_bytes.restype = ctypes.c_size_t
        for fn in (L.gdn_project_in_lora, L.gdn_project_out_lora):
            fn.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(ProjWeights), ctypes.POINTER(Lora), vp, vp, vp, vp,
                           ctypes.c_size_t, vp, vp]
            fn.restype = ip
        L.gdn_layer_verify_lora.argtypes = ([ctypes.POINTER(Dims), ctypes.POINTER(LayerParams),
                                             ctypes.POINTER(ProjWeights), ctypes.POINTER(Lora), ctypes.POINTER(Lora)] +
                                            [vp] * 8 + [ctypes.c_size_t, vp, vp])
        L.gdn_layer_verify_lora.restype = ip
        L.gdn_sample.argtypes = [ctypes.POINTER(SampleDims), ctypes.POINTER(SampleParams)] + [vp] * 6
        L.gdn_sample.restype = ip
        L.gdn_accept.argtypes = [ctypes.POINTER(Dims)] + [vp] * 8
        L.gdn_accept.restype = ip
        L.gdn_accept_tree.argtypes = [ctypes.POINTER(Dims)] + [vp] * 10
        L.gdn_accept_tree.restype = ip
        L.gdn_kv_append.argtypes = ([ctypes.POINTER(AttnDims), ctypes.POINTER(KvCache), ctypes.POINTER(QkParams)] +
                                    [vp] * 3 + [ctypes.c_longlong] * 3 + [vp] * 6)
        L.gdn_kv_append.restype = ip
        L.gdn_attend_workspace_bytes.argtypes = [ctypes.POINTER(AttnDims)]
        L.gdn_attend_workspace_bytes.restype = ctypes.c_size_t
        L.gdn_attend.argtypes = ([ctypes.POINTER(AttnDims), ctypes.POINTER(KvCache), ctypes.POINTER(AttnParams)] +
                                 [vp] * 5 + [ctypes.c_size_t, vp, vp])
        L.gdn_attend.restype = ip
        L.gdn_prefill_workspace_bytes.argtypes = [ctypes.POINTER(Dims)]
        L.gdn_prefill_workspace_bytes.restype = ctypes.c_size_t
        L.gdn_prefill_chunked.argtypes = ([ctypes.POINTER(Dims), ctypes.POINTER(LayerParams)] + [vp] * 8 +
                                          [ctypes.c_size_t, vp, vp])
        L.gdn_prefill_chunked.restype = ip
        L.gdn_prefill_chunked_static.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(LayerParams)] + [vp] * 9
        L.gdn_prefill_chunked_static.restype = ip
        L.gdn_prefill_static_scratch_bytes.argtypes = []
        L.gdn_prefill_static_scratch_bytes.restype = ctypes.c_size_t
        L.gdn_last_error.restype = ctypes.c_char_p
        L.gdn_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_current_stream = None


def _current_stream_call():
    """A function that returns the handle of torch's current stream on its current device."""
    import torch
    torch.cuda.current_stream()                  # initialises CUDA, or says why it cannot
    # asking for the handle itself takes 0.2 us where building the Stream object takes 3, more than a launch; a torch
    # without these two gets the public call
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or device is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    return lambda: raw(device())


def _stream(stream) -> Optional[int]:
    if stream is None:
        global _current_stream
        if _current_stream is None:
            _current_stream = _current_stream_call()
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int) -> None:
    if rc != GDN_OK:
        raise GdnError(rc, gdn_last_error())


def layer_params(conv_w, A_log, dt_bias, norm_w) -> LayerParams:
    return LayerParams(_ptr(conv_w), _ptr(A_log), _ptr(dt_bias), _ptr(norm_w))


def gdn_last_error() -> str:
    return lib().gdn_last_error().decode()


def gdn_version() -> str:
    return lib().gdn_version().decode()


def gdn_verify_forward(dims: Dims, params: LayerParams, qkv, z, alpha, beta_raw, state, conv_state,
                       cap_state=None, cap_conv=None, out=None, d_status=None, stream=None) -> None:
    _check(lib().gdn_verify_forward(ctypes.byref(dims), ctypes.byref(params), _ptr(qkv), _ptr(z),
                                    _ptr(alpha), _ptr(beta_raw), _ptr(state), _ptr(conv_state),
                                    _ptr(cap_state), _ptr(cap_conv), _ptr(out), _ptr(d_status),
                                    _stream(stream)))


def gdn_rollback(dims: Dims, d_trim, state, conv_state, cap_state, cap_conv, d_status=None,
                 stream=None) -> None:
    _check(lib().gdn_rollback(ctypes.byref(dims), _ptr(d_trim), _ptr(state), _ptr(conv_state),
                              _ptr(cap_state), _ptr(cap_conv), _ptr(d_status), _stream(stream)))


def pointer_table(tensors, device="cuda"):
    """A DEVICE int64 array of the tensors' data pointers (the tables gdn_rollback_layers reads)."""
    import torch
    return torch.tensor([t.data_ptr() for t in tensors], dtype=torch.int64, device=device)


def gdn_rollback_layers(dims: Dims, n_layers: int, d_trim, tab_state, tab_conv_state, tab_cap_state, tab_cap_conv,
                        d_status=None, stream=None) -> None:
    """gdn_rollback of n_layers layers in one launch; the tab_* are device pointer tables (pointer_table)."""
    _check(lib().gdn_rollback_layers(ctypes.byref(dims), int(n_layers), _ptr(d_trim), _ptr(tab_state),
                                     _ptr(tab_conv_state), _ptr(tab_cap_state), _ptr(tab_cap_conv), _ptr(d_status),
                                     _stream(stream)))


def gdn_rollback_tree_layers(dims: Dims, n_layers: int, d_accept, tab_state, tab_conv_state, tab_cap_state,
                             tab_cap_conv, d_status=None, stream=None) -> None:
    """gdn_rollback_tree of n_layers layers in one launch; the tab_* are device pointer tables (pointer_table)."""
    _check(lib().gdn_rollback_tree_layers(ctypes.byref(dims), int(n_layers), _ptr(d_accept), _ptr(tab_state),
                                          _ptr(tab_conv_state), _ptr(tab_cap_state), _ptr(tab_cap_conv),
                                          _ptr(d_status), _stream(stream)))


def gdn_verify_tree(dims: Dims, params: LayerParams, qkv, z, alpha, beta_raw, d_parent, state, conv_state,
                    cap_state, cap_conv, out, d_status=None, stream=None) -> None:
    _check(lib().gdn_verify_tree(ctypes.byref(dims), ctypes.byref(params), _ptr(qkv), _ptr(z), _ptr(alpha),
                                 _ptr(beta_raw), _ptr(d_parent), _ptr(state), _ptr(conv_state), _ptr(cap_state),
                                 _ptr(cap_conv), _ptr(out), _ptr(d_status), _stream(stream)))


def gdn_rollback_tree(dims: Dims, d_accept, state, conv_state, cap_state, cap_conv, d_status=None,
                      stream=None) -> None:
    _check(lib().gdn_rollback_tree(ctypes.byref(dims), _ptr(d_accept), _ptr(state), _ptr(conv_state),
                                   _ptr(cap_state), _ptr(cap_conv), _ptr(d_status), _stream(stream)))


def gdn_verify_after_rollback(dims: Dims, params: LayerParams, d_prev_trim, qkv, z, alpha, beta_raw, state,
                              conv_state, cap_state, cap_conv, out, d_status=None, stream=None) -> None:
    """Verify starting from what gdn_rollback(d_prev_trim) would leave, read from the
    previous batch's captures (which this call overwrites)."""
    _check(lib().gdn_verify_after_rollback(ctypes.byref(dims), ctypes.byref(params), _ptr(d_prev_trim), _ptr(qkv),
                                           _ptr(z), _ptr(alpha), _ptr(beta_raw), _ptr(state), _ptr(conv_state),
                                           _ptr(cap_state), _ptr(cap_conv), _ptr(out), _ptr(d_status),
                                           _stream(stream)))


def gdn_step_io_layout(dims: Dims) -> StepIO:
    io = StepIO()
    _check(lib().gdn_step_io_layout(ctypes.byref(dims), ctypes.byref(io)))
    return io


def gdn_verify_step_host(dims: Dims, params: LayerParams, rollback_first: int, h_in, h_out, d_io, d_io_bytes: int,
                         state, conv_state, cap_state, cap_conv, d_status=None, stream=None) -> None:
    """One verify step from host memory (packed pinned input block, output block)."""
    _check(lib().gdn_verify_step_host(ctypes.byref(dims), ctypes.byref(params), int(rollback_first), _ptr(h_in),
                                      _ptr(h_out), _ptr(d_io), int(d_io_bytes), _ptr(state), _ptr(conv_state),
                                      _ptr(cap_state), _ptr(cap_conv), _ptr(d_status), _stream(stream)))


def gdn_verify_lazy(dims: Dims, params: LayerParams, qkv, z, alpha, beta_raw, state, conv_state, out,
                    d_status=None, stream=None, prev_trim=None, prev_qkv=None, prev_alpha=None,
                    prev_beta_raw=None) -> None:
    """Outputs-only verify; with prev_trim (device int32[B]) it first commits the
    pending batch (prev_qkv, prev_alpha, prev_beta_raw) into state / conv_state."""
    _check(lib().gdn_verify_lazy(ctypes.byref(dims), ctypes.byref(params), _ptr(prev_trim), _ptr(prev_qkv),
                                 _ptr(prev_alpha), _ptr(prev_beta_raw), _ptr(qkv), _ptr(z), _ptr(alpha),
                                 _ptr(beta_raw), _ptr(state), _ptr(conv_state), _ptr(out), _ptr(d_status),
                                 _stream(stream)))


def gdn_commit_lazy(dims: Dims, params: LayerParams, d_trim, qkv, alpha, beta_raw, state, conv_state,
                    d_status=None, stream=None) -> None:
    _check(lib().gdn_commit_lazy(ctypes.byref(dims), ctypes.byref(params), _ptr(d_trim), _ptr(qkv),
                                 _ptr(alpha), _ptr(beta_raw), _ptr(state), _ptr(conv_state), _ptr(d_status),
                                 _stream(stream)))


def proj_weights(n_embd: int, w_in, w_out) -> "ProjWeights":
    """The projection weights of one layer (device tensors or pointers): w_in
    [C + H_v*d_v + 2*H_v][n_embd] (wqkv, wqkv_gate, ssm_alpha, ssm_beta rows),
    w_out [n_embd][H_v*d_v]; both bf16."""
    return ProjWeights(int(n_embd), _ptr(w_in), _ptr(w_out))


def gdn_proj_in_ld(dims: Dims) -> int:
    return int(lib().gdn_proj_in_ld(ctypes.byref(dims)))


def gdn_layer_workspace_bytes(dims: Dims, n_embd: int) -> int:
    return int(lib().gdn_layer_workspace_bytes(ctypes.byref(dims), int(n_embd)))


def gdn_project_in(dims: Dims, w: "ProjWeights", x, act, workspace, ws_bytes: int, stream=None) -> None:
    _check(lib().gdn_project_in(ctypes.byref(dims), ctypes.byref(w), _ptr(x), _ptr(act), _ptr(workspace),
                                int(ws_bytes), _stream(stream)))


def gdn_project_out(dims: Dims, w: "ProjWeights", out, y, workspace, ws_bytes: int, stream=None) -> None:
    _check(lib().gdn_project_out(ctypes.byref(dims), ctypes.byref(w), _ptr(out), _ptr(y), _ptr(workspace),
                                 int(ws_bytes), _stream(stream)))


def gdn_layer_verify(dims: Dims, params: LayerParams, w: "ProjWeights", x, state, conv_state, cap_state, cap_conv,
                     y, workspace, ws_bytes: int, d_status=None, stream=None) -> None:
    _check(lib().gdn_layer_verify(ctypes.byref(dims), ctypes.byref(params), ctypes.byref(w), _ptr(x), _ptr(state),
                                  _ptr(conv_state), _ptr(cap_state), _ptr(cap_conv), _ptr(y), _ptr(workspace),
                                  int(ws_bytes), _ptr(d_status), _stream(stream)))


def lora(n_adapters: int, rank: int, a, b, scale=None) -> Lora:
    """The low-rank adapters beside one projection of K input and N output columns (device tensors or pointers): a
    [n_adapters][rank][K] and b [n_adapters][N][rank] bf16, scale [n_adapters] f32 (None: 1)."""
    v = Lora(int(n_adapters), int(rank), _ptr(a), _ptr(b), _ptr(scale))
    v.tensors = (a, b, scale)            # the struct holds addresses: keep what they point to
    return v


def gdn_lora_workspace_bytes(dims: Dims, rank: int) -> int:
    return int(lib().gdn_lora_workspace_bytes(ctypes.byref(dims), int(rank)))


def gdn_project_in_lora(dims: Dims, w: "ProjWeights", lora: Lora, d_adapter, x, act, workspace, ws_bytes: int,
                        d_status=None, stream=None) -> None:
    """gdn_project_in, each slot's rows with the adapter d_adapter (device int32[B]) names beside it (-1: none)."""
    _check(lib().gdn_project_in_lora(ctypes.byref(dims), ctypes.byref(w), ctypes.byref(lora), _ptr(d_adapter), _ptr(x),
                                     _ptr(act), _ptr(workspace), int(ws_bytes), _ptr(d_status), _stream(stream)))


def gdn_project_out_lora(dims: Dims, w: "ProjWeights", lora: Lora, d_adapter, out, y, workspace, ws_bytes: int,
                         d_status=None, stream=None) -> None:
    """gdn_project_out with adapters, as gdn_project_in_lora."""
    _check(lib().gdn_project_out_lora(ctypes.byref(dims), ctypes.byref(w), ctypes.byref(lora), _ptr(d_adapter),
                                      _ptr(out), _ptr(y), _ptr(workspace), int(ws_bytes), _ptr(d_status),
                                      _stream(stream)))


def gdn_layer_lora_workspace_bytes(dims: Dims, n_embd: int, rank: int) -> int:
    return int(lib().gdn_layer_lora_workspace_bytes(ctypes.byref(dims), int(n_embd), int(rank)))


def gdn_layer_verify_lora(dims: Dims, params: LayerParams, w: "ProjWeights", lora_in: Optional[Lora],
                          lora_out: Optional[Lora], d_adapter, x, state, conv_state, cap_state, cap_conv, y, workspace,
                          ws_bytes: int, d_status=None, stream=None) -> None:
    """gdn_layer_verify with adapters beside its input projection, its output projection, or both."""
    ref = lambda v: None if v is None else ctypes.byref(v)  # noqa: E731
    _check(lib().gdn_layer_verify_lora(ctypes.byref(dims), ctypes.byref(params), ctypes.byref(w), ref(lora_in),
                                       ref(lora_out), _ptr(d_adapter), _ptr(x), _ptr(state), _ptr(conv_state),
                                       _ptr(cap_state), _ptr(cap_conv), _ptr(y), _ptr(workspace), int(ws_bytes),
                                       _ptr(d_status), _stream(stream)))


def make_sample_dims(n_slots: int, n_tokens: int, vocab: int, ld: Optional[int] = None,
                     dtype: int = GDN_F32) -> SampleDims:
    """Logits [n_slots * n_tokens][ld], the first vocab columns of each row used (ld None: vocab)."""
    return SampleDims(n_slots, n_tokens, vocab, dtype, vocab if ld is None else ld)


def sample_params(temperature=None, top_k=None, top_p=None, min_p=None) -> SampleParams:
    """Per-slot sampling parameters: device f32[B] (top_k: int32[B]); None: temperature 1, filter off."""
    v = SampleParams(_ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p))
    v.tensors = (temperature, top_k, top_p, min_p)
    return v


def gdn_sample(dims: SampleDims, params: SampleParams, logits, u, tokens, logprob=None, d_status=None,
               stream=None) -> None:
    """One token per row of logits from the uniforms u [B][T]; tokens [B][T] int32, logprob [B][T] f32 or None."""
    _check(lib().gdn_sample(ctypes.byref(dims), ctypes.byref(params), _ptr(logits), _ptr(u), _ptr(tokens),
                            _ptr(logprob), _ptr(d_status), _stream(stream)))


def gdn_accept(dims: Dims, draft, tokens, d_length, d_trim, d_next=None, d_emit=None, d_status=None,
               stream=None) -> None:
    """How much of its draft each slot keeps: d_trim [B] for the rollbacks, d_next [B], d_emit [B][T]."""
    _check(lib().gdn_accept(ctypes.byref(dims), _ptr(draft), _ptr(tokens), _ptr(d_length), _ptr(d_trim), _ptr(d_next),
                            _ptr(d_emit), _ptr(d_status), _stream(stream)))


def gdn_accept_tree(dims: Dims, d_parent, draft, tokens, d_length, d_accept, d_next=None, d_emit=None, d_path=None,
                    d_status=None, stream=None) -> None:
    """The accepted path of each slot's draft tree: d_accept [B] for gdn_rollback_tree, d_next [B], d_emit and
    d_path [B][T]."""
    _check(lib().gdn_accept_tree(ctypes.byref(dims), _ptr(d_parent), _ptr(draft), _ptr(tokens), _ptr(d_length),
                                 _ptr(d_accept), _ptr(d_next), _ptr(d_emit), _ptr(d_path), _ptr(d_status),
                                 _stream(stream)))


def make_attn_dims(n_slots: int, n_tokens: int, n_heads: int, n_kv_heads: int, d_head: int, page_tokens: int, n_pages: int,
                   max_pages: int, page_stride: Optional[int] = None, dtype: int = GDN_BF16) -> AttnDims:
    """A batch over a paged cache; page_stride None: pages follow one another."""
    stride = n_kv_heads * page_tokens * d_head if page_stride is None else page_stride
    return AttnDims(n_slots, n_tokens, n_heads, n_kv_heads, d_head, page_tokens, n_pages, max_pages, stride, dtype)


def kv_cache(k, v, page_table, past) -> KvCache:
    """One layer's pools [n_pages][n_kv_heads][page_tokens][d_head], the slots' pages [B][max_pages] and the positions
    they hold before the batch [B] (int32)."""
    c = KvCache(_ptr(k), _ptr(v), _ptr(page_table), _ptr(past))
    c.tensors = (k, v, page_table, past)
    return c


def qk_params(rope_dims: int, freq=None, q_norm=None, k_norm=None, norm_eps: float = 1e-6,
              adjacent: bool = False) -> QkParams:
    """Rotation (freq: device f32[rope_dims/2], radians a position) and the heads' norms (device f32[d_head], or None)."""
    p = QkParams(int(rope_dims), int(adjacent), _ptr(freq), _ptr(q_norm), _ptr(k_norm), norm_eps)
    p.tensors = (freq, q_norm, k_norm)
    return p


def attn_params(scale: float, window: int = 0, n_sink: int = 0) -> AttnParams:
    return AttnParams(scale, int(window), int(n_sink))


def gdn_kv_append(dims: AttnDims, cache: KvCache, params: QkParams, q, k, v, ld_q: int, ld_k: int, ld_v: int, q_out,
                  d_length=None, d_parent=None, d_path=None, d_status=None, stream=None) -> None:
    """Rotates q into q_out (both may be None) and k into the cache, and appends v; with d_path the accepted path of a
    tree goes to its final places."""
    _check(lib().gdn_kv_append(ctypes.byref(dims), ctypes.byref(cache), ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v),
                               int(ld_q), int(ld_k), int(ld_v), _ptr(q_out), _ptr(d_length), _ptr(d_parent),
                               _ptr(d_path), _ptr(d_status), _stream(stream)))


def gdn_attend_workspace_bytes(dims: AttnDims) -> int:
    return int(lib().gdn_attend_workspace_bytes(ctypes.byref(dims)))


def gdn_attend(dims: AttnDims, cache: KvCache, params: AttnParams, q, out, workspace, ws_bytes: int, d_length=None,
               d_parent=None, d_status=None, stream=None) -> None:
    """Attention of the batch's tokens over the cache: q and out [B][T][n_heads][d_head]."""
    _check(lib().gdn_attend(ctypes.byref(dims), ctypes.byref(cache), ctypes.byref(params), _ptr(q), _ptr(out),
                            _ptr(d_length), _ptr(d_parent), _ptr(workspace), int(ws_bytes), _ptr(d_status),
                            _stream(stream)))


def gdn_prefill_workspace_bytes(dims: Dims) -> int:
    return int(lib().gdn_prefill_workspace_bytes(ctypes.byref(dims)))


def gdn_prefill_chunked(dims: Dims, params: LayerParams, qkv, z, alpha, beta_raw, state, conv_state, out,
                        workspace=None, ws_bytes: int = 0, d_status=None, stream=None) -> None:
    _check(lib().gdn_prefill_chunked(ctypes.byref(dims), ctypes.byref(params), _ptr(qkv), _ptr(z),
                                     _ptr(alpha), _ptr(beta_raw), _ptr(state), _ptr(conv_state), _ptr(out),
                                     _ptr(workspace), ctypes.c_size_t(ws_bytes), _ptr(d_status),
                                     _stream(stream)))


def prefill_static_scratch_bytes() -> int:
    """Size of the library's built-in prefill scratch (GDN_PREFILL_STATIC_SCRATCH_BYTES), read from the library."""
    return int(lib().gdn_prefill_static_scratch_bytes())


def gdn_prefill_chunked_static(dims: Dims, params: LayerParams, qkv, z, alpha, beta_raw, state, conv_state, out,
                               d_status=None, stream=None) -> None:
    """gdn_prefill_chunked with the library's built-in scratch instead of a workspace."""
    _check(lib().gdn_prefill_chunked_static(ctypes.byref(dims), ctypes.byref(params), _ptr(qkv), _ptr(z),
                                            _ptr(alpha), _ptr(beta_raw), _ptr(state), _ptr(conv_state),
                                            _ptr(out), _ptr(d_status), _stream(stream)))
