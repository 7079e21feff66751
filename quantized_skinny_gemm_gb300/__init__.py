"""Python binding of libdg.so, the sm_103a decode-step skinny GEMV library.

Argument marshalling only: every function takes torch CUDA tensors, passes
their device pointers, shapes and the current CUDA stream to the C entry point
of the same name (``dg_<name>`` in include/dg.h) and raises ``DGError`` when it
returns a status other than DG_OK.  All arithmetic runs in the library's
kernels; there is no fallback of any kind, and using a function without the
built library raises.
"""
import ctypes
import os

__all__ = [
    "DGError", "Linear", "StepPlan", "F16", "BF16", "LINEAR_F16", "LINEAR_BF16",
    "LINEAR_W8A8", "LINEAR_W4A16", "LINEAR_W4A8", "gemv_f16", "gemv_w8a8", "gemv_w4",
    "quantize_act_i8", "lm_head_argmax", "lm_head_argmax_noalloc", "decode_step_weights", "workspace_bytes",
    "EPI_NONE", "EPI_RESIDUAL", "EPI_SWIGLU", "ACT_NONE", "ACT_SILU", "linear_forward", "swiglu",
    "residual_add", "causal_conv1d_update", "quantize_weights_i8", "quantize_weights_w4",
    "NORM_RMS", "NORM_LAYER", "MOE_SOFTMAX", "MOE_SIGMOID", "PagedKV", "Append", "Attention",
    "Norm", "Moe", "paged_kv", "append", "kv_append", "attention", "attn_decode",
    "attn_workspace_bytes", "norm", "norm_residual", "moe", "moe_forward", "moe_workspace_bytes",
    "PagedKV4", "HeadAppend", "KV4Rows", "Attention4", "PagePlan", "Logprobs", "paged_kv4", "head_append",
    "qkv_append", "kv4_rows", "kv4_read", "attention4", "attn4_decode", "attn4_workspace_bytes", "page_plan",
    "assign_pages", "pages_workspace_bytes", "logprobs", "token_logprobs", "logprobs_workspace_bytes",
    "check_device_status", "selftest_wait_timeout", "status_string", "probe_copy", "probe_read", "version",
    "library_path", "load",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libdg.so")

F16, BF16 = 0, 1
LINEAR_F16, LINEAR_BF16, LINEAR_W8A8, LINEAR_W4A16, LINEAR_W4A8 = range(5)
EPI_NONE, EPI_RESIDUAL, EPI_SWIGLU = range(3)
ACT_NONE, ACT_SILU = range(2)
NORM_RMS, NORM_LAYER = range(2)
MOE_SOFTMAX, MOE_SIGMOID = range(2)
_STATUS = ["DG_OK", "DG_ERR_INVALID_ARG", "DG_ERR_UNSUPPORTED", "DG_ERR_MISALIGNED",
           "DG_ERR_WORKSPACE", "DG_ERR_CUDA", "DG_ERR_TIMEOUT"]


class DGError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        name = _STATUS[status] if 0 <= status < len(_STATUS) else str(status)
        super().__init__("%s returned %s" % (where, name))


class Linear(ctypes.Structure):
    """Mirror of the C struct dg_linear."""
    _fields_ = [
        ("kind", ctypes.c_int32), ("M", ctypes.c_int32), ("N", ctypes.c_int32),
        ("K", ctypes.c_int32), ("group_size", ctypes.c_int32),
        ("W", ctypes.c_void_p), ("w_scale", ctypes.c_void_p), ("x", ctypes.c_void_p),
        ("x_i8", ctypes.c_void_p), ("x_scale", ctypes.c_void_p), ("y", ctypes.c_void_p),
        ("logits", ctypes.c_void_p), ("token", ctypes.c_void_p), ("acc_out", ctypes.c_void_p),
        ("epilogue", ctypes.c_int32), ("reserved", ctypes.c_int32), ("residual", ctypes.c_void_p),
        ("W2", ctypes.c_void_p), ("w2_scale", ctypes.c_void_p),
    ]


class PagedKV(ctypes.Structure):
    """Mirror of the C struct dg_paged_kv."""
    _fields_ = [
        ("type", ctypes.c_int32), ("batch", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("reserved", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64), ("block_table", ctypes.c_void_p),
        ("table_stride", ctypes.c_int64), ("seq_lens", ctypes.c_void_p),
    ]


class Append(ctypes.Structure):
    """Mirror of the C struct dg_append."""
    _fields_ = [
        ("kv", PagedKV), ("q_len", ctypes.c_int32), ("heads", ctypes.c_int32),
        ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
        ("max_pos", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("q_out", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64),
        ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p),
    ]


class Attention(ctypes.Structure):
    """Mirror of the C struct dg_attn."""
    _fields_ = [
        ("kv", PagedKV), ("q_len", ctypes.c_int32), ("heads", ctypes.c_int32),
        ("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("scale", ctypes.c_float),
        ("reserved", ctypes.c_int32), ("q", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
    ]


class Norm(ctypes.Structure):
    """Mirror of the C struct dg_norm."""
    _fields_ = [
        ("type", ctypes.c_int32), ("kind", ctypes.c_int32), ("rows", ctypes.c_int32),
        ("N", ctypes.c_int32), ("h_f32", ctypes.c_int32), ("gate_rows", ctypes.c_int32),
        ("alpha", ctypes.c_float), ("beta", ctypes.c_float), ("eps", ctypes.c_float),
        ("w_offset", ctypes.c_float), ("y", ctypes.c_void_p), ("w_post", ctypes.c_void_p),
        ("b_post", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("h", ctypes.c_void_p),
        ("w_pre", ctypes.c_void_p), ("b_pre", ctypes.c_void_p), ("h_out", ctypes.c_void_p),
        ("x_out", ctypes.c_void_p),
    ]


class Moe(ctypes.Structure):
    """Mirror of the C struct dg_moe."""
    _fields_ = [
        ("kind", ctypes.c_int32), ("M", ctypes.c_int32), ("K", ctypes.c_int32),
        ("I", ctypes.c_int32), ("E", ctypes.c_int32), ("top_k", ctypes.c_int32),
        ("group_size", ctypes.c_int32), ("score", ctypes.c_int32),
        ("renormalize", ctypes.c_int32), ("route_scale", ctypes.c_float),
        ("x", ctypes.c_void_p), ("router", ctypes.c_void_p), ("W_gate", ctypes.c_void_p),
        ("W_up", ctypes.c_void_p), ("W_down", ctypes.c_void_p), ("gate_scale", ctypes.c_void_p),
        ("up_scale", ctypes.c_void_p), ("down_scale", ctypes.c_void_p),
        ("residual", ctypes.c_void_p), ("y", ctypes.c_void_p), ("ids", ctypes.c_void_p),
        ("weights", ctypes.c_void_p),
    ]


class PagedKV4(ctypes.Structure):
    """Mirror of the C struct dg_paged_kv4."""
    _fields_ = [
        ("type", ctypes.c_int32), ("batch", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("reserved", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64), ("scale_page_stride", ctypes.c_int64),
        ("scale_token_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64),
        ("k_factor", ctypes.c_float), ("v_factor", ctypes.c_float),
        ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
        ("seq_lens", ctypes.c_void_p),
    ]


class HeadAppend(ctypes.Structure):
    """Mirror of the C struct dg_head_append."""
    _fields_ = [
        ("kv", PagedKV), ("kv4", PagedKV4), ("bits", ctypes.c_int32), ("q_len", ctypes.c_int32),
        ("tokens", ctypes.c_int32), ("heads", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32), ("max_pos", ctypes.c_int32), ("norm", ctypes.c_int32),
        ("eps", ctypes.c_float), ("w_offset", ctypes.c_float), ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
        ("q_out_stride", ctypes.c_int64), ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p),
        ("w_q", ctypes.c_void_p), ("w_k", ctypes.c_void_p), ("slots", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
    ]


class KV4Rows(ctypes.Structure):
    """Mirror of the C struct dg_kv4_rows."""
    _fields_ = [
        ("kv", PagedKV4), ("q_len", ctypes.c_int32), ("tokens", ctypes.c_int32),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64), ("slots", ctypes.c_void_p),
    ]


class Attention4(ctypes.Structure):
    """Mirror of the C struct dg_attn4."""
    _fields_ = [
        ("kv", PagedKV4), ("q_len", ctypes.c_int32), ("heads", ctypes.c_int32),
        ("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("scale", ctypes.c_float),
        ("reserved", ctypes.c_int32), ("q", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
    ]


class PagePlan(ctypes.Structure):
    """Mirror of the C struct dg_page_plan."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("pool_size", ctypes.c_int32), ("new_len", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
        ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p), ("new_lens", ctypes.c_void_p),
        ("lens_out", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("pool", ctypes.c_void_p),
        ("pool_state", ctypes.c_void_p), ("pool_state_out", ctypes.c_void_p),
        ("starts", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p),
    ]


class Logprobs(ctypes.Structure):
    """Mirror of the C struct dg_logprobs."""
    _fields_ = [
        ("type", ctypes.c_int32), ("logits_f32", ctypes.c_int32), ("rows", ctypes.c_int32),
        ("V", ctypes.c_int32), ("top_k", ctypes.c_int32), ("scale", ctypes.c_float),
        ("stride", ctypes.c_int64), ("logits", ctypes.c_void_p), ("tokens", ctypes.c_void_p),
        ("logprob", ctypes.c_void_p), ("rank", ctypes.c_void_p), ("entropy", ctypes.c_void_p),
        ("lse", ctypes.c_void_p), ("top_ids", ctypes.c_void_p), ("top_logprobs", ctypes.c_void_p),
    ]


_lib = None


def library_path():
    return _LIB_PATH


def load():
    """Loads libdg.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError("libdg.so is not built (%s); run __graft_entry__.build()" % _LIB_PATH)
    lib = ctypes.CDLL(_LIB_PATH)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    sig = {
        "dg_gemv_f16": [P, P, P, I, I, I, I, P, Z, P],
        "dg_gemv_w8a8": [P, P, P, P, P, P, I, I, I, P, Z, P],
        "dg_gemv_w4": [P, P, I, P, P, P, P, I, I, I, P, Z, P],
        "dg_quantize_act_i8": [P, P, P, I, I, P],
        "dg_lm_head_argmax": [P, P, Z, P],
        "dg_lm_head_argmax_noalloc": [P, P],
        "dg_decode_step_weights": [P, I, P, Z, P],
        "dg_check_device_status": [P],
        "dg_selftest_wait_timeout": [ctypes.c_uint, P],
        "dg_probe_copy": [P, P, Z, P],
        "dg_linear_forward": [P, P, Z, P],
        "dg_swiglu": [P, P, P, I, P],
        "dg_residual_add": [P, P, P, I, P],
        "dg_causal_conv1d_update": [P, P, P, P, P, I, I, I, I, P],
        "dg_quantize_weights_i8": [P, P, P, I, I, P],
        "dg_quantize_weights_w4": [P, P, P, I, I, I, P],
        "dg_probe_read": [P, Z, P, P],
        "dg_kv_append": [P, P],
        "dg_attn_decode": [P, P, Z, P],
        "dg_norm_residual": [P, P],
        "dg_moe_forward": [P, P, Z, P],
        "dg_qkv_append": [P, P],
        "dg_kv4_read": [P, P],
        "dg_attn4_decode": [P, P, Z, P],
        "dg_assign_pages": [P, P, Z, P],
        "dg_token_logprobs": [P, P, Z, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.dg_workspace_bytes.argtypes = [P, I]
    lib.dg_workspace_bytes.restype = Z
    for name in ("dg_attn_workspace_bytes", "dg_moe_workspace_bytes", "dg_attn4_workspace_bytes",
                 "dg_pages_workspace_bytes", "dg_logprobs_workspace_bytes"):
        getattr(lib, name).argtypes = [P]
        getattr(lib, name).restype = Z
    lib.dg_status_string.argtypes = [I]
    lib.dg_status_string.restype = ctypes.c_char_p
    lib.dg_version.argtypes = []
    lib.dg_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _ptr(t):
    return None if t is None else t.data_ptr()


_current = None


def _stream(stream):
    """The handle of a stream, or of the current one.  Asking torch for the raw
    handle takes 0.4 us, building its Stream object 3 us: half of a small call."""
    global _current
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    if _current is None:
        import torch
        torch.cuda.init()
        _current = (torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice)
    raw, device = _current
    return raw(device())


def _call(name, *args):
    st = getattr(load(), name)(*args)
    if st != 0:
        raise DGError(st, name)


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


# ---- entry points ----------------------------------------------------------------

def gemv_f16(W, x, y, dtype=F16, ws=None, stream=None):
    """y[M][N] = x[M][K] . W[N][K]^T for fp16 (dtype=F16) or bf16 (BF16) tensors."""
    N, K = W.shape
    M = x.numel() // K
    _call("dg_gemv_f16", _ptr(W), _ptr(x), _ptr(y), dtype, M, N, K, _ptr(ws), _nbytes(ws),
          _stream(stream))


def gemv_w8a8(W, w_scale, x_i8, x_scale, y=None, acc_out=None, ws=None, stream=None):
    N, K = W.shape
    M = x_i8.numel() // K
    _call("dg_gemv_w8a8", _ptr(W), _ptr(w_scale), _ptr(x_i8), _ptr(x_scale), _ptr(y),
          _ptr(acc_out), M, N, K, _ptr(ws), _nbytes(ws), _stream(stream))


def gemv_w4(Wq, scales, y, x_f16=None, x_i8=None, x_scale=None, group_size=32, ws=None,
            stream=None):
    """W4A16 when x_i8 is None, W4A8 otherwise.  Wq uint8 [N][K/2]."""
    N, K2 = Wq.shape
    K = 2 * K2
    xa = x_i8 if x_i8 is not None else x_f16
    M = xa.numel() // K
    _call("dg_gemv_w4", _ptr(Wq), _ptr(scales), group_size, _ptr(x_f16), _ptr(x_i8),
          _ptr(x_scale), _ptr(y), M, N, K, _ptr(ws), _nbytes(ws), _stream(stream))


def quantize_act_i8(x, xq, x_scale, stream=None):
    K = x.shape[-1]
    M = x.numel() // K
    _call("dg_quantize_act_i8", _ptr(x), _ptr(xq), _ptr(x_scale), M, K, _stream(stream))


def linear(kind, W, M, N, K, w_scale=None, x=None, x_i8=None, x_scale=None, y=None,
           logits=None, token=None, acc_out=None, group_size=32, epilogue=EPI_NONE,
           residual=None, W2=None, w2_scale=None):
    """Builds a Linear descriptor from tensors (pointers only; keep the tensors alive)."""
    return Linear(kind, M, N, K, group_size, _ptr(W), _ptr(w_scale), _ptr(x), _ptr(x_i8),
                  _ptr(x_scale), _ptr(y), _ptr(logits), _ptr(token), _ptr(acc_out), epilogue, 0,
                  _ptr(residual), _ptr(W2), _ptr(w2_scale))


def linear_forward(op, ws=None, stream=None):
    """Runs one op described by a Linear (any kind but an lm_head; any epilogue)."""
    _call("dg_linear_forward", ctypes.byref(op), _ptr(ws), _nbytes(ws), _stream(stream))


def swiglu(g, u, h, stream=None):
    """h = silu(g) * u elementwise (fp16)."""
    _call("dg_swiglu", _ptr(g), _ptr(u), _ptr(h), g.numel(), _stream(stream))


def residual_add(a, b, out, stream=None):
    """out = a + b elementwise (fp16)."""
    _call("dg_residual_add", _ptr(a), _ptr(b), _ptr(out), a.numel(), _stream(stream))


def causal_conv1d_update(x, state, w, y, bias=None, act=ACT_SILU, stream=None):
    """One causal-conv1d decode step: x [M][C], state [M][C][W-1] (updated in
    place), w [C][W], bias [C] or None, y [M][C]; all fp16."""
    C, width = w.shape
    M = x.numel() // C
    _call("dg_causal_conv1d_update", _ptr(x), _ptr(state), _ptr(w), _ptr(bias), _ptr(y), M, C,
          width, act, _stream(stream))


def quantize_weights_i8(W, Wq, w_scale, stream=None):
    """fp16 W [N][K] -> int8 Wq [N][K] + fp32 per-row scales (load-time packer)."""
    N, K = W.shape
    _call("dg_quantize_weights_i8", _ptr(W), _ptr(Wq), _ptr(w_scale), N, K, _stream(stream))


def quantize_weights_w4(W, Wq, scales, group_size=32, stream=None):
    """fp16 W [N][K] -> packed int4 Wq [N][K/2] + fp16 scales [N][K/group] (load-time packer)."""
    N, K = W.shape
    _call("dg_quantize_weights_w4", _ptr(W), _ptr(Wq), _ptr(scales), N, K, group_size,
          _stream(stream))


def lm_head_argmax(head, ws, stream=None):
    _call("dg_lm_head_argmax", ctypes.byref(head), _ptr(ws), _nbytes(ws), _stream(stream))


def lm_head_argmax_noalloc(head, stream=None):
    """lm_head + argmax with the library's own fixed scratch (no workspace)."""
    _call("dg_lm_head_argmax_noalloc", ctypes.byref(head), _stream(stream))


class StepPlan:
    """A decode step's ops, marshalled once into a C array of dg_linear."""

    def __init__(self, ops, keep=()):
        self.n = len(ops)
        self.array = (Linear * self.n)(*ops)
        self.keep = list(keep)  # tensors the descriptors point into

    def workspace_bytes(self):
        return int(load().dg_workspace_bytes(ctypes.cast(self.array, ctypes.c_void_p), self.n))


def decode_step_weights(plan, ws=None, stream=None):
    _call("dg_decode_step_weights", ctypes.cast(plan.array, ctypes.c_void_p), plan.n, _ptr(ws),
          _nbytes(ws), _stream(stream))


def workspace_bytes(ops):
    arr = (Linear * len(ops))(*ops)
    return int(load().dg_workspace_bytes(ctypes.cast(arr, ctypes.c_void_p), len(ops)))


# ---- the rest of a decoder layer ---------------------------------------------------
# Builders make a descriptor from tensors (pointers, shapes and strides only;
# keep the tensors alive), raising DGError where the tensors themselves do not
# fit together; the entry points of the same C name then run it.

def _fits(ok, where):
    if not ok:
        raise DGError(_STATUS.index("DG_ERR_INVALID_ARG"), where)


def _ftype(t, where):
    import torch
    _fits(t.dtype in (torch.float16, torch.bfloat16), where)
    return F16 if t.dtype == torch.float16 else BF16


def _contiguous(where, dtype, *tensors):
    for t in tensors:
        _fits(t is None or (t.dtype == dtype and t.is_contiguous()), where)


def _head_rows(t, tokens, heads, dim, dtype, where):
    """Elements between the tokens of t [tokens][heads][dim], heads adjacent."""
    if t.is_contiguous() and t.numel() == tokens * heads * dim:
        t = t.view(tokens, heads, dim)
    _fits(t.dtype == dtype and tuple(t.shape) == (tokens, heads, dim) and t.stride(2) == 1 and
          (heads == 1 or t.stride(1) == dim), where)
    return t.stride(0) if tokens > 1 else heads * dim


def paged_kv(k_cache, v_cache, block_table, seq_lens):
    """A paged cache: k_cache and v_cache [pages][page_size][kv_heads][head_dim]
    (any strides with the last dimension contiguous and both alike, so a
    [pages][kv_heads][page_size][head_dim] cache is passed transposed),
    block_table int32 [batch][max_pages] with rows at least max_pages apart (no
    expanded tables), seq_lens int32 [batch]."""
    import torch
    where = "paged_kv"
    kind = _ftype(k_cache, where)
    _fits(k_cache.dim() == 4 and k_cache.shape == v_cache.shape and
          k_cache.dtype == v_cache.dtype and k_cache.stride() == v_cache.stride() and
          k_cache.stride(3) == 1, where)
    _fits(block_table.dim() == 2 and block_table.dtype == torch.int32 and
          (block_table.shape[1] <= 1 or block_table.stride(1) == 1), where)
    _fits(seq_lens.dtype == torch.int32 and seq_lens.is_contiguous() and
          0 < seq_lens.numel() == block_table.shape[0], where)
    pages, page_size, heads, dim = k_cache.shape
    table_stride = block_table.stride(0) if block_table.shape[0] > 1 else block_table.shape[1]
    _fits(table_stride >= block_table.shape[1], where)
    return PagedKV(kind, block_table.shape[0], heads, dim, page_size, pages,
                   block_table.shape[1], 0, _ptr(k_cache), _ptr(v_cache), k_cache.stride(0),
                   k_cache.stride(1), k_cache.stride(2), _ptr(block_table), table_stride,
                   _ptr(seq_lens))


def _kv_dtype(kv):
    import torch
    return torch.float16 if kv.type == F16 else torch.bfloat16


def append(kv, q, k, v, q_out=None, q_len=1, cos=None, sin=None, interleaved=False):
    """Describes kv_append: q [batch * q_len][heads][head_dim] (or None), k and v
    with kv_heads heads; cos and sin fp32 [max_pos][rot_dim / 2], or None for no
    rotation; q_out is q itself by default."""
    import torch
    where, dt = "append", _kv_dtype(kv)
    _fits(q_len > 0, where)
    tokens, dim = kv.batch * q_len, kv.head_dim
    heads = 0 if q is None else q.numel() // (tokens * dim)
    q_out = q if q_out is None else q_out
    qs = qos = 0
    if q is not None:
        qs = _head_rows(q, tokens, heads, dim, dt, where)
        qos = _head_rows(q_out, tokens, heads, dim, dt, where)
    ks = _head_rows(k, tokens, kv.kv_heads, dim, dt, where)
    vs = _head_rows(v, tokens, kv.kv_heads, dim, dt, where)
    rot = max_pos = 0
    _fits((cos is None) == (sin is None), where)
    if cos is not None:
        _contiguous(where, torch.float32, cos, sin)
        _fits(cos.dim() == 2 and cos.shape == sin.shape, where)
        max_pos, rot = cos.shape[0], 2 * cos.shape[1]
    return Append(kv, q_len, heads, rot, int(interleaved), max_pos, 0, _ptr(q), _ptr(k), _ptr(v),
                  _ptr(q_out), qs, ks, vs, qos, _ptr(cos), _ptr(sin))


def kv_append(op, stream=None):
    """Rotates a step's q and k and writes k and v into their cache slots."""
    _call("dg_kv_append", ctypes.byref(op), _stream(stream))


def attention(kv, q, out, lse=None, q_len=1, scale=None, window=0, sinks=0):
    """Describes attn_decode: q and out [batch * q_len][heads][head_dim], lse
    fp32 [batch * q_len][heads] or None; scale defaults to head_dim ** -0.5."""
    import torch
    where, dt = "attention", _kv_dtype(kv)
    _fits(q_len > 0, where)
    tokens, dim = kv.batch * q_len, kv.head_dim
    heads = q.numel() // (tokens * dim)
    qs = _head_rows(q, tokens, heads, dim, dt, where)
    os_ = _head_rows(out, tokens, heads, dim, dt, where)
    _contiguous(where, torch.float32, lse)
    _fits(lse is None or lse.numel() == tokens * heads, where)
    return Attention(kv, q_len, heads, window, sinks, dim ** -0.5 if scale is None else scale, 0,
                     _ptr(q), _ptr(out), _ptr(lse), qs, os_)


def attn_workspace_bytes(op):
    return int(load().dg_attn_workspace_bytes(ctypes.byref(op)))


def attn_decode(op, ws, stream=None):
    """Attention of a step's new tokens over the paged cache."""
    _call("dg_attn_decode", ctypes.byref(op), _ptr(ws), _nbytes(ws), _stream(stream))


def norm(h, h_out, x_out, w_pre=None, b_pre=None, y=None, w_post=None, b_post=None, gate=None,
         alpha=1.0, beta=1.0, eps=1e-6, w_offset=0.0, kind=NORM_RMS):
    """Describes norm_residual: h' = alpha h + beta gate norm_post(y) into h_out,
    norm_pre(h') into x_out.  h and h_out in the type of the others or fp32;
    gate has y's shape, or one row."""
    import torch
    where = "norm"
    first = h if h is not None else y
    _fits(first is not None, where)
    shape = first.shape
    N = shape[-1]
    rows = first.numel() // N if N else 0
    small = next((t for t in (y, x_out, w_pre, h, h_out) if t is not None and
                  t.dtype != torch.float32), None)
    _fits(small is not None, where)
    dt, ftype = small.dtype, _ftype(small, where)
    res = [t for t in (h, h_out) if t is not None]
    h_f32 = int(bool(res) and res[0].dtype == torch.float32)
    _contiguous(where, torch.float32 if h_f32 else dt, h, h_out)
    _contiguous(where, dt, y, x_out, w_pre, b_pre, w_post, b_post, gate)
    for t in (h, h_out, y, x_out):
        _fits(t is None or t.numel() == rows * N, where)
    for t in (w_pre, b_pre, w_post, b_post):
        _fits(t is None or t.numel() == N, where)
    _fits(gate is None or (gate.numel() in (N, rows * N) and
                           (gate.dim() == 1 or gate.shape[-1] == N)), where)
    gate_rows = 0 if gate is None else gate.numel() // N
    return Norm(ftype, kind, rows, N, h_f32, gate_rows, alpha, beta, eps, w_offset, _ptr(y),
                _ptr(w_post), _ptr(b_post), _ptr(gate), _ptr(h), _ptr(w_pre), _ptr(b_pre),
                _ptr(h_out), _ptr(x_out))


def norm_residual(op, stream=None):
    """The norms around a block with its gate and residual scale."""
    _call("dg_norm_residual", ctypes.byref(op), _stream(stream))


def moe(kind, x, y, router, W_gate, W_up, W_down, top_k, gate_scale=None, up_scale=None,
        down_scale=None, residual=None, ids=None, weights=None, group_size=32,
        score=MOE_SOFTMAX, renormalize=False, route_scale=1.0):
    """Describes moe_forward: x, y, residual [M][K]; router [E][K]; W_gate, W_up
    [E][I][K], W_down [E][K][I] (int4: packed, with scales [E][rows][cols / group]);
    ids int32 and weights fp32 [M][top_k] receive the routing."""
    import torch
    where = "moe"
    w4 = kind == LINEAR_W4A16
    dt = torch.bfloat16 if kind == LINEAR_BF16 else torch.float16
    K = x.shape[-1]
    M = x.numel() // K if K else 0
    _fits(router.dim() == 2 and W_gate.dim() == 3 and W_down.dim() == 3, where)
    E, inter = router.shape[0], W_gate.shape[1]
    _contiguous(where, dt, x, y, router, residual, gate_scale, up_scale, down_scale)
    _contiguous(where, torch.uint8 if w4 else dt, W_gate, W_up, W_down)
    _contiguous(where, torch.int32, ids)
    _contiguous(where, torch.float32, weights)
    cut = 2 if w4 else 1
    _fits(router.shape[1] == K and tuple(W_gate.shape) == (E, inter, K // cut) and
          W_up.shape == W_gate.shape and tuple(W_down.shape) == (E, K, inter // cut), where)
    for t in (y, residual):
        _fits(t is None or t.numel() == M * K, where)
    for t in (ids, weights):
        _fits(t is None or t.numel() == M * top_k, where)
    if w4:
        _fits(group_size > 0, where)
        for t, rows, cols in ((gate_scale, inter, K), (up_scale, inter, K), (down_scale, K, inter)):
            _fits(t is not None and t.numel() == E * rows * (cols // group_size), where)
    return Moe(kind, M, K, inter, E, top_k, group_size if w4 else 0, score, int(renormalize),
               route_scale, _ptr(x), _ptr(router), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
               _ptr(gate_scale), _ptr(up_scale), _ptr(down_scale), _ptr(residual), _ptr(y),
               _ptr(ids), _ptr(weights))


def moe_workspace_bytes(op):
    return int(load().dg_moe_workspace_bytes(ctypes.byref(op)))


def moe_forward(op, ws, stream=None):
    """A mixture-of-experts layer for a few tokens."""
    _call("dg_moe_forward", ctypes.byref(op), _ptr(ws), _nbytes(ws), _stream(stream))


# ---- a serving step -----------------------------------------------------------------

def _i32(where, *numbers):
    """Whole numbers that a 32-bit field would cut off without a word."""
    _fits(all(-2 ** 31 <= n < 2 ** 31 for n in numbers), where)


def _paging(block_table, seq_lens, where):
    """batch, max_pages and table stride of a block table int32 [batch][max_pages]."""
    import torch
    _fits(block_table.dim() == 2 and block_table.dtype == torch.int32 and
          (block_table.shape[1] <= 1 or block_table.stride(1) == 1), where)
    batch, pages = block_table.shape
    _fits(seq_lens.dtype == torch.int32 and seq_lens.is_contiguous() and
          0 < seq_lens.numel() == batch, where)
    stride = block_table.stride(0) if batch > 1 else pages
    _fits(stride >= pages, where)
    return batch, pages, stride


def paged_kv4(k_codes, v_codes, k_scales, v_scales, block_table, seq_lens, dtype=None, k_factor=1.0,
              v_factor=1.0):
    """A paged cache held in 4 bits: codes uint8 [pages][page_size][kv_heads][head_dim / 2],
    scales uint8 or float8_e4m3fn [pages][page_size][kv_heads][head_dim / 16] (any
    strides with the last dimension contiguous, keys and values alike: a [pages][kv_heads]
    [page_size][..] cache, the faster order, is passed transposed); block_table and seq_lens
    as for paged_kv; dtype: of the q, k, v and out beside it (float16 by default)."""
    import torch
    where = "paged_kv4"
    dtype = torch.float16 if dtype is None else dtype
    _fits(dtype in (torch.float16, torch.bfloat16), where)
    _fits(k_codes.dim() == 4 and k_codes.shape == v_codes.shape and k_codes.stride() == v_codes.stride() and
          k_codes.stride(3) == 1 and k_codes.dtype == v_codes.dtype == torch.uint8, where)
    _fits(k_scales.dim() == 4 and k_scales.shape == v_scales.shape and
          k_scales.stride() == v_scales.stride() and (k_scales.shape[3] <= 1 or k_scales.stride(3) == 1) and
          k_scales.dtype in (torch.uint8, torch.float8_e4m3fn) and v_scales.dtype == k_scales.dtype, where)
    pages, page_size, heads, half = k_codes.shape
    _fits(half % 8 == 0 and tuple(k_scales.shape) == (pages, page_size, heads, half // 8), where)
    batch, max_pages, table_stride = _paging(block_table, seq_lens, where)
    return PagedKV4(F16 if dtype == torch.float16 else BF16, batch, heads, 2 * half, page_size, pages, max_pages, 0,
                    _ptr(k_codes), _ptr(v_codes), _ptr(k_scales), _ptr(v_scales), *k_codes.stride()[:3],
                    *k_scales.stride()[:3], k_factor, v_factor, _ptr(block_table), table_stride, _ptr(seq_lens))


def head_append(kv, q, k, v, q_out=None, q_len=None, cos=None, sin=None, interleaved=False, w_q=None, w_k=None,
                eps=1e-6, w_offset=0.0, kind=NORM_RMS, slots=None, positions=None):
    """Describes qkv_append into kv, a paged_kv or a paged_kv4: q [tokens][heads][head_dim]
    (or None), k and v with kv_heads heads; w_q and w_k [head_dim], or None for no norm;
    cos, sin, interleaved and q_out as for append.  Tokens are the last q_len (1 by
    default) of each sequence, or those of slots (int64) and positions (int32)."""
    import torch
    where, dt, dim = "head_append", _kv_dtype(kv), kv.head_dim
    by_map = slots is not None
    _fits(by_map == (positions is not None) and not (by_map and q_len is not None), where)
    if by_map:
        _contiguous(where, torch.int64, slots)
        _contiguous(where, torch.int32, positions)
        tokens, q_len = slots.numel(), 0
        _fits(0 < tokens < 2 ** 31 and positions.numel() == tokens, where)
    else:
        q_len = 1 if q_len is None else q_len
        _fits(q_len > 0, where)
        tokens = kv.batch * q_len
    heads = 0 if q is None else q.numel() // (tokens * dim)
    q_out = q if q_out is None else q_out
    qs = qos = 0
    if q is not None:
        qs = _head_rows(q, tokens, heads, dim, dt, where)
        qos = _head_rows(q_out, tokens, heads, dim, dt, where)
    ks = _head_rows(k, tokens, kv.kv_heads, dim, dt, where)
    vs = _head_rows(v, tokens, kv.kv_heads, dim, dt, where)
    rot = max_pos = 0
    _fits((cos is None) == (sin is None), where)
    if cos is not None:
        _contiguous(where, torch.float32, cos, sin)
        _fits(cos.dim() == 2 and cos.shape == sin.shape, where)
        max_pos, rot = cos.shape[0], 2 * cos.shape[1]
    _contiguous(where, dt, w_q, w_k)
    for w in (w_q, w_k):
        _fits(w is None or w.numel() == dim, where)
    four = isinstance(kv, PagedKV4)
    return HeadAppend(PagedKV() if four else kv, kv if four else PagedKV4(), 4 if four else 16, q_len,
                      tokens if by_map else 0, heads, rot, int(interleaved), max_pos, kind, eps, w_offset, _ptr(q),
                      _ptr(k), _ptr(v), _ptr(q_out), qs, ks, vs, qos, _ptr(cos), _ptr(sin), _ptr(w_q), _ptr(w_k),
                      _ptr(slots), _ptr(positions))


def qkv_append(op, stream=None):
    """Head norms, rotary positions and the append, to a 16-bit or a 4-bit cache."""
    _call("dg_qkv_append", ctypes.byref(op), _stream(stream))


def kv4_rows(kv, k=None, v=None, q_len=None, slots=None):
    """Describes kv4_read: k and v [tokens][kv_heads][head_dim] of the cache's dtype (or
    None) receive the last q_len positions of each sequence (1 by default), or what
    lies in slots (int64)."""
    import torch
    where, dt = "kv4_rows", _kv_dtype(kv)
    _fits(not (slots is not None and q_len is not None) and not (k is None and v is None), where)
    _contiguous(where, torch.int64, slots)
    if slots is None:
        q_len = 1 if q_len is None else q_len
    tokens = slots.numel() if slots is not None else kv.batch * q_len
    _fits(0 < tokens < 2 ** 31, where)
    ks, vs = (0 if t is None else _head_rows(t, tokens, kv.kv_heads, kv.head_dim, dt, where) for t in (k, v))
    for t, stride in ((k, ks), (v, vs)):
        _fits(t is None or stride >= kv.kv_heads * kv.head_dim, where)   # rows that overlap
    return KV4Rows(kv, 0 if slots is not None else q_len, tokens, _ptr(k), _ptr(v), ks, vs, _ptr(slots))


def kv4_read(op, stream=None):
    """A 4-bit cache's keys and values back in 16 bits."""
    _call("dg_kv4_read", ctypes.byref(op), _stream(stream))


def attention4(kv, q, out, lse=None, q_len=1, scale=None, window=0, sinks=0):
    """Describes attn4_decode over a paged_kv4; the rest as for attention."""
    import torch
    where, dt = "attention4", _kv_dtype(kv)
    _i32(where, window, sinks)
    _fits(q_len > 0, where)
    tokens, dim = kv.batch * q_len, kv.head_dim
    heads = q.numel() // (tokens * dim)
    qs = _head_rows(q, tokens, heads, dim, dt, where)
    os_ = _head_rows(out, tokens, heads, dim, dt, where)
    _contiguous(where, torch.float32, lse)
    _fits(lse is None or lse.numel() == tokens * heads, where)
    return Attention4(kv, q_len, heads, window, sinks, dim ** -0.5 if scale is None else scale, 0,
                      _ptr(q), _ptr(out), _ptr(lse), qs, os_)


def attn4_workspace_bytes(op):
    return int(load().dg_attn4_workspace_bytes(ctypes.byref(op)))


def attn4_decode(op, ws, stream=None):
    """Attention of a step's new tokens over the paged 4-bit cache."""
    _call("dg_attn4_decode", ctypes.byref(op), _ptr(ws), _nbytes(ws), _stream(stream))


def page_plan(lens, block_table, pool, pool_state, page_size, new_lens=None, new_len=1, lens_out=None,
              pool_state_out=None, starts=None, slots=None, positions=None):
    """Describes assign_pages: lens and new_lens int32 [batch] (new_len for every sequence
    without), block_table int32 [batch][max_pages], pool int32 [..] with pool_state
    int32 (first, count); lens and pool_state are updated in place unless given an
    output; starts int32 [batch + 1], slots int64 and positions int32 [tokens] or None."""
    import torch
    where = "page_plan"
    _i32(where, page_size, new_len)
    batch, max_pages, stride = _paging(block_table, lens, where)
    lens_out = lens if lens_out is None else lens_out
    pool_state_out = pool_state if pool_state_out is None else pool_state_out
    _contiguous(where, torch.int32, new_lens, lens_out, pool, pool_state, pool_state_out, starts, positions)
    _contiguous(where, torch.int64, slots)
    for t, n in ((new_lens, batch), (lens_out, batch), (pool_state, 2), (pool_state_out, 2), (starts, batch + 1)):
        _fits(t is None or t.numel() == n, where)
    tokens = 0 if slots is None else slots.numel()
    _fits(max(tokens, pool.numel(), max_pages) < 2 ** 31, where)
    _fits(positions is None or positions.numel() == tokens, where)
    return PagePlan(batch, page_size, max_pages, pool.numel(), new_len, tokens, stride, _ptr(lens), _ptr(new_lens),
                    _ptr(lens_out), _ptr(block_table), _ptr(pool), _ptr(pool_state), _ptr(pool_state_out),
                    _ptr(starts), _ptr(slots), _ptr(positions))


def pages_workspace_bytes(op):
    return int(load().dg_pages_workspace_bytes(ctypes.byref(op)))


def assign_pages(op, ws=None, stream=None):
    """Pages for a step's tokens, and the slots where they go."""
    _call("dg_assign_pages", ctypes.byref(op), _ptr(ws), _nbytes(ws), _stream(stream))


def logprobs(logits, tokens=None, logprob=None, rank=None, entropy=None, lse=None, top_ids=None,
             top_logprobs=None, scale=1.0):
    """Describes token_logprobs: logits [rows][V] (or [V]) fp16, bf16 or fp32, rows any
    stride apart; tokens int32 [rows]; outputs, each optional: logprob, entropy, lse
    fp32 [rows], rank int32 [rows], top_ids int32 and top_logprobs fp32 [rows][top_k]."""
    import torch
    where = "logprobs"
    f32 = logits.dtype == torch.float32
    kind = F16 if f32 else _ftype(logits, where)
    _fits(logits.dim() in (1, 2) and logits.numel() > 0 and (logits.shape[-1] == 1 or logits.stride(-1) == 1), where)
    rows, V = (1, logits.shape[0]) if logits.dim() == 1 else logits.shape
    _fits(max(rows, V) < 2 ** 31, where)
    stride = logits.stride(0) if rows > 1 else V
    _contiguous(where, torch.int32, tokens, rank, top_ids)
    _contiguous(where, torch.float32, logprob, entropy, lse, top_logprobs)
    for t in (tokens, rank, logprob, entropy, lse):
        _fits(t is None or t.numel() == rows, where)
    top = top_ids if top_ids is not None else top_logprobs
    top_k = 0 if top is None else top.numel() // rows
    for t in (top_ids, top_logprobs):
        _fits(t is None or t.numel() == rows * top_k, where)
    return Logprobs(kind, int(f32), rows, V, top_k, scale, stride, _ptr(logits), _ptr(tokens), _ptr(logprob),
                    _ptr(rank), _ptr(entropy), _ptr(lse), _ptr(top_ids), _ptr(top_logprobs))


def logprobs_workspace_bytes(op):
    return int(load().dg_logprobs_workspace_bytes(ctypes.byref(op)))


def token_logprobs(op, ws=None, stream=None):
    """Log probabilities of given tokens, entropy and the best alternatives."""
    _call("dg_token_logprobs", ctypes.byref(op), _ptr(ws), _nbytes(ws), _stream(stream))


def check_device_status(stream=None):
    _call("dg_check_device_status", _stream(stream))


def selftest_wait_timeout(spin_limit, stream=None):
    """Launches the bounded-wait self test (see include/dg.h)."""
    _call("dg_selftest_wait_timeout", spin_limit, _stream(stream))


def status_string(s):
    return load().dg_status_string(s).decode()


def probe_copy(src, dst, stream=None):
    _call("dg_probe_copy", _ptr(src), _ptr(dst), _nbytes(src), _stream(stream))


def probe_read(src, sink, stream=None):
    _call("dg_probe_read", _ptr(src), _nbytes(src), _ptr(sink), _stream(stream))


def version():
    return load().dg_version().decode()
