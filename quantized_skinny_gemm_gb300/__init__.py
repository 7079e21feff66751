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
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.dg_workspace_bytes.argtypes = [P, I]
    lib.dg_workspace_bytes.restype = Z
    for name in ("dg_attn_workspace_bytes", "dg_moe_workspace_bytes"):
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
