// C entry points of the decoder-layer operators around the weight stream:
// host-side checks, then the launch.
#include <algorithm>
#include <cmath>

#include "dg_internal.cuh"

namespace dg {

static bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

static bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + bn && y < x + an;
}

static dg_status status_of(cudaError_t e) { return e == cudaSuccess ? DG_OK : DG_ERR_CUDA; }

static constexpr int kMaxBatch = 1 << 20, kMaxHeads = 1024, kMaxQLen = 16;

static dg_status check_kv(const dg_paged_kv& kv, int q_len, int heads) {
    if (kv.type != DG_F16 && kv.type != DG_BF16) return DG_ERR_INVALID_ARG;
    if (kv.batch < 1 || kv.kv_heads < 1 || kv.head_dim < 1 || kv.page_size < 1 || kv.num_pages < 1 ||
        kv.max_pages < 1 || q_len < 1 || kv.reserved)
        return DG_ERR_INVALID_ARG;
    if (!kv.k || !kv.v || !kv.block_table || !kv.seq_lens) return DG_ERR_INVALID_ARG;
    if (kv.page_stride < 0 || kv.token_stride < 0 || kv.head_stride < 0) return DG_ERR_INVALID_ARG;
    if (kv.table_stride < (kv.batch > 1 ? kv.max_pages : 0)) return DG_ERR_INVALID_ARG;
    if (kv.batch > kMaxBatch || kv.kv_heads > kMaxHeads || heads > kMaxHeads || q_len > kMaxQLen)
        return DG_ERR_UNSUPPORTED;
    if (kv.head_dim % 8 || kv.head_dim > 256) return DG_ERR_UNSUPPORTED;
    if (!aligned(kv.block_table, 4) || !aligned(kv.seq_lens, 4)) return DG_ERR_MISALIGNED;
    return DG_OK;
}

static dg_status check_append(const dg_append& op) {
    const dg_status st = check_kv(op.kv, op.q_len, op.heads);
    if (st != DG_OK) return st;
    if (op.reserved || op.heads < 0 || (op.heads > 0) != (op.q != nullptr) ||
        (op.heads > 0) != (op.q_out != nullptr) || !op.k || !op.v)
        return DG_ERR_INVALID_ARG;
    if (op.interleaved != 0 && op.interleaved != 1) return DG_ERR_INVALID_ARG;
    if (op.rot_dim < 0 || op.rot_dim % 2 || op.rot_dim > op.kv.head_dim) return DG_ERR_INVALID_ARG;
    if (op.rot_dim && (!op.cos || !op.sin || op.max_pos < 1)) return DG_ERR_INVALID_ARG;
    if (op.q_stride < 0 || op.k_stride < 0 || op.v_stride < 0) return DG_ERR_INVALID_ARG;
    if (op.heads && op.q_out_stride < (int64_t)op.heads * op.kv.head_dim) return DG_ERR_INVALID_ARG;
    if (op.heads && op.q_out == op.q && op.q_out_stride != op.q_stride) return DG_ERR_INVALID_ARG;
    const void* p2[] = {op.q, op.k, op.v, op.q_out, op.kv.k, op.kv.v};
    for (const void* p : p2)
        if (!aligned(p, 2)) return DG_ERR_MISALIGNED;
    if (op.rot_dim && (!aligned(op.cos, 4) || !aligned(op.sin, 4))) return DG_ERR_MISALIGNED;
    return DG_OK;
}

static dg_status check_attn(const dg_attn& op) {
    const dg_status st = check_kv(op.kv, op.q_len, op.heads);
    if (st != DG_OK) return st;
    if (op.reserved || op.heads < 1 || !op.q || !op.out) return DG_ERR_INVALID_ARG;
    // scores are held in units of log2(e)
    if (op.heads % op.kv.kv_heads || op.window < 0 || op.sinks < 0 || !std::isfinite(op.scale * 1.4426950408889634f))
        return DG_ERR_INVALID_ARG;
    if ((int64_t)op.kv.batch * op.q_len * op.heads > 0x7fffffff) return DG_ERR_UNSUPPORTED;
    const int64_t row = (int64_t)op.heads * op.kv.head_dim;
    if (op.q_stride < 0 || op.out_stride < row) return DG_ERR_INVALID_ARG;
    if (!aligned(op.q, 16) || !aligned(op.out, 16) || !aligned(op.kv.k, 16) || !aligned(op.kv.v, 16))
        return DG_ERR_MISALIGNED;
    if (op.q_stride % 8 || op.out_stride % 8 || op.kv.page_stride % 8 || op.kv.token_stride % 8 ||
        op.kv.head_stride % 8)
        return DG_ERR_MISALIGNED;
    if (op.lse && !aligned(op.lse, 4)) return DG_ERR_MISALIGNED;
    return DG_OK;
}

static dg_status check_norm(const dg_norm& op) {
    if (op.type != DG_F16 && op.type != DG_BF16) return DG_ERR_INVALID_ARG;
    if (op.kind != DG_NORM_RMS && op.kind != DG_NORM_LAYER) return DG_ERR_INVALID_ARG;
    if (op.rows < 1 || op.N < 1 || (op.h_f32 != 0 && op.h_f32 != 1)) return DG_ERR_INVALID_ARG;
    if (!op.y && (!op.h || op.w_post || op.gate)) return DG_ERR_INVALID_ARG;
    if ((op.b_post && !op.w_post) || (op.b_pre && !op.w_pre)) return DG_ERR_INVALID_ARG;
    if ((!op.h_out && !op.x_out) || (op.x_out && !op.w_pre)) return DG_ERR_INVALID_ARG;
    if (op.gate ? (op.gate_rows != 1 && op.gate_rows != op.rows) : op.gate_rows != 0)
        return DG_ERR_INVALID_ARG;
    if (!(op.eps >= 0.f) || !std::isfinite(op.eps) || !std::isfinite(op.alpha) ||
        !std::isfinite(op.beta) || !std::isfinite(op.w_offset))
        return DG_ERR_INVALID_ARG;
    if (op.N > 32768) return DG_ERR_UNSUPPORTED;
    const unsigned ha = op.h_f32 ? 4 : 2;
    if (!aligned(op.h, ha) || !aligned(op.h_out, ha)) return DG_ERR_MISALIGNED;
    const void* p2[] = {op.y, op.w_post, op.b_post, op.gate, op.w_pre, op.b_pre, op.x_out};
    for (const void* p : p2)
        if (!aligned(p, 2)) return DG_ERR_MISALIGNED;
    // an output may be an input of its own type, element by element; nothing else
    const size_t n = (size_t)op.rows * op.N, row = (size_t)op.N * 2, hb = n * (op.h_f32 ? 4 : 2);
    struct In {
        const void* p;
        size_t bytes;
        bool same_as_h, same_as_x;  // whole [rows][N] array of h_out's / x_out's type
    };
    const In in[] = {{op.y, n * 2, !op.h_f32, true},
                     {op.h, hb, true, !op.h_f32},
                     {op.gate, op.gate_rows == 1 ? row : n * 2,
                      op.gate_rows == op.rows && !op.h_f32, op.gate_rows == op.rows},
                     {op.w_post, row, false, false},
                     {op.b_post, row, false, false},
                     {op.w_pre, row, false, false},
                     {op.b_pre, row, false, false}};
    for (const In& i : in) {
        if (overlap(i.p, i.bytes, op.h_out, hb) && !(i.p == op.h_out && i.same_as_h))
            return DG_ERR_INVALID_ARG;
        if (overlap(i.p, i.bytes, op.x_out, n * 2) && !(i.p == op.x_out && i.same_as_x))
            return DG_ERR_INVALID_ARG;
    }
    if (overlap(op.h_out, hb, op.x_out, n * 2)) return DG_ERR_INVALID_ARG;
    return DG_OK;
}

static dg_status check_moe(const dg_moe& op) {
    const bool w4 = op.kind == DG_LINEAR_W4A16;
    if (op.kind < DG_LINEAR_F16 || op.kind > DG_LINEAR_W4A8) return DG_ERR_INVALID_ARG;
    if (op.kind != DG_LINEAR_F16 && op.kind != DG_LINEAR_BF16 && !w4) return DG_ERR_UNSUPPORTED;
    if (op.M < 1 || op.K < 1 || op.I < 1 || op.E < 1 || op.top_k < 1) return DG_ERR_INVALID_ARG;
    if (op.top_k > op.E) return DG_ERR_INVALID_ARG;
    if (op.score != DG_MOE_SOFTMAX && op.score != DG_MOE_SIGMOID) return DG_ERR_INVALID_ARG;
    if ((op.renormalize != 0 && op.renormalize != 1) || !std::isfinite(op.route_scale))
        return DG_ERR_INVALID_ARG;
    if (!op.x || !op.router || !op.W_gate || !op.W_up || !op.W_down || !op.y) return DG_ERR_INVALID_ARG;
    if (w4 && (!op.gate_scale || !op.up_scale || !op.down_scale)) return DG_ERR_INVALID_ARG;
    if (op.M > 16 || op.E > 1024 || op.top_k > 16 || op.K > 65536 || op.I > 65536)
        return DG_ERR_UNSUPPORTED;
    if (w4) {
        if (op.group_size < 32 || op.group_size % 32 || op.K % op.group_size || op.I % op.group_size)
            return DG_ERR_UNSUPPORTED;
        if (!aligned(op.gate_scale, 2) || !aligned(op.up_scale, 2) || !aligned(op.down_scale, 2))
            return DG_ERR_MISALIGNED;
    } else if (op.K % 8 || op.I % 8) {
        return DG_ERR_MISALIGNED;
    }
    const void* p16[] = {op.x, op.router, op.W_gate, op.W_up, op.W_down, op.y};
    for (const void* p : p16)
        if (!aligned(p, 16)) return DG_ERR_MISALIGNED;
    if (!aligned(op.residual, 2) || !aligned(op.ids, 4) || !aligned(op.weights, 4))
        return DG_ERR_MISALIGNED;
    return DG_OK;
}

// ---- a serving step ---------------------------------------------------------------------

// (table and lengths belong to a cache also where an op has slots)
static dg_status check_kv4(const dg_paged_kv4& kv, int heads) {
    if (kv.type != DG_F16 && kv.type != DG_BF16) return DG_ERR_INVALID_ARG;
    if (kv.batch < 1 || kv.kv_heads < 1 || kv.head_dim < 1 || kv.page_size < 1 || kv.num_pages < 1 ||
        kv.max_pages < 1 || kv.reserved)
        return DG_ERR_INVALID_ARG;
    if (!kv.k || !kv.v || !kv.k_scale || !kv.v_scale || !kv.block_table || !kv.seq_lens) return DG_ERR_INVALID_ARG;
    if (kv.page_stride < 0 || kv.token_stride < 0 || kv.head_stride < 0 || kv.scale_page_stride < 0 ||
        kv.scale_token_stride < 0 || kv.scale_head_stride < 0)
        return DG_ERR_INVALID_ARG;
    if (!(kv.k_factor > 0.f) || !(kv.v_factor > 0.f) || !std::isfinite(7.f * kv.k_factor) ||
        !std::isfinite(16.f * kv.v_factor))
        return DG_ERR_INVALID_ARG;
    if (kv.table_stride < (kv.batch > 1 ? kv.max_pages : 0)) return DG_ERR_INVALID_ARG;
    if (kv.batch > kMaxBatch || kv.kv_heads > kMaxHeads || heads > kMaxHeads) return DG_ERR_UNSUPPORTED;
    if (kv.head_dim % 16 || kv.head_dim > 256) return DG_ERR_UNSUPPORTED;
    // (the kernels multiply by strides of 32 bits)
    const int64_t strides[] = {kv.page_stride,       kv.token_stride,       kv.head_stride,
                               kv.scale_page_stride, kv.scale_token_stride, kv.scale_head_stride};
    for (const int64_t x : strides)
        if (x > 0xffffffffll) return DG_ERR_UNSUPPORTED;
    if (!aligned(kv.block_table, 4) || !aligned(kv.seq_lens, 4) || !aligned(kv.k, 8) || !aligned(kv.v, 8) ||
        kv.page_stride % 8 || kv.token_stride % 8 || kv.head_stride % 8)
        return DG_ERR_MISALIGNED;
    return DG_OK;
}

static dg_status check_head_append(const dg_head_append& op) {
    if (op.bits != 16 && op.bits != 4) return DG_ERR_INVALID_ARG;
    if (op.slots ? op.tokens < 1 || op.q_len || !op.positions : op.tokens || op.q_len < 1 || op.positions)
        return DG_ERR_INVALID_ARG;
    if (op.q_len > kMaxQLen) return DG_ERR_UNSUPPORTED;
    const dg_status st = op.bits == 4 ? check_kv4(op.kv4, op.heads) : check_kv(op.kv, 1, op.heads);
    if (st != DG_OK) return st;
    const int D = op.bits == 4 ? op.kv4.head_dim : op.kv.head_dim, kvh = op.bits == 4 ? op.kv4.kv_heads : op.kv.kv_heads;
    const int batch = op.bits == 4 ? op.kv4.batch : op.kv.batch;
    if (op.heads < 0 || (op.heads > 0) != (op.q != nullptr) || (op.heads > 0) != (op.q_out != nullptr) || !op.k || !op.v)
        return DG_ERR_INVALID_ARG;
    if ((op.w_q && !op.q) || (op.norm != DG_NORM_RMS && op.norm != DG_NORM_LAYER) || !(op.eps >= 0.f) ||
        !std::isfinite(op.eps) || !std::isfinite(op.w_offset))
        return DG_ERR_INVALID_ARG;
    if (op.interleaved != 0 && op.interleaved != 1) return DG_ERR_INVALID_ARG;
    if (op.rot_dim < 0 || op.rot_dim % 2 || op.rot_dim > D) return DG_ERR_INVALID_ARG;
    if (op.rot_dim && (!op.cos || !op.sin || op.max_pos < 1)) return DG_ERR_INVALID_ARG;
    if (op.q_stride < 0 || op.k_stride < 0 || op.v_stride < 0) return DG_ERR_INVALID_ARG;
    if (op.heads && op.q_out_stride < (int64_t)op.heads * D) return DG_ERR_INVALID_ARG;
    if (op.heads && op.q_out == op.q && op.q_out_stride != op.q_stride) return DG_ERR_INVALID_ARG;
    // a warp takes a head at least
    const int64_t tokens = op.slots ? op.tokens : (int64_t)batch * op.q_len;
    if (tokens * (op.heads + 2 * kvh) > 0x7fffffff) return DG_ERR_UNSUPPORTED;
    const void* p2[] = {op.q, op.k, op.v, op.q_out, op.w_q, op.w_k, op.bits == 16 ? op.kv.k : nullptr,
                        op.bits == 16 ? op.kv.v : nullptr};
    for (const void* p : p2)
        if (!aligned(p, 2)) return DG_ERR_MISALIGNED;
    if (op.rot_dim && (!aligned(op.cos, 4) || !aligned(op.sin, 4))) return DG_ERR_MISALIGNED;
    if (!aligned(op.slots, 8) || !aligned(op.positions, 4)) return DG_ERR_MISALIGNED;
    return DG_OK;
}

static dg_status check_kv4_rows(const dg_kv4_rows& op) {
    const dg_status st = check_kv4(op.kv, 0);
    if (st != DG_OK) return st;
    if (op.tokens < 1 || (!op.k && !op.v)) return DG_ERR_INVALID_ARG;
    if (op.slots ? op.q_len != 0 : op.q_len < 1 || op.tokens != (int64_t)op.kv.batch * op.q_len)
        return DG_ERR_INVALID_ARG;
    const int64_t row = (int64_t)op.kv.kv_heads * op.kv.head_dim;
    if ((op.k && op.k_stride < row) || (op.v && op.v_stride < row)) return DG_ERR_INVALID_ARG;
    if (!aligned(op.k, 2) || !aligned(op.v, 2) || !aligned(op.slots, 8)) return DG_ERR_MISALIGNED;
    return DG_OK;
}

static dg_status check_attn4(const dg_attn4& op) {
    const dg_status st = check_kv4(op.kv, op.heads);
    if (st != DG_OK) return st;
    if (op.reserved || op.q_len < 1 || op.heads < 1 || !op.q || !op.out) return DG_ERR_INVALID_ARG;
    if (op.q_len > kMaxQLen) return DG_ERR_UNSUPPORTED;
    if (op.heads % op.kv.kv_heads || op.window < 0 || op.sinks < 0 ||
        !std::isfinite(op.scale * 1.4426950408889634f * 16.f) ||
        !std::isfinite(op.scale * 1.4426950408889634f * 16.f * op.kv.k_factor))
        return DG_ERR_INVALID_ARG;
    if ((int64_t)op.kv.batch * op.q_len * op.heads > 0x7fffffff) return DG_ERR_UNSUPPORTED;
    if (op.q_stride < 0 || op.out_stride < (int64_t)op.heads * op.kv.head_dim) return DG_ERR_INVALID_ARG;
    if (!aligned(op.q, 16) || !aligned(op.out, 16) || op.q_stride % 8 || op.out_stride % 8 ||
        (op.lse && !aligned(op.lse, 4)))
        return DG_ERR_MISALIGNED;
    return DG_OK;
}

static dg_status check_plan(const dg_page_plan& op) {
    if (op.batch < 1 || op.page_size < 1 || op.max_pages < 1 || op.pool_size < 1 || op.max_tokens < 0)
        return DG_ERR_INVALID_ARG;
    if (!op.lens || !op.lens_out || !op.block_table || !op.pool || !op.pool_state || !op.pool_state_out)
        return DG_ERR_INVALID_ARG;
    if ((op.slots != nullptr) != (op.max_tokens > 0) || (op.positions && !op.slots)) return DG_ERR_INVALID_ARG;
    if (op.table_stride < (op.batch > 1 ? op.max_pages : 0)) return DG_ERR_INVALID_ARG;
    if (op.batch > kMaxBatch) return DG_ERR_UNSUPPORTED;
    const void* p4[] = {op.lens, op.new_lens, op.lens_out, op.block_table, op.pool, op.pool_state, op.pool_state_out,
                        op.starts, op.positions};
    for (const void* p : p4)
        if (!aligned(p, 4)) return DG_ERR_MISALIGNED;
    if (!aligned(op.slots, 8)) return DG_ERR_MISALIGNED;
    // what is written apart from what is read and from each other; lens_out may be lens
    // and pool_state_out pool_state
    const size_t B = (size_t)op.batch * 4,
                 table = ((size_t)(op.batch - 1) * op.table_stride + op.max_pages) * 4;
    struct Area {
        const void* p;
        size_t bytes;
    };
    const Area out[] = {{op.lens_out, B}, {op.pool_state_out, 8}, {op.block_table, table},
                        {op.pool, (size_t)op.pool_size * 4}, {op.starts, B + 4},
                        {op.slots, (size_t)op.max_tokens * 8}, {op.positions, (size_t)op.max_tokens * 4}};
    const Area in[] = {{op.lens, B}, {op.pool_state, 8}, {op.new_lens, B}};
    for (const Area& o : out) {
        for (const Area& i : in)
            if (overlap(o.p, o.bytes, i.p, i.bytes) && !(o.p == i.p && &o - out == &i - in && &i - in < 2))
                return DG_ERR_INVALID_ARG;
        for (const Area& x : out)
            if (&x != &o && overlap(o.p, o.bytes, x.p, x.bytes)) return DG_ERR_INVALID_ARG;
    }
    return DG_OK;
}

static dg_status check_logprobs(const dg_logprobs& op) {
    if (op.type != DG_F16 && op.type != DG_BF16) return DG_ERR_INVALID_ARG;
    if ((op.logits_f32 != 0 && op.logits_f32 != 1) || op.rows < 1 || op.V < 1 || op.top_k < 0 || op.top_k > op.V)
        return DG_ERR_INVALID_ARG;
    if (!op.logits || op.stride < (op.rows > 1 ? op.V : 0) || !(op.scale > 0.f) ||
        !std::isfinite(op.scale * 1.4426950408889634f))
        return DG_ERR_INVALID_ARG;
    if ((!op.tokens && (op.logprob || op.rank)) || (op.top_k > 0) != (op.top_ids || op.top_logprobs))
        return DG_ERR_INVALID_ARG;
    if (!op.logprob && !op.rank && !op.entropy && !op.lse && !op.top_k) return DG_ERR_INVALID_ARG;
    if (op.top_k > 32 || op.rows > (1 << 22) || op.V > (1 << 30)) return DG_ERR_UNSUPPORTED;
    if (!aligned(op.logits, op.logits_f32 ? 4 : 2)) return DG_ERR_MISALIGNED;
    const void* p4[] = {op.tokens, op.logprob, op.rank, op.entropy, op.lse, op.top_ids, op.top_logprobs};
    for (const void* p : p4)
        if (!aligned(p, 4)) return DG_ERR_MISALIGNED;
    return DG_OK;
}

static dg_status check_ws(const void* ws, size_t have, size_t need) {
    if (!ws || have < need) return DG_ERR_WORKSPACE;
    return aligned(ws, 16) ? DG_OK : DG_ERR_MISALIGNED;
}

}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_kv_append(const dg_append* op, dg_stream stream) {
    if (!op) return DG_ERR_INVALID_ARG;
    const dg_status st = check_append(*op);
    return st != DG_OK ? st : status_of(launch_kv_append(*op, stream));
}

size_t dg_attn_workspace_bytes(const dg_attn* op) {
    return op && check_attn(*op) == DG_OK ? attn_ws_bytes(*op) : 0;
}

dg_status dg_attn_decode(const dg_attn* op, void* ws, size_t ws_bytes, dg_stream stream) {
    if (!op) return DG_ERR_INVALID_ARG;
    dg_status st = check_attn(*op);
    if (st != DG_OK) return st;
    if ((st = check_ws(ws, ws_bytes, attn_ws_bytes(*op))) != DG_OK) return st;
    return status_of(launch_attn(*op, ws, stream));
}

dg_status dg_norm_residual(const dg_norm* op, dg_stream stream) {
    if (!op) return DG_ERR_INVALID_ARG;
    const dg_status st = check_norm(*op);
    return st != DG_OK ? st : status_of(launch_norm(*op, stream));
}

size_t dg_moe_workspace_bytes(const dg_moe* op) {
    return op && check_moe(*op) == DG_OK ? moe_ws_bytes(*op) : 0;
}

dg_status dg_moe_forward(const dg_moe* op, void* ws, size_t ws_bytes, dg_stream stream) {
    if (!op) return DG_ERR_INVALID_ARG;
    dg_status st = check_moe(*op);
    if (st != DG_OK) return st;
    if ((st = check_ws(ws, ws_bytes, moe_ws_bytes(*op))) != DG_OK) return st;
    return status_of(launch_moe(*op, ws, stream));
}

dg_status dg_qkv_append(const dg_head_append* op, dg_stream stream) {
    if (!op) return DG_ERR_INVALID_ARG;
    const dg_status st = check_head_append(*op);
    return st != DG_OK ? st : status_of(launch_head_append(*op, stream));
}

dg_status dg_kv4_read(const dg_kv4_rows* op, dg_stream stream) {
    if (!op) return DG_ERR_INVALID_ARG;
    const dg_status st = check_kv4_rows(*op);
    return st != DG_OK ? st : status_of(launch_kv4_read(*op, stream));
}

size_t dg_attn4_workspace_bytes(const dg_attn4* op) {
    return op && check_attn4(*op) == DG_OK ? attn4_ws_bytes(*op) : 0;
}

dg_status dg_attn4_decode(const dg_attn4* op, void* ws, size_t ws_bytes, dg_stream stream) {
    if (!op) return DG_ERR_INVALID_ARG;
    dg_status st = check_attn4(*op);
    if (st != DG_OK) return st;
    if ((st = check_ws(ws, ws_bytes, attn4_ws_bytes(*op))) != DG_OK) return st;
    return status_of(launch_attn4(*op, ws, stream));
}

size_t dg_pages_workspace_bytes(const dg_page_plan* op) {
    return op && check_plan(*op) == DG_OK ? plan_ws_bytes(*op) : 0;
}

dg_status dg_assign_pages(const dg_page_plan* op, void* ws, size_t ws_bytes, dg_stream stream) {
    if (!op) return DG_ERR_INVALID_ARG;
    dg_status st = check_plan(*op);
    if (st != DG_OK) return st;
    const size_t need = plan_ws_bytes(*op);
    if (need && (st = check_ws(ws, ws_bytes, need)) != DG_OK) return st;
    return status_of(launch_plan(*op, ws, stream));
}

size_t dg_logprobs_workspace_bytes(const dg_logprobs* op) {
    return op && check_logprobs(*op) == DG_OK ? lp_ws_bytes(*op) : 0;
}

dg_status dg_token_logprobs(const dg_logprobs* op, void* ws, size_t ws_bytes, dg_stream stream) {
    if (!op) return DG_ERR_INVALID_ARG;
    dg_status st = check_logprobs(*op);
    if (st != DG_OK) return st;
    const size_t need = lp_ws_bytes(*op);
    if (need && (st = check_ws(ws, ws_bytes, need)) != DG_OK) return st;
    return status_of(launch_logprobs(*op, ws, stream));
}

}  // extern "C"
