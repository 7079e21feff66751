// Rotary positions on a step's q and k, with k and v written into their pages.
#include "elem.cuh"

namespace dg {

// One token per CTA.  Its values are cut into pieces of U = 8 or 1: first those
// that are copied, four at a time, from the last thread down, then the pairs of
// pieces of q and k that rotate, from the first thread up (so that hardly a
// warp does both).  A thread reads all of a pair before it writes any, so q_out
// may be q.
//
// Bound by latency: one token is a few KB behind two dependent reads, length ->
// page id (2.8 us back to back); of many tokens each small CTA waits for length ->
// page id -> copy in turn, with half of an SM's warps resident (8 tokens of 256
// sequences, 32 + 2 x 8 heads of 128: 11.3 us, 4.5 TB/s of traffic that L2 mostly
// holds, DRAM 26 %; one piece at a time 14.1).
constexpr int kAppendThreads = 128;
template <int U>
struct PieceOf {
    using type = uint16_t;
};
template <>
struct PieceOf<8> {
    using type = uint4;
};
struct AppendParams {
    dg_append op;
    FastDiv q_len, page_size, pairs, plain, whole;
};
template <bool BF16, int U>
__global__ void __launch_bounds__(kAppendThreads) k_kv_append(const AppendParams prm) {
    griddep_launch_dependents();
    griddep_wait();
    const dg_append& op = prm.op;
    const int t = blockIdx.x, b = t / prm.q_len;
    const int D = op.kv.head_dim, half = op.rot_dim / 2, kvh = op.kv.kv_heads;
    // a length below zero is none: no position may wrap around
    const int p = max(0, op.kv.seq_lens[b]) - op.q_len + (t - b * op.q_len);
    const bool live = p >= 0 && (op.rot_dim == 0 || p < op.max_pos);
    int at = 0;
    const int page = live ? page_slot(op.kv, prm.page_size, b, p, at) : -1;
    const long long slot = page < 0 ? 0 : page * op.kv.page_stride + at * op.kv.token_stride;
    const uint16_t* q = static_cast<const uint16_t*>(op.q) + t * op.q_stride;
    const uint16_t* k = static_cast<const uint16_t*>(op.k) + t * op.k_stride;
    const uint16_t* v = static_cast<const uint16_t*>(op.v) + t * op.v_stride;
    uint16_t* qo = static_cast<uint16_t*>(op.q_out) + t * op.q_out_stride;
    uint16_t* ko = static_cast<uint16_t*>(op.kv.k) + slot;
    uint16_t* vo = static_cast<uint16_t*>(op.kv.v) + slot;
    const int turned = op.heads + kvh, pairs = half / U, plain = (D - op.rot_dim) / U, whole = D / U;
    const int n_pair = turned * pairs, n_copy = turned * plain + kvh * whole;
    using Piece = typename PieceOf<U>::type;
    for (int i0 = blockDim.x - 1 - threadIdx.x; i0 < n_copy; i0 += 4 * blockDim.x) {
        Piece x[4];
        uint16_t* dst[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            int j = i0 + w * blockDim.x;
            dst[w] = nullptr;
            if (j >= n_copy) continue;
            const uint16_t* src;
            bool is_q = false;
            if (j < turned * plain) {
                const int h = j / prm.plain, d = op.rot_dim + (j - h * plain) * U;
                is_q = h < op.heads;
                src = is_q ? q + h * D + d : k + (h - op.heads) * D + d;
                dst[w] = is_q ? qo + h * D + d : ko + (h - op.heads) * op.kv.head_stride + d;
            } else {
                j -= turned * plain;
                const int h = j / prm.whole, d = (j - h * whole) * U;
                src = v + h * D + d;
                dst[w] = vo + h * op.kv.head_stride + d;
            }
            if (!is_q && page < 0) dst[w] = nullptr;   // nowhere to put it
            if (live)
                x[w] = *reinterpret_cast<const Piece*>(src);
            else
                memset(&x[w], 0, sizeof(Piece));
        }
#pragma unroll
        for (int w = 0; w < 4; ++w)
            if (dst[w]) *reinterpret_cast<Piece*>(dst[w]) = x[w];
    }
    for (int i = threadIdx.x; i < n_pair; i += blockDim.x) {
        const int h = i / prm.pairs, u = i - h * pairs;
        const bool is_q = h < op.heads;
        if (!is_q && page < 0) continue;   // nowhere to put it
        const uint16_t* src = is_q ? q + h * D : k + (h - op.heads) * D;
        uint16_t* dst = is_q ? qo + h * D : ko + (h - op.heads) * op.kv.head_stride;
        const int d0 = op.interleaved ? 2 * u * U : u * U, d1 = d0 + (op.interleaved ? U : half);
        const float* cp = op.cos + (long long)p * half + u * U;
        const float* sp = op.sin + (long long)p * half + u * U;
        if constexpr (U == 8) {
            uint4 a = make_uint4(0, 0, 0, 0), c = a;
            if (live) {
                a = *reinterpret_cast<const uint4*>(src + d0);
                c = *reinterpret_cast<const uint4*>(src + d1);
                float x[8], y[8], cs[8], sn[8];
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    *reinterpret_cast<float4*>(cs + j) = __ldg(reinterpret_cast<const float4*>(cp + j));
                    *reinterpret_cast<float4*>(sn + j) = __ldg(reinterpret_cast<const float4*>(sp + j));
                }
                if (op.interleaved) {   // pairs (x, y) lie side by side
                    const uint32_t w[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
                    uint32_t o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 f = pair_f32<BF16>(w[j]);
                        o[j] = pair_16<BF16>(f.x * cs[j] - f.y * sn[j], f.y * cs[j] + f.x * sn[j]);
                    }
                    a = make_uint4(o[0], o[1], o[2], o[3]);
                    c = make_uint4(o[4], o[5], o[6], o[7]);
                } else {
                    unpack8<BF16>(a, x);
                    unpack8<BF16>(c, y);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float x0 = x[j];
                        x[j] = x0 * cs[j] - y[j] * sn[j];
                        y[j] = y[j] * cs[j] + x0 * sn[j];
                    }
                    a = pack8<BF16>(x);
                    c = pack8<BF16>(y);
                }
            }
            *reinterpret_cast<uint4*>(dst + d0) = a;
            *reinterpret_cast<uint4*>(dst + d1) = c;
        } else {
            uint16_t a = 0, c = 0;
            if (live) {
                const float x = elem_f32<BF16>(src[d0]), y = elem_f32<BF16>(src[d1]);
                const float cs = __ldg(cp), sn = __ldg(sp);
                a = elem_16<BF16>(x * cs - y * sn);
                c = elem_16<BF16>(y * cs + x * sn);
            }
            dst[d0] = a;
            dst[d1] = c;
        }
    }
}

static bool vec_ok(const void* p, int64_t stride) {
    return ((uintptr_t)p & 15u) == 0 && stride % 8 == 0;
}

cudaError_t launch_kv_append(const dg_append& op, cudaStream_t s) {
    const dg_paged_kv& kv = op.kv;
    const bool vec = op.rot_dim % 16 == 0 && kv.head_dim % 8 == 0 && vec_ok(op.k, op.k_stride) &&
                     vec_ok(op.v, op.v_stride) && vec_ok(kv.k, kv.page_stride) &&
                     vec_ok(kv.v, kv.token_stride) && kv.head_stride % 8 == 0 &&
                     (!op.heads || (vec_ok(op.q, op.q_stride) && vec_ok(op.q_out, op.q_out_stride))) &&
                     (!op.rot_dim || (vec_ok(op.cos, 0) && vec_ok(op.sin, 0)));
    const int U = vec ? 8 : 1;
    const int turned = op.heads + kv.kv_heads;
    const int units = turned * (op.rot_dim / 2 / U) + turned * ((kv.head_dim - op.rot_dim) / U) +
                      kv.kv_heads * (kv.head_dim / U);
    const dim3 grid(kv.batch * op.q_len);
    const int threads = units < kAppendThreads ? (units + 31) / 32 * 32 : kAppendThreads;
    AppendParams p{op,
                   fast_div(op.q_len),
                   fast_div(kv.page_size),
                   fast_div(op.rot_dim / 2 / U),
                   fast_div((kv.head_dim - op.rot_dim) / U),
                   fast_div(kv.head_dim / U)};
    const bool bf = kv.type == DG_BF16;
    const void* fn = vec ? (bf ? (const void*)k_kv_append<true, 8> : (const void*)k_kv_append<false, 8>)
                         : (bf ? (const void*)k_kv_append<true, 1> : (const void*)k_kv_append<false, 1>);
    void* args[] = {&p};
    return launch_pdl(fn, grid, dim3(threads), 0, s, args);
}

}  // namespace dg
