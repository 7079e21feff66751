// Norms of queries and keys for each head, rotary positions, and the append to a 16-bit
// or 4-bit paged cache; and the 4-bit cache read back.
//
// A head's values of one token are a team's: 8, 16 or 32 lanes of 8 values each, so
// that a norm is one exchange between lanes, a rotated pair's other half another, and
// the 16 values of a scale group two neighbouring lanes.  q, k and v go through
// once, in registers, whatever the cache holds.  A 4-bit value is divided by its scale
// with one rounding, not multiplied by a reciprocal: 16-bit inputs meet halves of a scale
// often enough for ties to show (they go to the even code).
#include "elem.cuh"

namespace dg {

constexpr int kHeadThreads = 128;

struct HeadParams {
    dg_head_append op;
    int batch, kvh, D, page_size, num_pages;   // of the cache meant
    int tokens, chunks;                        // CTAs of a token
    float k_div, v_div;                        // 7 x factor
    FastDiv by_chunks, by_q_len, by_page;
};

__device__ __forceinline__ uint32_t e4m3_of(float v) {   // to nearest even, at most 448
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
    return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_f32(uint32_t byte) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)byte));
    return __half2float(__ushort_as_half((uint16_t)h));
}

// Where a token's keys and values go: page -1: nowhere.
struct Place {
    int page, at;
};
__device__ __forceinline__ Place place_of(const int64_t* slots, const int32_t* table, int64_t table_stride,
                                          int max_pages, int num_pages, int page_size, FastDiv by_page, int t, int b,
                                          int p) {
    Place w = {-1, 0};
    if (slots) {
        const long long s = slots[t];
        if (s >= 0 && s < (long long)num_pages * page_size) {
            w.page = s >> 31 ? (int)(s / page_size) : (int)s / by_page;
            w.at = (int)(s - (long long)w.page * page_size);
        }
    } else {
        const int i = p / by_page;
        if (i < max_pages) {
            const int page = table[b * table_stride + i];   // the kernel before may have written it
            if (page >= 0 && page < num_pages) w = {page, p - i * page_size};
        }
    }
    return w;
}

// VEC: 16-byte rows and a rotation of whole vectors; else values one by one and pairs
// through shared memory.
template <bool BF16, bool Q4, int TEAM, bool VEC>
__global__ void __launch_bounds__(kHeadThreads) k_head_append(const HeadParams p) {
    constexpr int kTeams = kHeadThreads / TEAM;
    __shared__ float shared[VEC ? 1 : kTeams][VEC ? 1 : TEAM * 8];
    griddep_launch_dependents();
    griddep_wait();
    const dg_head_append& op = p.op;
    const int t = (int)blockIdx.x / p.by_chunks, chunk = blockIdx.x - t * p.chunks;
    const int team = threadIdx.x / TEAM, i = threadIdx.x % TEAM, task = chunk * kTeams + team;
    const int D = p.D, d0 = i * 8, heads = op.heads;
    const int kind = task < heads ? 0 : task < heads + p.kvh ? 1 : 2;   // q, k, v
    const int h = kind == 0 ? task : kind == 1 ? task - heads : task - heads - p.kvh;
    const bool mine = task < heads + 2 * p.kvh && d0 < D;
    const uint16_t* src = kind == 0   ? static_cast<const uint16_t*>(op.q) + t * op.q_stride
                          : kind == 1 ? static_cast<const uint16_t*>(op.k) + t * op.k_stride
                                      : static_cast<const uint16_t*>(op.v) + t * op.v_stride;
    src += (long long)h * D + d0;
    const uint16_t* w = static_cast<const uint16_t*>(kind == 0 ? op.w_q : kind == 1 ? op.w_k : nullptr);
    const int left = min(8, D - d0);
    float x[8], g[8];
    auto load8 = [&](const uint16_t* at, float (&f)[8]) {
        if (VEC) {
            unpack8<BF16>(*reinterpret_cast<const uint4*>(at), f);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = e < left ? elem_f32<BF16>(at[e]) : 0.f;
        }
    };
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = g[e] = 0.f;
    if (mine) {
        load8(src, x);
        if (w) load8(w + d0, g);
    }
    // ---- the token's position and place ---------------------------------------------------
    int pos, b = 0;
    if (op.slots) {
        pos = op.positions[t];
    } else {
        b = t / p.by_q_len;
        const int32_t* lens = Q4 ? op.kv4.seq_lens : op.kv.seq_lens;
        pos = max(0, lens[b]) - op.q_len + (t - b * op.q_len);   // a length below zero is none
    }
    const bool live = pos >= 0 && (op.rot_dim == 0 || pos < op.max_pos);
    Place at = {-1, 0};
    if (live && kind != 0)
        at = place_of(op.slots, Q4 ? op.kv4.block_table : op.kv.block_table,
                      Q4 ? op.kv4.table_stride : op.kv.table_stride, Q4 ? op.kv4.max_pages : op.kv.max_pages,
                      p.num_pages, p.page_size, p.by_page, t, b, pos);

    // ---- norm over the head -----------------------------------------------------------------
    auto team_sum = [&](float v) {
#pragma unroll
        for (int o = TEAM / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    const float inv_d = 1.f / (float)D;
    if (op.w_q || op.w_k) {   // (the lanes of a warp take part together)
        float mean = 0.f;
        if (op.norm == DG_NORM_LAYER) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += x[e];
            mean = team_sum(s) * inv_d;
        }
        float u[8], sq = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            u[e] = mine && e < left ? x[e] - mean : 0.f;
            sq = fmaf(u[e], u[e], sq);
        }
        const float k = 1.f / sqrtf(team_sum(sq) * inv_d + op.eps);
        if (w) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = u[e] * k * (op.w_offset + g[e]);
        }
    }
    // ---- rotation ---------------------------------------------------------------------------
    const int half = op.rot_dim / 2;
    if (half) {
        const float* cos = op.cos + (long long)(live ? pos : 0) * half;
        const float* sin = op.sin + (long long)(live ? pos : 0) * half;
        const bool turn = kind != 2 && live;
        if (VEC) {
            const int lanes = half / 8;   // of one half of the pairs
            const int other = op.interleaved ? i : i < lanes ? i + lanes : i - lanes;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)   // lanes past the rotated dims read from anywhere in the team
                y[e] = __shfl_sync(0xffffffffu, x[e], other & (TEAM - 1), TEAM);
            if (turn && mine && d0 < op.rot_dim) {
                float c[8], s[8];
                if (op.interleaved) {
                    const int j = d0 / 2;   // four pairs
                    *reinterpret_cast<float4*>(c) = __ldg(reinterpret_cast<const float4*>(cos + j));
                    *reinterpret_cast<float4*>(s) = __ldg(reinterpret_cast<const float4*>(sin + j));
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float a = x[e], z = x[e + 1];
                        x[e] = a * c[e / 2] - z * s[e / 2];
                        x[e + 1] = z * c[e / 2] + a * s[e / 2];
                    }
                } else {
                    const bool low = d0 < half;
                    const int j = low ? d0 : d0 - half;
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        *reinterpret_cast<float4*>(c + e) = __ldg(reinterpret_cast<const float4*>(cos + j + e));
                        *reinterpret_cast<float4*>(s + e) = __ldg(reinterpret_cast<const float4*>(sin + j + e));
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float sn = low ? -s[e] : s[e];
                        x[e] = x[e] * c[e] + y[e] * sn;
                    }
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) shared[team][d0 + e] = x[e];
            __syncwarp();
            if (turn && mine) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int d = d0 + e;
                    if (d >= op.rot_dim) continue;
                    const bool low = op.interleaved ? !(d & 1) : d < half;
                    const int j = op.interleaved ? d / 2 : low ? d : d - half;
                    const int o = op.interleaved ? d ^ 1 : low ? d + half : d - half;
                    const float c = __ldg(cos + j), s = __ldg(sin + j);
                    x[e] = x[e] * c + shared[team][o] * (low ? -s : s);
                }
            }
        }
    }
    auto store8 = [&](uint16_t* to) {
        if (VEC) {
            *reinterpret_cast<uint4*>(to) = pack8<BF16>(x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) to[e] = elem_16<BF16>(x[e]);
        }
    };
    if (kind == 0) {
        if (!mine) return;
        if (!live)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.f;
        store8(static_cast<uint16_t*>(op.q_out) + t * op.q_out_stride + (long long)h * D + d0);
        return;
    }
    if (!Q4) {
        if (mine && at.page >= 0)
            store8(static_cast<uint16_t*>(kind == 1 ? op.kv.k : op.kv.v) + at.page * op.kv.page_stride +
                   at.at * op.kv.token_stride + h * op.kv.head_stride + d0);
        return;
    }
    // ---- sixteen values and their scale, by two lanes ------------------------------------------
    float top = 0.f;
    bool odd = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        top = fmaxf(top, fabsf(x[e]));
        odd = odd || !(fabsf(x[e]) <= 3.402823466e38f);
    }
    const unsigned pair = 3u << (threadIdx.x & 30);   // (teams part ways above: q's return)
    top = fmaxf(top, __shfl_xor_sync(pair, top, 1));
    odd = __shfl_xor_sync(pair, (int)odd, 1) | (int)odd;
    if (!mine || at.page < 0) return;
    const float factor = kind == 1 ? op.kv4.k_factor : op.kv4.v_factor;
    const uint32_t byte = odd ? 0x7Fu : e4m3_of(__fdiv_rn(top, kind == 1 ? p.k_div : p.v_div));
    const float step = odd ? 0.f : e4m3_f32(byte) * factor;
    uint32_t codes = 0;
    if (step > 0.f) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            codes |= (uint32_t)(max(-7, min(7, __float2int_rn(__fdiv_rn(x[e], step)))) & 15) << (4 * e);
    }
    uint8_t* c = (kind == 1 ? op.kv4.k : op.kv4.v) + at.page * op.kv4.page_stride + at.at * op.kv4.token_stride +
                 h * op.kv4.head_stride + d0 / 2;
    *reinterpret_cast<uint32_t*>(c) = codes;
    if ((i & 1) == 0)
        (kind == 1 ? op.kv4.k_scale : op.kv4.v_scale)[at.page * op.kv4.scale_page_stride +
                                                       at.at * op.kv4.scale_token_stride +
                                                       h * op.kv4.scale_head_stride + i / 2] = (uint8_t)byte;
}

template <bool BF16, bool Q4, int TEAM>
static const void* head_kernel(bool vec) {
    return vec ? (const void*)k_head_append<BF16, Q4, TEAM, true> : (const void*)k_head_append<BF16, Q4, TEAM, false>;
}
template <bool BF16, bool Q4>
static const void* head_kernel(int team, bool vec) {
    return team == 8 ? head_kernel<BF16, Q4, 8>(vec) : team == 16 ? head_kernel<BF16, Q4, 16>(vec)
                                                                  : head_kernel<BF16, Q4, 32>(vec);
}

static bool vec_row(const void* p, int64_t stride) { return ((uintptr_t)p & 15u) == 0 && stride % 8 == 0; }

cudaError_t launch_head_append(const dg_head_append& op, cudaStream_t s) {
    const bool q4 = op.bits == 4;
    HeadParams p;
    p.op = op;
    p.batch = q4 ? op.kv4.batch : op.kv.batch;
    p.kvh = q4 ? op.kv4.kv_heads : op.kv.kv_heads;
    p.D = q4 ? op.kv4.head_dim : op.kv.head_dim;
    p.page_size = q4 ? op.kv4.page_size : op.kv.page_size;
    p.num_pages = q4 ? op.kv4.num_pages : op.kv.num_pages;
    p.tokens = op.slots ? op.tokens : p.batch * op.q_len;
    p.k_div = (float)(7.0 * op.kv4.k_factor);
    p.v_div = (float)(7.0 * op.kv4.v_factor);
    const bool bf = (q4 ? op.kv4.type : op.kv.type) == DG_BF16;
    const bool vec = op.rot_dim % (op.interleaved ? 8 : 16) == 0 && p.D % 8 == 0 && vec_row(op.k, op.k_stride) &&
                     vec_row(op.v, op.v_stride) && vec_row(op.w_q, 0) && vec_row(op.w_k, 0) &&
                     (!op.heads || (vec_row(op.q, op.q_stride) && vec_row(op.q_out, op.q_out_stride))) &&
                     (!op.rot_dim || (vec_row(op.cos, 0) && vec_row(op.sin, 0))) &&
                     (q4 || (vec_row(op.kv.k, op.kv.page_stride) && vec_row(op.kv.v, op.kv.token_stride) &&
                             op.kv.head_stride % 8 == 0));
    const int team = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32, teams = kHeadThreads / team;
    p.chunks = (op.heads + 2 * p.kvh + teams - 1) / teams;
    p.by_chunks = fast_div((uint32_t)p.chunks);
    p.by_q_len = fast_div((uint32_t)(op.slots ? 1 : op.q_len));
    p.by_page = fast_div((uint32_t)p.page_size);
    const void* fn = bf ? (q4 ? head_kernel<true, true>(team, vec) : head_kernel<true, false>(team, vec))
                        : (q4 ? head_kernel<false, true>(team, vec) : head_kernel<false, false>(team, vec));
    void* args[] = {&p};
    return launch_pdl(fn, dim3((unsigned)(p.tokens * p.chunks)), dim3(kHeadThreads), 0, s, args);
}

// ---- the 4-bit cache read back -------------------------------------------------------------
struct ReadParams {
    dg_kv4_rows op;
    int pieces;          // of 8 dims in a head
    long long units;     // tokens x heads x pieces, of k and of v each
    FastDiv by_q_len, by_page;
};

template <bool BF16>
__global__ void __launch_bounds__(256) k_kv4_read(const ReadParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const dg_kv4_rows& op = p.op;
    const dg_paged_kv4& kv = op.kv;
    const long long stride = (long long)gridDim.x * blockDim.x, per = (long long)kv.kv_heads * p.pieces;
    for (long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x; u < p.units; u += stride) {
        const int t = (int)(u / per), r = (int)(u - t * per), h = r / p.pieces, c = r - h * p.pieces;
        int pos = 0, b = 0;
        if (!op.slots) {
            b = t / p.by_q_len;
            pos = max(0, kv.seq_lens[b]) - op.q_len + (t - b * op.q_len);
        }
        Place at = {-1, 0};
        if (pos >= 0)
            at = place_of(op.slots, kv.block_table, kv.table_stride, kv.max_pages, kv.num_pages, kv.page_size,
                          p.by_page, t, b, pos);
        const long long code = at.page * kv.page_stride + at.at * kv.token_stride + h * kv.head_stride + c * 4;
        const long long scale =
            at.page * kv.scale_page_stride + at.at * kv.scale_token_stride + h * kv.scale_head_stride + c / 2;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            uint16_t* to = static_cast<uint16_t*>(which ? op.v : op.k);
            if (!to) continue;
            to += t * (which ? op.v_stride : op.k_stride) + (long long)h * kv.head_dim + c * 8;
            float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (at.page >= 0) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>((which ? kv.v : kv.k) + code);
                const float s = e4m3_f32((which ? kv.v_scale : kv.k_scale)[scale]) * (which ? kv.v_factor : kv.k_factor);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = (float)((int)(w << (28 - 4 * e)) >> 28) * s;
            }
            if (((uintptr_t)to & 15) == 0) {
                *reinterpret_cast<uint4*>(to) = pack8<BF16>(f);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) to[e] = elem_16<BF16>(f[e]);
            }
        }
    }
}

cudaError_t launch_kv4_read(const dg_kv4_rows& op, cudaStream_t s) {
    ReadParams p;
    p.op = op;
    p.pieces = op.kv.head_dim / 8;
    p.units = (long long)op.tokens * op.kv.kv_heads * p.pieces;
    p.by_q_len = fast_div((uint32_t)(op.slots ? 1 : op.q_len));
    p.by_page = fast_div((uint32_t)op.kv.page_size);
    const long long want = (p.units + 255) / 256, most = sm_count() * 16ll;
    void* args[] = {&p};
    return launch_pdl(op.kv.type == DG_BF16 ? (const void*)k_kv4_read<true> : (const void*)k_kv4_read<false>,
                      dim3((unsigned)(want < most ? want : most)), dim3(256), 0, s, args);
}

}  // namespace dg
