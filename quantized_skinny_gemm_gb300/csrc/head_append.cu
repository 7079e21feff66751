// Norms of queries and keys for each head, rotary positions, and the append to a 16-bit
// or 4-bit paged cache; and the 4-bit cache read back.
//
// A head's values of one token are a team's: 8, 16 or 32 lanes of 8 values each, so
// that a norm is one exchange between lanes, a rotated pair's other half another, and
// the 16 values of a scale group two neighbouring lanes.  A warp takes one or four rounds of heads of one
// token, all of q, of k or of v: their position and place, the norm's weights, the cosines and sines
// and the addresses are worked out once for all of them, and all heads are loaded before the
// first is used.  (A head a team and a launch-wide list of heads: 450 instructions a warp,
// bound by issue, 80 us for 6700 tokens of 32 + 2 x 8 heads of 128.)  A 4-bit value
// is divided by its scale with one rounding, not just multiplied by a reciprocal: 16-bit inputs meet halves of
// a scale often enough for ties to show (they go to the even code).
#include "elem.cuh"

namespace dg {

constexpr int kHeadThreads = 128, kHeadWarps = kHeadThreads / 32;

struct HeadParams {
    dg_head_append op;
    int batch, kvh, D, page_size, num_pages;   // of the cache meant
    int q_warps, k_warps, units;               // warps of a token for q, and for k (and v); of all tokens
    float k_div, v_div;                        // 7 x factor
    FastDiv by_warps, by_q_len, by_page;
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

// The larger of two, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// VEC: 16-byte rows and a rotation of whole vectors; else values one by one and pairs
// through shared memory.
template <bool BF16, bool Q4, int TEAM, bool VEC, int kRounds>
__global__ void __launch_bounds__(kHeadThreads, kRounds == 1 ? 8 : 6) k_head_append(const HeadParams p) {
    constexpr int kTeams = 32 / TEAM;   // of a warp
    __shared__ float shared[VEC ? 1 : kHeadThreads / TEAM][VEC ? 1 : TEAM * 8];
    griddep_launch_dependents();
    griddep_wait();
    const dg_head_append& op = p.op;
    const int unit = blockIdx.x * kHeadWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (unit >= p.units) return;
    const int warps = p.q_warps + 2 * p.k_warps, t = unit / p.by_warps, part = unit - t * warps;
    const int kind = part < p.q_warps ? 0 : part < p.q_warps + p.k_warps ? 1 : 2;   // q, k, v
    const int heads = kind == 0 ? op.heads : p.kvh;
    const int chunk = kind == 0 ? part : kind == 1 ? part - p.q_warps : part - p.q_warps - p.k_warps;
    const int team = lane / TEAM, i = lane % TEAM, h0 = chunk * kTeams * kRounds + team;
    const int D = p.D, d0 = i * 8;
    const bool mine = d0 < D;   // (head sizes are multiples of 8)
    const uint16_t* src = kind == 0   ? static_cast<const uint16_t*>(op.q) + t * op.q_stride
                          : kind == 1 ? static_cast<const uint16_t*>(op.k) + t * op.k_stride
                                      : static_cast<const uint16_t*>(op.v) + t * op.v_stride;
    src += (long long)h0 * D + d0;
    const uint16_t* w = static_cast<const uint16_t*>(kind == 0 ? op.w_q : kind == 1 ? op.w_k : nullptr);
    auto load8 = [&](const uint16_t* at) {
        if (VEC) return *reinterpret_cast<const uint4*>(at);
        uint32_t r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = at[2 * e] | (uint32_t)at[2 * e + 1] << 16;
        return make_uint4(r[0], r[1], r[2], r[3]);
    };
    auto store8 = [&](uint16_t* to, const float (&x)[8]) {
        const uint4 v = pack8<BF16>(x);
        if (VEC) {
            *reinterpret_cast<uint4*>(to) = v;
        } else {
            const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                to[2 * e] = (uint16_t)r[e];
                to[2 * e + 1] = (uint16_t)(r[e] >> 16);
            }
        }
    };
    uint4 raw[kRounds];
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
        raw[u] = make_uint4(0, 0, 0, 0);
        if (mine && h0 + u * kTeams < heads) raw[u] = load8(src + u * kTeams * D);
    }
    float g[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = 0.f;
    if (w && mine) unpack8<BF16>(load8(w + d0), g);
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
    if (kind != 0 && at.page < 0) return;   // nowhere to put it (the same for the whole warp)
    if (!live) {
        const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < kRounds; ++u)
            if (mine && h0 + u * kTeams < heads)
                store8(static_cast<uint16_t*>(op.q_out) + t * op.q_out_stride + (long long)(h0 + u * kTeams) * D + d0,
                       zero);
        return;
    }
    // ---- cosines and sines of this lane's dims: x c + (the other of the pair) s --------------------
    const int half = op.rot_dim / 2;
    const bool turn = kind != 2 && mine && d0 < op.rot_dim;
    const int lanes = half / 8, other = op.interleaved ? i : i < lanes ? i + lanes : i - lanes;   // VEC
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = 1.f, s[e] = 0.f;
    if (turn) {
        const float* cos = op.cos + (long long)pos * half;
        const float* sin = op.sin + (long long)pos * half;
        if (VEC && !op.interleaved) {
            const bool low = d0 < half;
            const int j = low ? d0 : d0 - half;
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                *reinterpret_cast<float4*>(c + e) = __ldg(reinterpret_cast<const float4*>(cos + j + e));
                const float4 v = __ldg(reinterpret_cast<const float4*>(sin + j + e));
                s[e] = low ? -v.x : v.x, s[e + 1] = low ? -v.y : v.y;
                s[e + 2] = low ? -v.z : v.z, s[e + 3] = low ? -v.w : v.w;
            }
        } else if (VEC) {   // four pairs
            const float4 v = __ldg(reinterpret_cast<const float4*>(cos + d0 / 2));
            const float4 z = __ldg(reinterpret_cast<const float4*>(sin + d0 / 2));
            c[0] = c[1] = v.x, c[2] = c[3] = v.y, c[4] = c[5] = v.z, c[6] = c[7] = v.w;
            s[0] = -z.x, s[1] = z.x, s[2] = -z.y, s[3] = z.y, s[4] = -z.z, s[5] = z.z, s[6] = -z.w, s[7] = z.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = d0 + e;
                if (d >= op.rot_dim) continue;
                const bool low = op.interleaved ? !(d & 1) : d < half;
                const int j = op.interleaved ? d / 2 : low ? d : d - half;
                c[e] = __ldg(cos + j);
                const float v = __ldg(sin + j);
                s[e] = low ? -v : v;
            }
        }
    }
    // x = k (u g) for a normed head, u the (centred) values; then x c + y s with y the other of the
    // pair: k (u (g c) + u' (g' s)), the products in brackets once for all heads
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = w ? g[e] + op.w_offset : 1.f;
    if (VEC) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float z = op.interleaved ? g[e ^ 1] : __shfl_sync(0xffffffffu, g[e], other & (TEAM - 1), TEAM);
            s[e] *= turn ? z : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] *= c[e];
    }
    auto team_sum = [&](float v) {
#pragma unroll
        for (int o = TEAM / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    const float inv_d = 1.f / (float)D;
    // where the first head goes, and the next one
    uint16_t* out = nullptr;
    uint8_t *codes = nullptr, *scales = nullptr;
    long long next = 0, next_scale = 0;
    if (kind == 0) {
        out = static_cast<uint16_t*>(op.q_out) + t * op.q_out_stride + (long long)h0 * D + d0;
        next = (long long)kTeams * D;
    } else if (!Q4) {
        out = static_cast<uint16_t*>(kind == 1 ? op.kv.k : op.kv.v) + at.page * op.kv.page_stride +
              at.at * op.kv.token_stride + h0 * op.kv.head_stride + d0;
        next = kTeams * op.kv.head_stride;
    } else {
        codes = (kind == 1 ? op.kv4.k : op.kv4.v) + at.page * op.kv4.page_stride + at.at * op.kv4.token_stride +
                h0 * op.kv4.head_stride + d0 / 2;
        scales = (kind == 1 ? op.kv4.k_scale : op.kv4.v_scale) + at.page * op.kv4.scale_page_stride +
                 at.at * op.kv4.scale_token_stride + h0 * op.kv4.scale_head_stride + i / 2;
        next = kTeams * op.kv4.head_stride;
        next_scale = kTeams * op.kv4.scale_head_stride;
    }
    const float factor = kind == 1 ? op.kv4.k_factor : op.kv4.v_factor, divisor = kind == 1 ? p.k_div : p.v_div;

#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
        if (chunk * kTeams * kRounds + u * kTeams >= heads) break;   // (no team of the warp has one)
        const bool have = mine && h0 + u * kTeams < heads;
        float x[8];
        unpack8<BF16>(raw[u], x);
        const float2 one = make_float2(1.f, 1.f), zero = make_float2(0.f, 0.f);
        auto two = [&](int e) { return make_float2(x[e], x[e + 1]); };
        auto put = [&](int e, float2 v) {
            x[e] = v.x;
            x[e + 1] = v.y;
        };
        float k = 1.f;
        if (w) {
            if (op.norm == DG_NORM_LAYER) {
                const float2 sum = fma2(fma2(two(0), one, two(2)), one, fma2(two(4), one, two(6)));
                const float mean = team_sum(sum.x + sum.y) * inv_d, off = mine ? -mean : 0.f;
#pragma unroll
                for (int e = 0; e < 8; e += 2) put(e, fma2(two(e), one, make_float2(off, off)));
            }
            float2 sq = zero;
#pragma unroll
            for (int e = 0; e < 8; e += 2) sq = fma2(two(e), two(e), sq);
            k = rsqrtf(team_sum(sq.x + sq.y) * inv_d + op.eps);
        }
        if (VEC) {
            if (kind != 2) {
                float y[8];
                if (half) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)   // lanes past the rotated dims read from anywhere in the team
                        y[e] = op.interleaved ? x[e ^ 1] : __shfl_sync(0xffffffffu, x[e], other & (TEAM - 1), TEAM);
                }
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    float2 v = fma2(two(e), make_float2(g[e], g[e + 1]), zero);
                    if (turn) v = fma2(make_float2(y[e], y[e + 1]), make_float2(s[e], s[e + 1]), v);
                    put(e, fma2(v, make_float2(k, k), zero));
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * k * g[e];
            if (half && kind != 2) {
                float* row = shared[(threadIdx.x >> 5) * kTeams + team];
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) row[d0 + e] = x[e];
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int d = d0 + e, o = op.interleaved ? d ^ 1 : d < half ? d + half : d - half;
                    if (turn && d < op.rot_dim) x[e] = x[e] * c[e] + row[o] * s[e];
                }
            }
        }
        if (!Q4 || kind == 0) {
            if (have) store8(out, x);
            out += next;
            continue;
        }
        // ---- sixteen values and their scale, by two lanes ------------------------------------------
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(x[e]));
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
        const bool odd = !(top <= 3.402823466e38f);
        const uint32_t byte = odd ? 0x7Fu : e4m3_of(__fdiv_rn(top, divisor));
        const float step = odd ? 0.f : e4m3_f32(byte) * factor;
        uint32_t word = 0;
        if (step > 1e-30f && step < 1e30f && top < 7.49f * step) {
            // x / step rounded once: a quotient by the reciprocal and its remainder.  Added to 1.5 2^23 it
            // leaves the nearest whole number, ties to even, in the last bits; the sum of these times
            // 16^e with 8 added to each, and the eights taken off again, is the codes.
            const float inv = __frcp_rn(step);
            const float2 r = make_float2(inv, inv), minus = make_float2(-step, -step);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 y = fma2(two(e), r, zero);
                const float2 z = fma2(fma2(y, minus, two(e)), r, y);
                const float2 n = fma2(z, one, make_float2(12582912.f, 12582912.f));
                word += (__float_as_uint(n.x) + 16u * __float_as_uint(n.y)) << (4 * e);
            }
            constexpr uint32_t kBias = 0x4B400000u;   // 12582912 as a number of 32 bits
            word = (word - kBias * 0x11111111u + 0x88888888u) ^ 0x88888888u;
        } else if (step > 0.f) {
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
                float v = 0.f;
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    if (d == e) v = x[d];
                word |= (uint32_t)(max(-7, min(7, __float2int_rn(__fdiv_rn(v, step)))) & 15) << (4 * e);
            }
        }
        if (have) {
            *reinterpret_cast<uint32_t*>(codes) = word;
            if ((i & 1) == 0) *scales = (uint8_t)byte;
        }
        codes += next;
        scales += next_scale;
    }
}

template <bool BF16, bool Q4, int TEAM>
static const void* head_kernel(bool vec, int rounds) {
    if (!vec) return (const void*)k_head_append<BF16, Q4, TEAM, false, 1>;
    return rounds == 1 ? (const void*)k_head_append<BF16, Q4, TEAM, true, 1>
                       : (const void*)k_head_append<BF16, Q4, TEAM, true, 4>;
}
template <bool BF16, bool Q4>
static const void* head_kernel(int team, bool vec, int rounds) {
    return team == 8    ? head_kernel<BF16, Q4, 8>(vec, rounds)
           : team == 16 ? head_kernel<BF16, Q4, 16>(vec, rounds)
                        : head_kernel<BF16, Q4, 32>(vec, rounds);
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
    p.k_div = (float)(7.0 * op.kv4.k_factor);
    p.v_div = (float)(7.0 * op.kv4.v_factor);
    const bool bf = (q4 ? op.kv4.type : op.kv.type) == DG_BF16;
    const bool vec = op.rot_dim % (op.interleaved ? 8 : 16) == 0 && p.D % 8 == 0 && vec_row(op.k, op.k_stride) &&
                     vec_row(op.v, op.v_stride) && vec_row(op.w_q, 0) && vec_row(op.w_k, 0) &&
                     (!op.heads || (vec_row(op.q, op.q_stride) && vec_row(op.q_out, op.q_out_stride))) &&
                     (!op.rot_dim || (vec_row(op.cos, 0) && vec_row(op.sin, 0))) &&
                     (q4 || (vec_row(op.kv.k, op.kv.page_stride) && vec_row(op.kv.v, op.kv.token_stride) &&
                             op.kv.head_stride % 8 == 0));
    // Few tokens are bound by latency (one of 12 + 2 x 2 heads: 2.2 us with a round a warp, 2.9 with four), many
    // by what a warp does once (6825 tokens of 32 + 2 x 8: 80 and 59).
    const int team = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32, tokens = op.slots ? op.tokens : p.batch * op.q_len;
    const long long teams = (long long)tokens * (op.heads + 2 * p.kvh);
    const int rounds = vec && teams * team / 32 > 32ll * sm_count() ? 4 : 1;
    const int heads = 32 / team * rounds;   // of a warp
    p.q_warps = (op.heads + heads - 1) / heads;
    p.k_warps = (p.kvh + heads - 1) / heads;
    const int warps = p.q_warps + 2 * p.k_warps;
    p.units = tokens * warps;
    p.by_warps = fast_div((uint32_t)warps);
    p.by_q_len = fast_div((uint32_t)(op.slots ? 1 : op.q_len));
    p.by_page = fast_div((uint32_t)p.page_size);
    const void* fn = bf ? (q4 ? head_kernel<true, true>(team, vec, rounds) : head_kernel<true, false>(team, vec, rounds))
                        : (q4 ? head_kernel<false, true>(team, vec, rounds) : head_kernel<false, false>(team, vec, rounds));
    void* args[] = {&p};
    return launch_pdl(fn, dim3((unsigned)((p.units + kHeadWarps - 1) / kHeadWarps)), dim3(kHeadThreads), 0, s, args);
}

// ---- the 4-bit cache read back -------------------------------------------------------------
struct ReadParams {
    dg_kv4_rows op;
    int pieces;          // of 8 dims in a head
    long long units;     // tokens x heads x pieces, of k and of v each
    FastDiv by_q_len, by_page, by_token, by_head;
};

template <bool BF16>
__global__ void __launch_bounds__(256) k_kv4_read(const ReadParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const dg_kv4_rows& op = p.op;
    const dg_paged_kv4& kv = op.kv;
    const long long stride = (long long)gridDim.x * blockDim.x, per = (long long)kv.kv_heads * p.pieces;
    for (long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x; u < p.units; u += stride) {
        const int t = u >> 31 ? (int)(u / per) : (int)u / p.by_token;
        const int r = (int)(u - t * per), h = r / p.by_head, c = r - h * p.pieces;
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
    p.by_token = fast_div((uint32_t)(op.kv.kv_heads * p.pieces));
    p.by_head = fast_div((uint32_t)p.pieces);
    p.by_q_len = fast_div((uint32_t)(op.slots ? 1 : op.q_len));
    p.by_page = fast_div((uint32_t)op.kv.page_size);
    const long long want = (p.units + 255) / 256, most = sm_count() * 16ll;
    void* args[] = {&p};
    return launch_pdl(op.kv.type == DG_BF16 ? (const void*)k_kv4_read<true> : (const void*)k_kv4_read<false>,
                      dim3((unsigned)(want < most ? want : most)), dim3(256), 0, s, args);
}

}  // namespace dg
