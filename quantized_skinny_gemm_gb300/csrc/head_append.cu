// Norms of queries and keys for each head, rotary positions, and the append to a 16-bit
// or 4-bit paged cache; and the 4-bit cache read back.
//
// A head's values of one token are a team's: 8, 16 or 32 lanes of 8 values each, so
// that a norm is one exchange between lanes, a rotated pair's other half another, and
// the 16 values of a scale group two neighbouring lanes.  A warp takes one or four rounds of heads of one
// token, all of q, of k or of v: their position and place, the norm's weights, the cosines and sines
// and the addresses are worked out once for all of them, and all heads are loaded before the
// first is used.  (A head a team and a launch-wide list of heads: 450 instructions a warp,
// bound by issue, 80 us for 6700 tokens of 32 + 2 x 8 heads of 128.)  Where pairs are half a
// rotation apart a lane has four dims of either half, so that it turns them by itself, and lanes
// change to neighbouring dims just before a key becomes codes.  (Eight neighbouring dims, and
// the other of each pair by an exchange: 57 us for 6825 tokens of 32 + 2 x 8 into 4 bits and 47 into 16;
// these 47 and 36.  The 72 and 64 registers are what seven and eight CTAs an SM leave: into 4 bits the kernels of four
// rounds spill 12 to 68 bytes a thread, into 16 bits none, or 36 to 64 where pairs are neighbours or absent; 4 % of the
// instructions at 8 tokens of 256 sequences of 32 + 2 x 8 heads, interleaved, 16 us.)  A 4-bit value
// is divided by its scale with one rounding, not just multiplied by a reciprocal: 16-bit inputs meet halves of
// a scale often enough for ties to show (they go to the even code).
#include "elem.cuh"

namespace dg {

constexpr int kHeadThreads = 128, kHeadWarps = kHeadThreads / 32;

struct HeadParams {
    dg_head_append op;
    int batch, kvh, D, page_size, num_pages;   // of the cache meant
    int q_warps, k_warps, units;               // warps of a token for q, and for k (and v); of all tokens
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
// through shared memory.  SPLIT (VEC, not interleaved): a lane's dims below rot_dim are four of
// either half.
template <bool BF16, bool Q4, int TEAM, bool VEC, int kRounds, bool SPLIT>
__global__ void __launch_bounds__(kHeadThreads, kRounds == 1 || !Q4 ? 8 : 7) k_head_append(const HeadParams p) {
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
    const int D = p.D, half = op.rot_dim / 2;
    // dims d0 .. d0 + 3 and d1 .. d1 + 3
    const bool pair = SPLIT && kind != 2 && i * 8 < op.rot_dim;
    const int d0 = pair ? i * 4 : i * 8, d1 = pair ? half + i * 4 : d0 + 4;
    const bool mine = i * 8 < D;   // (head sizes are multiples of 8)
    const uint16_t* src = kind == 0   ? static_cast<const uint16_t*>(op.q) + t * op.q_stride
                          : kind == 1 ? static_cast<const uint16_t*>(op.k) + t * op.k_stride
                                      : static_cast<const uint16_t*>(op.v) + t * op.v_stride;
    src += (long long)h0 * D;
    const uint16_t* w = static_cast<const uint16_t*>(kind == 0 ? op.w_q : kind == 1 ? op.w_k : nullptr);
    auto load8 = [&](const uint16_t* at) {   // of a head that starts at `at`
        if (SPLIT) {
            const uint2 a = *reinterpret_cast<const uint2*>(at + d0), b = *reinterpret_cast<const uint2*>(at + d1);
            return make_uint4(a.x, a.y, b.x, b.y);
        }
        at += d0;
        if (VEC) return *reinterpret_cast<const uint4*>(at);
        uint32_t r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = at[2 * e] | (uint32_t)at[2 * e + 1] << 16;
        return make_uint4(r[0], r[1], r[2], r[3]);
    };
    auto store8 = [&](uint16_t* to, const float (&x)[8]) {
        const uint4 v = pack8<BF16>(x);
        if (SPLIT) {
            *reinterpret_cast<uint2*>(to + d0) = make_uint2(v.x, v.y);
            *reinterpret_cast<uint2*>(to + d1) = make_uint2(v.z, v.w);
            return;
        }
        to += d0;
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
    if (w && mine) unpack8<BF16>(load8(w), g);
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
                store8(static_cast<uint16_t*>(op.q_out) + t * op.q_out_stride + (long long)(h0 + u * kTeams) * D, zero);
        return;
    }
    // ---- cosines and sines of this lane's dims: x c + (the other of the pair) s --------------------
    const bool turn = kind != 2 && mine && i * 8 < op.rot_dim;
    const int lanes = half / 8, other = op.interleaved ? i : i < lanes ? i + lanes : i - lanes;   // VEC
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = 1.f, s[e] = 0.f;
    if (turn) {
        const float* cos = op.cos + (long long)pos * half;
        const float* sin = op.sin + (long long)pos * half;
        if (SPLIT) {   // pairs (e, e + 4)
            *reinterpret_cast<float4*>(c) = __ldg(reinterpret_cast<const float4*>(cos + d0));
            *reinterpret_cast<float4*>(s) = __ldg(reinterpret_cast<const float4*>(sin + d0));
        } else if (VEC && !op.interleaved) {
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
    if (SPLIT) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float z = s[e], y = turn ? c[e] : 1.f;
            s[e] = -z * g[e + 4];
            s[e + 4] = z * g[e];
            g[e] *= y;
            g[e + 4] *= y;
        }
    } else if (VEC) {
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
    const int d8 = !pair ? i * 8 : i & 1 ? half + (i - 1) * 4 : i * 4;   // the eight dims that this lane makes codes of
    unsigned char* to;   // (of codes: this lane's)
    uint8_t* scales = nullptr;
    long long next, next_scale = 0;   // bytes
    if (kind == 0) {
        to = static_cast<unsigned char*>(op.q_out) + 2 * (t * op.q_out_stride + (long long)h0 * D);
        next = 2ll * kTeams * D;
    } else if (!Q4) {
        to = static_cast<unsigned char*>(kind == 1 ? op.kv.k : op.kv.v) +
             2 * (at.page * op.kv.page_stride + at.at * op.kv.token_stride + h0 * op.kv.head_stride);
        next = 2 * kTeams * op.kv.head_stride;
    } else {
        to = (kind == 1 ? op.kv4.k : op.kv4.v) + at.page * op.kv4.page_stride + at.at * op.kv4.token_stride +
             h0 * op.kv4.head_stride + d8 / 2;
        scales = (kind == 1 ? op.kv4.k_scale : op.kv4.v_scale) + at.page * op.kv4.scale_page_stride +
                 at.at * op.kv4.scale_token_stride + h0 * op.kv4.scale_head_stride + d8 / 16;
        next = kTeams * op.kv4.head_stride;
        next_scale = kTeams * op.kv4.scale_head_stride;
    }
    const float factor = kind == 1 ? op.kv4.k_factor : op.kv4.v_factor;

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
            if (SPLIT && kind != 2) {
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float2 a = two(e), b = two(e + 4), kk = make_float2(k, k);
                    float2 v = fma2(a, make_float2(g[e], g[e + 1]), zero), z = fma2(b, make_float2(g[e + 4], g[e + 5]), zero);
                    if (turn) {
                        v = fma2(b, make_float2(s[e], s[e + 1]), v);
                        z = fma2(a, make_float2(s[e + 4], s[e + 5]), z);
                    }
                    put(e, fma2(v, kk, zero));
                    put(e + 4, fma2(z, kk, zero));
                }
            } else if (kind != 2) {
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
            if (have) store8(reinterpret_cast<uint16_t*>(to), x);
            to += next;
            continue;
        }
        // ---- sixteen values and their scale, by two lanes ------------------------------------------
        if (SPLIT && kind == 1) {   // a lane takes the low halves of two, its neighbour the high ones
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float z = __shfl_xor_sync(0xffffffffu, i & 1 ? x[e] : x[e + 4], 1);
                if (pair && (i & 1)) x[e] = z;
                if (pair && !(i & 1)) x[e + 4] = z;
            }
        }
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(x[e]));
        top = max_nan(top, SPLIT ? __shfl_sync(0xffffffffu, top, lane ^ (pair ? 2 : 1)) : __shfl_xor_sync(0xffffffffu, top, 1));
        const bool odd = !(top <= 3.402823466e38f);
        const uint32_t byte = odd ? 0x7Fu : e4m3_of(__fdiv_rn(top, __fmul_rn(7.f, factor)));
        const float step = odd ? 0.f : e4m3_f32(byte) * factor;
        uint32_t word = 0;
        if (step > 1e-30f && step < 1e30f && top < 7.49f * step) {
            // x / step rounded once: a quotient by the correctly rounded reciprocal, corrected by its remainder, which
            // one fused operation gives exactly (P. Markstein, Computation of elementary functions on the IBM RISC
            // System/6000 processor, IBM J. Res. Dev. 34, 1990).  Added to 1.5 2^23 it
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
            *reinterpret_cast<uint32_t*>(to) = word;
            if ((d8 & 8) == 0) *scales = (uint8_t)byte;
        }
        to += next;
        scales += next_scale;
    }
}

template <bool BF16, bool Q4, int TEAM>
static const void* head_kernel(bool vec, int rounds, bool split) {
    if (!vec) return (const void*)k_head_append<BF16, Q4, TEAM, false, 1, false>;
    return rounds == 1 ? (const void*)k_head_append<BF16, Q4, TEAM, true, 1, false>
           : split     ? (const void*)k_head_append<BF16, Q4, TEAM, true, 4, true>
                       : (const void*)k_head_append<BF16, Q4, TEAM, true, 4, false>;
}
template <bool BF16, bool Q4>
static const void* head_kernel(int team, bool vec, int rounds, bool split) {
    return team == 8    ? head_kernel<BF16, Q4, 8>(vec, rounds, split)
           : team == 16 ? head_kernel<BF16, Q4, 16>(vec, rounds, split)
                        : head_kernel<BF16, Q4, 32>(vec, rounds, split);
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
    // (a half of whole scale groups: four lanes have two groups between them)
    const bool split = !op.interleaved && op.rot_dim && op.rot_dim % (q4 ? 32 : 16) == 0;
    const auto kernel = bf ? (q4 ? head_kernel<true, true> : head_kernel<true, false>)
                           : (q4 ? head_kernel<false, true> : head_kernel<false, false>);
    const void* fn = kernel(team, vec, rounds, split);
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

// Bound by issue (79 % of the slots in the middle of 6825 tokens of 2 x 8 heads of 128: 11 us, of which the bytes are 5; a
// piece of eight values finds its token, head and page by itself): as many threads as pieces.
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
        uint32_t word[2] = {0, 0}, byte[2] = {0, 0};
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if (at.page < 0 || !(which ? op.v : op.k)) continue;
            word[which] = *reinterpret_cast<const uint32_t*>((which ? kv.v : kv.k) + code);
            byte[which] = (which ? kv.v_scale : kv.k_scale)[scale];
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            uint16_t* to = static_cast<uint16_t*>(which ? op.v : op.k);
            if (!to) continue;
            to += t * (which ? op.v_stride : op.k_stride) + (long long)h * kv.head_dim + c * 8;
            // code times scale is exact; scale times factor might pass fp32 beside a code of zero
            const float s = e4m3_f32(byte[which]), factor = which ? kv.v_factor : kv.k_factor;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = (float)((int)(word[which] << (28 - 4 * e)) >> 28) * s * factor;
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
    const long long want = (p.units + 255) / 256, most = 1 << 30;
    void* args[] = {&p};
    return launch_pdl(op.kv.type == DG_BF16 ? (const void*)k_kv4_read<true> : (const void*)k_kv4_read<false>,
                      dim3((unsigned)(want < most ? want : most)), dim3(256), 0, s, args);
}

}  // namespace dg
