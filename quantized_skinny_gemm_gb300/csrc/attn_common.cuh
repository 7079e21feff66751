// Attention over a paged cache, what the 16-bit and the 4-bit kernels share: the visible
// positions and their split into one equal range of blocks per CTA, the weights as
// two 16-bit numbers, and the join of units that were cut between CTAs.
#pragma once

#include <algorithm>
#include <cfloat>
#include <climits>

#include "mma16.cuh"
#include "tc_common.cuh"

namespace dg {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kBlockKeys = 128;
constexpr int kAttnMaxCtas = 640;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttnParams {
    dg_attn op;
    int groups;          // row groups per (sequence, head)
    int rows;            // q_len * heads / kv_heads
    int2* info;          // [units] a unit's first part and the number of its parts
    float* part;         // [grid][2] parts of a row group
    FastDiv page_size;
    float out_factor;    // of the sums over the weights' sum: 1, or what a 4-bit cache's values are counted in
};
// Floats of a part: a maximum and a sum for each row, then the rows.
constexpr int part_floats(int rows, int dp) { return rows * (dp + 2); }

__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The matrix instruction takes weights of 16 bits; one would cost 2^-12 (fp16) or
// 2^-9 (bf16) of a weight, as much as the output's own rounding.  Each weight is
// therefore the sum of two, hi + lo, 2^-21 (fp16) or 2^-16 (bf16) off.  hi is cut
// off below the weight, so that lo is above zero too and a value of infinity meets
// no zero and no minus.  fp16 ends at 2^-24: weights are taken 2^kLift times, up to
// 2^15, so that what is lost of one lies 2^-32 below the strongest key's.
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;
template <bool BF16>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t& hi, uint32_t& lo) {
    constexpr float kBelow = 1.f - 1.f / 4096;
    constexpr float kStep = BF16 ? 0.f : 5.9604645e-8f * kBelow;   // just below the smallest fp16 number
    const float2 w = make_float2(a, b), c = fma2(w, make_float2(kBelow, kBelow), make_float2(-kStep, -kStep));
    if (BF16)
        hi = __byte_perm(__float_as_uint(c.x), __float_as_uint(c.y), 0x7632);
    else
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(c.y), "f"(c.x));
    const float2 l = fma2(pair_f32<BF16>(hi), make_float2(-1.f, -1.f), w);
    lo = pair_16<BF16>(l.x, l.y);
}

// log sum e^z from the greatest score in units of log2(e) and the sum of the
// weights 2^(kLift + ..).
template <bool BF16>
__device__ __forceinline__ float lse_of(float top, float sum) {
    return sum == 0.f ? -INFINITY : (top + (log2f(sum) - kLift<BF16>)) * kLn2;
}

// The positions some token of sequence b sees: [0, seen_sinks) and [seen_lo,
// end).  They are walked in two pieces that start and end at multiples of 16,
// [0, sinks) and [lo, end), so that with pages of a multiple of 16 positions a
// stage lies in one page.
struct Span {
    int first;   // position of the step's first token (negative: before the start)
    int sinks, lo, end, seen_sinks, seen_lo;
    __device__ __forceinline__ int count() const { return end - lo + sinks; }
    __device__ __forceinline__ int position(int c) const { return c < sinks ? c : c - sinks + lo; }
    __device__ __forceinline__ bool seen(int j) const { return j >= seen_lo || j < seen_sinks; }
};
__device__ __forceinline__ Span span_of(const dg_attn& op, int b) {
    const int len = max(0, op.kv.seq_lens[b]);   // a step's own writes: no read-only loads
    const long long cap = (long long)op.kv.max_pages * op.kv.page_size;
    Span s;
    s.first = len - op.q_len;
    s.end = (int)min((long long)len, cap);
    const long long lo = op.window ? (long long)s.first - op.window + 1 : 0;
    s.seen_lo = (int)max(0ll, min(lo, (long long)s.end));
    s.lo = s.seen_lo & ~15;
    s.seen_sinks = min(op.sinks, s.seen_lo);
    s.sinks = (int)min(((unsigned)s.seen_sinks + 15u) & ~15u, (unsigned)s.lo);
    return s;
}
__device__ __forceinline__ int blocks_of(const Span& s) {
    return max(1, (int)(((long long)s.count() + kBlockKeys - 1) / kBlockKeys));
}

// First block of CTA c's range: floor(c * total / ctas).
__device__ __forceinline__ long long range_at(long long c, long long total, int ctas) {
    if (total < (1 << 22)) return (unsigned)c * (unsigned)total / (unsigned)ctas;
    return c * total / ctas;
}
__device__ __forceinline__ int quotient(long long a, int b) {
    return (unsigned long long)a >> 32 ? (int)(a / b) : (int)((unsigned)a / (unsigned)b);
}

// A CTA's equal range [begin, end) of the call's `total` blocks, cut into `ctas` ranges,
// and the sequence that its first block belongs to.  The blocks of one head are counted
// over the sequences: by every warp for itself up to 32, else 128 at a time by the CTA,
// in two passes past 128 (the second finds the sequence of the range's first block).
// heads: units per sequence.
struct CtaRange {
    long long total, begin, end;
    int ctas, b;
    long long seq_at;   // first block of sequence b
};
struct RangeScan {
    long long warps[kAttnWarps], found[2];
};
__device__ __forceinline__ CtaRange find_range(const dg_attn& op, int heads, RangeScan& s) {
    CtaRange r = {};
    const int B = op.kv.batch, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto take_range = [&] {
        r.ctas = (int)min((long long)gridDim.x, r.total);
        r.begin = range_at(blockIdx.x, r.total, r.ctas);
        r.end = blockIdx.x < r.ctas ? range_at(blockIdx.x + 1, r.total, r.ctas) : r.begin;
    };
    if (B <= 32) {
        const int n = lane < B ? blocks_of(span_of(op, lane)) : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        r.total = (long long)__shfl_sync(0xffffffffu, inc, 31) * heads;
        take_range();
        const long long lo = (long long)(inc - n) * heads, hi = (long long)inc * heads;
        const unsigned here = __ballot_sync(0xffffffffu, r.begin >= lo && r.begin < hi);
        r.b = max(0, __ffs(here) - 1);
        r.seq_at = __shfl_sync(0xffffffffu, lo, r.b);
    } else {
        const int passes = B <= kAttnThreads ? 1 : 2;
        for (int pass = 0; pass < passes; ++pass) {
            long long carry = 0;
            for (int b0 = 0; b0 < B; b0 += kAttnThreads) {
                const int n = b0 + tid < B ? blocks_of(span_of(op, b0 + tid)) : 0;
                long long inc = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += t;
                }
                if (lane == 31) s.warps[warp] = inc;
                __syncthreads();
                long long before = carry, sum = 0;
#pragma unroll
                for (int w = 0; w < kAttnWarps; ++w) {
                    if (w < warp) before += s.warps[w];
                    sum += s.warps[w];
                }
                const long long at = before + inc - n;
                carry += sum;
                if (pass == 0 && b0 + kAttnThreads >= B) {
                    r.total = carry * heads;
                    take_range();
                }
                if (pass == passes - 1 && n && r.begin >= at * heads && r.begin < (at + n) * heads) {
                    s.found[0] = b0 + tid;
                    s.found[1] = at;
                }
                __syncthreads();
            }
        }
        r.b = (int)s.found[0];
        r.seq_at = s.found[1] * heads;
    }
    return r;
}

// A unit's first part and the number of its parts, by the CTA that holds its first block
// blk, of nb blocks, up to block ke.  They lie in this CTA's first or second part and the
// first ones of the following CTAs; the last is the largest c with
// floor(c * total / ctas) <= u1, that is c * total < (u1 + 1) * ctas.
__device__ __forceinline__ int2 unit_parts(const CtaRange& r, long long blk, int nb, int ke, bool first) {
    int c = blockIdx.x;
    if (ke < nb) {
        const long long top = (blk + nb) * r.ctas;
        c = max(c, min(r.ctas - 1, __float2int_rz(__fdividef((float)top, (float)r.total))));
        while (c * r.total >= top) --c;
        while ((c + 1) * r.total < top) ++c;
    }
    return make_int2(blockIdx.x * 2 + (first ? 0 : 1), c - (int)blockIdx.x + 1);
}

// The parts of a unit that was cut between CTAs, joined in CTA order.  A CTA has
// `per` rows of the unit: its eight warps share them where the parts are few (32
// or less), else they share each row, every eighth part a warp and then the
// warps' in order.  per is 8 where the call has about as many units as CTAs, and
// 1 where few units have many parts.
constexpr int kJoinWarps = 8;
// ROWS: of a part; W16: how the weights were lifted (kLift).
template <bool BF16, int DP, int ROWS, bool W16>
__global__ void __launch_bounds__(kJoinWarps * 32) k_attn_join(const AttnParams p, int per) {
    constexpr int kPart = part_floats(ROWS, DP);
    constexpr int kPairs = DP / 64;   // pairs of output values of a lane, 64 apart
    // Parts under way: eight where a part is few registers (8 tokens of 8 sequences on windows of 4096, 16 bits, 64 dims:
    // 31.5 us, with four 33.0), four from 192 dims on (50000 positions of 5 x 192, 16 bits: 41.4 us, with eight 43.0).
    constexpr int kAhead = DP <= 128 ? 8 : 4;
    __shared__ float2 acc[kJoinWarps][kPairs][32];
    __shared__ float tops[kJoinWarps], sums[kJoinWarps];
    griddep_launch_dependents();
    griddep_wait();
    const dg_attn& op = p.op;
    const int2 info = __ldcg(p.info + blockIdx.x);
    const int n = info.y;
    if (n == 1) return;  // finished in place
    const int G = op.heads / op.kv.kv_heads, heads = op.kv.kv_heads * p.groups;
    const int b = blockIdx.x / heads, hg = blockIdx.x - b * heads, D = op.kv.head_dim;
    const int hk = hg / p.groups, base_row = (hg - hk * p.groups) * ROWS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float* parts = p.part + (size_t)(info.x >> 1) * 2 * kPart;
    const int skip = (info.x & 1) * kPart;
    const bool few = per > 1 && n <= 32;
    const int last = min(min(ROWS, p.rows - base_row), (int)(blockIdx.y + 1) * per);
    for (int r = blockIdx.y * per + (few ? warp : 0); r < last; r += few ? kJoinWarps : 1) {
        float top = -INFINITY, sum = 0.f;
        float2 v[kPairs];
#pragma unroll
        for (int x = 0; x < kPairs; ++x) v[x] = make_float2(0.f, 0.f);
        auto add = [&](float m, float l, const float2 (&w)[kPairs]) {
            const float nt = fmaxf(top, m), base = nt == -INFINITY ? 0.f : nt;
            const float f = exp2_fast(top - base), k = exp2_fast(m - base);
            top = nt;
            sum = sum * f + l * k;
#pragma unroll
            for (int x = 0; x < kPairs; ++x) {
                v[x].x = v[x].x * f + w[x].x * k;
                v[x].y = v[x].y * f + w[x].y * k;
            }
        };
#pragma unroll kAhead
        for (int i = few ? 0 : warp; i < n; i += few ? 1 : kJoinWarps) {
            const float* q = parts + (size_t)i * 2 * kPart + (i == 0 ? skip : 0);
            const float2* o = reinterpret_cast<const float2*>(q + 2 * ROWS + r * DP) + lane;
            float2 w[kPairs];
#pragma unroll
            for (int x = 0; x < kPairs; ++x)
                w[x] = x * 64 + lane * 2 < D ? __ldcg(o + x * 32) : make_float2(0.f, 0.f);
            add(__ldcg(q + r), __ldcg(q + ROWS + r), w);
        }
        if (!few) {
            if (lane == 0) {
                tops[warp] = top;
                sums[warp] = sum;
            }
#pragma unroll
            for (int x = 0; x < kPairs; ++x) acc[warp][x][lane] = v[x];
            __syncthreads();
            if (warp == 0) {
                for (int w = 1; w < kJoinWarps; ++w) {
                    float2 o[kPairs];
#pragma unroll
                    for (int x = 0; x < kPairs; ++x) o[x] = acc[w][x][lane];
                    add(tops[w], sums[w], o);
                }
            }
        }
        if (few || warp == 0) {
            const int row = base_row + r, tok = row / G, h = hk * G + row - tok * G;
            const long long t = (long long)b * op.q_len + tok;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(op.out) + t * op.out_stride +
                                                        (long long)h * D);
#pragma unroll
            for (int x = 0; x < kPairs; ++x)
                if (x * 64 + lane * 2 < D)
                    out[x * 32 + lane] = pair_16<BF16>(v[x].x * inv * p.out_factor, v[x].y * inv * p.out_factor);
            if (lane == 0 && op.lse)
                op.lse[t * op.heads + h] = lse_of<W16>(top, sum);
        }
        if (!few) __syncthreads();
    }
}

template <bool BF16, int DP, int ROWS, bool W16>
cudaError_t launch_join(const AttnParams& p, int grid, cudaStream_t s) {
    const long long units = (long long)p.op.kv.batch * p.op.kv.kv_heads * p.groups;
    int per = units * kJoinWarps >= grid ? kJoinWarps : 1;
    void* args[] = {const_cast<AttnParams*>(&p), &per};
    return launch_pdl((const void*)k_attn_join<BF16, DP, ROWS, W16>,
                      dim3((unsigned)units, (std::min(p.rows, ROWS) + per - 1) / per), dim3(kJoinWarps * 32), 0, s,
                      args);
}

inline long long max_blocks(const dg_attn& op, int groups) {
    const long long cap = (long long)op.kv.max_pages * op.kv.page_size;
    return (long long)op.kv.batch * op.kv.kv_heads * groups * ((cap + kBlockKeys - 1) / kBlockKeys);
}
inline bool never_split(const dg_attn& op) {
    return (long long)op.kv.max_pages * op.kv.page_size <= kBlockKeys;
}
inline size_t info_bytes(const dg_attn& op, int groups) {
    return ((size_t)op.kv.batch * op.kv.kv_heads * groups * 8 + 255) & ~(size_t)255;
}

}  // namespace dg
