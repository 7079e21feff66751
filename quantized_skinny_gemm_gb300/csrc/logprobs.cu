// Log probabilities of given tokens, entropy, rank and the best alternatives of rows of
// logits, in one pass over them.
//
// A row (or a part of it, where the rows are few) is a CTA's, taken in tiles of 512
// 16-byte vectors, four a thread, the next tile loading while one is used.  Small CTAs, eight an SM
// (fp32: five): while one looks for its row's best the others stream (2047 x 128255 bf16 with
// everything and one alternative: 101 us, with four CTAs of 256 threads 110; 95, 5.5 TB/s, since lanes
// take one base before their sums are added).  Bound by issue; one row of 128256 fp32 with five alternatives
// by two launches, 7.9 us.  Each thread
// keeps a base m and, with c = scale log2(e) and B = m c rounded, the sums l of w = 2^(x c - B)
// and a of w (x c - B): an exponent is one fused multiply-add, rounded once, B
// being a number like any other (a softmax of scale c / log2(e), 2^-24 off).  The base
// follows the maximum only when that has grown by 2^8.  lse = ln 2 (B + log2 l), the entropy is
// ln 2 (log2 l - a / l); the base may lie up to 8 below the row's maximum, and then both terms are 8 larger than the
// result: an entropy near 0 is up to 1e-6 off, not a part of itself.  Past |m c| = 2^22, where
// B's rounding nears a whole power of two (rows of nothing but masks, mostly), bases stand and the sums are taken
// again with exponents (x - m) c.  Sums of either kind join by what their weights were counted from, B or m c itself:
// parts of a row may lie on both sides.
//
// Rows may start anywhere: the vectors are aligned ones, and the logits before the first and behind
// the last are a thread's each.
//
// The rank is counted where a thread's four vectors hold something that is not below the token's
// logit, 16-bit logits two at a time, by one comparison: what equals the token and comes before it
// is what is above the next number below.  The best top_k cost the stream next to nothing: a thread only keeps its
// maximum, and that of each sixteenth of its tiles.  The top_k-th largest of 64 groups' maxima is
// then a floor that about top_k logits of the row reach; the sixteenths that
// reach it are read once more (from L2, mostly), by all threads at once, and what does is listed.
// (Sums and 20 alternatives: 94 us, each thread its own sixteenths 116; with one alternative 95 both ways.)  Keys are (logit, lowest index)
// in one 64-bit number, no two alike: what is chosen depends on no order.  (Lists that each warp kept while it
// streamed, cut to top_k again and again: 173 us for one alternative and 376 for 20, 2048 x
// 128256 bf16, where the sums alone take 94.)
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

#include "elem.cuh"

namespace dg {

constexpr int kLpThreads = 128, kLpVecs = 4, kLpTile = kLpThreads * kLpVecs;   // vectors of a tile
constexpr int kLpWarps = kLpThreads / 32, kLpMaxParts = 64;
constexpr int kLpGroups = 64, kLpTeam = kLpThreads / kLpGroups;   // groups of threads: more than top_k
constexpr int kLpSlices = 16;                 // of a part's tiles, with a maximum of a thread each
constexpr int kLpList = 1024;                 // candidates; where more reach the floor it is raised
constexpr float kNan = __builtin_nanf("");
constexpr float kLpLog2e = 1.4426950408889634f, kLpLn2 = 0.6931471805599453f;
using Key = unsigned long long;
template <int TYPE>
constexpr int kLpCtas = TYPE == 2 ? 5 : 8;   // of an SM

struct LpPart {
    float m, l, a;
    int before;
};
struct LpParams {
    dg_logprobs op;
    int whole, parts;   // rows that are a CTA's each; parts of the others
    float c, grow;      // scale * log2(e); how far the maximum may pass the base
    float most;         // bases up to this size have |m c| <= 2^22
    uint32_t low;       // bf16: a pair of -2^k, 2^24 <= 2^k c < 2^25: no weight beside any base, and finite
    int always_far;     // there is no such k (a temperature of 2^102)
    LpPart* part;       // [rows - whole][parts]
    Key* keys;          // [rows - whole][parts][top_k]
    FastDiv by_parts;
};

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float mul_rn(float a, float b) {   // (never part of a fused operation)
    float r;
    asm("mul.rn.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Larger logit first, then lower index; NaN below every number; 0: nothing.
__device__ __forceinline__ Key key_of(float v, int i) {
    const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
    const uint32_t o = v != v ? 1u : (u & 0x80000000u) ? ~u : u | 0x80000000u;   // -infinity is 0x007FFFFF
    return (Key)o << 32 | (0xffffffffu - (uint32_t)i);
}
__device__ __forceinline__ int index_of(Key k) { return (int)(0xffffffffu - (uint32_t)k); }
__device__ __forceinline__ float logit_of(Key k) {
    const uint32_t o = (uint32_t)(k >> 32);
    if (o <= 1u) return kNan;
    return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}

// The sums of a set of logits; an empty set's base is -infinity.  Their weights are counted from m c rounded where
// |m| <= most, else from m c.
struct Sums {
    float m, l, a;
    // what rounding left of m c
    __device__ __forceinline__ static float rest(float m, const LpParams& p) {
        return fabsf(m) <= p.most ? fmaf(m, p.c, -mul_rn(m, p.c)) : 0.f;
    }
    // other's base seen from this one's, in powers of two
    __device__ __forceinline__ static float distance(float from, float to, const LpParams& p) {
        const float near = mul_rn(from, p.c) - mul_rn(to, p.c);
        if (__builtin_expect(fabsf(from) <= p.most && fabsf(to) <= p.most, 1)) return near;
        return (from - to) * p.c - rest(from, p) + rest(to, p);
    }
    __device__ __forceinline__ void move(float to, const LpParams& p) {
        if (m == to) return;
        const float d = distance(m, to, p), f = ex2(d);
        a = f == 0.f || l == 0.f ? 0.f : f * (a + d * l);   // (d may be -infinity)
        l = f * l;
        m = to;
    }
    __device__ __forceinline__ void join(Sums o, const LpParams& p) {
        const float top = fmaxf(m, o.m);
        move(top, p);
        o.move(top, p);
        l += o.l;
        a += o.a;
    }
    // Those of LANES neighbouring lanes: one base for all first, so that each moves once.
    template <int LANES = 32>
    __device__ __forceinline__ void join_warp(const LpParams& p) {
        float top = m;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        move(top, p);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) {
            l += __shfl_xor_sync(0xffffffffu, l, o);
            a += __shfl_xor_sync(0xffffffffu, a, o);
        }
    }
};

template <int TYPE>   // 0 fp16, 1 bf16, 2 fp32
__device__ __forceinline__ float logit_at(const void* p, long long i) {
    if (TYPE == 2) return static_cast<const float*>(p)[i];
    return elem_f32<TYPE == 1>(static_cast<const uint16_t*>(p)[i]);
}

// A row's numbers from its sums; those of a row of only -infinity stand in the header.
struct Row {
    Sums s;
    float log_l, base, scale, c;
    bool near;
    __device__ __forceinline__ Row(const Sums& sums, const LpParams& p)
        : s(sums), log_l(log2f(sums.l)), base(mul_rn(sums.m, p.c)), scale(p.op.scale), c(p.c),
          near(fabsf(sums.m) <= p.most) {}
    __device__ __forceinline__ float lse() const {
        if (s.l == 0.f) return -INFINITY;
        return near ? (base + log_l) * kLpLn2 : fmaf(scale, s.m, log_l * kLpLn2);
    }
    __device__ __forceinline__ float logprob(float x) const {
        if (s.l == 0.f) return -INFINITY;
        const float d = fmaf(x, c, -base);   // (may pass fp32 where the result does not)
        if (near && fabsf(d) <= FLT_MAX) return (d - log_l) * kLpLn2;
        const float z = x - s.m;   // (passes fp32 for two finite numbers of different signs only: nothing cancels)
        return (z < -FLT_MAX && x >= -FLT_MAX ? scale * x - scale * s.m : scale * z) - log_l * kLpLn2;
    }
    __device__ __forceinline__ float entropy() const { return s.l == 0.f ? 0.f : (log_l - s.a / s.l) * kLpLn2; }
};

// The given token, -1 where there is none inside the row, and its logit.
struct Given {
    int tok;
    float logit;
};
template <int TYPE>
__device__ __forceinline__ Given given(const dg_logprobs& op, int row, const void* x) {
    Given g = {-1, kNan};
    if (!op.tokens) return g;
    const int tok = op.tokens[row];
    if (tok >= 0 && tok < op.V) g = {tok, logit_at<TYPE>(x, tok)};
    return g;
}
__device__ __forceinline__ void write_row(const LpParams& p, const Row& r, int row, int before, Given g) {
    const dg_logprobs& op = p.op;
    if (op.lse) op.lse[row] = r.lse();
    if (op.entropy) op.entropy[row] = r.entropy();
    if (op.rank) op.rank[row] = g.tok >= 0 ? before : op.V;
    // of a row of NaN everything is NaN
    if (op.logprob) op.logprob[row] = g.tok >= 0 ? r.logprob(g.logit) : r.s.l != r.s.l ? r.s.l : -INFINITY;
}

// The largest of a vector; NaN only where all are.
template <int TYPE>
__device__ __forceinline__ float vec_max(uint4 v) {
    if (TYPE == 2)
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    uint32_t m, n;
    if (TYPE == 1) {
        asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(v.x), "r"(v.y));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(n) : "r"(v.z), "r"(v.w));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(n));
    } else {
        asm("max.f16x2 %0, %1, %2;" : "=r"(m) : "r"(v.x), "r"(v.y));
        asm("max.f16x2 %0, %1, %2;" : "=r"(n) : "r"(v.z), "r"(v.w));
        asm("max.f16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(n));
    }
    const float2 f = pair_f32<TYPE == 1>(m);
    return fmaxf(f.x, f.y);
}

// How many of a vector's logits are above one of their kind (16-bit ones twice in a word), which
// 16-bit ones count as pairs of ones.
template <int TYPE>
__device__ __forceinline__ void count_above(uint4 v, uint32_t than, uint32_t& pairs, int& n) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (TYPE == 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) n += __uint_as_float(w[e]) > __uint_as_float(than);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (TYPE == 1) {
            __nv_bfloat162 a, b, c;
            memcpy(&a, &w[e], 4);
            memcpy(&b, &than, 4);
            memcpy(&c, &pairs, 4);
            c = __hadd2(c, __hgt2(a, b));
            memcpy(&pairs, &c, 4);
        } else {
            pairs = h2_as_u32(__hadd2(u32_as_h2(pairs), __hgt2(u32_as_h2(w[e]), u32_as_h2(than))));
        }
    }
}
// The next number below a finite one, as bits of its type.
__device__ __forceinline__ uint32_t bits_below(uint32_t u, uint32_t sign) {
    return u == 0 || u == sign ? sign + 1 : u & sign ? u + 1 : u - 1;
}
// 16-bit pairs, -infinity (and what has no weight in any sum) raised to `low`; NaN stays.
__device__ __forceinline__ uint32_t raise_bf16x2(uint32_t v, uint32_t low) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(low));
    return r;
}


template <int TYPE>
__global__ void __launch_bounds__(kLpThreads, kLpCtas<TYPE>) k_logprobs(const LpParams p) {
    constexpr int kEl = TYPE == 2 ? 4 : 8, kSize = TYPE == 2 ? 4 : 2;   // of a vector; bytes of a logit
    constexpr uint32_t kNone = TYPE == 2 ? 0xFF800000u : TYPE == 1 ? 0xFF80FF80u : 0xFC00FC00u;   // -infinity
    __shared__ Key list[kLpList];
    __shared__ __align__(16) Key group_key[kLpGroups];
    __shared__ __align__(16) float group_max[kLpGroups];
    __shared__ float slice_max[kLpSlices][kLpThreads];
    __shared__ Sums red[kLpWarps];
    __shared__ unsigned odd[kLpWarps];
    __shared__ int ranked_ahead[kLpWarps];   // what a warp saw before the token
    __shared__ Key s_floor;
    __shared__ int s_n, s_hot;
    __shared__ uint16_t hot[kLpSlices * kLpThreads];
    const dg_logprobs& op = p.op;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cut = (int)blockIdx.x - p.whole, parts = cut < 0 ? 1 : p.parts;   // whole rows first, then the cut ones
    const int row = cut < 0 ? blockIdx.x : p.whole + cut / p.by_parts, part = cut < 0 ? 0 : cut - (row - p.whole) * parts;
    const int V = op.V, K = op.top_k;
    griddep_launch_dependents();
    griddep_wait();
    const unsigned char* x = static_cast<const unsigned char*>(op.logits) + (long long)row * op.stride * kSize;
    // vectors [first, last) lie inside the row, vector v holding logits [v * kEl - skew, ..)
    const int skew = (int)(((uintptr_t)x & 15) / kSize);
    const uint4* vecs = reinterpret_cast<const uint4*>(x - skew * kSize);
    const int first = skew ? 1 : 0, last = (int)(((long long)V + skew) / kEl);
    const int tiles = (last - first + kLpTile - 1) / kLpTile;   // 0 where last < first
    const int tile0 = (int)((long long)part * tiles / parts), tile1 = (int)((long long)(part + 1) * tiles / parts);
    const int full = min(tile1, (last - first) / kLpTile);   // tiles before this one need no bounds
    uint4 next[kLpVecs];
    auto fetch = [&](int tile) {
        const uint4* from = vecs + (first + tile * kLpTile + tid);
        auto load = [](const uint4* v) { return TYPE == 2 ? *v : __ldcs(v); };
        if (tile < full) {
#pragma unroll
            for (int q = 0; q < kLpVecs; ++q) next[q] = load(from + q * kLpThreads);
        } else if (tile < tile1) {
#pragma unroll
            for (int q = 0; q < kLpVecs; ++q) {
                next[q] = make_uint4(kNone, kNone, kNone, kNone);
                if (first + tile * kLpTile + q * kLpThreads + tid < last) next[q] = load(from + q * kLpThreads);
            }
        }
    };
    fetch(tile0);
    if (tid == 0) s_floor = 0;   // (the sums' barriers lie before its next use)
    const Given token = given<TYPE>(op, row, x);   // (now: at the row's end all of the CTA would wait for it)
    const int tok = op.rank ? token.tok : -1;
    const float mine = token.logit;
    const bool nan_token = tok >= 0 && mine != mine;
    auto before = [&](float v, int i) {   // whether logit v of word i comes before the token
        if (nan_token) return v == v || i < tok;
        return v > mine || (v == mine && i < tok);
    };
    // Vectors before the token's own count what is above `below`, the next number below its logit,
    // others what is above the logit itself.  Tokens of NaN or -infinity have their own pass.
    const bool ranked = tok >= 0 && mine > -INFINITY, pass = tok >= 0 && !ranked;
    const uint32_t bits = TYPE == 2 ? __float_as_uint(mine) : pair_16<TYPE == 1>(mine, mine);   // (it has 16 bits)
    const uint32_t below = TYPE == 2 ? bits_below(bits, 0x80000000u) : bits_below(bits & 0xFFFFu, 0x8000u) * 0x10001u;
    const int tok_vec = (tok + skew) / kEl;
    // the thread's sums: weights of 2^(x c - base), base m c rounded, or most c with m's sign past it
    float m = -INFINITY, base = 0.f;
    float2 l = make_float2(0.f, 0.f), a = l;
    auto base_of = [&](float v) { return mul_rn(fminf(fmaxf(v, -p.most), p.most), p.c); };
    int ahead = 0;
    // ---- the logits outside the vectors, by the first part ---------------------------------------
    const int head = min(V, skew ? kEl - skew : 0), tail = max(head, last * kEl - skew);
    const bool end = part == 0 && tid < head + (V - tail);
    const int end_i = tid < head ? tid : tail + tid - head;
    if (end) {
        const float v = logit_at<TYPE>(x, end_i);
        if (v > -INFINITY) {
            m = v;
            base = base_of(v);
            const float d = fmaf(v, p.c, -base);
            l.x = ex2(d);
            a.x = l.x * fmaxf(d, -FLT_MAX);
        }
        if (v != v || v == INFINITY) l.x = kNan;
        ahead = tok >= 0 && before(v, end_i);
        list[tid] = key_of(v, end_i);   // always a candidate
    }
    const int ends = part == 0 ? head + (V - tail) : 0;
    if (ranked && tid < kEl && tok_vec >= first + tile0 * kLpTile && tok_vec < min(last, first + tile1 * kLpTile)) {
        const int i = tok_vec * kEl - skew + tid;   // in the token's own vector, before it
        if (i < tok) ahead += logit_at<TYPE>(x, i) == mine;
    }
    // logit e of a vector; the index of the first of this thread's vector q; where vectors end
    auto logit = [&](const uint4& v, int e) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if (TYPE == 2) return __uint_as_float(w[e & 3]);
        return elem_f32<TYPE == 1>((uint16_t)(w[e / 2 & 3] >> (e & 1) * 16));
    };
    auto index = [&](int tile, int q) { return (first + tile * kLpTile + q * kLpThreads + tid) * kEl - skew; };
    const int inside = last * kEl - skew;
    const float2 c2 = make_float2(p.c, p.c), one = make_float2(1.f, 1.f);
    float greatest = -INFINITY, sliced = -INFINITY;   // of the thread's vectors, and of this slice of tiles
    int greatest_at = tile0, slice = 0;
    const int per_slice = max(1, (tile1 - tile0 + kLpSlices - 1) / kLpSlices);
    int slice_end = tile0 + per_slice;
    for (int tile = tile0; tile < tile1; ++tile) {
        uint4 now[kLpVecs];
#pragma unroll
        for (int q = 0; q < kLpVecs; ++q) now[q] = next[q];
        fetch(tile + 1);
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < kLpVecs; ++q) top = fmaxf(top, vec_max<TYPE>(now[q]));
        if (K) {
            if (top > greatest) {   // the first tile that holds it
                greatest = top;
                greatest_at = tile;
            }
            sliced = fmaxf(sliced, top);
            if (tile + 1 == slice_end || tile + 1 == tile1) {
                slice_max[slice++][tid] = sliced;
                sliced = -INFINITY;
                slice_end += per_slice;
            }
        }
        if (top > m + p.grow) {
            // (bases past 2^22 stand there; the sums are taken again if that was the part's maximum)
            const float to = base_of(top);
            const float d = base - to, k = ex2(d);
            const bool none = m == -INFINITY;   // then l is 0, or NaN, and a is 0
            a = none ? make_float2(0.f, 0.f) : make_float2(k * (a.x + d * l.x), k * (a.y + d * l.y));
            l = none ? make_float2(l.x * 0.f, l.y * 0.f) : make_float2(l.x * k, l.y * k);
            m = top;
            base = to;
        }
        const float2 off = make_float2(-base, -base);
#pragma unroll
        for (int q = 0; q < kLpVecs; ++q) {
            const uint32_t w[4] = {now[q].x, now[q].y, now[q].z, now[q].w};
#pragma unroll
            for (int e = 0; e < kEl / 2; ++e) {
                const float2 f = TYPE == 2 ? make_float2(__uint_as_float(w[2 * e & 3]), __uint_as_float(w[(2 * e + 1) & 3]))
                                           : pair_f32<TYPE == 1>(TYPE == 1 ? raise_bf16x2(w[e], p.low) : w[e]);
                const float2 d = fma2(f, c2, off);
                const float2 t = make_float2(ex2(d.x), ex2(d.y));
                l = fma2(t, one, l);
                // -infinity has no part: 0 times a number
                a = fma2(t, TYPE == 1 ? d : make_float2(fmaxf(d.x, -FLT_MAX), fmaxf(d.y, -FLT_MAX)), a);
            }
        }
        if (ranked && top >= mine) {
            uint32_t pairs = 0;   // at most 16 each
#pragma unroll
            for (int q = 0; q < kLpVecs; ++q)
                count_above<TYPE>(now[q], first + tile * kLpTile + q * kLpThreads + tid < tok_vec ? below : bits, pairs,
                                  ahead);
            if (TYPE != 2) {
                const float2 f = pair_f32<TYPE == 1>(pairs);
                ahead += (int)(f.x + f.y);
            }
        }
    }
    const long long i0 = (long long)(first + tile0 * kLpTile) * kEl - skew;   // the part's vectors
    const long long i1 = (long long)min(last, first + tile1 * kLpTile) * kEl - skew;
    if (pass)
        for (long long i = i0 + tid; i < i1; i += kLpThreads) ahead += before(logit_at<TYPE>(x, i), (int)i);
    // ---- the part's sums ------------------------------------------------------------------
    Sums s = {m, l.x + l.y, a.x + a.y};
    if (m == INFINITY) s.l = kNan;
    else if (m > -INFINITY) s.m = fminf(fmaxf(m, -p.most), p.most);   // as its base
    auto whole = [&] {   // the CTA's, in every thread
        s.join_warp(p);
        if (lane == 0) red[warp] = s;
        __syncthreads();
        s = red[lane % kLpWarps];
        s.join_warp<kLpWarps>(p);
    };
    // a place for each warp, read behind the sums' barrier: nobody has to clear a common one first
    ahead = warp_sum(ahead);
    if (lane == 0) ranked_ahead[warp] = ahead;
    // where the threads' maxima lie (those that their bases follow, up to 2^8 below the true ones)
    const unsigned past = __any_sync(0xffffffffu, m < INFINITY && m > p.most);
    const unsigned some = __any_sync(0xffffffffu, m > -INFINITY);
    const unsigned inside_most = __any_sync(0xffffffffu, m >= -p.most);
    if (lane == 0) odd[warp] = past | some << 1 | inside_most << 2;
    if (K) {
        float group = greatest;
#pragma unroll
        for (int o = 1; o < kLpTeam; o <<= 1) group = fmaxf(group, __shfl_xor_sync(0xffffffffu, group, o));
        if (tid % kLpTeam == 0) group_max[tid / kLpTeam] = group;
    }
    whole();
    unsigned any = 0;
#pragma unroll
    for (int w = 0; w < kLpWarps; ++w) any |= odd[w];
    // A maximum past most has weights that pass fp32 beside its base; with all of them below -most the best one's may be so
    // small that weaker ones vanish.
    const bool far = p.always_far || (any & 1u) || (any & 6u) == 2u;
    if (far) {   // exponents as differences, or from the true maximum's base
        auto all = [&](auto&& use) {
            if (end) use(logit_at<TYPE>(x, end_i));
            for (long long i = i0 + tid; i < i1; i += kLpThreads) use(logit_at<TYPE>(x, i));
        };
        __syncthreads();   // red has been read
        s = {-INFINITY, 0.f, 0.f};
        all([&](float v) { s.m = fmaxf(s.m, v); });
        const bool near = fabsf(s.m) <= p.most;
        const float from = mul_rn(s.m, p.c);
        all([&](float v) {
            const float d = near ? fmaf(v, p.c, -from) : (v - s.m) * p.c, t = ex2(d);
            if (v == -INFINITY) return;
            s.l += t;
            s.a = fmaf(t, fmaxf(d, -FLT_MAX), s.a);
        });
        whole();
    }
    const Row r(s, p);
    if (tid == 0) {
        int all_ahead = 0;
#pragma unroll
        for (int w = 0; w < kLpWarps; ++w) all_ahead += ranked_ahead[w];
        if (cut < 0) write_row(p, r, row, all_ahead, token);
        else p.part[cut] = {s.m, s.l, s.a, all_ahead};
    }
    if (K == 0) return;
    // ---- the best -------------------------------------------------------------------------------
    // K groups' maxima are not below the floor
    if (tid < kLpGroups) {
        const float v = group_max[tid];
        int above = 0, same = 0;
#pragma unroll 4
        for (int j = 0; j < kLpGroups; j += 4) {
            const float4 o = *reinterpret_cast<const float4*>(group_max + j);
            above += (o.x > v) + (o.y > v) + (o.z > v) + (o.w > v);
            same += (o.x == v) + (o.y == v) + (o.z == v) + (o.w == v);
        }
        // (a maximum of -infinity may be of NaN only)
        if (above < K && above + same >= K) s_floor = v > -INFINITY ? key_of(v, -1) : 0;
    }
    int n;
    for (int turn = 0;; ++turn) {
        if (tid == 0) {
            s_n = ends;
            s_hot = 0;
        }
        __syncthreads();
        const Key floor = s_floor;
        float at_least = floor ? logit_of(floor) : -INFINITY;
        if (at_least != at_least) at_least = -INFINITY;   // a floor of NaN: any logit may reach it
        // which threads' slices hold something that may: all of them first, then all threads read those
        // vectors, so that no thread waits for memory as often as it has such slices
        if (greatest >= at_least)
            for (int h = 0; h < slice; ++h)
                if (slice_max[h][tid] >= at_least) hot[atomicAdd(&s_hot, 1)] = (uint16_t)(h * kLpThreads + tid);
        __syncthreads();
        const int per_hot = per_slice * kLpVecs, vectors = s_hot * per_hot;
        for (int at = tid; at < vectors; at += kLpThreads * kLpVecs) {
            uint4 v[kLpVecs];
            int i[kLpVecs];
#pragma unroll
            for (int q = 0; q < kLpVecs; ++q) {
                const int u = at + q * kLpThreads, w = u / per_hot, rest = u - w * per_hot;
                i[q] = INT_MAX;
                if (u >= vectors) continue;
                const int h = hot[w] / kLpThreads, t = hot[w] % kLpThreads, tile = tile0 + h * per_slice + rest / kLpVecs;
                const int vec = first + tile * kLpTile + rest % kLpVecs * kLpThreads + t;
                if (tile >= tile1 || vec >= last) continue;
                i[q] = vec * kEl - skew;
                v[q] = vecs[vec];
            }
#pragma unroll
            for (int q = 0; q < kLpVecs; ++q) {
                if (i[q] == INT_MAX || vec_max<TYPE>(v[q]) < at_least) continue;   // (not where all are NaN)
#pragma unroll
                for (int e = 0; e < kEl; ++e) {
                    const Key k = key_of(logit(v[q], e), i[q] + e);
                    if (k < floor) continue;
                    const int to_list = atomicAdd(&s_n, 1);
                    if (to_list < kLpList) list[to_list] = k;
                }
            }
        }
        __syncthreads();
        n = s_n;
        if (n <= kLpList) break;
        // too many: next time from the groups' keys (equal logits differ there), and then from the
        // top_k-th of those that found room
        if (turn == 0) {
            Key largest = 0;
            if (tile0 < tile1) {
#pragma unroll
                for (int q = 0; q < kLpVecs; ++q) {
                    const int i = index(greatest_at, q);
                    if (i >= inside) break;
                    const uint4 v = vecs[first + greatest_at * kLpTile + q * kLpThreads + tid];
#pragma unroll
                    for (int e = 0; e < kEl; ++e) largest = max(largest, key_of(logit(v, e), i + e));
                }
            }
#pragma unroll
            for (int o = 1; o < kLpTeam; o <<= 1) largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, o));
            if (tid % kLpTeam == 0) group_key[tid / kLpTeam] = largest;
            __syncthreads();
            if (tid < kLpGroups) {
                const Key k = group_key[tid];
                int above = 0;
                for (int j = 0; j < kLpGroups; ++j) above += group_key[j] > k;
                if (k && above == K - 1) s_floor = max(s_floor, k);
            }
        } else {
            for (int i = tid; i < kLpList; i += kLpThreads) {
                const Key k = list[i];
                int above = 0;
                for (int j = 0; j < kLpList; ++j) above += list[j] > k;
                if (above == K - 1) s_floor = k;
            }
        }
        __syncthreads();
    }
    Key* keys = cut < 0 ? nullptr : p.keys + (size_t)cut * K;
    for (int i = tid; i < n; i += kLpThreads) {
        const Key k = list[i];
        int place = 0;
        for (int j = 0; j < n; ++j) place += list[j] > k;
        if (place >= K) continue;
        if (keys) {
            keys[place] = k;
            continue;
        }
        const long long at = (long long)row * K + place;
        if (op.top_ids) op.top_ids[at] = index_of(k);
        if (op.top_logprobs) op.top_logprobs[at] = r.logprob(logit_of(k));
    }
    if (keys)   // a part of fewer logits than top_k
        for (int i = n + tid; i < K; i += kLpThreads) keys[i] = 0;
}

// The parts of a row, a CTA a row: its first warp joins their sums, while the second takes top_k times the
// largest of the parts' next keys, when all have brought those to shared memory.
constexpr int kLpJoinThreads = 128;
template <int TYPE>
__global__ void __launch_bounds__(kLpJoinThreads) k_logprobs_join(const LpParams p) {
    __shared__ Key keys[kLpMaxParts * 32];
    __shared__ Sums total;
    griddep_launch_dependents();
    griddep_wait();
    const dg_logprobs& op = p.op;
    const int cut = blockIdx.x, row = p.whole + cut, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, K = op.top_k,
              n = p.parts;
    const unsigned char* x = static_cast<const unsigned char*>(op.logits) + (long long)row * op.stride * (TYPE == 2 ? 4 : 2);
    for (int i = threadIdx.x; i < n * K; i += kLpJoinThreads) keys[i] = p.keys[(size_t)cut * n * K + i];
    const Given token = warp == 0 ? given<TYPE>(op, row, x) : Given{-1, kNan};
    __syncthreads();
    Key mine = 0;   // of this lane's place
    if (warp == 0) {
        Sums s = {-INFINITY, 0.f, 0.f};
        int before = 0;
        for (int i = lane; i < n; i += 32) {   // (two parts a lane at most)
            const LpPart q = p.part[(size_t)cut * n + i];
            s.join({q.m, q.l, q.a}, p);
            before += q.before;
        }
        s.join_warp(p);
        before = warp_sum(before);
        if (lane == 0) {
            total = s;
            write_row(p, Row(s, p), row, before, token);
        }
    } else if (warp == 1 && K) {
        int at[2] = {0, 0};
        Key head[2];   // the two lists' next keys
#pragma unroll
        for (int h = 0; h < 2; ++h) head[h] = lane + 32 * h < n ? keys[(lane + 32 * h) * K] : 0;
        for (int i = 0; i < K; ++i) {
            const int h = head[1] > head[0];
            const Key best = h ? head[1] : head[0];
            const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
            const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
            const Key win = (Key)hi << 32 | lo;
            if (lane == i) mine = win;
            if (win == best && win) {   // keys are unique: one lane
                const int next = h ? ++at[1] : ++at[0];
                const Key k = next < K ? keys[(lane + 32 * h) * K + next] : 0;
                if (h) head[1] = k;
                else head[0] = k;
            }
        }
    }
    if (K == 0) return;
    __syncthreads();
    if (warp == 1 && lane < K && mine) {
        const Row r(total, p);
        const long long to = (long long)row * K + lane;
        if (op.top_ids) op.top_ids[to] = index_of(mine);
        if (op.top_logprobs) op.top_logprobs[to] = r.logprob(logit_of(mine));
    }
}

// Rows come in rounds of as many CTAs as the 152 SMs hold (a workspace's size must not depend on the device that asks for
// it, so this is no question to one; with other numbers of SMs only the time changes).  Those of a last round that would leave half of
// the places empty, or of a call of so few, are cut into parts.
struct LpSplit {
    int whole, parts;
};
static LpSplit lp_split(const dg_logprobs& op) {
    const int el = op.logits_f32 ? 4 : 8, places = 152 * (op.logits_f32 ? kLpCtas<2> : kLpCtas<0>);
    const int rest = op.rows % places;
    if (rest == 0 || rest * 2 > places) return {op.rows, 1};
    const long long tiles = ((long long)op.V + el - 1) / el / kLpTile + 1, want = places / rest;
    const int parts = (int)std::min({want, tiles, (long long)kLpMaxParts});
    return parts == 1 ? LpSplit{op.rows, 1} : LpSplit{op.rows - rest, parts};
}

size_t lp_ws_bytes(const dg_logprobs& op) {
    const LpSplit c = lp_split(op);
    return (size_t)(op.rows - c.whole) * c.parts * (sizeof(LpPart) + sizeof(Key) * op.top_k);
}

template <int TYPE>
static cudaError_t launch_lp(const dg_logprobs& op, void* ws, cudaStream_t s) {
    LpParams p;
    p.op = op;
    const LpSplit split = lp_split(op);
    p.whole = split.whole;
    p.parts = split.parts;
    const int cut = op.rows - p.whole;
    p.c = op.scale * kLpLog2e;
    p.grow = fminf(8.f / p.c, FLT_MAX);   // finite: the first maximum is always taken
    p.most = fminf(4194304.f / p.c, FLT_MAX);
    const int k = 24 - std::ilogb(p.c);
    p.always_far = TYPE == 1 && k > 126;
    p.low = (0x8000u | (uint32_t)(127 + std::min(k, 126)) << 7) * 0x10001u;
    p.part = static_cast<LpPart*>(ws);
    p.keys = reinterpret_cast<Key*>(static_cast<char*>(ws) + (size_t)cut * p.parts * sizeof(LpPart));
    p.by_parts = fast_div((uint32_t)p.parts);
    void* args[] = {&p};
    const cudaError_t e = launch_pdl((const void*)k_logprobs<TYPE>, dim3((unsigned)(p.whole + cut * p.parts)),
                                     dim3(kLpThreads), 0, s, args);
    if (e != cudaSuccess || cut == 0) return e;
    return launch_pdl((const void*)k_logprobs_join<TYPE>, dim3(cut), dim3(kLpJoinThreads), 0, s, args);
}

cudaError_t launch_logprobs(const dg_logprobs& op, void* ws, cudaStream_t s) {
    return op.logits_f32 ? launch_lp<2>(op, ws, s)
                         : op.type == DG_BF16 ? launch_lp<1>(op, ws, s) : launch_lp<0>(op, ws, s);
}

}  // namespace dg
