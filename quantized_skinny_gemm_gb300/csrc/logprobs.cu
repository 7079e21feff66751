// Log probabilities of given tokens, entropy, rank and the best alternatives of rows of
// logits, in one pass over them.
//
// A row (or a part of it, where the rows are few) is a CTA's, taken in tiles of 1024
// 16-byte vectors, four a thread, the next tile loading while one is used.  Each thread
// keeps a base m, l = sum 2^((x - m) c) and a = sum 2^((x - m) c) (x - m) of its own, c =
// scale log2(e); the base follows the maximum only when that has grown by 2^8, so that a
// logit costs a difference, a product and one exponential; the entropy is ln l - scale a / l,
// whose terms have the size of the result.  Rows may start anywhere: the
// vectors are aligned ones, those at the row's ends are read one logit at a time.
//
// The best top_k: a candidate list in shared memory and a threshold that every candidate
// reaches.  Where more than 32 threads of a tile hold something above it, it is
// raised first to the top_k-th largest of the threads' maxima, so that
// hardly more than top_k logits of a tile are ever put in the list.  Keys are (logit,
// lowest index) in one 64-bit number, no two alike: what is chosen depends on no order.
#include <cfloat>
#include <climits>

#include "elem.cuh"

namespace dg {

constexpr int kLpThreads = 256, kLpVecs = 4, kLpTile = kLpThreads * kLpVecs;   // vectors of a tile
constexpr int kLpMaxParts = 64;
constexpr int kLpRaise = 32;                  // threads above the threshold before it is raised
constexpr int kLpKeep = 256;                  // candidates before the list is cut to top_k
constexpr int kLpList = kLpKeep + kLpRaise * kLpVecs * 8;
constexpr float kLpLog2e = 1.4426950408889634f;
using Key = unsigned long long;

struct LpPart {
    float m, l, a;
    int before;
};
struct LpParams {
    dg_logprobs op;
    int parts;
    float c, grow;      // scale * log2(e); how far the maximum may pass the base
    LpPart* part;       // [rows][parts]
    Key* keys;          // [rows][parts][top_k]
    FastDiv by_parts;
};

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
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
    if (o <= 1u) return __uint_as_float(0x7fffffffu);
    return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}

// (m, l, a) of two sets of logits.  An empty set's base is -infinity.
__device__ __forceinline__ void join(float& m, float& l, float& a, float m2, float l2, float a2, float c) {
    const float top = fmaxf(m, m2);
    auto moved = [&](float& mm, float& ll, float& aa) {
        if (mm == top) return;
        const float d = mm - top, f = ex2(d * c);   // ll 0: nothing to move (d may be -infinity)
        aa = ll == 0.f ? 0.f : f * (aa + d * ll);
        ll = f * ll;
    };
    moved(m, l, a);
    moved(m2, l2, a2);
    m = top;
    l += l2;
    a += a2;
}

template <int TYPE>   // 0 fp16, 1 bf16, 2 fp32
__device__ __forceinline__ float logit_at(const void* p, long long i) {
    if (TYPE == 2) return static_cast<const float*>(p)[i];
    return elem_f32<TYPE == 1>(static_cast<const uint16_t*>(p)[i]);
}

// A row's numbers from its sums; those of a row of only -infinity stand in the header.
struct Row {
    float m, l, log_l, scale;
    __device__ __forceinline__ Row(float m_, float l_, float s) : m(m_), l(l_), log_l(logf(l_)), scale(s) {}
    __device__ __forceinline__ float lse() const { return l == 0.f ? -INFINITY : fmaf(scale, m, log_l); }
    __device__ __forceinline__ float logprob(float x) const { return l == 0.f ? -INFINITY : scale * (x - m) - log_l; }
    __device__ __forceinline__ float entropy(float a) const { return l == 0.f ? 0.f : log_l - scale * (a / l); }
};

template <int TYPE>
__device__ __forceinline__ void write_row(const dg_logprobs& op, int row, float m, float l, float a, int before,
                                          const void* x) {
    const Row r(m == -INFINITY ? 0.f : m, l, op.scale);
    if (op.lse) op.lse[row] = r.lse();
    if (op.entropy) op.entropy[row] = r.entropy(a);
    if (!op.tokens) return;
    const int tok = op.tokens[row];
    const bool there = tok >= 0 && tok < op.V;
    if (op.rank) op.rank[row] = there ? before : op.V;
    // of a row of NaN everything is NaN
    if (op.logprob) op.logprob[row] = there ? r.logprob(logit_at<TYPE>(x, tok)) : l != l ? l : -INFINITY;
}

template <int TYPE>
__global__ void __launch_bounds__(kLpThreads) k_logprobs(const LpParams p) {
    constexpr int kEl = TYPE == 2 ? 4 : 8, kSize = TYPE == 2 ? 4 : 2;   // of a vector; bytes of a logit
    __shared__ Key list[kLpList];
    __shared__ Key maxima[kLpThreads];
    __shared__ float red[3][kLpThreads / 32];
    __shared__ Key s_floor;
    __shared__ int s_n, s_before;
    const dg_logprobs& op = p.op;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = (int)blockIdx.x / p.by_parts, part = blockIdx.x - row * p.parts;
    const int V = op.V, K = op.top_k;
    griddep_launch_dependents();
    griddep_wait();
    const unsigned char* x = static_cast<const unsigned char*>(op.logits) + (long long)row * op.stride * kSize;
    // vector v holds logits [v * kEl - skew, ..) of the row
    const int skew = (int)(((uintptr_t)x & 15) / kSize);
    const uint4* vecs = reinterpret_cast<const uint4*>(x - skew * kSize);
    const int nvec = (int)(((long long)V + skew + kEl - 1) / kEl);
    const int tiles = (nvec + kLpTile - 1) / kLpTile;
    const int tile0 = (int)((long long)part * tiles / p.parts), tile1 = (int)((long long)(part + 1) * tiles / p.parts);
    if (tid == 0) {
        s_n = s_before = 0;
        s_floor = 0;
    }
    int tok = -1;
    float mine = 0.f;   // the given token's logit
    if (op.rank && op.tokens) {
        tok = op.tokens[row];
        if (tok < 0 || tok >= V) tok = -1;
        else mine = logit_at<TYPE>(x, tok);
    }
    const bool count = tok >= 0;
    auto before = [&](float v, int i) {   // whether logit v of word i comes before the token
        if (mine != mine) return v == v || i < tok;
        return v > mine || (v == mine && i < tok);
    };
    auto whole = [&](int v) { return v * (long long)kEl >= skew && (v + 1) * (long long)kEl - skew <= V; };
    uint4 next[kLpVecs];
    auto fetch = [&](int tile) {
#pragma unroll
        for (int q = 0; q < kLpVecs; ++q) {
            const int v = tile * kLpTile + q * kLpThreads + tid;
            if (tile < tile1 && v < nvec && whole(v)) next[q] = __ldcs(vecs + v);
        }
    };
    float m = -INFINITY, base = 0.f;
    float2 l = make_float2(0.f, 0.f), a = l;
    int ahead = 0;
    Key floor = 0;
    float floor_logit = -INFINITY;
    fetch(tile0);
    __syncthreads();
    for (int tile = tile0; tile < tile1; ++tile) {
        uint4 now[kLpVecs];
#pragma unroll
        for (int q = 0; q < kLpVecs; ++q) now[q] = next[q];
        fetch(tile + 1);
        float tile_max = -INFINITY;
        bool any = false;
        auto unpack = [&](int q, float (&f)[kEl]) {
            if constexpr (TYPE == 2) {
                f[0] = __uint_as_float(now[q].x), f[1] = __uint_as_float(now[q].y);
                f[2] = __uint_as_float(now[q].z), f[3] = __uint_as_float(now[q].w);
            } else {
                unpack8<TYPE == 1>(now[q], f);
            }
        };
#pragma unroll
        for (int q = 0; q < kLpVecs; ++q) {
            const int v = tile * kLpTile + q * kLpThreads + tid;
            if (v >= nvec) continue;
            float f[kEl];
            const int i0 = v * kEl - skew;
            if (whole(v)) {
                unpack(q, f);
            } else {   // an end of the row: what is not there has no part in anything
#pragma unroll
                for (int e = 0; e < kEl; ++e)
                    f[e] = i0 + e >= 0 && i0 + e < V ? logit_at<TYPE>(x, i0 + e) : -INFINITY;
            }
            any = true;
            float top = f[0];
#pragma unroll
            for (int e = 1; e < kEl; ++e) top = fmaxf(top, f[e]);
            tile_max = fmaxf(tile_max, top);
            if (top > m + p.grow) {
                const float d = m - top, k = ex2(d * p.c);
                const bool none = m == -INFINITY;   // then l is 0, or NaN, and a is 0
                a = none ? make_float2(0.f, 0.f) : make_float2(k * (a.x + d * l.x), k * (a.y + d * l.y));
                l.x *= k;
                l.y *= k;
                m = base = top;
            }
#pragma unroll
            for (int e = 0; e < kEl; e += 2) {
                const float2 one = make_float2(1.f, 1.f);
                const float2 d = fma2(make_float2(f[e], f[e + 1]), one, make_float2(-base, -base));
                const float2 w = make_float2(ex2(d.x * p.c), ex2(d.y * p.c));
                l = fma2(w, one, l);
                a = fma2(w, make_float2(fmaxf(d.x, -FLT_MAX), fmaxf(d.y, -FLT_MAX)), a);   // -infinity has no part
            }
            if (count) {
                const bool edge = !whole(v) || mine != mine || (i0 <= tok && tok < i0 + kEl);
                if (edge) {
#pragma unroll
                    for (int e = 0; e < kEl; ++e)
                        ahead += i0 + e >= 0 && i0 + e < V && before(f[e], i0 + e);
                } else if (i0 < tok) {
#pragma unroll
                    for (int e = 0; e < kEl; ++e) ahead += f[e] >= mine;
                } else {
#pragma unroll
                    for (int e = 0; e < kEl; ++e) ahead += f[e] > mine;
                }
            }
        }
        if (K == 0) continue;
        const int above = __syncthreads_count(any && (floor == 0 || tile_max >= floor_logit));
        if (above == 0) continue;
        // every logit of this thread's vectors, with its index
        auto each = [&](auto&& use) {
#pragma unroll
            for (int q = 0; q < kLpVecs; ++q) {
                const int v = tile * kLpTile + q * kLpThreads + tid;
                if (v >= nvec) continue;
                float f[kEl];
                const int i0 = v * kEl - skew;
                const bool in = whole(v);
                if (in) unpack(q, f);
#pragma unroll
                for (int e = 0; e < kEl; ++e) {
                    const int i = i0 + e;
                    if (in) use(f[e], i);
                    else if (i >= 0 && i < V) use(logit_at<TYPE>(x, i), i);
                }
            }
        };
        if (s_n > kLpKeep) {   // (the same for all threads: read between two barriers)
            const int n = s_n;
            Key kept[kLpList / kLpThreads + 1];
            int rank[kLpList / kLpThreads + 1], have = 0;
            for (int i = tid; i < n; i += kLpThreads, ++have) {
                const Key k = list[i];
                int r = 0;
                for (int j = 0; j < n; ++j) r += list[j] > k;
                kept[have] = k;
                rank[have] = r;
            }
            __syncthreads();
            have = 0;
            for (int i = tid; i < n; i += kLpThreads, ++have)
                if (rank[have] < K) {
                    list[rank[have]] = kept[have];
                    if (rank[have] == K - 1) s_floor = max(s_floor, kept[have]);
                }
            if (tid == 0) s_n = K;
            __syncthreads();
        }
        if (above > kLpRaise) {
            Key best = 0;
            each([&](float v, int i) { best = max(best, key_of(v, i)); });
            maxima[tid] = best;
            __syncthreads();
            int r = 0;
#pragma unroll 8
            for (int j = 0; j < kLpThreads; ++j) r += maxima[j] > best;
            if (best && r == K - 1) s_floor = max(s_floor, best);
        }
        __syncthreads();
        floor = s_floor;
        floor_logit = floor ? logit_of(floor) : -INFINITY;
        if (floor_logit != floor_logit) floor_logit = -INFINITY;   // a floor of NaN: all reach it
        if (any && (floor == 0 || tile_max >= floor_logit))
            each([&](float v, int i) {
                const Key k = key_of(v, i);
                if (k >= floor) list[atomicAdd(&s_n, 1)] = k;
            });
        __syncthreads();
    }
    // ---- the part's sums ------------------------------------------------------------------
    float sl = l.x + l.y, sa = a.x + a.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, sl, o);
        const float a2 = __shfl_xor_sync(0xffffffffu, sa, o);
        join(m, sl, sa, m2, l2, a2, p.c);
    }
    if (count) {
        ahead = warp_sum(ahead);
        if (lane == 0 && ahead) atomicAdd(&s_before, ahead);
    }
    if (lane == 0) {
        red[0][warp] = m;
        red[1][warp] = sl;
        red[2][warp] = sa;
    }
    __syncthreads();
    m = red[0][0];
    sl = red[1][0];
    sa = red[2][0];
    for (int w = 1; w < kLpThreads / 32; ++w) join(m, sl, sa, red[0][w], red[1][w], red[2][w], p.c);
    if (tid == 0) {
        if (p.parts == 1) write_row<TYPE>(op, row, m, sl, sa, s_before, x);
        else p.part[blockIdx.x] = {m, sl, sa, s_before};
    }
    if (K == 0) return;
    const int n = s_n;
    const Row r(m == -INFINITY ? 0.f : m, sl, op.scale);
    Key* keys = p.parts == 1 ? nullptr : p.keys + (size_t)blockIdx.x * K;
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

// The parts of a row: their sums in order, and top_k times the largest of the parts' next
// keys.  A warp a row.
template <int TYPE>
__global__ void __launch_bounds__(32) k_logprobs_join(const LpParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const dg_logprobs& op = p.op;
    const int row = blockIdx.x, lane = threadIdx.x, K = op.top_k, n = p.parts;
    const unsigned char* x = static_cast<const unsigned char*>(op.logits) + (long long)row * op.stride * (TYPE == 2 ? 4 : 2);
    float m = -INFINITY, l = 0.f, a = 0.f;
    int before = 0;
    for (int i = lane; i < n; i += 32) {   // (two parts a lane at most)
        const LpPart q = p.part[(size_t)row * n + i];
        join(m, l, a, q.m, q.l, q.a, p.c);
        before += q.before;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
        const float a2 = __shfl_xor_sync(0xffffffffu, a, o);
        join(m, l, a, m2, l2, a2, p.c);
    }
    before = warp_sum(before);
    if (lane == 0) write_row<TYPE>(op, row, m, l, a, before, x);
    if (K == 0) return;
    const Row r(m == -INFINITY ? 0.f : m, l, op.scale);
    const Key* keys = p.keys + (size_t)row * n * K;
    int at[2] = {0, 0};
    Key head[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) head[h] = lane + 32 * h < n ? keys[(size_t)(lane + 32 * h) * K] : 0;
    for (int i = 0; i < K; ++i) {
        const int h = head[1] > head[0];
        Key best = h ? head[1] : head[0];
        const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
        const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
        const Key win = (Key)hi << 32 | lo;
        if (win == best && win) {   // keys are unique: one lane
            const long long to = (long long)row * K + i;
            if (op.top_ids) op.top_ids[to] = index_of(win);
            if (op.top_logprobs) op.top_logprobs[to] = r.logprob(logit_of(win));
            ++at[h];
            head[h] = at[h] < K ? keys[(size_t)(lane + 32 * h) * K + at[h]] : 0;
        }
    }
}

static int lp_parts(const dg_logprobs& op) {
    // as many CTAs as the SMs hold, where the rows alone are fewer
    const int el = op.logits_f32 ? 4 : 8;
    const long long tiles = ((long long)op.V + el - 1) / el / kLpTile + 1, want = (4ll * 152 + op.rows - 1) / op.rows;
    long long n = want < tiles ? want : tiles;
    return (int)(n > kLpMaxParts ? kLpMaxParts : n);
}

size_t lp_ws_bytes(const dg_logprobs& op) {
    const int parts = lp_parts(op);
    return parts == 1 ? 0 : (size_t)op.rows * parts * (sizeof(LpPart) + sizeof(Key) * op.top_k);
}

template <int TYPE>
static cudaError_t launch_lp(const dg_logprobs& op, void* ws, cudaStream_t s) {
    LpParams p;
    p.op = op;
    p.parts = lp_parts(op);
    p.c = op.scale * kLpLog2e;
    p.grow = fminf(8.f / p.c, FLT_MAX);   // finite: the first maximum is always taken
    p.part = static_cast<LpPart*>(ws);
    p.keys = reinterpret_cast<Key*>(static_cast<char*>(ws) + (size_t)op.rows * p.parts * sizeof(LpPart));
    p.by_parts = fast_div((uint32_t)p.parts);
    void* args[] = {&p};
    const cudaError_t e = launch_pdl((const void*)k_logprobs<TYPE>, dim3((unsigned)op.rows * p.parts),
                                     dim3(kLpThreads), 0, s, args);
    if (e != cudaSuccess || p.parts == 1) return e;
    return launch_pdl((const void*)k_logprobs_join<TYPE>, dim3(op.rows), dim3(32), 0, s, args);
}

cudaError_t launch_logprobs(const dg_logprobs& op, void* ws, cudaStream_t s) {
    return op.logits_f32 ? launch_lp<2>(op, ws, s)
                         : op.type == DG_BF16 ? launch_lp<1>(op, ws, s) : launch_lp<0>(op, ws, s);
}

}  // namespace dg
