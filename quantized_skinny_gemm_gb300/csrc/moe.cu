// A mixture-of-experts layer for a few tokens, in three launches: router
// scores; gate and up products with SwiGLU; down products with the weighted
// sum over experts.
//
// The cost is the chosen experts' weights (6 * I * K bytes each at 16 bits,
// 1.7 * I * K at int4), read once whatever the number of tokens, so the
// products stream weights and spend the matrix instruction (m16n8k16: 16
// weight rows x 8 token columns) on few tokens: it costs no more for eight
// than for one.  Weights go from global memory straight into the
// instruction's registers: a lane's 16 bytes are 8 columns of its row, and
// the order of columns inside an instruction is free as long as the tokens'
// values follow it.  A warp keeps one chunk (16 rows x 256 columns, 8 KB at
// 16 bits) in flight and reloads each register as soon as it is used.
//
//   up:   a CTA takes 8 gate and the same 8 up rows of an expert at a time, so
//         that silu(gate) * up meets in one thread; its warps deal the row
//         tile's chunks along K among themselves, without a break from one
//         tile to the next, and their sums are added in warp order.
//   down: a CTA takes 16 output rows at a time; its warps deal the chunks of
//         all chosen experts, each adding weight * sum into its own fp32 rows
//         [token], which are summed in warp order.
//
// h goes from one to the other as two 16-bit values, hi + lo, that are two
// columns of the matrix instruction: fp16 hi = h / 256 and lo = the rest x 2048
// (22 bits, |h| up to 2^24), bf16 hi and lo (16 bits); the products keep fp32
// sums.  int4 codes become fp16 by bit operations (exact).  A group of 32
// codes must be summed on its own before its scale, but a quad's lanes hold
// parts of several groups (PH = 2 of 8-byte pieces, or 4 of 16-byte ones): each
// token gets PH columns, column f carrying the token's values for the lanes
// whose codes belong to group f and zero for the others, so that one
// instruction sums the groups apart.
#include "mma16.cuh"
#include "tc_common.cuh"

namespace dg {

constexpr int kMoeMaxSlots = 256;   // tokens x choices
constexpr int kMoeWarps = 8;

// Workspace: scores [M][E], ids and weights [256], x in int4 order [M][K], h
// [slots][2][I].
struct MoeWs {
    float* scores;
    int* ids;
    float* wts;
    uint16_t* xp;
    uint16_t* h;
};

struct MoeParams {
    dg_moe op;
    MoeWs ws;
    int pair_scales;  // int4: two groups' scales are one aligned 4-byte load
};

// ---- router scores ------------------------------------------------------------------------

// Where value i of eight lies in the order the int4 unpacking gives its codes:
// (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ int int4_place(int i) { return i < 4 ? 2 * i : 2 * i - 7; }

// One CTA per expert and four tokens: their scores.  The first row of CTAs also
// writes x in the int4 order, which the up products read.
constexpr int kScoreTokens = 4;
template <bool BF16>
__global__ void __launch_bounds__(256) k_moe_scores(const MoeParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const dg_moe& op = p.op;
    const int e = blockIdx.x, m0 = blockIdx.y * kScoreTokens;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K8 = op.K / 8;
    const uint4* r = static_cast<const uint4*>(op.router) + (size_t)e * K8;
    const uint4* x = static_cast<const uint4*>(op.x);
    float z[kScoreTokens];
#pragma unroll
    for (int m = 0; m < kScoreTokens; ++m) z[m] = 0.f;
#pragma unroll 2
    for (int k = tid; k < K8; k += 256) {
        float w[8];
        const uint4 wv = __ldg(r + k);
        uint4 xv[kScoreTokens];
#pragma unroll
        for (int m = 0; m < kScoreTokens; ++m) xv[m] = __ldcg(x + (size_t)min(m0 + m, op.M - 1) * K8 + k);
        unpack8<BF16>(wv, w);
#pragma unroll
        for (int m = 0; m < kScoreTokens; ++m) {
            float v[8];
            unpack8<BF16>(xv[m], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[m] = fmaf(w[i], v[i], z[m]);
        }
    }
    __shared__ float part[8][kScoreTokens];
#pragma unroll
    for (int m = 0; m < kScoreTokens; ++m) {
        const float v = warp_sum(z[m]);
        if (lane == 0) part[warp][m] = v;
    }
    __syncthreads();
    if (tid < kScoreTokens && m0 + tid < op.M) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += part[w][tid];
        p.ws.scores[(size_t)(m0 + tid) * op.E + e] = v;
    }
    if (op.kind == DG_LINEAR_W4A16 && m0 == 0) {
        const int n8 = op.M * K8;
        for (int i = e * 256 + tid; i < n8; i += gridDim.x * 256) {
            const uint4 v = __ldcg(x + i);
            reinterpret_cast<uint4*>(p.ws.xp)[i] =
                make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                           __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
        }
    }
}

// ---- routing ------------------------------------------------------------------------------

// One warp: a token's probabilities from its scores (prob: E floats of shared
// memory), its top_k experts and their weights.  Selection compares integers:
// 0 nothing, 1 NaN, then the probability's bits (it is not negative).
__device__ void route_token(const dg_moe& op, const float* scores, float* prob, int* ids, float* wts) {
    const int lane = threadIdx.x & 31, E = op.E;
    if (op.score == DG_MOE_SOFTMAX) {
        float top = -INFINITY, sum = 0.f;
        for (int e = lane; e < E; e += 32) top = fmaxf(top, prob[e] = __ldcg(scores + e));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        for (int e = lane; e < E; e += 32) sum += prob[e] = expf(prob[e] - top);
        sum = warp_sum(sum);
        for (int e = lane; e < E; e += 32) prob[e] = prob[e] / sum;
    } else {
        for (int e = lane; e < E; e += 32) prob[e] = 1.f / (1.f + expf(-__ldcg(scores + e)));
    }
    float mine = 0.f, total = 0.f;   // lane c holds choice c
    int id = 0;
    for (int c = 0; c < op.top_k; ++c) {
        unsigned best = 0;
        int at = 0x7fffffff;
        for (int e = lane; e < E; e += 32) {
            const float v = prob[e];
            const unsigned key = v != v ? 1u : v < 0.f ? 0u : __float_as_uint(v) + 2u;
            if (key > best) {
                best = key;
                at = e;
            }
        }
        const unsigned top = __reduce_max_sync(0xffffffffu, best);
        const int e = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7fffffff);
        const float v = prob[e];   // this lane's or another's: nobody has changed it yet
        __syncwarp();
        if (lane == (e & 31)) prob[e] = -1.f;
        if (lane == c) {
            mine = v;
            id = e;
        }
        total += v;
        __syncwarp();
    }
    if (lane < op.top_k) {
        ids[lane] = id;
        wts[lane] = (op.renormalize ? mine / total : mine) * op.route_scale;
    }
}

// The chosen experts in ascending order and each one's slots (token * top_k +
// choice) in token order.
struct Lists {
    int count;
    uint16_t expert[kMoeMaxSlots];
    uint8_t tokens[kMoeMaxSlots];          // slots of the expert
    uint8_t slot[kMoeMaxSlots][16];
    uint8_t token_of[kMoeMaxSlots];        // of a slot
    int ids[kMoeMaxSlots];
    float wts[kMoeMaxSlots];
    unsigned mask[1024];                   // tokens of every expert
    uint16_t at[1024];                     // its place among the chosen
};

// From L.ids (filled, synchronized) by all threads of the CTA.
__device__ void build_lists(const dg_moe& op, Lists& L) {
    const int tid = threadIdx.x, slots = op.M * op.top_k;
    for (int e = tid; e < op.E; e += blockDim.x) L.mask[e] = 0;
    __syncthreads();
    for (int s = tid; s < slots; s += blockDim.x) {
        const int m = s / op.top_k;
        L.token_of[s] = (uint8_t)m;
        atomicOr(&L.mask[L.ids[s]], 1u << m);
    }
    __syncthreads();
    if (tid < 32) {
        int n = 0;
        for (int e0 = 0; e0 < op.E; e0 += 32) {
            const int e = e0 + tid;
            const unsigned mk = e < op.E ? L.mask[e] : 0u;
            const unsigned b = __ballot_sync(0xffffffffu, mk != 0);
            if (mk) {
                const int at = n + __popc(b & ((1u << tid) - 1));
                L.expert[at] = (uint16_t)e;
                L.tokens[at] = (uint8_t)__popc(mk);
                L.at[e] = (uint16_t)at;
            }
            n += __popc(b);
        }
        if (tid == 0) L.count = n;
    }
    __syncthreads();
    for (int s = tid; s < slots; s += blockDim.x) {
        const int e = L.ids[s], m = L.token_of[s];
        L.slot[L.at[e]][__popc(L.mask[e] & ((1u << m) - 1))] = (uint8_t)s;
    }
    __syncthreads();
}

// ---- weight chunks --------------------------------------------------------------------------

// Four fp16 pairs from eight int4 codes: (0, 4), (1, 5), (2, 6), (3, 7).
// 0x6400 + u is the fp16 number 1024 + u; the code's sign bit is flipped, so u
// = q + 8.
__device__ __forceinline__ void int4_pairs(uint32_t w, uint32_t (&v)[4]) {
    const uint32_t h = w >> 8;
    const __half2 k1032 = __float2half2_rn(1032.f), k16 = __float2half2_rn(0.0625f),
                  k72 = __float2half2_rn(-72.f);
    v[0] = h2_as_u32(__hsub2(u32_as_h2(and_xor(w, 0x000F000Fu, 0x64086408u)), k1032));
    v[1] = h2_as_u32(__hfma2(u32_as_h2(and_xor(w, 0x00F000F0u, 0x64806480u)), k16, k72));
    v[2] = h2_as_u32(__hsub2(u32_as_h2(and_xor(h, 0x000F000Fu, 0x64086408u)), k1032));
    v[3] = h2_as_u32(__hfma2(u32_as_h2(and_xor(h, 0x00F000F0u, 0x64806480u)), k16, k72));
}

// A chunk is 16 rows x kCols columns in kSteps steps of kStep; a lane (g =
// lane / 4, t = lane % 4) holds kLane columns of rows g and g + 8 per step,
// from column t * kLane of the step on.  PH: phases of int4 (1 for 16-bit).
template <int KIND, int PH>
struct Shape {
    static constexpr bool kInt4 = KIND == DG_LINEAR_W4A16;
    static constexpr int kLane = kInt4 ? (PH == 4 ? 32 : 16) : 8;
    static constexpr int kStep = 4 * kLane;
    static constexpr int kCols = kInt4 ? 512 : 256;
    static constexpr int kSteps = kCols / kStep;
    static constexpr int kWords = kInt4 ? kLane / 8 : 4;   // 32-bit registers of a row and step
    static constexpr int kTokens = 8 / PH;                 // token rows of 8 columns
};

// Rows g and g + 8 of a row tile at this lane's first column, and their scales.
struct Src {
    const char* w[2];
    const uint16_t* s[2];
    int k0;   // first column of the chunk
};

template <int KIND, int PH>
struct Chunk {
    using S = Shape<KIND, PH>;
    uint32_t v[S::kSteps][2][S::kWords];
    uint32_t sc[S::kInt4 ? S::kSteps : 1][2];   // this thread's two columns' scales

    __device__ __forceinline__ void load_step(const MoeParams& p, const Src& q, int i, int Kd) {
        const int t = threadIdx.x & 3;
        const bool in = q.k0 + i * S::kStep + t * S::kLane < Kd;
        const size_t at = S::kInt4 ? (q.k0 + i * S::kStep) / 2 : (size_t)(q.k0 + i * S::kStep) * 2;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (S::kWords == 4) {
                const uint4 x = in ? ld_stream16(q.w[r] + at) : make_uint4(0, 0, 0, 0);
                v[i][r][0] = x.x, v[i][r][1] = x.y;
                v[i][r][S::kWords - 2] = x.z, v[i][r][S::kWords - 1] = x.w;
            } else {
                uint2 x = make_uint2(0, 0);
                if (in)
                    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                                 : "=r"(x.x), "=r"(x.y)
                                 : "l"(q.w[r] + at));
                v[i][r][0] = x.x, v[i][r][1] = x.y;
            }
            if (S::kInt4) {
                // columns 2 t and 2 t + 1: groups f and f + 1 of the step's PH
                const int grp = (q.k0 + i * S::kStep) / 32 + (PH == 4 ? (t & 1) * 2 : 0);
                uint32_t two = 0;
                if (p.pair_scales) {
                    if (grp * 32 < Kd)
                        asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];"
                                     : "=r"(two)
                                     : "l"(q.s[r] + grp));
                } else {
                    // any group size, count or alignment
                    if (grp * 32 < Kd) two = ld_stream_u16(q.s[r] + grp * 32 / p.op.group_size);
                    if (grp * 32 + 32 < Kd)
                        two |= (uint32_t)ld_stream_u16(q.s[r] + (grp * 32 + 32) / p.op.group_size) << 16;
                }
                sc[i][r] = two;
            }
        }
    }

    __device__ __forceinline__ void load(const MoeParams& p, const Src& q, int Kd) {
#pragma unroll
        for (int i = 0; i < S::kSteps; ++i) load_step(p, q, i, Kd);
    }

    // acc[j] += (16 weight rows) x (token rows j * kTokens ..), the chunk's
    // columns; each step's registers are then reloaded from `next` (if any).
    // x[j]: the token row of this lane's column of block j, from column 0 on.
    template <int NT>
    __device__ __forceinline__ void mma(const MoeParams& p, const uint16_t* const (&x)[NT], int R, int k0,
                                        int Kd, float (&acc)[NT][4], const Src& next, bool more) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const bool mine = PH == 1 || (PH == 2 ? (g & 1) == (t >> 1) : (g & 3) == t);
#pragma unroll
        for (int i = 0; i < S::kSteps; ++i) {
            const int k = k0 + i * S::kStep + t * S::kLane;
            const bool in = mine && k < Kd;
            if (S::kInt4) {
                uint32_t lo[S::kWords][4], hi[S::kWords][4];
#pragma unroll
                for (int w = 0; w < S::kWords; ++w) {
                    int4_pairs(v[i][0][w], lo[w]);
                    int4_pairs(v[i][1][w], hi[w]);
                }
                const float2 f0 = __half22float2(u32_as_h2(sc[i][0])), f1 = __half22float2(u32_as_h2(sc[i][1]));
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    if (j * S::kTokens < R) {
                        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int w = 0; w < S::kWords; ++w) {
                            uint4 b = make_uint4(0, 0, 0, 0);
                            if (in) b = __ldg(reinterpret_cast<const uint4*>(x[j] + k + w * 8));
                            const uint32_t a0[4] = {lo[w][0], hi[w][0], lo[w][1], hi[w][1]};
                            const uint32_t a1[4] = {lo[w][2], hi[w][2], lo[w][3], hi[w][3]};
                            mma16816<false>(c, a0, b.x, b.y);
                            mma16816<false>(c, a1, b.z, b.w);
                        }
                        acc[j][0] = fmaf(f0.x, c[0], acc[j][0]);
                        acc[j][1] = fmaf(f0.y, c[1], acc[j][1]);
                        acc[j][2] = fmaf(f1.x, c[2], acc[j][2]);
                        acc[j][3] = fmaf(f1.y, c[3], acc[j][3]);
                    }
                }
            } else {
                constexpr bool BF = KIND == DG_LINEAR_BF16;
                const uint32_t a0[4] = {v[i][0][0], v[i][1][0], v[i][0][1], v[i][1][1]};
                const uint32_t a1[4] = {v[i][0][S::kWords - 2], v[i][1][S::kWords - 2],
                                        v[i][0][S::kWords - 1], v[i][1][S::kWords - 1]};
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    if (j * S::kTokens < R) {
                        uint4 b = make_uint4(0, 0, 0, 0);
                        if (in) b = __ldg(reinterpret_cast<const uint4*>(x[j] + k));
                        mma16816<BF>(acc[j], a0, b.x, b.y);
                        mma16816<BF>(acc[j], a1, b.z, b.w);
                    }
                }
            }
            if (more) load_step(p, next, i, Kd);
        }
    }

    // The sums of token row n of block j in acc, after all chunks: for 16-bit
    // weights columns 2 t and 2 t + 1 are two tokens; for int4 their phases'
    // sums belong together.  sum(q, h): token row q of this thread's (q < 2 for
    // PH 1, else 0), weight row g + 8 h.
    __device__ __forceinline__ static float sum(const float (&a)[4], int q, int h) {
        if (PH == 1) return a[2 * h + q];
        const float two = a[2 * h] + a[2 * h + 1];
        return PH == 2 ? two : two + __shfl_xor_sync(0xffffffffu, two, 1);
    }
};

// The token row behind column g of block j (what a lane loads), and behind
// this thread's accumulators.
template <int PH>
__device__ __forceinline__ int column_row(int j) {
    return j * (8 / PH) + ((threadIdx.x & 31) >> 2) / PH;
}

// ---- gate and up ----------------------------------------------------------------------------

template <int KIND>
__device__ __forceinline__ size_t row_bytes_of(int cols) {
    return KIND == DG_LINEAR_W4A16 ? (size_t)cols / 2 : (size_t)cols * 2;
}

template <int KIND, int PH, int NT>
__global__ void __launch_bounds__(kMoeWarps * 32, NT >= 8 ? 1 : 2) k_moe_up(const MoeParams p) {
    using S = Shape<KIND, PH>;
    constexpr bool BF = KIND == DG_LINEAR_BF16;
    constexpr int kTok = NT * S::kTokens;   // token rows of the accumulators
    extern __shared__ __align__(16) float dyn[];
    __shared__ Lists L;
    const dg_moe& op = p.op;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    griddep_launch_dependents();
    griddep_wait();
    for (int m = warp; m < op.M; m += kMoeWarps)
        route_token(op, p.ws.scores + (size_t)m * op.E, dyn + (size_t)warp * op.E, L.ids + m * op.top_k,
                    L.wts + m * op.top_k);
    __syncthreads();
    build_lists(op, L);
    if (blockIdx.x == 0)
        for (int s = tid; s < op.M * op.top_k; s += blockDim.x) {
            p.ws.ids[s] = L.ids[s];
            p.ws.wts[s] = L.wts[s];
            if (op.ids) op.ids[s] = L.ids[s];
            if (op.weights) op.weights[s] = L.wts[s];
        }

    // the warps' sums of a row tile, [2 tiles in turn][warps][kTok][16 rows]
    float* part = dyn;
    const int tiles = op.I / 8, total = L.count * tiles, n = (op.K + S::kCols - 1) / S::kCols;
    const size_t rb = row_bytes_of<KIND>(op.K);
    const uint16_t* x = S::kInt4 ? p.ws.xp : static_cast<const uint16_t*>(op.x);

    // the next chunk to load: chunk fk of the n of row tile `fi`
    int fi = blockIdx.x, fk = warp;
    auto settle = [&] {
        while (fk >= n) {
            fk -= n;
            fi += gridDim.x;
        }
    };
    Src src{};
    auto find = [&] {
        const int li = fi / tiles, tile = fi - li * tiles;
        const size_t row = (size_t)L.expert[li] * op.I + tile * 8 + g;
        src.k0 = fk * S::kCols;
        src.w[0] = static_cast<const char*>(op.W_gate) + row * rb + (S::kInt4 ? t * S::kLane / 2 : t * S::kLane * 2);
        src.w[1] = static_cast<const char*>(op.W_up) + row * rb + (S::kInt4 ? t * S::kLane / 2 : t * S::kLane * 2);
        if (S::kInt4) {
            const size_t at = row * (op.K / op.group_size);
            src.s[0] = static_cast<const uint16_t*>(op.gate_scale) + at;
            src.s[1] = static_cast<const uint16_t*>(op.up_scale) + at;
        }
    };
    Chunk<KIND, PH> ch;
    settle();
    if (fi < total) {
        find();
        ch.load(p, src, op.K);
    }
    int k = warp, turn = 0;
    for (int item = blockIdx.x; item < total; item += gridDim.x) {
        const int li = item / tiles, tile = item - li * tiles, R = L.tokens[li];
        const uint16_t* xr[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
            xr[j] = x + (size_t)L.token_of[L.slot[li][min(column_row<PH>(j), R - 1)]] * op.K;
        float acc[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
        for (; k < n; k += kMoeWarps) {
            fk += kMoeWarps;
            settle();
            const bool more = fi < total;
            if (more) find();
            ch.mma(p, xr, R, k * S::kCols, op.K, acc, src, more);
        }
        k -= n;
        float* mine = part + (size_t)(turn * kMoeWarps + warp) * kTok * 16;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (PH == 1) {
                    mine[(j * 8 + t * 2) * 16 + g + 8 * h] = ch.sum(acc[j], 0, h);
                    mine[(j * 8 + t * 2 + 1) * 16 + g + 8 * h] = ch.sum(acc[j], 1, h);
                } else {
                    const float v = ch.sum(acc[j], 0, h);
                    if (PH == 2 || (t & 1) == 0)
                        mine[(j * S::kTokens + (PH == 2 ? t : t >> 1)) * 16 + g + 8 * h] = v;
                }
            }
        __syncthreads();
        for (int i = tid; i < R * 8; i += kMoeWarps * 32) {
            const int tok = i >> 3, r = i & 7;
            const float* q = part + (size_t)turn * kMoeWarps * kTok * 16 + tok * 16 + r;
            float gate = 0.f, up = 0.f;
#pragma unroll
            for (int w = 0; w < kMoeWarps; ++w) {
                gate += q[w * kTok * 16];
                up += q[w * kTok * 16 + 8];
            }
            const float v = silu_f32(gate) * up;
            uint16_t* h = p.ws.h + (size_t)L.slot[li][tok] * 2 * op.I + tile * 8 +
                          (S::kInt4 ? int4_place(r) : r);
            const float s = BF ? v : v * 0.00390625f;
            const uint16_t hi = elem_16<BF>(s);
            h[0] = hi;
            h[op.I] = elem_16<BF>((s - elem_f32<BF>(hi)) * (BF ? 1.f : 2048.f));
        }
        turn ^= 1;
    }
}

// ---- down and the weighted sum ----------------------------------------------------------------

template <int KIND, int PH, int NT>
__global__ void __launch_bounds__(kMoeWarps * 32, NT >= 8 ? 1 : 2) k_moe_down(const MoeParams p) {
    using S = Shape<KIND, PH>;
    constexpr bool BF = KIND == DG_LINEAR_BF16;
    extern __shared__ __align__(16) float dyn[];
    __shared__ Lists L;
    const dg_moe& op = p.op;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int M = op.M, tiles = (op.K + 15) / 16, n = (op.I + S::kCols - 1) / S::kCols;
    float* sums = dyn;   // [warps][M][16]
    griddep_launch_dependents();
    for (int i = tid; i < kMoeWarps * 16 * M; i += blockDim.x) sums[i] = 0.f;
    griddep_wait();
    for (int s = tid; s < M * op.top_k; s += blockDim.x) {
        L.ids[s] = __ldcg(p.ws.ids + s);
        L.wts[s] = __ldcg(p.ws.wts + s);
    }
    __syncthreads();
    build_lists(op, L);
    const size_t rb = row_bytes_of<KIND>(op.I);
    float* mine = sums + warp * 16 * M;

    // the next chunk to load: chunk fk of the n of expert fl in row tile ft
    int ft = blockIdx.x, fl = 0, fk = warp;
    auto settle = [&] {
        while (fk >= n) {
            fk -= n;
            if (++fl == L.count) {
                fl = 0;
                ft += gridDim.x;
            }
        }
    };
    Src src{};
    auto find = [&] {
        // op.K is a multiple of 8: a last tile may lack its second half
        const size_t row = (size_t)L.expert[fl] * op.K + ft * 16 + g;
        const int half = ft * 16 + 8 < op.K ? 8 : 0;
        src.k0 = fk * S::kCols;
        src.w[0] = static_cast<const char*>(op.W_down) + row * rb + (S::kInt4 ? t * S::kLane / 2 : t * S::kLane * 2);
        src.w[1] = src.w[0] + half * rb;
        if (S::kInt4) {
            const int srow = op.I / op.group_size;
            src.s[0] = static_cast<const uint16_t*>(op.down_scale) + row * srow;
            src.s[1] = src.s[0] + half * srow;
        }
    };
    Chunk<KIND, PH> ch;
    settle();
    if (ft < tiles) {
        find();
        ch.load(p, src, op.I);
    }
    int k = warp;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        for (int li = 0; li < L.count; ++li) {
            if (k >= n) {   // nothing of this expert is this warp's
                k -= n;
                continue;
            }
            const int R = 2 * L.tokens[li];
            const uint16_t* xr[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int r = min(column_row<PH>(j), R - 1);
                xr[j] = p.ws.h + ((size_t)L.slot[li][r >> 1] * 2 + (r & 1)) * op.I;
            }
            float acc[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
            for (; k < n; k += kMoeWarps) {
                fk += kMoeWarps;
                settle();
                const bool more = ft < tiles;
                if (more) find();
                ch.mma(p, xr, R, k * S::kCols, op.I, acc, src, more);
            }
            k -= n;
            // token rows 2 i and 2 i + 1 are hi and lo of the expert's token i
#pragma unroll
            for (int j = 0; j < NT; ++j) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float hi, lo;
                    int i;
                    if (PH == 1) {
                        hi = ch.sum(acc[j], 0, h), lo = ch.sum(acc[j], 1, h);
                        i = j * 4 + t;
                    } else {
                        const int over = PH == 2 ? 1 : 2;   // the lane with the next token row
                        hi = ch.sum(acc[j], 0, h);
                        lo = __shfl_xor_sync(0xffffffffu, hi, over);
                        i = PH == 2 ? ((t & 1) ? 16 : j * 2 + (t >> 1)) : (t ? 16 : j);
                    }
                    if (2 * i < R) {
                        const int s = L.slot[li][i];
                        const float v = BF ? hi + lo : fmaf(lo, 1.f / 2048.f, hi) * 256.f;
                        float* to = mine + L.token_of[s] * 16 + g + 8 * h;
                        *to = fmaf(L.wts[s], v, *to);
                    }
                }
            }
        }
        __syncthreads();
        for (int i = tid; i < 16 * M; i += blockDim.x) {
            const int m = i >> 4, row = tile * 16 + (i & 15);
            float y = 0.f;
#pragma unroll
            for (int w = 0; w < kMoeWarps; ++w) {
                y += sums[w * 16 * M + i];
                sums[w * 16 * M + i] = 0.f;
            }
            if (row >= op.K) continue;
            const size_t at = (size_t)m * op.K + row;
            if (op.residual) y += elem_f32<BF>(static_cast<const uint16_t*>(op.residual)[at]);
            static_cast<uint16_t*>(op.y)[at] = elem_16<BF>(y);
        }
        __syncthreads();
    }
}

// ---- host side --------------------------------------------------------------------------------

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

static size_t place(const dg_moe& op, void* base, MoeWs* w) {
    char* b = static_cast<char*>(base);
    size_t at = 0;
    auto take = [&](size_t n) {
        char* r = b + at;
        at += up256(n);
        return r;
    };
    w->scores = reinterpret_cast<float*>(take((size_t)op.M * op.E * 4));
    w->ids = reinterpret_cast<int*>(take(kMoeMaxSlots * 4));
    w->wts = reinterpret_cast<float*>(take(kMoeMaxSlots * 4));
    w->xp = reinterpret_cast<uint16_t*>(take(op.kind == DG_LINEAR_W4A16 ? (size_t)op.M * op.K * 2 : 0));
    w->h = reinterpret_cast<uint16_t*>(take((size_t)op.M * op.top_k * 2 * op.I * 2));
    return at;
}

size_t moe_ws_bytes(const dg_moe& op) {
    MoeWs w;
    return place(op, nullptr, &w);
}

// Kernels of each format by their token blocks: NT blocks of 8 / PH token rows.
template <int KIND>
static const void* up_kernel(int M) {
    if constexpr (KIND == DG_LINEAR_W4A16) {
        if (M == 1) return (const void*)k_moe_up<KIND, 4, 1>;
        return M <= 4   ? (const void*)k_moe_up<KIND, 2, 1>
               : M <= 8 ? (const void*)k_moe_up<KIND, 2, 2> : (const void*)k_moe_up<KIND, 2, 4>;
    } else {
        return M <= 8 ? (const void*)k_moe_up<KIND, 1, 1> : (const void*)k_moe_up<KIND, 1, 2>;
    }
}
template <int KIND>
static const void* down_kernel(int M) {
    if constexpr (KIND == DG_LINEAR_W4A16) {
        if (M == 1) return (const void*)k_moe_down<KIND, 4, 1>;
        return M <= 2   ? (const void*)k_moe_down<KIND, 2, 1>
               : M <= 4 ? (const void*)k_moe_down<KIND, 2, 2>
               : M <= 8 ? (const void*)k_moe_down<KIND, 2, 4> : (const void*)k_moe_down<KIND, 2, 8>;
    } else {
        return M <= 4   ? (const void*)k_moe_down<KIND, 1, 1>
               : M <= 8 ? (const void*)k_moe_down<KIND, 1, 2> : (const void*)k_moe_down<KIND, 1, 4>;
    }
}

template <int KIND>
static cudaError_t launch_moe_kind(const dg_moe& op, void* ws, cudaStream_t s) {
    MoeParams p;
    p.op = op;
    place(op, ws, &p.ws);
    const bool g32 = KIND == DG_LINEAR_W4A16 && op.group_size == 32;
    auto al4 = [](const void* q) { return ((uintptr_t)q & 3u) == 0; };
    void* args[] = {&p};
    p.pair_scales = 0;
    cudaError_t e = launch_pdl((const void*)k_moe_scores<KIND == DG_LINEAR_BF16>,
                               dim3(op.E, (op.M + kScoreTokens - 1) / kScoreTokens), dim3(256), 0, s, args);
    if (e != cudaSuccess) return e;

    // two CTAs per SM
    p.pair_scales = g32 && op.K % 64 == 0 && al4(op.gate_scale) && al4(op.up_scale);
    const int tok = op.M <= 8 ? 8 : 16;
    size_t smem = (size_t)2 * kMoeWarps * tok * 16 * 4;
    if (smem < (size_t)kMoeWarps * op.E * 4) smem = (size_t)kMoeWarps * op.E * 4;
    const void* fn = up_kernel<KIND>(op.M);
    if ((e = tc::smem_attr_once(fn, smem)) != cudaSuccess) return e;
    const int ctas = 2 * sm_count();
    if ((e = launch_pdl(fn, dim3(ctas), dim3(kMoeWarps * 32), smem, s, args)) != cudaSuccess) return e;

    p.pair_scales = g32 && op.I % 64 == 0 && al4(op.down_scale);
    const int tiles = (op.K + 15) / 16;
    return launch_pdl(down_kernel<KIND>(op.M), dim3(tiles < ctas ? tiles : ctas), dim3(kMoeWarps * 32),
                      (size_t)kMoeWarps * 16 * op.M * 4, s, args);
}

cudaError_t launch_moe(const dg_moe& op, void* ws, cudaStream_t s) {
    switch (op.kind) {
        case DG_LINEAR_F16: return launch_moe_kind<DG_LINEAR_F16>(op, ws, s);
        case DG_LINEAR_BF16: return launch_moe_kind<DG_LINEAR_BF16>(op, ws, s);
        default: return launch_moe_kind<DG_LINEAR_W4A16>(op, ws, s);
    }
}

}  // namespace dg
