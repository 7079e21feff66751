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
// values follow it.  A warp loads one chunk (16 rows x 128 columns, 4 KB at 16
// bits) with its tokens' values at once, then computes it; what keeps HBM busy
// meanwhile are the SM's other warps (32 where registers allow).  A copy of
// 1 GB in this pattern reads 6.7 TB/s with 32 warps of 4 KB per SM and 6.0 with
// 16 of 8 KB; rows brought by the bulk copy engine (256 or 512 bytes each)
// reached 2.9, cp.async rings of 8 warps 4.6.
//
//   up:   one, two, four or eight warps take 8 gate and the same 8 up rows of
//         an expert at a time, so that silu(gate) * up meets in one thread;
//         they deal the row tile's chunks along K among themselves and their
//         sums are added in warp order.
//   down: a CTA takes 16 output rows at a time; its warps deal the chunks of
//         all chosen experts, each adding weight * sum into its own fp32 rows
//         [token], which are summed in warp order.
//
// h goes from one to the other as two 16-bit values, hi + lo, that are two
// columns of the matrix instruction: fp16 hi = h / 256 and lo = the rest x 2048
// (22 bits from 2^-6 to 2^24; below, where hi is subnormal, steps of 2^-27, an
// eighth of an fp16 output's finest), bf16 hi and lo (16 bits); the products keep
// fp32 sums.  int4 codes become fp16 by bit operations (exact).  A group of 32
// codes must be summed on its own before its scale, but a quad's lanes hold
// parts of several groups (PH = 2 of 8-byte pieces, or 4 of 16-byte ones): each
// token gets PH columns, column f carrying the token's values for the lanes
// whose codes belong to group f and zero for the others, so that one
// instruction sums the groups apart.
//
// Measured: 16 tokens, 4096 x 14336 bf16, 2 of 8 experts: 436 to 449 us, 6.2 to 6.4
// TB/s; one token, fp16 (101 MB): 28.4 us, 3.6 TB/s, of which the scores and the routing at
// the head of `up` take 6; int4, one token, 4096 x 14336, 2 of 8: 57 us, 3.5
// TB/s, bound by unpacking and by the latency of 16 warps' chunks.
#include <algorithm>

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
    int scale_pairs;    // int4: groups of 32 whose scales can be loaded two at a time
    FastDiv group_32s;  // int4: group_size / 32
    int split;          // up: warps sharing a row tile's columns (1, 2, 4 or 8)
    int stage;          // byte of dynamic shared memory where the warps' token rows are staged
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
        const int n8 = op.M * K8, first = e * 256 + tid, stride = gridDim.x * 256;
        uint4* xp = reinterpret_cast<uint4*>(p.ws.xp);
        for (int i = first; i < n8; i += stride) {
            const uint4 v = __ldcg(x + i);
            xp[i] = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                               __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
        }
    }
}

// ---- routing ------------------------------------------------------------------------------

// One warp: a token's probabilities from its scores, its top_k experts and
// their weights.  Selection compares integers: 0 nothing, 1 NaN, otherwise the
// probability's bits + 2 (it is not negative).  A lane keeps the experts lane,
// lane + 32, .. of up to 256 in registers, more in `more` (E words of shared
// memory).
__device__ __forceinline__ unsigned route_key(float v) { return v != v ? 1u : __float_as_uint(v) + 2u; }
__device__ void route_token(const dg_moe& op, const float* scores, unsigned* more, int* ids, float* wts) {
    constexpr int kReg = 8;
    const int lane = threadIdx.x & 31, E = op.E;
    float v[kReg];
    unsigned key[kReg];
#pragma unroll
    for (int j = 0; j < kReg; ++j) v[j] = lane + 32 * j < E ? __ldcg(scores + lane + 32 * j) : -INFINITY;
    if (op.score == DG_MOE_SOFTMAX) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int j = 0; j < kReg; ++j) top = fmaxf(top, v[j]);
        for (int e = lane + 32 * kReg; e < E; e += 32) top = fmaxf(top, __ldcg(scores + e));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
        for (int j = 0; j < kReg; ++j) {
            v[j] = lane + 32 * j < E ? expf(v[j] - top) : 0.f;
            sum += v[j];
        }
        for (int e = lane + 32 * kReg; e < E; e += 32) sum += expf(__ldcg(scores + e) - top);
        sum = warp_sum(sum);
#pragma unroll
        for (int j = 0; j < kReg; ++j) key[j] = lane + 32 * j < E ? route_key(v[j] / sum) : 0u;
        for (int e = lane + 32 * kReg; e < E; e += 32) more[e] = route_key(expf(__ldcg(scores + e) - top) / sum);
    } else {
#pragma unroll
        for (int j = 0; j < kReg; ++j) key[j] = lane + 32 * j < E ? route_key(1.f / (1.f + expf(-v[j]))) : 0u;
        for (int e = lane + 32 * kReg; e < E; e += 32) more[e] = route_key(1.f / (1.f + expf(-__ldcg(scores + e))));
    }
    float mine = 0.f, total = 0.f;   // lane c holds choice c
    int id = 0;
    for (int c = 0; c < op.top_k; ++c) {
        unsigned best = 0;
        int at = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < kReg; ++j)
            if (key[j] > best) {
                best = key[j];
                at = lane + 32 * j;
            }
        for (int e = lane + 32 * kReg; e < E; e += 32)
            if (more[e] > best) {
                best = more[e];
                at = e;
            }
        const unsigned top = __reduce_max_sync(0xffffffffu, best);
        const int e = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7fffffff);
        if (at == e) {   // this lane's: taken
#pragma unroll
            for (int j = 0; j < kReg; ++j)
                if (e == lane + 32 * j) key[j] = 0;
            if (e >= 32 * kReg) more[e] = 0;
        }
        const float prob = top == 1u ? NAN : __uint_as_float(top - 2u);
        if (lane == c) {
            mine = prob;
            id = e;
        }
        total += prob;
    }
    if (lane < op.top_k) {
        ids[lane] = id;
        wts[lane] = (op.renormalize ? mine / total : mine) * op.route_scale;
    }
}

// The chosen experts in ascending order and each one's slots (token * top_k +
// choice) in token order.  An expert of more tokens than the kernel takes at a
// time (CAP) is listed twice.
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
template <int CAP>
__device__ void build_lists(const dg_moe& op, Lists& L) {
    static_assert(CAP >= 8, "16 tokens make two parts at most");
    const int tid = threadIdx.x, slots = op.M * op.top_k;
    if (slots <= 32) {   // one warp's lanes: a slot each
        if (tid < 32) {
            const int e = tid < slots ? L.ids[tid] : -1 - tid;
            const unsigned same = __match_any_sync(0xffffffffu, e);
            const int rank = __popc(same & ((1u << tid) - 1)), key = e * 2 + rank / CAP;
            const bool first = e >= 0 && rank % CAP == 0;
            const unsigned firsts = __ballot_sync(0xffffffffu, first);
            int at = 0;
            for (unsigned f = firsts; f; f &= f - 1) at += __shfl_sync(0xffffffffu, key, __ffs(f) - 1) < key;
            if (e >= 0) {
                L.token_of[tid] = (uint8_t)(tid / op.top_k);
                L.slot[at][rank % CAP] = (uint8_t)tid;
                if (first) {
                    L.expert[at] = (uint16_t)e;
                    L.tokens[at] = (uint8_t)min(__popc(same) - rank, CAP);
                }
            }
            if (tid == 0) L.count = __popc(firsts);
        }
        __syncthreads();
        return;
    }
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
            const int e = e0 + tid, tokens = e < op.E ? __popc(L.mask[e]) : 0;
            const unsigned one = __ballot_sync(0xffffffffu, tokens > 0), two = __ballot_sync(0xffffffffu, tokens > CAP);
            if (tokens) {
                const unsigned below = (1u << tid) - 1;
                const int at = n + __popc(one & below) + __popc(two & below);
                L.at[e] = (uint16_t)at;
                L.expert[at] = (uint16_t)e;
                L.tokens[at] = (uint8_t)min(tokens, CAP);
                if (tokens > CAP) {
                    L.expert[at + 1] = (uint16_t)e;
                    L.tokens[at + 1] = (uint8_t)(tokens - CAP);
                }
            }
            n += __popc(one) + __popc(two);
        }
        if (tid == 0) L.count = n;
    }
    __syncthreads();
    for (int s = tid; s < slots; s += blockDim.x) {
        const int e = L.ids[s], m = L.token_of[s], rank = __popc(L.mask[e] & ((1u << m) - 1));
        L.slot[L.at[e] + rank / CAP][rank % CAP] = (uint8_t)s;
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
    static constexpr int kCols = PH == 4 ? 512 : kInt4 ? 256 : 128;
    static constexpr int kSteps = kCols / kStep;
    static constexpr int kWords = kInt4 ? kLane / 8 : 4;   // 32-bit registers of a row and step
    static constexpr int kTokens = 8 / PH;                 // token rows of 8 columns
    static constexpr int kGroups = kCols / 128;            // int4: scale groups of a lane and row
    static constexpr bool kStaged = PH == 2;               // token rows through shared memory
    static constexpr int kPitch = kCols * 2;               // bytes of a staged token row
};

// Streaming loads; the predicated forms give zero where `in` is false.  WIDE asks
// L2 for the whole 256 bytes: better for long streams (16 tokens, 2.8 GB bf16: 436 to
// 449 us, 450 to 461 without; one token, 198 MB int4: 56.8, 57.6; 4 tokens, 310 MB
// int4: 91 both), worse for the short ones of one block of tokens at 16 bits (one
// token, 101 MB: 29.4, 28.6 without).
template <bool WIDE>
__device__ __forceinline__ void ld_weights16(uint32_t (&v)[4], const void* p) {
    if (WIDE)
        asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "l"(p));
    else
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "l"(p));
}
__device__ __forceinline__ void ld_weights(uint32_t (&v)[2], const void* p) {
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p));
}
__device__ __forceinline__ void ld_weights(uint32_t& v, const void* p) {
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
}
__device__ __forceinline__ void ld_weights(uint32_t (&v)[4], const void* p, bool in) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
        "mov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "=&r"(v[0]), "=&r"(v[1]), "=&r"(v[2]), "=&r"(v[3])
        : "l"(p), "r"((int)in));
}
__device__ __forceinline__ void ld_weights(uint32_t (&v)[2], const void* p, bool in) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];\n\t}"
        : "=&r"(v[0]), "=&r"(v[1])
        : "l"(p), "r"((int)in));
}
__device__ __forceinline__ void ld_weights(uint32_t& v, const void* p, bool in) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.u32 %0, [%1];\n\t}"
        : "=&r"(v)
        : "l"(p), "r"((int)in));
}
// Eight values of a token row (kept in L1: other row tiles want them too).  The
// kernel before wrote them, perhaps while this one had already started: no
// read-only loads.
__device__ __forceinline__ uint4 ld_token(const uint16_t* p, bool in) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
        "mov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t@p ld.global.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((int)in));
    return v;
}

// The same, leaving v as it is where `in` is false.
__device__ __forceinline__ void ld_token_keep(uint4& v, const uint16_t* p, bool in) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p ld.global.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "l"(p), "r"((int)in));
}
// Eight values from shared memory, likewise.
__device__ __forceinline__ void lds_token_keep(uint4& v, uint32_t at, bool in) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
                 : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
                 : "r"(at), "r"((int)in));
}

// Rows g and g + 8 of a row tile at this lane's first column, and their scales.
struct Src {
    const char* w[2];
    const uint16_t* s[2];
};

// The token row behind column g of block j.
template <int PH>
__device__ __forceinline__ int column_row(int j) {
    return j * (8 / PH) + ((threadIdx.x & 31) >> 2) / PH;
}

template <int KIND, int PH>
struct Chunk {
    using S = Shape<KIND, PH>;

    // acc[j] += (16 weight rows) x (token rows j * kTokens ..), columns [k0,
    // k0 + kCols) of Kd.  x[j]: the token row of this lane's column of block j.
    // Two phases (experts of three tokens or more) have the warp copy the chunk of
    // their R token rows row(r) to shared memory at xs beside the weight loads,
    // so that they are not fetched step by step (16 tokens, 4096 x 2048, 2 of 8
    // experts: 93 -> 82 us); one or two rows are faster from L1 (one token, 4096
    // x 14336, 2 of 8: 56 us, staged 66).
    // FULL: all of the chunk's columns exist and int4 scales come in pairs.
    template <bool FULL, int NT, class Row>
    __device__ __forceinline__ static void add_cols(const MoeParams& p, const Src& q, const uint16_t* const (&x)[NT],
                                                    const Row& row, uint32_t xs, int R, int k0, int Kd,
                                                    float (&acc)[NT][4]) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        uint32_t v[S::kSteps][2][S::kWords], sc[2][2];
        if constexpr (S::kStaged) {
            __syncwarp();   // the last chunk's values have been read
            for (int r = 0; r < R; ++r) {
                const uint16_t* from = row(r) + k0;
#pragma unroll
                for (int c = lane * 8; c < S::kCols; c += 256)
                    cp_async16(xs + r * S::kPitch + c * 2, from + (FULL || k0 + c < Kd ? c : 0), FULL || k0 + c < Kd);
            }
            cp_commit();
        }
        const size_t at = S::kInt4 ? k0 / 2 : (size_t)k0 * 2;
#pragma unroll
        for (int r = 0; r < 2; ++r) {   // a row's 256 bytes one after the other: whole lines
#pragma unroll
            for (int i = 0; i < S::kSteps; ++i) {
                const bool in = k0 + i * S::kStep + t * S::kLane < Kd;
                const char* w = q.w[r] + at + (S::kInt4 ? i * S::kStep / 2 : i * S::kStep * 2);
                if constexpr (!FULL)
                    ld_weights(v[i][r], w, in);
                else if constexpr (S::kWords == 4)
                    ld_weights16<S::kInt4 || (NT > 1)>(v[i][r], w);
                else
                    ld_weights(v[i][r], w);
            }
        }
        if constexpr (S::kInt4) {
            // the chunk's scales of a row, in order over the quad's lanes: lane t
            // holds groups t * kGroups .. + kGroups - 1 of the chunk
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int w = 0; w < S::kGroups / 2; ++w) {
                    const int j = k0 / 32 + t * S::kGroups + 2 * w;   // which 32 columns
                    if (FULL) {
                        ld_weights(sc[r][w], q.s[r] + j);
                    } else if (p.scale_pairs) {
                        ld_weights(sc[r][w], q.s[r] + j, j * 32 < Kd);
                    } else {   // any group size, count or alignment
                        uint32_t two = 0;
                        if (j * 32 < Kd) two = ld_stream_u16(q.s[r] + j / p.group_32s);
                        if (j * 32 + 32 < Kd) two |= (uint32_t)ld_stream_u16(q.s[r] + (j + 1) / p.group_32s) << 16;
                        sc[r][w] = two;
                    }
                }
        }
        if constexpr (S::kInt4) {
            if constexpr (S::kStaged) {
                cp_wait<0>();
                __syncwarp();
            }
            // columns of other groups than this lane's codes are zero
            const bool mine = PH == 2 ? (g & 1) == (t >> 1) : (g & 3) == t;
            uint32_t xl[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) xl[j] = xs + min(column_row<PH>(j), R - 1) * S::kPitch + t * S::kLane * 2;
            uint4 b[2][S::kWords];   // stays zero in lanes that load nothing
#pragma unroll
            for (int w = 0; w < 2 * S::kWords; ++w) b[w / S::kWords][w % S::kWords] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < S::kSteps; ++i) {
                const int k = k0 + i * S::kStep + t * S::kLane;
                float c[NT][4];
#pragma unroll
                for (int j = 0; j < NT; ++j) c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.f;
#pragma unroll
                for (int w = 0; w < S::kWords; ++w) {
                    uint32_t lo[4], hi[4];
                    int4_pairs(v[i][0][w], lo);
                    int4_pairs(v[i][1][w], hi);
                    const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]};
                    const uint32_t a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        if (j == 0 || j * S::kTokens < R) {
                            uint4& q = b[NT == 1 ? i & 1 : j & 1][w];
                            if (S::kStaged)
                                lds_token_keep(q, xl[j] + (i * S::kStep + w * 8) * 2, mine);
                            else if (FULL)
                                ld_token_keep(q, x[j] + k + w * 8, mine);
                            else
                                q = ld_token(x[j] + k + w * 8, mine && k < Kd);
                            mma16816<false>(c[j], a0, q.x, q.y);
                            mma16816<false>(c[j], a1, q.z, q.w);
                        }
                    }
                }
                // columns 2 t and 2 t + 1: groups f and f + 1 of the step's PH
                float2 f[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint32_t two;
                    if (PH == 4) {   // step i's four groups are lane i's
                        const uint32_t lo = __shfl_sync(0xffffffffu, sc[r][0], i, 4);
                        const uint32_t hi = __shfl_sync(0xffffffffu, sc[r][1], i, 4);
                        two = (t & 1) ? hi : lo;
                    } else {         // step i's two groups are lane i's
                        two = __shfl_sync(0xffffffffu, sc[r][0], i, 4);
                    }
                    f[r] = __half22float2(u32_as_h2(two));
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    acc[j][0] = fmaf(f[0].x, c[j][0], acc[j][0]);
                    acc[j][1] = fmaf(f[0].y, c[j][1], acc[j][1]);
                    acc[j][2] = fmaf(f[1].x, c[j][2], acc[j][2]);
                    acc[j][3] = fmaf(f[1].y, c[j][3], acc[j][3]);
                }
            }
        } else {
            constexpr bool BF = KIND == DG_LINEAR_BF16;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j == 0 || j * S::kTokens < R) {
                    uint4 b[S::kSteps];
#pragma unroll
                    for (int i = 0; i < S::kSteps; ++i) {
                        const int k = k0 + i * S::kStep + t * S::kLane;
                        b[i] = FULL ? *reinterpret_cast<const uint4*>(x[j] + k) : ld_token(x[j] + k, k < Kd);
                    }
#pragma unroll
                    for (int i = 0; i < S::kSteps; ++i) {
                        const uint32_t a0[4] = {v[i][0][0], v[i][1][0], v[i][0][1], v[i][1][1]};
                        const uint32_t a1[4] = {v[i][0][2], v[i][1][2], v[i][0][3], v[i][1][3]};
                        mma16816<BF>(acc[j], a0, b[i].x, b[i].y);
                        mma16816<BF>(acc[j], a1, b[i].z, b[i].w);
                    }
                }
            }
        }
    }

    template <int NT, class Row>
    __device__ __forceinline__ static void add(const MoeParams& p, const Src& q, const uint16_t* const (&x)[NT],
                                               const Row& row, uint32_t xs, int R, int k0, int Kd,
                                               float (&acc)[NT][4]) {
        if (k0 + S::kCols <= Kd && (!S::kInt4 || p.scale_pairs))
            add_cols<true>(p, q, x, row, xs, R, k0, Kd, acc);
        else
            add_cols<false>(p, q, x, row, xs, R, k0, Kd, acc);
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

// Warps per SM that the kernels' registers are held to.  NT 0 (int4, one token):
// four phases only.
__host__ __device__ constexpr int moe_warps(int KIND, int NT) {
    return KIND == DG_LINEAR_W4A16 ? 16 : NT <= 1 ? 32 : NT == 2 ? 24 : 16;
}

// Bytes of a warp's staged token rows.
__host__ __device__ constexpr int moe_stage(int KIND, int NT) {
    return KIND == DG_LINEAR_W4A16 ? NT * Shape<DG_LINEAR_W4A16, 2>::kTokens * Shape<DG_LINEAR_W4A16, 2>::kPitch : 0;
}

// ---- gate and up ----------------------------------------------------------------------------

template <int KIND>
__device__ __forceinline__ size_t row_bytes_of(int cols) {
    return KIND == DG_LINEAR_W4A16 ? (size_t)cols / 2 : (size_t)cols * 2;
}

// This warp's chunks k, k + split, .. of row tile `tile` of expert li: its sums
// to mine [token][16 rows].
template <int KIND, int PH, int NT>
__device__ __forceinline__ void up_tile(const MoeParams& p, const Lists& L, int li, int tile, int& k, int split,
                                        uint32_t xs, float* mine) {
    using S = Shape<KIND, PH>;
    using C = Chunk<KIND, PH>;
    const dg_moe& op = p.op;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, R = L.tokens[li];
    const int n = (op.K + S::kCols - 1) / S::kCols;
    const size_t row = (size_t)L.expert[li] * op.I + tile * 8 + g;
    const size_t at = row * row_bytes_of<KIND>(op.K) + (S::kInt4 ? t * S::kLane / 2 : t * S::kLane * 2);
    Src src{};
    src.w[0] = static_cast<const char*>(op.W_gate) + at;
    src.w[1] = static_cast<const char*>(op.W_up) + at;
    if (S::kInt4) {
        src.s[0] = static_cast<const uint16_t*>(op.gate_scale) + row * (op.K / op.group_size);
        src.s[1] = static_cast<const uint16_t*>(op.up_scale) + row * (op.K / op.group_size);
    }
    const uint16_t* x = S::kInt4 ? p.ws.xp : static_cast<const uint16_t*>(op.x);
    auto token = [&](int r) { return x + (size_t)L.token_of[L.slot[li][r]] * op.K; };
    const uint16_t* xr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) xr[j] = token(min(column_row<PH>(j), R - 1));
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    for (; k < n; k += split) C::add(p, src, xr, token, xs, R, k * S::kCols, op.K, acc);
    k -= n;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (PH == 1) {
                mine[(j * 8 + t * 2) * 16 + g + 8 * h] = C::sum(acc[j], 0, h);
                mine[(j * 8 + t * 2 + 1) * 16 + g + 8 * h] = C::sum(acc[j], 1, h);
            } else {
                const float v = C::sum(acc[j], 0, h);
                if (PH == 2 || (t & 1) == 0)
                    mine[(j * S::kTokens + (PH == 2 ? t : t >> 1)) * 16 + g + 8 * h] = v;
            }
        }
}

// NT: blocks of eight columns for all of an expert's token rows (int4: two
// phases; experts with one or two token rows take four).
template <int KIND, int NT>
__global__ void __launch_bounds__(kMoeWarps * 32, moe_warps(KIND, NT) / kMoeWarps) k_moe_up(const MoeParams p) {
    constexpr bool BF = KIND == DG_LINEAR_BF16, kInt4 = KIND == DG_LINEAR_W4A16;
    constexpr int kTok = !kInt4 ? NT * 8 : NT ? NT * 4 : 2;   // token rows at a time
    extern __shared__ __align__(16) float dyn[];
    __shared__ Lists L;
    const dg_moe& op = p.op;
    const int tid = threadIdx.x, warp = tid >> 5;
    griddep_launch_dependents();
    griddep_wait();
    for (int m = warp; m < op.M; m += kMoeWarps)
        route_token(op, p.ws.scores + (size_t)m * op.E, reinterpret_cast<unsigned*>(dyn) + (size_t)warp * op.E, L.ids + m * op.top_k,
                    L.wts + m * op.top_k);
    __syncthreads();
    build_lists<kTok < 8 ? 16 : kTok>(op, L);   // fewer than 8: so are the tokens
    if (blockIdx.x == 0)
        for (int s = tid; s < op.M * op.top_k; s += blockDim.x) {
            p.ws.ids[s] = L.ids[s];
            p.ws.wts[s] = L.wts[s];
            if (op.ids) op.ids[s] = L.ids[s];
            if (op.weights) op.weights[s] = L.wts[s];
        }

    // warps [team * split, ..) share a row tile; their sums of it lie in part
    // [2 tiles in turn][kTok][16 rows] of each warp
    const int split = p.split, team = warp / split, first = team * split, teams = kMoeWarps / split;
    constexpr int kPart = kTok * 16;
    float* part = dyn + first * 2 * kPart;
    const uint32_t xs = (uint32_t)__cvta_generic_to_shared(dyn) + p.stage + warp * moe_stage(KIND, NT);
    const int tiles = op.I / 8, total = L.count * tiles;
    int k = warp - first, turn = 0;   // this warp's next chunk of the row tile
    for (int item = blockIdx.x + team * gridDim.x; item < total; item += teams * gridDim.x) {
        const int li = item / tiles, tile = item - li * tiles, R = L.tokens[li];
        float* mine = part + ((warp - first) * 2 + turn) * kPart;
        if constexpr (kInt4) {
            if (R <= 2)
                up_tile<KIND, 4, 1>(p, L, li, tile, k, split, xs, mine);
            else if constexpr (NT > 0)
                up_tile<KIND, 2, NT>(p, L, li, tile, k, split, xs, mine);
        } else {
            up_tile<KIND, 1, NT>(p, L, li, tile, k, split, xs, mine);
        }
        if (split == 1)
            __syncwarp();
        else
            tc::named_sync(1 + team, split * 32);
        for (int i = tid - first * 32; i < R * 8; i += split * 32) {
            const int tok = i >> 3, r = i & 7;
            const float* q = part + turn * kPart + tok * 16 + r;
            float gate = 0.f, up = 0.f;
            for (int w = 0; w < split; ++w) {
                gate += q[w * 2 * kPart];
                up += q[w * 2 * kPart + 8];
            }
            const float v = silu_f32(gate) * up;
            uint16_t* h = p.ws.h + (size_t)L.slot[li][tok] * 2 * op.I + tile * 8 +
                          (kInt4 ? int4_place(r) : r);
            const float s = BF ? v : v * 0.00390625f;
            const uint16_t hi = elem_16<BF>(s);
            const float rest = s - elem_f32<BF>(hi);   // not finite beside a hi that is not
            h[0] = hi;
            h[op.I] = elem_16<BF>(fabsf(rest) < INFINITY ? rest * (BF ? 1.f : 2048.f) : 0.f);
        }
        turn ^= 1;
    }
}

// ---- down and the weighted sum ----------------------------------------------------------------

// This warp's chunks k, k + warps, .. of expert li for output rows tile * 16 ..:
// weight * sum added to mine [token][16 rows].
template <int KIND, int PH, int NT>
__device__ __forceinline__ void down_expert(const MoeParams& p, const Lists& L, int li, int tile, int& k, int warps,
                                            uint32_t xs, float* mine) {
    using S = Shape<KIND, PH>;
    using C = Chunk<KIND, PH>;
    constexpr bool BF = KIND == DG_LINEAR_BF16;
    const dg_moe& op = p.op;
    const int n = (op.I + S::kCols - 1) / S::kCols;
    if (k >= n) {   // nothing of this expert is this warp's
        k -= n;
        return;
    }
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, R = 2 * L.tokens[li];
    // op.K is a multiple of 8: a last tile may lack its second half
    const int half = tile * 16 + 8 < op.K ? 8 : 0;
    const size_t row = (size_t)L.expert[li] * op.K + tile * 16 + g, rb = row_bytes_of<KIND>(op.I);
    Src src{};
    src.w[0] = static_cast<const char*>(op.W_down) + row * rb + (S::kInt4 ? t * S::kLane / 2 : t * S::kLane * 2);
    src.w[1] = src.w[0] + half * rb;
    if (S::kInt4) {
        const int srow = op.I / op.group_size;
        src.s[0] = static_cast<const uint16_t*>(op.down_scale) + row * srow;
        src.s[1] = src.s[0] + half * srow;
    }
    auto token = [&](int r) { return p.ws.h + ((size_t)L.slot[li][r >> 1] * 2 + (r & 1)) * op.I; };
    const uint16_t* xr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) xr[j] = token(min(column_row<PH>(j), R - 1));
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    for (; k < n; k += warps) C::add(p, src, xr, token, xs, R, k * S::kCols, op.I, acc);
    k -= n;
    // token rows 2 i and 2 i + 1 are hi and lo of the expert's token i.  In the expert
    // before, another lane may have held this token: its sums must have arrived.
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float hi, lo;
            int i;
            if (PH == 1) {
                hi = C::sum(acc[j], 0, h), lo = C::sum(acc[j], 1, h);
                i = j * 4 + t;
            } else {
                const int over = PH == 2 ? 1 : 2;   // the lane with the next token row
                hi = C::sum(acc[j], 0, h);
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

template <int KIND, int NT>
__global__ void __launch_bounds__(moe_warps(KIND, NT) * 32) k_moe_down(const MoeParams p) {
    constexpr bool BF = KIND == DG_LINEAR_BF16;
    constexpr int kTok = KIND == DG_LINEAR_W4A16 ? NT * 2 : NT * 4;   // tokens at a time
    extern __shared__ __align__(16) float dyn[];
    __shared__ Lists L;
    const dg_moe& op = p.op;
    const int tid = threadIdx.x, warp = tid >> 5, warps = blockDim.x >> 5;
    const int M = op.M, tiles = (op.K + 15) / 16;
    float* sums = dyn;   // [warps][M][16]
    griddep_launch_dependents();
    for (int i = tid; i < warps * 16 * M; i += blockDim.x) sums[i] = 0.f;
    griddep_wait();
    for (int s = tid; s < M * op.top_k; s += blockDim.x) {
        L.ids[s] = __ldcg(p.ws.ids + s);
        L.wts[s] = __ldcg(p.ws.wts + s);
    }
    __syncthreads();
    build_lists<kTok < 8 ? 16 : kTok>(op, L);   // fewer than 8: so are the tokens
    float* mine = sums + warp * 16 * M;
    const uint32_t xs = (uint32_t)__cvta_generic_to_shared(dyn) + p.stage + warp * moe_stage(KIND, NT);

    int k = warp;   // this warp's next chunk of the expert
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        for (int li = 0; li < L.count; ++li) {
            if constexpr (KIND == DG_LINEAR_W4A16) {
                if (L.tokens[li] == 1)
                    down_expert<KIND, 4, 1>(p, L, li, tile, k, warps, xs, mine);
                else if constexpr (NT > 0)
                    down_expert<KIND, 2, NT>(p, L, li, tile, k, warps, xs, mine);
            } else {
                down_expert<KIND, 1, NT>(p, L, li, tile, k, warps, xs, mine);
            }
        }
        __syncthreads();
        for (int i = tid; i < 16 * M; i += blockDim.x) {
            const int m = i >> 4, row = tile * 16 + (i & 15);
            float y = 0.f;
            for (int w = 0; w < warps; ++w) {
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

// Token blocks of the kernels, enough for `tokens` of `rows` token rows each (up:
// one; down: hi and lo).
template <int KIND>
static int token_blocks(int tokens, int rows) {
    if (KIND == DG_LINEAR_W4A16 && tokens == 1) return 0;
    const int per = KIND == DG_LINEAR_W4A16 ? 4 : 8, nt = (tokens * rows + per - 1) / per;
    return nt <= 2 ? nt : 4;
}
template <int KIND>
static const void* up_kernel(int nt) {
    if constexpr (KIND == DG_LINEAR_W4A16)
        return nt == 0   ? (const void*)k_moe_up<KIND, 0>
               : nt == 1 ? (const void*)k_moe_up<KIND, 1> : (const void*)k_moe_up<KIND, 2>;
    else
        return nt == 1 ? (const void*)k_moe_up<KIND, 1> : (const void*)k_moe_up<KIND, 2>;
}
template <int KIND>
static const void* down_kernel(int nt) {
    if constexpr (KIND == DG_LINEAR_W4A16)
        return nt == 0   ? (const void*)k_moe_down<KIND, 0>
               : nt == 1 ? (const void*)k_moe_down<KIND, 1>
               : nt == 2 ? (const void*)k_moe_down<KIND, 2> : (const void*)k_moe_down<KIND, 4>;
    else
        return nt == 1   ? (const void*)k_moe_down<KIND, 1>
               : nt == 2 ? (const void*)k_moe_down<KIND, 2> : (const void*)k_moe_down<KIND, 4>;
}

template <int KIND>
static cudaError_t launch_moe_kind(const dg_moe& op, void* ws, cudaStream_t s) {
    MoeParams p;
    p.op = op;
    place(op, ws, &p.ws);
    const bool g32 = KIND == DG_LINEAR_W4A16 && op.group_size == 32;
    auto al4 = [](const void* q) { return ((uintptr_t)q & 3u) == 0; };
    void* args[] = {&p};
    p.group_32s = fast_div(KIND == DG_LINEAR_W4A16 ? op.group_size / 32 : 1);
    cudaError_t e = launch_pdl((const void*)k_moe_scores<KIND == DG_LINEAR_BF16>,
                               dim3(op.E, (op.M + kScoreTokens - 1) / kScoreTokens), dim3(256), 0, s, args);
    if (e != cudaSuccess) return e;

    p.scale_pairs = g32 && op.K % 64 == 0 && al4(op.gate_scale) && al4(op.up_scale);
    // Tokens of an expert at a time: registers for sixteen cost warps, a second
    // part reads the expert's weights again (mostly from L2).  int4 always takes
    // eight (16 tokens, 4096 x 2048, 2 of 8 experts: 94 us, sixteen 142; all 16 on
    // one expert of 2048 x 2048: 29, 44), 16-bit weights where experts of more are
    // rare (12 tokens, 2048 x 1024, 8 of 64: 125, 134; but 16 tokens, 4096 x
    // 14336, 2 of 8: 536 to 584, 436 to 449).
    const bool few = KIND == DG_LINEAR_W4A16 || op.M * op.top_k <= 2 * op.E;
    const int tokens = few ? std::min(op.M, 8) : op.M;
    const int nt = token_blocks<KIND>(tokens, 1), ctas = sm_count() * (moe_warps(KIND, nt) / kMoeWarps);
    // as few warps to a row tile as leave no SM without work: each split costs a
    // meeting per tile
    const int chunk = KIND == DG_LINEAR_W4A16 ? 512 : 128, experts = std::min(op.E, op.M * op.top_k);
    p.split = 1;
    while (p.split < kMoeWarps && (long long)experts * (op.I / 8) * p.split < 3ll * ctas * kMoeWarps &&
           p.split * chunk < op.K)
        p.split *= 2;
    size_t smem = (size_t)2 * kMoeWarps * (tokens <= 8 ? 8 : 16) * 16 * 4;
    if (smem < (size_t)kMoeWarps * op.E * 4) smem = (size_t)kMoeWarps * op.E * 4;
    p.stage = (int)((smem + 15) & ~(size_t)15);
    smem = p.stage + (size_t)kMoeWarps * moe_stage(KIND, nt);
    const void* fn = up_kernel<KIND>(nt);
    if ((e = tc::smem_attr_once(fn, smem)) != cudaSuccess) return e;
    if ((e = launch_pdl(fn, dim3(ctas), dim3(kMoeWarps * 32), smem, s, args)) != cudaSuccess) return e;

    // down: one CTA a row tile and the SM's warps divided among its CTAs, down
    // to 8 warps; more tiles than that gives follow one another
    p.scale_pairs = g32 && op.I % 64 == 0 && al4(op.down_scale);
    const int tiles = (op.K + 15) / 16, sms = sm_count(), dt = token_blocks<KIND>(tokens, 2);
    const int most = moe_warps(KIND, dt);
    const int per_sm = std::min((tiles + sms - 1) / sms, most / kMoeWarps), warps = most / per_sm;
    const int grid = std::min(tiles, sms * per_sm);
    p.stage = (int)((size_t)warps * 16 * op.M * 4);
    smem = p.stage + (size_t)warps * moe_stage(KIND, dt);
    fn = down_kernel<KIND>(dt);
    if ((e = tc::smem_attr_once(fn, smem)) != cudaSuccess) return e;
    return launch_pdl(fn, dim3(grid), dim3(warps * 32), smem, s, args);
}

cudaError_t launch_moe(const dg_moe& op, void* ws, cudaStream_t s) {
    switch (op.kind) {
        case DG_LINEAR_F16: return launch_moe_kind<DG_LINEAR_F16>(op, ws, s);
        case DG_LINEAR_BF16: return launch_moe_kind<DG_LINEAR_BF16>(op, ws, s);
        default: return launch_moe_kind<DG_LINEAR_W4A16>(op, ws, s);
    }
}

}  // namespace dg
