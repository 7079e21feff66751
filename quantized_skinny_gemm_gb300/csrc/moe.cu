// A mixture-of-experts layer for a few tokens, in three launches: router
// scores; gate and up products with SwiGLU; down products with the weighted
// sum over experts.
//
// The cost is the chosen experts' weights (6 * I * K bytes each at 16 bits,
// 1.7 * I * K at int4), read once whatever the number of tokens, so the
// products stream weights through shared memory and spend the matrix
// instruction (m16n8k16: 16 weight rows x 8 tokens) on few tokens: it costs
// no more for eight than for one.  Each warp has its own ring of cp.async
// stages (16 weight rows and the expert's token rows, kc columns) and never
// waits for another warp while it streams.
//
//   up:   one warp takes 8 gate and the same 8 up rows of an expert over the
//         whole of K, so that silu(gate) * up is in one thread's registers.
//   down: the warps of a CTA share 16 output rows and deal the stages of all
//         chosen experts among themselves; each adds weight * sum into its own
//         fp32 rows [token], which are summed in warp order at the end.
//
// h goes from one to the other as two 16-bit values, hi + lo, that are two
// columns of the matrix instruction: fp16 hi = h / 256 and lo = the rest x 2048
// (22 bits, |h| up to 2^24), bf16 hi and lo (16 bits); the products keep fp32
// sums.  int4 codes become fp16 by bit operations (exact); each group of 32
// codes is one pair of matrix instructions whose fp32 sum is then scaled.
#include "mma16.cuh"
#include "tc_common.cuh"

namespace dg {

constexpr int kMoeStages = 4;
constexpr int kMoeMaxSlots = 256;   // tokens x choices
constexpr int kMoeMaxWarps = 12;

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
    int slot_bytes;   // of a ring stage
    int vec_scales;   // int4: scales come by cp.async
};

// ---- router scores ------------------------------------------------------------------------

// Where value i of eight lies in the order the int4 unpacking gives its codes:
// (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ int int4_place(int i) { return i < 4 ? 2 * i : 2 * i - 7; }

// One CTA per expert: its score for every token.  The CTAs also write x in the
// int4 order, which the up products read.
template <bool BF16>
__global__ void __launch_bounds__(256) k_moe_scores(const MoeParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const dg_moe& op = p.op;
    const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint16_t* r = static_cast<const uint16_t*>(op.router) + (size_t)e * op.K;
    const uint16_t* x = static_cast<const uint16_t*>(op.x);
    float z[16];
#pragma unroll
    for (int m = 0; m < 16; ++m) z[m] = 0.f;
    for (int k = tid * 8; k < op.K; k += 2048) {
        float w[8];
        unpack8<BF16>(ld_nc16(r + k), w);
#pragma unroll
        for (int m = 0; m < 16; ++m) {
            if (m < op.M) {
                float v[8];
                unpack8<BF16>(ld_cg16(x + (size_t)m * op.K + k), v);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[m] = fmaf(w[i], v[i], z[m]);
            }
        }
    }
    __shared__ float part[8][16];
#pragma unroll
    for (int m = 0; m < 16; ++m)
        if (m < op.M) {
            const float v = warp_sum(z[m]);
            if (lane == 0) part[warp][m] = v;
        }
    __syncthreads();
    if (tid < op.M) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += part[w][tid];
        p.ws.scores[(size_t)tid * op.E + e] = v;
    }
    if (op.kind == DG_LINEAR_W4A16) {
        const int n8 = op.M * (op.K / 8);
        for (int i = e * 256 + tid; i < n8; i += gridDim.x * 256) {
            const uint4 v = ld_cg16(x + (size_t)i * 8);
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

// ---- ring stages ----------------------------------------------------------------------------

// A stage holds 16 weight rows and R token rows of kc columns.  kc shrinks as
// R grows, so that one stage size serves every expert.  Row pitches put eight
// rows' 16-byte pieces (ldmatrix; int4 token rows) or 4-byte pieces (int4
// codes) in different banks.
template <int KIND>
struct Stage {
    static constexpr bool kInt4 = KIND == DG_LINEAR_W4A16;
    __host__ __device__ static int kc(int R) {
        return kInt4 ? (R <= 8 ? 256 : R <= 16 ? 128 : 64) : (R <= 8 ? 128 : 64);
    }
    __host__ __device__ static int w_pitch(int kc) { return kInt4 ? kc / 2 + 16 : kc * 2 + 16; }
    __host__ __device__ static int x_pitch(int kc) { return kInt4 ? kc * 2 + 64 : kc * 2 + 16; }
    __host__ __device__ static int bytes(int R) {
        return 16 * w_pitch(kc(R)) + R * x_pitch(kc(R));
    }
};

// Copies 2^log_pieces 16-byte pieces of each of `rows` rows, from byte `from` of
// a row of row_bytes bytes on; pieces past its end read as zero.  row(r) is row
// r's address.
template <class Row>
__device__ __forceinline__ void copy_rows(uint32_t dst, int pitch, int rows, int log_pieces, int from,
                                          int row_bytes, Row row) {
    const int lane = threadIdx.x & 31;
    for (int i = lane; i < rows << log_pieces; i += 32) {
        const int r = i >> log_pieces, at = (i & ((1 << log_pieces) - 1)) * 16;
        const bool in = from + at < row_bytes;
        cp_async16(dst + r * pitch + at, reinterpret_cast<const char*>(row(r)) + (in ? from + at : 0), in);
    }
}

// Fetches one stage: weight rows row_w(0..15) (null: none), their scales, and
// R token rows row_x(r), columns [k0, k0 + kc) of Kd.
template <int KIND, class RowW, class RowS, class RowX>
__device__ __forceinline__ void fetch_stage(const MoeParams& p, uint32_t dst, int R, int kc, int k0, int Kd,
                                            RowW row_w, RowS row_s, RowX row_x) {
    using St = Stage<KIND>;
    const int wp = St::w_pitch(kc), xp = St::x_pitch(kc);
    if (St::kInt4) {
        const int lg = kc == 256 ? 3 : kc == 128 ? 2 : 1;   // 16-byte pieces of a row of codes
        copy_rows(dst, wp, 16, lg, k0 / 2, Kd / 2, row_w);
        const int lane = threadIdx.x & 31;
        if (p.vec_scales) {
            if (lane < 16) {
                const char* s = reinterpret_cast<const char*>(row_s(lane)) + k0 / 16;
                const uint32_t d = dst + lane * wp + kc / 2;
                if (kc == 256)
                    cp_async16(d, s, true);
                else if (kc == 128)
                    cp_async_small<8>(d, s);
                else
                    cp_async_small<4>(d, s);
            }
        } else {
            // any group size, count or alignment: plain loads, one per 32 columns
            for (int i = lane; i < 16 << lg; i += 32) {
                const int r = i >> lg, b = i & ((1 << lg) - 1), k = k0 + b * 32;
                uint16_t v = 0;
                if (k < Kd) v = ld_stream_u16(reinterpret_cast<const uint16_t*>(row_s(r)) + k / p.op.group_size);
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + r * wp + kc / 2 + b * 2), "h"(v) : "memory");
            }
        }
        copy_rows(dst + 16 * wp, xp, R, lg + 2, k0 * 2, Kd * 2, row_x);
    } else {
        const int lg = kc == 128 ? 4 : 3;
        copy_rows(dst, wp, 16, lg, k0 * 2, Kd * 2, row_w);
        copy_rows(dst + 16 * wp, xp, R, lg, k0 * 2, Kd * 2, row_x);
    }
}

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

// acc[j] += (16 weight rows) x (token rows 8 j ..), columns of one stage.
template <int KIND, int NT>
__device__ __forceinline__ void mma_stage(uint32_t st, int R, int kc, int cols, float (&acc)[NT][4]) {
    using St = Stage<KIND>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int wp = St::w_pitch(kc), xp = St::x_pitch(kc);
    const uint32_t xs = st + 16 * wp;
    if (St::kInt4) {
        const uint32_t wa = st + g * wp + t * 4;
        uint32_t xa[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) xa[j] = xs + min(j * 8 + g, R - 1) * xp + t * 16;
        const int groups = min(cols, kc) / 32;
#pragma unroll 2
        for (int b = 0; b < groups; ++b) {
            uint32_t lo[4], hi[4];
            int4_pairs(lds32(wa + b * 16), lo);
            int4_pairs(lds32(wa + 8 * wp + b * 16), hi);
            uint16_t s0, s1;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(s0) : "r"(st + g * wp + kc / 2 + b * 2) : "memory");
            asm volatile("ld.shared.u16 %0, [%1];"
                         : "=h"(s1)
                         : "r"(st + (g + 8) * wp + kc / 2 + b * 2)
                         : "memory");
            const float f0 = elem_f32<false>(s0), f1 = elem_f32<false>(s1);
            const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j * 8 < R) {
                    const uint4 x = lds128(xa[j] + b * 64);
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
                    mma16816<false>(c, a0, x.x, x.y);
                    mma16816<false>(c, a1, x.z, x.w);
                    acc[j][0] = fmaf(f0, c[0], acc[j][0]);
                    acc[j][1] = fmaf(f0, c[1], acc[j][1]);
                    acc[j][2] = fmaf(f1, c[2], acc[j][2]);
                    acc[j][3] = fmaf(f1, c[3], acc[j][3]);
                }
            }
        }
    } else {
        constexpr bool BF = KIND == DG_LINEAR_BF16;
        const uint32_t wa = st + ((lane & 7) + ((lane >> 3) & 1) * 8) * wp + (lane >> 4) * 16;
        uint32_t xa[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) xa[j] = xs + min(j * 8 + (lane & 7), R - 1) * xp + (lane >> 3) * 16;
        const int steps = kc / 32;
#pragma unroll 2
        for (int k = 0; k < steps; ++k) {
            uint32_t a0[4], a1[4];
            ldsm4(a0, wa + k * 64);
            ldsm4(a1, wa + k * 64 + 32);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j * 8 < R) {
                    uint32_t x[4];
                    ldsm4(x, xa[j] + k * 64);
                    mma16816<BF>(acc[j], a0, x[0], x[1]);
                    mma16816<BF>(acc[j], a1, x[2], x[3]);
                }
            }
        }
    }
}

// ---- gate and up ----------------------------------------------------------------------------

template <int KIND>
__device__ __forceinline__ size_t row_bytes_of(int cols) {
    return KIND == DG_LINEAR_W4A16 ? (size_t)cols / 2 : (size_t)cols * 2;
}

template <int KIND, int NT>
__global__ void __launch_bounds__(kMoeMaxWarps * 32) k_moe_up(const MoeParams p) {
    using St = Stage<KIND>;
    constexpr bool BF = KIND == DG_LINEAR_BF16;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Lists L;
    const dg_moe& op = p.op;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    griddep_launch_dependents();
    griddep_wait();
    // the ring, not yet in use, holds the probabilities
    for (int m = warp; m < op.M; m += warps)
        route_token(op, p.ws.scores + (size_t)m * op.E, reinterpret_cast<float*>(smem) + (size_t)warp * op.E,
                    L.ids + m * op.top_k, L.wts + m * op.top_k);
    __syncthreads();
    build_lists(op, L);
    if (blockIdx.x == 0)
        for (int s = tid; s < op.M * op.top_k; s += blockDim.x) {
            p.ws.ids[s] = L.ids[s];
            p.ws.wts[s] = L.wts[s];
            if (op.ids) op.ids[s] = L.ids[s];
            if (op.weights) op.weights[s] = L.wts[s];
        }

    const int tiles = op.I / 8, total = L.count * tiles, stride = warps * gridDim.x;
    const size_t rb = row_bytes_of<KIND>(op.K);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * kMoeStages * p.slot_bytes;
    const uint16_t* x = KIND == DG_LINEAR_W4A16 ? p.ws.xp : static_cast<const uint16_t*>(op.x);

    // the stage to fetch next, and the stage to compute next
    struct Cursor {
        int item, k0;
    } f = {(int)(warp * gridDim.x + blockIdx.x), 0}, c = f;
    int fs = 0, cs = 0;
    auto fetch = [&] {
        if (f.item < total) {
            const int li = f.item / tiles, tile = f.item - li * tiles;
            const int R = L.tokens[li], kc = St::kc(R);
            const size_t row0 = (size_t)L.expert[li] * op.I + tile * 8;
            auto row_w = [&](int r) {
                return static_cast<const char*>(r < 8 ? op.W_gate : op.W_up) + (row0 + (r & 7)) * rb;
            };
            auto row_s = [&](int r) {
                return static_cast<const char*>(r < 8 ? op.gate_scale : op.up_scale) +
                       (row0 + (r & 7)) * (op.K / op.group_size) * 2;
            };
            auto row_x = [&](int r) { return x + (size_t)L.token_of[L.slot[li][r]] * op.K; };
            fetch_stage<KIND>(p, ring + fs * p.slot_bytes, R, kc, f.k0, op.K, row_w, row_s, row_x);
            f.k0 += kc;
            if (f.k0 >= op.K) {
                f.k0 = 0;
                f.item += stride;
            }
            fs = fs + 1 == kMoeStages ? 0 : fs + 1;
        }
        cp_commit();
    };
    for (int i = 0; i < kMoeStages - 1; ++i) fetch();
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    while (c.item < total) {
        const int li = c.item / tiles, tile = c.item - li * tiles;
        const int R = L.tokens[li], kc = St::kc(R);
        cp_wait<kMoeStages - 2>();
        __syncwarp();
        fetch();
        mma_stage<KIND, NT>(ring + cs * p.slot_bytes, R, kc, op.K - c.k0, acc);
        cs = cs + 1 == kMoeStages ? 0 : cs + 1;
        c.k0 += kc;
        if (c.k0 < op.K) continue;
        // rows g (gate) and g + 8 (up) of tokens 2 t and 2 t + 1: one thread's
        const int g = lane >> 2, t = lane & 3;
        const int i = tile * 8 + (KIND == DG_LINEAR_W4A16 ? int4_place(g) : g);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int n = j * 8 + t * 2 + q;
                if (n < R) {
                    const float v = silu_f32(acc[j][q]) * acc[j][2 + q];
                    uint16_t* h = p.ws.h + (size_t)L.slot[li][n] * 2 * op.I + i;
                    const float s = BF ? v : v * 0.00390625f;
                    const uint16_t hi = elem_16<BF>(s);
                    h[0] = hi;
                    h[op.I] = elem_16<BF>((s - elem_f32<BF>(hi)) * (BF ? 1.f : 2048.f));
                }
            }
            acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
        }
        c.k0 = 0;
        c.item += stride;
    }
    cp_wait<0>();
}

// ---- down and the weighted sum ----------------------------------------------------------------

template <int KIND, int NT>
__global__ void __launch_bounds__(kMoeMaxWarps * 32) k_moe_down(const MoeParams p) {
    using St = Stage<KIND>;
    constexpr bool BF = KIND == DG_LINEAR_BF16;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Lists L;
    const dg_moe& op = p.op;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int M = op.M, n0 = blockIdx.x * 16;
    float* sums = reinterpret_cast<float*>(smem + warps * kMoeStages * p.slot_bytes);  // [warps][16][M]
    griddep_launch_dependents();
    for (int i = tid; i < warps * 16 * M; i += blockDim.x) sums[i] = 0.f;
    griddep_wait();
    for (int s = tid; s < M * op.top_k; s += blockDim.x) {
        L.ids[s] = __ldcg(p.ws.ids + s);
        L.wts[s] = __ldcg(p.ws.wts + s);
    }
    __syncthreads();
    build_lists(op, L);
    const size_t rb = row_bytes_of<KIND>(op.I);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * kMoeStages * p.slot_bytes;
    float* mine = sums + warp * 16 * M;

    // the experts' stages in one sequence, dealt to the warps in turn
    struct Cursor {
        int li, k;   // stage k of expert li
    } f = {0, warp}, c = f;
    auto settle = [&](Cursor& q) {
        while (q.li < L.count) {
            const int kc = St::kc(2 * L.tokens[q.li]), n = (op.I + kc - 1) / kc;
            if (q.k < n) return;
            q.k -= n;
            ++q.li;
        }
    };
    settle(f);
    c = f;
    int fs = 0, cs = 0;
    auto fetch = [&] {
        if (f.li < L.count) {
            const int li = f.li, R = 2 * L.tokens[li], kc = St::kc(R);
            const size_t row0 = (size_t)L.expert[li] * op.K;
            const int last = op.K - 1;   // rows past the end repeat the last one
            auto row_w = [&](int r) {
                return static_cast<const char*>(op.W_down) + (row0 + min(n0 + r, last)) * rb;
            };
            auto row_s = [&](int r) {
                return static_cast<const char*>(op.down_scale) +
                       (row0 + min(n0 + r, last)) * (op.I / op.group_size) * 2;
            };
            auto row_x = [&](int r) {
                return p.ws.h + ((size_t)L.slot[li][r >> 1] * 2 + (r & 1)) * op.I;
            };
            fetch_stage<KIND>(p, ring + fs * p.slot_bytes, R, kc, f.k * kc, op.I, row_w, row_s, row_x);
            f.k += warps;
            settle(f);
            fs = fs + 1 == kMoeStages ? 0 : fs + 1;
        }
        cp_commit();
    };
    for (int i = 0; i < kMoeStages - 1; ++i) fetch();
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    while (c.li < L.count) {
        const int li = c.li, R = 2 * L.tokens[li], kc = St::kc(R);
        cp_wait<kMoeStages - 2>();
        __syncwarp();
        fetch();
        mma_stage<KIND, NT>(ring + cs * p.slot_bytes, R, kc, op.I - c.k * kc, acc);
        cs = cs + 1 == kMoeStages ? 0 : cs + 1;
        c.k += warps;
        settle(c);
        if (c.li == li) continue;
        // columns 2 i and 2 i + 1 are hi and lo of the expert's token i
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int i = j * 4 + t;
            if (2 * i < R) {
                const int s = L.slot[li][i], m = L.token_of[s];
                const float w = L.wts[s];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float v = BF ? acc[j][2 * q] + acc[j][2 * q + 1]
                                       : fmaf(acc[j][2 * q + 1], 1.f / 2048.f, acc[j][2 * q]) * 256.f;
                    mine[(g + 8 * q) * M + m] = fmaf(w, v, mine[(g + 8 * q) * M + m]);
                }
            }
            acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
        }
    }
    cp_wait<0>();
    __syncthreads();
    for (int i = tid; i < 16 * M; i += blockDim.x) {
        const int m = i >> 4, r = i & 15;
        if (n0 + r >= op.K) continue;
        float y = 0.f;
        for (int w = 0; w < warps; ++w) y += sums[(w * 16 + r) * M + m];
        const size_t at = (size_t)m * op.K + n0 + r;
        if (op.residual) y += elem_f32<BF>(static_cast<const uint16_t*>(op.residual)[at]);
        static_cast<uint16_t*>(op.y)[at] = elem_16<BF>(y);
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

template <int KIND>
static cudaError_t launch_moe_kind(const dg_moe& op, void* ws, cudaStream_t s) {
    using St = Stage<KIND>;
    constexpr int kList = sizeof(Lists);
    MoeParams p;
    p.op = op;
    place(op, ws, &p.ws);
    const int g = op.group_size;
    auto vec16 = [](const void* q) { return ((uintptr_t)q & 15u) == 0; };
    void* args[] = {&p};

    p.slot_bytes = p.vec_scales = 0;
    cudaError_t e = launch_pdl((const void*)k_moe_scores<KIND == DG_LINEAR_BF16>, dim3(op.E), dim3(256), 0, s, args);
    if (e != cudaSuccess) return e;

    auto stage_for = [](int most) {   // the largest stage of 1..most token rows
        int b = 0;
        for (int r = 1; r <= most; ++r) b = St::bytes(r) > b ? St::bytes(r) : b;
        return b;
    };
    // up: one CTA per SM, as many warps as their rings fit
    const int sms = sm_count();
    p.slot_bytes = stage_for(op.M);
    int warps = (int)((smem_optin_limit() - kList - 1024) / (kMoeStages * p.slot_bytes));
    if (warps > kMoeMaxWarps) warps = kMoeMaxWarps;
    if (warps < 1) return cudaErrorInvalidConfiguration;
    size_t smem = (size_t)warps * kMoeStages * p.slot_bytes;
    if (smem < (size_t)warps * op.E * 4) smem = (size_t)warps * op.E * 4;
    p.vec_scales = St::kInt4 && g == 32 && op.K % 256 == 0 && vec16(op.gate_scale) && vec16(op.up_scale);
    const void* fn = op.M <= 8 ? (const void*)k_moe_up<KIND, 1> : (const void*)k_moe_up<KIND, 2>;
    if ((e = tc::smem_attr_once(fn, smem)) != cudaSuccess) return e;
    if ((e = launch_pdl(fn, dim3(sms), dim3(warps * 32), smem, s, args)) != cudaSuccess) return e;

    // down: two CTAs per SM (more row tiles than SMs then run side by side)
    p.slot_bytes = stage_for(2 * op.M);
    warps = (int)((114 * 1024 - kList - 2048) / (kMoeStages * p.slot_bytes + 64 * op.M));
    if (warps > kMoeMaxWarps) warps = kMoeMaxWarps;
    if (warps < 1) return cudaErrorInvalidConfiguration;
    smem = (size_t)warps * (kMoeStages * p.slot_bytes + 64 * op.M);
    p.vec_scales = St::kInt4 && g == 32 && op.I % 256 == 0 && vec16(op.down_scale);
    fn = op.M <= 4 ? (const void*)k_moe_down<KIND, 1>
         : op.M <= 8 ? (const void*)k_moe_down<KIND, 2> : (const void*)k_moe_down<KIND, 4>;
    if ((e = tc::smem_attr_once(fn, smem)) != cudaSuccess) return e;
    return launch_pdl(fn, dim3((op.K + 15) / 16), dim3(warps * 32), smem, s, args);
}

cudaError_t launch_moe(const dg_moe& op, void* ws, cudaStream_t s) {
    switch (op.kind) {
        case DG_LINEAR_F16: return launch_moe_kind<DG_LINEAR_F16>(op, ws, s);
        case DG_LINEAR_BF16: return launch_moe_kind<DG_LINEAR_BF16>(op, ws, s);
        default: return launch_moe_kind<DG_LINEAR_W4A16>(op, ws, s);
    }
}

}  // namespace dg
