// The norms around a block, fused with its gate and residual scale.
#include <algorithm>

#include "elem.cuh"
#include "tc_common.cuh"

namespace dg {

// The threads that share a row: L lanes of a warp, or the CTA.  sum() gives all of
// them the total; the CTA's alternates between two halves of `red` from call to
// call, so that one barrier per call is enough.
template <int L>
struct LaneTeam {
    static constexpr int kLanes = L;
    __device__ __forceinline__ explicit LaneTeam(float (*)[32]) {}
    __device__ __forceinline__ int id() const { return threadIdx.x & (L - 1); }
    __device__ __forceinline__ int size() const { return L; }
    __device__ __forceinline__ float sum(float v) {
        const uint32_t mates = L == 32 ? ~0u : ((1u << (L & 31)) - 1) << (threadIdx.x & 31 & ~(L - 1));
#pragma unroll
        for (int d = L / 2; d; d /= 2) v += __shfl_xor_sync(mates, v, d);
        return v;
    }
};
struct CtaTeam {
    static constexpr int kLanes = 0;
    float (*red)[32];
    int turn = 0;
    __device__ __forceinline__ explicit CtaTeam(float (*red)[32]) : red(red) {}
    __device__ __forceinline__ int id() const { return threadIdx.x; }
    __device__ __forceinline__ int size() const { return blockDim.x; }
    __device__ __forceinline__ float sum(float v) {
        v = warp_sum(v);
        float* r = red[turn];
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
        __syncthreads();
        const int lane = threadIdx.x & 31;
        return warp_sum(lane < (int)(blockDim.x >> 5) ? r[lane] : 0.f);
    }
};

// Value j of vector c of a thread is element ((c * team.size() + team.id()) * U + j).
template <int U, int C>
struct RowRegs {
    float v[C][U];
};

// Vector c of a row, zero past its end.
template <bool BF16, int U>
__device__ __forceinline__ void load_part(const CtaTeam& team, const void* p, int N, int c, float (&f)[U]) {
    const uint16_t* e = static_cast<const uint16_t*>(p);
    const int n = (c * team.size() + team.id()) * U;
    if constexpr (U == 8) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (n < N) v = *reinterpret_cast<const uint4*>(e + n);
        unpack8<BF16>(v, f);
    } else if constexpr (U == 2) {
        const uint32_t v = n < N ? *reinterpret_cast<const uint32_t*>(e + n) : 0u;
        const float2 x = pair_f32<BF16>(v);
        f[0] = x.x, f[1] = x.y;
    } else {
        f[0] = n < N ? elem_f32<BF16>(e[n]) : 0.f;
    }
}
template <int U>
__device__ __forceinline__ void load_part_f32(const CtaTeam& team, const float* p, int N, int c, float (&f)[U]) {
    const int n = (c * team.size() + team.id()) * U;
#pragma unroll
    for (int j = 0; j < U; ++j) f[j] = 0.f;
    if (n >= N) return;
    if constexpr (U == 8) {
        const float4 a = *reinterpret_cast<const float4*>(p + n), b = *reinterpret_cast<const float4*>(p + n + 4);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else if constexpr (U == 2) {
        const float2 a = *reinterpret_cast<const float2*>(p + n);
        f[0] = a.x, f[1] = a.y;
    } else {
        f[0] = p[n];
    }
}

template <bool BF16, int U, int C>
__device__ __forceinline__ void store_row(const CtaTeam& team, void* p, int N, const RowRegs<U, C>& r) {
    uint16_t* e = static_cast<uint16_t*>(p);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int n = (c * team.size() + team.id()) * U;
        if (n >= N) continue;
        if constexpr (U == 8)
            *reinterpret_cast<uint4*>(e + n) = pack8<BF16>(r.v[c]);
        else if constexpr (U == 2)
            *reinterpret_cast<uint32_t*>(e + n) = pair_16<BF16>(r.v[c][0], r.v[c][1]);
        else
            e[n] = elem_16<BF16>(r.v[c][0]);
    }
}

template <int U, int C>
__device__ __forceinline__ void store_row_f32(const CtaTeam& team, float* p, int N, const RowRegs<U, C>& r) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int n = (c * team.size() + team.id()) * U;
        if (n >= N) continue;
        if constexpr (U == 8) {
            *reinterpret_cast<float4*>(p + n) = make_float4(r.v[c][0], r.v[c][1], r.v[c][2], r.v[c][3]);
            *reinterpret_cast<float4*>(p + n + 4) = make_float4(r.v[c][4], r.v[c][5], r.v[c][6], r.v[c][7]);
        } else if constexpr (U == 2) {
            *reinterpret_cast<float2*>(p + n) = make_float2(r.v[c][0], r.v[c][1]);
        } else {
            p[n] = r.v[c][0];
        }
    }
}

// r <- norm(r; w, b) of dg_norm.  The row sits in registers, so the mean and
// the centred squares are two exact passes over it, not one with cancellation.
template <bool BF16, int U, int C>
__device__ __forceinline__ void norm_row(const dg_norm& op, const void* w, const void* b, RowRegs<U, C>& r,
                                         CtaTeam& team) {
    const int N = op.N;
    if (op.kind == DG_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < U; ++j) s += r.v[c][j];
        const float mean = team.sum(s) / (float)N;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < U; ++j)
                if ((c * team.size() + team.id()) * U < N) r.v[c][j] -= mean;
    }
    float q = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < U; ++j) q = fmaf(r.v[c][j], r.v[c][j], q);
    const float k = 1.f / sqrtf(team.sum(q) / (float)N + op.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float g[U];
        load_part<BF16>(team, w, N, c, g);
#pragma unroll
        for (int j = 0; j < U; ++j) r.v[c][j] = r.v[c][j] * k * (op.w_offset + g[j]);
        if (b) {
            load_part<BF16>(team, b, N, c, g);
#pragma unroll
            for (int j = 0; j < U; ++j) r.v[c][j] += g[j];
        }
    }
}

// One CTA per row, the row held in registers (U values per vector, C vectors per
// thread), so y and h are read once and h' and x written once: for few rows, and
// for pointers or weights that k_norm_flat cannot take.
template <bool BF16, int U, int C>
__global__ void __launch_bounds__(C > 16 ? 512 : 1024) k_norm(const dg_norm op) {
    __shared__ float red[2][32];
    griddep_launch_dependents();
    griddep_wait();
    CtaTeam team(red);
    const int row = blockIdx.x;
    const int N = op.N;
    const size_t at = (size_t)row * N;
    RowRegs<U, C> r;
    const uint16_t* y = static_cast<const uint16_t*>(op.y) + at;
    const uint16_t* gate = static_cast<const uint16_t*>(op.gate) + (op.gate_rows == 1 ? 0 : at);
    if (op.y) {
#pragma unroll
        for (int c = 0; c < C; ++c) load_part<BF16>(team, y, N, c, r.v[c]);
        if (op.w_post) norm_row<BF16>(op, op.w_post, op.b_post, r, team);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float h[U], g[U];
        if (op.h) {
            if (op.h_f32)
                load_part_f32(team, static_cast<const float*>(op.h) + at, N, c, h);
            else
                load_part<BF16>(team, static_cast<const uint16_t*>(op.h) + at, N, c, h);
        }
        if (op.gate) load_part<BF16>(team, gate, N, c, g);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            float v = r.v[c][j];
            if (op.gate) v *= g[j];
            const float a = h[j] * op.alpha;
            r.v[c][j] = !op.y ? a : op.h ? fmaf(op.beta, v, a) : op.beta * v;
        }
    }
    if (op.h_out) {
        if (op.h_f32)
            store_row_f32(team, static_cast<float*>(op.h_out) + at, N, r);
        else
            store_row<BF16>(team, static_cast<uint16_t*>(op.h_out) + at, N, r);
    }
    if (op.x_out) {
        norm_row<BF16>(op, op.w_pre, op.b_pre, r, team);
        store_row<BF16>(team, static_cast<uint16_t*>(op.x_out) + at, N, r);
    }
}

// Rows of any width, in aligned vectors of eight values.  Row r begins
// (r * N) mod 8 = shift values into such a vector, so its first and last vectors
// may reach into the neighbouring rows; what they hold of those is masked, and
// only the row's own values are stored.  A team takes every step-th row, step a
// multiple of eight, so that its shift never changes: it lays the weights out in
// shared memory once, vector by vector as it will need them.  With one vector a
// thread (AHEAD) the next row's y, h and gate are loaded before this one is
// reduced, so that HBM stays busy over the sums.  HBM bounds it: 4096 x 4096
// bf16 with both norms, gate and fp32 residual 42.0 us, 5.6 TB/s of the copy's
// 6.8; odd rows add the edges' instructions, the wide ones a row's latency
// (41371 x 115 with a gate: 3.1 TB/s, 2000 x 6143: 4.2, 900 x 16383: 1.6; in
// single values, one row after the other, they ran at 0.7 to 1.0).
struct RawVec {
    uint4 y, gate, h[2];
};
constexpr int kFlatThreads = 256;   // of a CTA of lane teams
constexpr int kFlatArrays = 5;      // w_post, b_post, w_pre, b_pre, a gate of one row

// Eight values from `at` on; those past the tensor's end, which a row's last
// vector may reach, are zero.
template <bool EVEN>
__device__ __forceinline__ uint4 flat_load(const void* base, size_t at, size_t total) {
    const uint16_t* p = static_cast<const uint16_t*>(base);
    if (EVEN || at + 8 <= total) return __ldcs(reinterpret_cast<const uint4*>(p + at));
    uint16_t e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = at + j < total ? p[at + j] : (uint16_t)0;
    uint4 v;
    memcpy(&v, e, 16);
    return v;
}

template <bool BF16, bool EVEN, int C, class T>
struct Flat {
    static constexpr bool AHEAD = C == 1;
    const dg_norm& op;
    T team;
    int shift;
    uint4* lay;
    size_t total;

    // First value of vector c in its row; the vector is of use if any value is.
    __device__ __forceinline__ int first(int c) const {
        return (c * team.size() + team.id()) * 8 - (EVEN ? 0 : shift);
    }
    __device__ __forceinline__ bool inside(int n) const { return EVEN || (n >= 0 && n + 8 <= op.N); }
    // Where vector c of array `which` lies; only the arrays in use have room.
    __device__ __forceinline__ uint4* laid(int which, int c) const {
        int slot = which;
        if (which > 0) slot -= !op.w_post;
        if (which > 1) slot -= !op.b_post;
        if (which > 2) slot -= !op.w_pre;
        if (which > 3) slot -= !op.b_pre;
        return lay + (slot * C + c) * team.size() + team.id();
    }

    __device__ __forceinline__ void fetch_gate(unsigned row, int c, RawVec& q) const {
        const int n = first(c);
        if (n >= op.N) return;
        if (op.gate)
            q.gate = op.gate_rows == 1 ? *laid(4, c) : flat_load<EVEN>(op.gate, (size_t)row * op.N + n, total);
    }
    __device__ __forceinline__ void fetch_y(unsigned row, int c, RawVec& q) const {
        const int n = first(c);
        if (n < op.N && op.y) q.y = flat_load<EVEN>(op.y, (size_t)row * op.N + n, total);
    }
    __device__ __forceinline__ void fetch_h(unsigned row, int c, RawVec& q) const {
        const int n = first(c);
        if (n >= op.N || !op.h) return;
        const size_t at = (size_t)row * op.N + n;
        if (!op.h_f32) {
            q.h[0] = flat_load<EVEN>(op.h, at, total);
            return;
        }
        const float* h = static_cast<const float*>(op.h) + at;
        if (EVEN || at + 8 <= total) {
            q.h[0] = __ldcs(reinterpret_cast<const uint4*>(h));
            q.h[1] = __ldcs(reinterpret_cast<const uint4*>(h) + 1);
        } else {
            float e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = at + j < total ? h[j] : 0.f;
            memcpy(q.h, e, 32);
        }
    }

    // Zeroes what is not of this row.
    __device__ __forceinline__ void mask(float (&r)[8], int c) const {
        const int n = first(c);
        if (n >= 0 && n + 8 <= op.N) return;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if ((unsigned)(n + j) >= (unsigned)op.N) r[j] = 0.f;
    }
    // r <- norm(r) by the weights `which` and the biases behind them.
    __device__ __forceinline__ void norm(float (&r)[C][8], int which, bool bias) {
        const int N = op.N;
        if (op.kind == DG_NORM_LAYER) {
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) s += r[c][j];
            const float mean = team.sum(s) / (float)N;
#pragma unroll
            for (int c = 0; c < C; ++c) {
#pragma unroll
                for (int j = 0; j < 8; ++j) r[c][j] -= mean;
                mask(r[c], c);
            }
        }
        float q = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) q = fmaf(r[c][j], r[c][j], q);
        const float k = 1.f / sqrtf(team.sum(q) / (float)N + op.eps);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float g[8];
            unpack8<BF16>(*laid(which, c), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[c][j] = r[c][j] * k * (op.w_offset + g[j]);
            if (bias) {
                unpack8<BF16>(*laid(which + 1, c), g);
#pragma unroll
                for (int j = 0; j < 8; ++j) r[c][j] += g[j];
            }
        }
    }
    __device__ __forceinline__ void store(void* out, size_t at, const float (&r)[8], int n) const {
        uint16_t* p = static_cast<uint16_t*>(out) + at;
        if (inside(n)) {
            *reinterpret_cast<uint4*>(p) = pack8<BF16>(r);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((unsigned)(n + j) < (unsigned)op.N) p[j] = elem_16<BF16>(r[j]);
        }
    }
    __device__ __forceinline__ void store_f32(void* out, size_t at, const float (&r)[8], int n) const {
        float* p = static_cast<float*>(out) + at;
        if (inside(n)) {
            reinterpret_cast<float4*>(p)[0] = make_float4(r[0], r[1], r[2], r[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(r[4], r[5], r[6], r[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((unsigned)(n + j) < (unsigned)op.N) p[j] = r[j];
        }
    }

    __device__ __forceinline__ void run(unsigned row, unsigned step) {
        const unsigned rows = op.rows;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        RawVec q{zero, zero, {zero, zero}};
        if (AHEAD && row < rows) fetch_y(row, 0, q), fetch_h(row, 0, q), fetch_gate(row, 0, q);
        for (; row < rows; row += step) {
            float r[C][8];
            RawVec v[C];
            if constexpr (AHEAD) {
                v[0] = q;
                if (row + step < rows)
                    fetch_y(row + step, 0, q), fetch_h(row + step, 0, q), fetch_gate(row + step, 0, q);
                unpack8<BF16>(v[0].y, r[0]);
            } else {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    v[c] = RawVec{zero, zero, {zero, zero}};
                    fetch_y(row, c, v[c]);
                    unpack8<BF16>(v[c].y, r[c]);
                }
            }
            if (op.y && op.w_post) {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (!EVEN) mask(r[c], c);
                norm(r, 0, op.b_post != nullptr);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if constexpr (!AHEAD) fetch_h(row, c, v[c]), fetch_gate(row, c, v[c]);
                float h[8], g[8];
                unpack8<BF16>(v[c].gate, g);
                if (op.h_f32)
                    memcpy(h, v[c].h, 32);
                else
                    unpack8<BF16>(v[c].h[0], h);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float x = r[c][j];
                    if (op.gate) x *= g[j];
                    const float a = h[j] * op.alpha;
                    r[c][j] = !op.y ? a : op.h ? fmaf(op.beta, x, a) : op.beta * x;
                }
                if (!EVEN) mask(r[c], c);   // else zeros were loaded
            }
            const size_t at = (size_t)row * op.N;
            if (op.h_out) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int n = first(c);
                    if (n >= op.N) continue;
                    if (op.h_f32)
                        store_f32(op.h_out, at + n, r[c], n);
                    else
                        store(op.h_out, at + n, r[c], n);
                }
            }
            if (op.x_out) {
                norm(r, 2, op.b_pre != nullptr);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int n = first(c);
                    if (n < op.N) store(op.x_out, at + n, r[c], n);
                }
            }
        }
    }
};

template <bool BF16, bool EVEN, int C, class T>
__global__ void __launch_bounds__(T::kLanes ? kFlatThreads : 1024, T::kLanes ? 3 : 1) k_norm_flat(const dg_norm op) {
    extern __shared__ __align__(16) uint4 flat_smem[];
    __shared__ float red[2][32];
    griddep_launch_dependents();
    griddep_wait();
    const int L = T::kLanes ? T::kLanes : (int)blockDim.x, teams = blockDim.x / L, mine = threadIdx.x / L;
    const unsigned row = blockIdx.x * teams + mine;
    const int arrays = !!op.w_post + !!op.b_post + !!op.w_pre + !!op.b_pre + (op.gate && op.gate_rows == 1);
    Flat<BF16, EVEN, C, T> f{op, T(red), (int)(row * (unsigned)op.N & 7u), flat_smem + mine * arrays * C * L,
                             (size_t)op.rows * op.N};
    const void* src[kFlatArrays] = {op.w_post, op.b_post, op.w_pre, op.b_pre, op.gate_rows == 1 ? op.gate : nullptr};
#pragma unroll
    for (int w = 0; w < kFlatArrays; ++w) {
        if (!src[w]) continue;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int n = f.first(c);
            uint16_t e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                e[j] = (unsigned)(n + j) < (unsigned)op.N ? static_cast<const uint16_t*>(src[w])[n + j] : (uint16_t)0;
            memcpy(f.laid(w, c), e, 16);   // only this thread reads it
        }
    }
    f.run(row, gridDim.x * teams);
}

// Vectors of U values, C of them a thread.
template <bool BF16, int U>
static const void* norm_fn(int C) {
    if (C <= 1) return (const void*)k_norm<BF16, U, 1>;
    if (C <= 2) return (const void*)k_norm<BF16, U, 2>;
    if (C <= 4) return (const void*)k_norm<BF16, U, 4>;
    if constexpr (U < 8) {
        if (C <= 8) return (const void*)k_norm<BF16, U, 8>;
        if (C <= 16) return (const void*)k_norm<BF16, U, 16>;
    }
    if constexpr (U < 2)
        if (C <= 64) return (const void*)k_norm<BF16, U, 64>;
    return nullptr;
}
template <bool BF16>
static const void* norm_fn_u(int U, int C) {
    return U == 8 ? norm_fn<BF16, 8>(C) : U == 2 ? norm_fn<BF16, 2>(C) : norm_fn<BF16, 1>(C);
}

// lanes a row (0: a CTA's, C vectors each)
template <bool BF16, bool EVEN>
static const void* flat_fn(int lanes, int C) {
    if (lanes == 16) return (const void*)k_norm_flat<BF16, EVEN, 1, LaneTeam<16>>;
    if (lanes == 32) return (const void*)k_norm_flat<BF16, EVEN, 1, LaneTeam<32>>;
    if (C == 1) return (const void*)k_norm_flat<BF16, EVEN, 1, CtaTeam>;
    if (C == 2) return (const void*)k_norm_flat<BF16, EVEN, 2, CtaTeam>;
    return (const void*)k_norm_flat<BF16, EVEN, 4, CtaTeam>;
}

cudaError_t launch_norm(const dg_norm& op, cudaStream_t s) {
    const bool bf = op.type == DG_BF16;
    const int sms = sm_count();
    void* args[] = {const_cast<dg_norm*>(&op)};
    const uintptr_t rows_at = (uintptr_t)op.y | (uintptr_t)op.h | (uintptr_t)op.h_out | (uintptr_t)op.x_out |
                              (op.gate_rows == 1 ? 0 : (uintptr_t)op.gate);
    if (rows_at % 16 == 0 && op.N <= 32752) {
        const bool even = op.N % 8 == 0;
        const int vecs = even ? op.N / 8 : (op.N + 14) / 8;   // that a row of any shift touches
        // Lanes of a warp where they suffice (109692 x 108: a CTA of one warp each
        // 111 us, 16 lanes each 27.4), else a CTA with as few vectors a thread as
        // its 1024 threads allow (2000 x 8192 bf16: one 35.8 us, two 41.5).
        const int lanes = vecs <= 16 ? 16 : vecs <= 32 ? 32 : 0;
        const int C = lanes || vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4;
        const int threads = lanes ? kFlatThreads : ((vecs + C - 1) / C + 31) / 32 * 32;
        const int teams = lanes ? threads / lanes : 1;
        const int arrays = !!op.w_post + !!op.b_post + !!op.w_pre + !!op.b_pre + (op.gate && op.gate_rows == 1);
        const size_t smem = (size_t)arrays * C * threads * 16, room = 220000;
        // by registers (lane teams have up to 80 a thread, others 64), and by shared memory
        int resident = lanes ? 3 : 1024 / threads;
        if (smem) resident = std::min(resident, std::max(1, (int)(room / (smem + 1024))));
        // A row for every team at most: laying the weights out does not pay where
        // k_norm's vectors are as wide, or its rows short (300 x 2222: 4.8 us by
        // k_norm, 5.2 so; 44 x 12761: 12.1 and 7.0).
        const bool few = op.rows <= sms * resident * teams;
        if (smem <= room && !(few && (even || op.N <= 4096))) {
            const void* fn = bf ? even ? flat_fn<true, true>(lanes, C) : flat_fn<true, false>(lanes, C)
                                : even ? flat_fn<false, true>(lanes, C) : flat_fn<false, false>(lanes, C);
            const cudaError_t e = tc::smem_attr_once(fn, smem);
            if (e != cudaSuccess) return e;
            // a multiple of eight CTAs, but for a row a team at most
            const int ctas = few ? (op.rows + teams - 1) / teams : sms * resident / 8 * 8;
            return launch_pdl(fn, dim3(ctas), dim3(threads), smem, s, args);
        }
    }
    // 16-byte vectors where rows and pointers allow, pairs for even widths, else
    // single values
    uintptr_t low = (uintptr_t)op.N * 2, wide = (uintptr_t)op.h | (uintptr_t)op.h_out;
    const void* p16[] = {op.y, op.w_post, op.b_post, op.gate, op.w_pre, op.b_pre, op.x_out};
    for (const void* p : p16) low |= (uintptr_t)p;
    const int U = (low | wide) % 16 == 0 ? 8 : low % 4 == 0 && wide % (op.h_f32 ? 8 : 4) == 0 ? 2 : 1;
    const int vecs = (op.N + U - 1) / U;
    int threads = std::min((vecs + 31) / 32 * 32, 1024);
    if (vecs > threads * 16) threads = 512;   // up to 64 single values a thread
    const int C = (vecs + threads - 1) / threads;
    return launch_pdl(bf ? norm_fn_u<true>(U, C) : norm_fn_u<false>(U, C), dim3(op.rows), dim3(threads), 0, s, args);
}

}  // namespace dg
