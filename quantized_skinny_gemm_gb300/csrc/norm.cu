// The norms around a block, fused with its gate and residual scale.
#include "elem.cuh"

namespace dg {

// Sum over the CTA, the same in every thread.  `red` alternates between two
// halves from call to call, so one barrier per call is enough.
__device__ __forceinline__ float cta_sum(float v, float (*red)[32], int& turn) {
    v = warp_sum(v);
    float* r = red[turn];
    turn ^= 1;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return warp_sum(lane < warps ? r[lane] : 0.f);
}

// Value j of chunk c of this thread is element ((c * blockDim.x + threadIdx.x) * U + j).
template <int U, int C>
struct RowRegs {
    float v[C][U];
};

// Vector c of a row, zero past its end.
template <bool BF16, int U>
__device__ __forceinline__ void load_part(const void* p, int N, int c, float (&f)[U]) {
    const uint16_t* e = static_cast<const uint16_t*>(p);
    const int n = (c * blockDim.x + threadIdx.x) * U;
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
__device__ __forceinline__ void load_part_f32(const float* p, int N, int c, float (&f)[U]) {
    const int n = (c * blockDim.x + threadIdx.x) * U;
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
__device__ __forceinline__ void store_row(void* p, int N, const RowRegs<U, C>& r) {
    uint16_t* e = static_cast<uint16_t*>(p);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int n = (c * blockDim.x + threadIdx.x) * U;
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
__device__ __forceinline__ void store_row_f32(float* p, int N, const RowRegs<U, C>& r) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int n = (c * blockDim.x + threadIdx.x) * U;
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
__device__ __forceinline__ void norm_row(const dg_norm& op, const void* w, const void* b,
                                         RowRegs<U, C>& r, float (*red)[32], int& turn) {
    const int N = op.N;
    if (op.kind == DG_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < U; ++j) s += r.v[c][j];
        const float mean = cta_sum(s, red, turn) / (float)N;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < U; ++j)
                if ((c * (int)blockDim.x + (int)threadIdx.x) * U < N) r.v[c][j] -= mean;
    }
    float q = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < U; ++j) q = fmaf(r.v[c][j], r.v[c][j], q);
    const float k = 1.f / sqrtf(cta_sum(q, red, turn) / (float)N + op.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float g[U];
        load_part<BF16>(w, N, c, g);
#pragma unroll
        for (int j = 0; j < U; ++j) r.v[c][j] = r.v[c][j] * k * (op.w_offset + g[j]);
        if (b) {
            load_part<BF16>(b, N, c, g);
#pragma unroll
            for (int j = 0; j < U; ++j) r.v[c][j] += g[j];
        }
    }
}

// One CTA per row, the row held in registers (U values per vector, C vectors
// per thread), so y and h are read once and h' and x written once.
template <bool BF16, int U, int C>
__global__ void __launch_bounds__(1024) k_norm(const dg_norm op) {
    __shared__ float red[2][32];
    int turn = 0;
    griddep_launch_dependents();
    griddep_wait();
    const int N = op.N;
    const size_t at = (size_t)blockIdx.x * N;
    RowRegs<U, C> r;
    const uint16_t* y = static_cast<const uint16_t*>(op.y) + at;
    const uint16_t* gate = static_cast<const uint16_t*>(op.gate) + (op.gate_rows == 1 ? 0 : at);
    if (op.y) {
#pragma unroll
        for (int c = 0; c < C; ++c) load_part<BF16>(y, N, c, r.v[c]);
        if (op.w_post) norm_row<BF16>(op, op.w_post, op.b_post, r, red, turn);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float h[U], g[U];
        if (op.h) {
            if (op.h_f32)
                load_part_f32(static_cast<const float*>(op.h) + at, N, c, h);
            else
                load_part<BF16>(static_cast<const uint16_t*>(op.h) + at, N, c, h);
        }
        if (op.gate) load_part<BF16>(gate, N, c, g);
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
            store_row_f32(static_cast<float*>(op.h_out) + at, N, r);
        else
            store_row<BF16>(static_cast<uint16_t*>(op.h_out) + at, N, r);
    }
    if (op.x_out) {
        norm_row<BF16>(op, op.w_pre, op.b_pre, r, red, turn);
        store_row<BF16>(static_cast<uint16_t*>(op.x_out) + at, N, r);
    }
}

// The same for many rows of up to 8192 values in vectors of eight, one vector a
// thread: each CTA takes every gridDim.x-th row and loads the next row's y, h
// and gate before it reduces this one, so that HBM stays busy over the CTA-wide
// sums (4096 x 4096 bf16 with an fp32 residual, both norms and a gate, 235 MB: one
// CTA per row 47.9 us).
struct RowRaw {
    uint4 y, gate, h[2];
};
template <bool BF16>
__device__ __forceinline__ void fetch_row(const dg_norm& op, int row, RowRaw& q) {
    const int n = threadIdx.x * 8;
    if (row >= op.rows || n >= op.N) return;
    const size_t at = (size_t)row * op.N + n;
    if (op.y) q.y = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(op.y) + at));
    if (op.gate && op.gate_rows != 1)
        q.gate = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(op.gate) + at));
    if (op.h) {
        if (op.h_f32) {
            const uint4* h = reinterpret_cast<const uint4*>(static_cast<const float*>(op.h) + at);
            q.h[0] = __ldcs(h);
            q.h[1] = __ldcs(h + 1);
        } else {
            q.h[0] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(op.h) + at));
        }
    }
}

template <bool BF16>
__global__ void __launch_bounds__(1024) k_norm_rows(const dg_norm op) {
    __shared__ float red[2][32];
    int turn = 0;
    griddep_launch_dependents();
    griddep_wait();
    const int N = op.N, n = threadIdx.x * 8;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    RowRaw next{zero, zero, {zero, zero}};
    if (op.gate && op.gate_rows == 1 && n < N)
        next.gate = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(op.gate) + n);
    fetch_row<BF16>(op, blockIdx.x, next);
    for (int row = blockIdx.x; row < op.rows; row += gridDim.x) {
        RowRegs<8, 1> r;
        {
            float y[8], h[8], g[8];
            unpack8<BF16>(next.y, y);
            unpack8<BF16>(next.gate, g);
            if (op.h_f32) {
                memcpy(h, next.h, 32);
            } else {
                unpack8<BF16>(next.h[0], h);
            }
            fetch_row<BF16>(op, row + gridDim.x, next);
#pragma unroll
            for (int j = 0; j < 8; ++j) r.v[0][j] = y[j];
            if (op.y && op.w_post) norm_row<BF16>(op, op.w_post, op.b_post, r, red, turn);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float v = r.v[0][j];
                if (op.gate) v *= g[j];
                const float a = h[j] * op.alpha;
                r.v[0][j] = !op.y ? a : op.h ? fmaf(op.beta, v, a) : op.beta * v;
            }
        }
        const size_t at = (size_t)row * N;
        if (op.h_out) {
            if (op.h_f32)
                store_row_f32(static_cast<float*>(op.h_out) + at, N, r);
            else
                store_row<BF16>(static_cast<uint16_t*>(op.h_out) + at, N, r);
        }
        if (op.x_out) {
            norm_row<BF16>(op, op.w_pre, op.b_pre, r, red, turn);
            store_row<BF16>(static_cast<uint16_t*>(op.x_out) + at, N, r);
        }
    }
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
    if constexpr (U < 2) return (const void*)k_norm<BF16, U, 32>;
    return nullptr;
}

cudaError_t launch_norm(const dg_norm& op, cudaStream_t s) {
    // 16-byte vectors where rows and pointers allow, pairs for even widths, else
    // single values
    const void* p16[] = {op.y, op.w_post, op.b_post, op.gate, op.w_pre, op.b_pre, op.x_out};
    uintptr_t low = (uintptr_t)op.N * 2, wide = 0;
    for (const void* p : p16) low |= (uintptr_t)p;
    wide = (uintptr_t)op.h | (uintptr_t)op.h_out;
    const int U = (low | wide) % 16 == 0 ? 8 : low % 4 == 0 && wide % (op.h_f32 ? 8 : 4) == 0 ? 2 : 1;
    const int vecs = (op.N + U - 1) / U;
    int threads = (vecs + 31) / 32 * 32;
    if (threads > 1024) threads = 1024;
    const int C = (vecs + threads - 1) / threads;
    const bool bf = op.type == DG_BF16;
    const void* fn = U == 8   ? (bf ? norm_fn<true, 8>(C) : norm_fn<false, 8>(C))
                     : U == 2 ? (bf ? norm_fn<true, 2>(C) : norm_fn<false, 2>(C))
                              : (bf ? norm_fn<true, 1>(C) : norm_fn<false, 1>(C));
    void* args[] = {const_cast<dg_norm*>(&op)};
    // 64 registers a thread: as many CTAs as an SM's 65536 hold
    const int resident = sm_count() * (1024 / threads);
    if (U == 8 && C == 1 && op.rows > resident)
        return launch_pdl(bf ? (const void*)k_norm_rows<true> : (const void*)k_norm_rows<false>,
                          dim3(resident), dim3(threads), 0, s, args);
    return launch_pdl(fn, dim3(op.rows), dim3(threads), 0, s, args);
}

}  // namespace dg
