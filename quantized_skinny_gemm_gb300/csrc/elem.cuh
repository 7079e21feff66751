// 16-bit element access shared by the layer kernels, for fp16 and bf16.
#pragma once

#include "dg_internal.cuh"

namespace dg {

template <bool BF16>
__device__ __forceinline__ float elem_f32(uint16_t v) {
    if (BF16) return __uint_as_float((uint32_t)v << 16);
    return __half2float(__ushort_as_half(v));
}

// Round to nearest even into the 16-bit type.
template <bool BF16>
__device__ __forceinline__ uint16_t elem_16(float v) {
    if (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    return __half_as_ushort(__float2half_rn(v));
}

template <bool BF16>
__device__ __forceinline__ float2 pair_f32(uint32_t v) {
    if (BF16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    return __half22float2(u32_as_h2(v));
}

// (a in the low half, b in the high half)
template <bool BF16>
__device__ __forceinline__ uint32_t pair_16(float a, float b) {
    if (BF16) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
        uint32_t u;
        memcpy(&u, &p, 4);
        return u;
    }
    return h2_as_u32(__floats2half2_rn(a, b));
}

// Products of two pairs, each rounded to the 16-bit type.
template <bool BF16>
__device__ __forceinline__ uint32_t mul_16(uint32_t a, uint32_t b) {
    uint32_t r;
    if (BF16)
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = pair_f32<BF16>(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pair_16<BF16>(f[0], f[1]), pair_16<BF16>(f[2], f[3]),
                      pair_16<BF16>(f[4], f[5]), pair_16<BF16>(f[6], f[7]));
}

// Division of 0 <= j < 2^31 by a fixed d >= 1: with s = ceil(log2 d) and mul =
// floor(2^(31 + s) / d) + 1 < 2^32, the high word of j * mul shifted by s - 1 is
// floor(j / d) exactly: mul is 2^(31 + s) / d + e with 0 < e <= 1, so j mul / 2^(31 + s)
// = j / d + j e / 2^(31 + s), and the last term is below 2^-s <= 1 / d.  mul 0: d = 1.
struct FastDiv {
    uint32_t mul;
    int shift;
};
inline FastDiv fast_div(uint32_t d) {
    if (d <= 1) return {0, 0};
    int log = 1;
    while ((1ull << log) < d) ++log;
    return {(uint32_t)((1ull << (31 + log)) / d + 1), log - 1};
}
__device__ __forceinline__ int operator/(int j, FastDiv f) {
    return f.mul ? (int)(__umulhi((uint32_t)j, f.mul) >> f.shift) : j;
}

// The page of position j >= 0 of sequence b and its slot there; page -1: none.  The
// table may be the work of the kernel before, which ran while this one had already
// started: no read-only load.
__device__ __forceinline__ int page_slot(const dg_paged_kv& kv, FastDiv page_size, int b, int j, int& slot) {
    const int at = j / page_size;
    slot = j - at * kv.page_size;
    if (at >= kv.max_pages) return -1;
    const int page = kv.block_table[(long long)b * kv.table_stride + at];
    return page >= 0 && page < kv.num_pages ? page : -1;
}

}  // namespace dg
