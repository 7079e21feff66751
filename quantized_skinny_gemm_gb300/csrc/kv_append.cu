// Rotary positions on a step's q and k, with k and v written into their pages.
#include "elem.cuh"

namespace dg {

// One token per grid row.  Its heads (q, then k, then v) are cut into units of
// U = 8 or 1 values: in the rotated part a unit is U pairs (U values and their
// U partners), elsewhere U plain values.  Each unit is one thread's, which
// reads all of it before it writes, so q_out may be q.
//
// Bound by latency at decode sizes (one token: a few KB, two dependent reads,
// length -> page id) and by HBM at large ones.
template <bool BF16, int U>
__global__ void __launch_bounds__(256) k_kv_append(const dg_append op) {
    griddep_launch_dependents();
    griddep_wait();
    const int t = blockIdx.x;
    const int b = t / op.q_len;
    const int D = op.kv.head_dim, half = op.rot_dim / 2;
    const int rot_units = half / U, units = rot_units + (D - op.rot_dim) / U;
    const int heads = op.heads + 2 * op.kv.kv_heads;
    const int at = blockIdx.y * blockDim.x + threadIdx.x;
    if (at >= heads * units) return;
    const int h = at / units, u = at - h * units;
    const int p = op.kv.seq_lens[b] - op.q_len + t % op.q_len;
    const bool live = p >= 0 && (op.rot_dim == 0 || p < op.max_pos);
    const bool is_q = h < op.heads, is_v = h >= op.heads + op.kv.kv_heads;
    const uint16_t* src;
    uint16_t* dst;
    if (is_q) {
        src = static_cast<const uint16_t*>(op.q) + t * op.q_stride + (long long)h * D;
        dst = static_cast<uint16_t*>(op.q_out) + t * op.q_out_stride + (long long)h * D;
    } else {
        const int page = live ? page_of(op.kv, b, p) : -1;
        if (page < 0) return;
        const int hk = h - op.heads - (is_v ? op.kv.kv_heads : 0);
        src = is_v ? static_cast<const uint16_t*>(op.v) + t * op.v_stride + (long long)hk * D
                   : static_cast<const uint16_t*>(op.k) + t * op.k_stride + (long long)hk * D;
        dst = static_cast<uint16_t*>(is_v ? op.kv.v : op.kv.k) + page * op.kv.page_stride +
              (p % op.kv.page_size) * op.kv.token_stride + hk * op.kv.head_stride;
    }
    // where this unit's values lie: first[i] at d0 + i, or (a pair) also at d1 + i
    const bool pair = u < rot_units;
    int d0, d1;
    if (!pair) {
        d0 = d1 = op.rot_dim + (u - rot_units) * U;
    } else if (op.interleaved) {
        d0 = 2 * u * U;
        d1 = d0 + U;
    } else {
        d0 = u * U;
        d1 = d0 + half;
    }
    if (U == 8) {
        const uint4 a = *reinterpret_cast<const uint4*>(src + d0);
        if (!pair) {
            *reinterpret_cast<uint4*>(dst + d0) = live ? a : make_uint4(0, 0, 0, 0);
            return;
        }
        const uint4 c = *reinterpret_cast<const uint4*>(src + d1);
        if (!live || is_v) {
            const uint4 z = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(dst + d0) = live ? a : z;
            *reinterpret_cast<uint4*>(dst + d1) = live ? c : z;
            return;
        }
        float f[2][8], cs[8], sn[8];
        unpack8<BF16>(a, f[0]);
        unpack8<BF16>(c, f[1]);
        const float* cp = op.cos + (long long)p * half + u * 8;
        const float* sp = op.sin + (long long)p * half + u * 8;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            *reinterpret_cast<float4*>(cs + i) = __ldg(reinterpret_cast<const float4*>(cp + i));
            *reinterpret_cast<float4*>(sn + i) = __ldg(reinterpret_cast<const float4*>(sp + i));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // interleaved: the 16 values in order are 8 neighbouring pairs
            float& x = op.interleaved ? f[i >> 2][2 * (i & 3)] : f[0][i];
            float& y = op.interleaved ? f[i >> 2][2 * (i & 3) + 1] : f[1][i];
            const float x0 = x, y0 = y;
            x = x0 * cs[i] - y0 * sn[i];
            y = y0 * cs[i] + x0 * sn[i];
        }
        *reinterpret_cast<uint4*>(dst + d0) = pack8<BF16>(f[0]);
        *reinterpret_cast<uint4*>(dst + d1) = pack8<BF16>(f[1]);
    } else {
        const uint16_t a = src[d0], c = src[d1];
        if (!pair || !live || is_v) {
            dst[d0] = live ? a : (uint16_t)0;
            if (pair) dst[d1] = live ? c : (uint16_t)0;
            return;
        }
        const float x = elem_f32<BF16>(a), y = elem_f32<BF16>(c);
        const float cs = op.cos[(long long)p * half + u], sn = op.sin[(long long)p * half + u];
        dst[d0] = elem_16<BF16>(x * cs - y * sn);
        dst[d1] = elem_16<BF16>(y * cs + x * sn);
    }
}

static bool vec_ok(const void* p, int64_t stride) {
    return ((uintptr_t)p & 15u) == 0 && stride % 8 == 0;
}

cudaError_t launch_kv_append(const dg_append& op, cudaStream_t s) {
    const dg_paged_kv& kv = op.kv;
    const bool vec = op.rot_dim % 16 == 0 && kv.head_dim % 8 == 0 && vec_ok(op.k, op.k_stride) &&
                     vec_ok(op.v, op.v_stride) && vec_ok(kv.k, kv.page_stride) &&
                     vec_ok(kv.v, kv.token_stride) && kv.head_stride % 8 == 0 &&
                     (!op.heads || (vec_ok(op.q, op.q_stride) && vec_ok(op.q_out, op.q_out_stride))) &&
                     (!op.rot_dim || (vec_ok(op.cos, 0) && vec_ok(op.sin, 0)));
    const int U = vec ? 8 : 1, half = op.rot_dim / 2;
    const int units = (half + kv.head_dim - op.rot_dim) / U * (op.heads + 2 * kv.kv_heads);
    const dim3 grid(kv.batch * op.q_len, (units + 255) / 256);
    const int threads = units < 256 ? (units + 31) / 32 * 32 : 256;
    const bool bf = kv.type == DG_BF16;
    const void* fn = vec ? (bf ? (const void*)k_kv_append<true, 8> : (const void*)k_kv_append<false, 8>)
                         : (bf ? (const void*)k_kv_append<true, 1> : (const void*)k_kv_append<false, 1>);
    void* args[] = {const_cast<dg_append*>(&op)};
    return launch_pdl(fn, grid, dim3(threads), 0, s, args);
}

}  // namespace dg
