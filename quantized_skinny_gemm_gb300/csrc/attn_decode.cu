// Attention of a step's new tokens over the paged key-value cache.
#include "elem.cuh"

namespace dg {

constexpr int kAttnThreads = 128;

// One CTA per query row (token and head); its threads share the positions,
// each keeping its own running maximum, sum and output, joined at the end.
template <bool BF16>
__global__ void __launch_bounds__(kAttnThreads) k_attn_rows(const dg_attn op) {
    griddep_launch_dependents();
    griddep_wait();
    const int D = op.kv.head_dim, t = blockIdx.x, h = blockIdx.y;
    const int b = t / op.q_len;
    const int p = op.kv.seq_lens[b] - op.q_len + t % op.q_len;
    const int g = h / (op.heads / op.kv.kv_heads);
    __shared__ float q[256], part[kAttnThreads][33];
    __shared__ float smax[kAttnThreads], ssum[kAttnThreads];
    const uint16_t* qr = static_cast<const uint16_t*>(op.q) + t * op.q_stride + (long long)h * D;
    for (int d = threadIdx.x; d < D; d += kAttnThreads) q[d] = elem_f32<BF16>(qr[d]);
    __syncthreads();
    float m = -INFINITY, l = 0.f;
    const int last = (int)min((long long)p, (long long)op.kv.max_pages * op.kv.page_size - 1);
    const int lo = op.window ? max(0, p - op.window + 1) : 0;
    // the positions are walked once for the maximum and sum, then once per 32 dims
    for (int pass = -1; pass < (D + 31) / 32; ++pass) {
        float o[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0.f;
        for (int j = threadIdx.x; j <= last; j += kAttnThreads) {
            if (j < lo && j >= op.sinks) continue;
            const int page = page_of(op.kv, b, j);
            if (page < 0) continue;
            const long long at = page * op.kv.page_stride +
                                 (j % op.kv.page_size) * op.kv.token_stride + g * op.kv.head_stride;
            const uint16_t* k = static_cast<const uint16_t*>(op.kv.k) + at;
            const uint16_t* v = static_cast<const uint16_t*>(op.kv.v) + at;
            float z = 0.f;
            for (int d = 0; d < D; ++d) z = fmaf(q[d], elem_f32<BF16>(k[d]), z);
            z *= op.scale;
            if (pass < 0) {
                const float nm = fmaxf(m, z);
                if (z != z) {
                    l = z;
                } else if (nm != -INFINITY) {
                    l = l * expf(m - nm) + expf(z - nm);
                    m = nm;
                }
            } else {
                const float w = z != z ? z : m == -INFINITY ? 0.f : expf(z - m);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (pass * 32 + i < D) o[i] = fmaf(w, elem_f32<BF16>(v[pass * 32 + i]), o[i]);
            }
        }
        if (pass < 0) {
            smax[threadIdx.x] = m;
            ssum[threadIdx.x] = l;
            __syncthreads();
            float top = -INFINITY, sum = 0.f;
            for (int i = 0; i < kAttnThreads; ++i) top = fmaxf(top, smax[i]);
            for (int i = 0; i < kAttnThreads; ++i)
                if (smax[i] != -INFINITY) sum += ssum[i] * expf(smax[i] - top);
                else if (ssum[i] != ssum[i]) sum = ssum[i];
            m = top;
            l = sum;
            if (threadIdx.x == 0 && op.lse)
                op.lse[(long long)t * op.heads + h] = l == 0.f ? -INFINITY : m + logf(l);
        } else {
            for (int i = 0; i < 32; ++i) part[threadIdx.x][i] = o[i];
            __syncthreads();
            if (threadIdx.x < 32 && pass * 32 + (int)threadIdx.x < D) {
                float s = 0.f;
                for (int i = 0; i < kAttnThreads; ++i) s += part[i][threadIdx.x];
                uint16_t* out = static_cast<uint16_t*>(op.out) + t * op.out_stride + (long long)h * D;
                out[pass * 32 + threadIdx.x] = elem_16<BF16>(l == 0.f ? 0.f : s / l);
            }
            __syncthreads();
        }
    }
}

size_t attn_ws_bytes(const dg_attn&) { return 16; }

cudaError_t launch_attn(const dg_attn& op, void*, cudaStream_t s) {
    const void* fn = op.kv.type == DG_BF16 ? (const void*)k_attn_rows<true> : (const void*)k_attn_rows<false>;
    void* args[] = {const_cast<dg_attn*>(&op)};
    return launch_pdl(fn, dim3(op.kv.batch * op.q_len, op.heads), dim3(kAttnThreads), 0, s, args);
}

}  // namespace dg
