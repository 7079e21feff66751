// A mixture-of-experts layer for a few tokens: router and top-k, gate and up
// products with SwiGLU, down product with the weighted sum over experts.
#include "elem.cuh"

namespace dg {

// One CTA per token: router scores, probabilities, and the top_k choices.
template <bool BF16>
__global__ void __launch_bounds__(256) k_moe_route(const dg_moe op, int* ids, float* wts) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float prob[1024];
    const int m = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t* x = static_cast<const uint16_t*>(op.x) + (size_t)m * op.K;
    for (int e = warp; e < op.E; e += 8) {
        const uint16_t* r = static_cast<const uint16_t*>(op.router) + (size_t)e * op.K;
        float z = 0.f;
        for (int k = lane; k < op.K; k += 32) z = fmaf(elem_f32<BF16>(x[k]), elem_f32<BF16>(r[k]), z);
        z = warp_sum(z);
        if (lane == 0) prob[e] = z;
    }
    __syncthreads();
    if (threadIdx.x) return;
    if (op.score == DG_MOE_SOFTMAX) {
        float top = -INFINITY, sum = 0.f;
        for (int e = 0; e < op.E; ++e) top = fmaxf(top, prob[e]);
        for (int e = 0; e < op.E; ++e) sum += prob[e] = expf(prob[e] - top);
        for (int e = 0; e < op.E; ++e) prob[e] /= sum;
    } else {
        for (int e = 0; e < op.E; ++e) prob[e] = 1.f / (1.f + expf(-prob[e]));
    }
    float total = 0.f, chosen[16];
    int id[16];
    for (int k = 0; k < op.top_k; ++k) {
        float bv = NAN;
        int bi = -1;
        for (int e = 0; e < op.E; ++e) {
            bool taken = false;
            for (int i = 0; i < k; ++i) taken = taken || id[i] == e;
            if (!taken && (bi < 0 || arg_better(prob[e], e, bv, bi))) {
                bv = prob[e];
                bi = e;
            }
        }
        id[k] = bi;
        chosen[k] = bv;
        total += bv;
    }
    for (int k = 0; k < op.top_k; ++k) {
        const float w = (op.renormalize ? chosen[k] / total : chosen[k]) * op.route_scale;
        ids[m * op.top_k + k] = id[k];
        wts[m * op.top_k + k] = w;
        if (op.ids) op.ids[m * op.top_k + k] = id[k];
        if (op.weights) op.weights[m * op.top_k + k] = w;
    }
}

// Element k of row `row` of a matrix [rows][cols].
template <int KIND>
__device__ __forceinline__ float moe_w(const void* W, const void* scale, size_t row, int cols, int k,
                                       int group) {
    if (KIND == DG_LINEAR_W4A16) {
        const uint8_t byte = static_cast<const uint8_t*>(W)[row * (cols / 2) + k / 2];
        const int q = (((k & 1) ? byte >> 4 : byte & 15) ^ 8) - 8;
        return (float)q * __half2float(static_cast<const __half*>(scale)[row * (cols / group) + k / group]);
    }
    return elem_f32<KIND == DG_LINEAR_BF16>(static_cast<const uint16_t*>(W)[row * cols + k]);
}

// One warp per (token, choice, intermediate row).
template <int KIND>
__global__ void __launch_bounds__(256) k_moe_up(const dg_moe op, const int* ids, float* h) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, slot = blockIdx.y;
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= op.I) return;
    const uint16_t* x = static_cast<const uint16_t*>(op.x) + (size_t)(slot / op.top_k) * op.K;
    const size_t row = (size_t)ids[slot] * op.I + i;
    float g = 0.f, u = 0.f;
    for (int k = lane; k < op.K; k += 32) {
        const float v = elem_f32<KIND == DG_LINEAR_BF16>(x[k]);
        g = fmaf(moe_w<KIND>(op.W_gate, op.gate_scale, row, op.K, k, op.group_size), v, g);
        u = fmaf(moe_w<KIND>(op.W_up, op.up_scale, row, op.K, k, op.group_size), v, u);
    }
    g = warp_sum(g);
    u = warp_sum(u);
    if (lane == 0) h[(size_t)slot * op.I + i] = silu_f32(g) * u;
}

// One warp per (token, output row).
template <int KIND>
__global__ void __launch_bounds__(256) k_moe_down(const dg_moe op, const int* ids, const float* wts,
                                                  const float* h) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, m = blockIdx.y;
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (n >= op.K) return;
    float y = 0.f;
    for (int c = 0; c < op.top_k; ++c) {
        const int slot = m * op.top_k + c;
        const size_t row = (size_t)ids[slot] * op.K + n;
        float s = 0.f;
        for (int i = lane; i < op.I; i += 32)
            s = fmaf(moe_w<KIND>(op.W_down, op.down_scale, row, op.I, i, op.group_size),
                     h[(size_t)slot * op.I + i], s);
        y = fmaf(wts[slot], warp_sum(s), y);
    }
    constexpr bool BF = KIND == DG_LINEAR_BF16;
    if (lane == 0) {
        const size_t at = (size_t)m * op.K + n;
        if (op.residual) y += elem_f32<BF>(static_cast<const uint16_t*>(op.residual)[at]);
        static_cast<uint16_t*>(op.y)[at] = elem_16<BF>(y);
    }
}

size_t moe_ws_bytes(const dg_moe& op) {
    const size_t slots = (size_t)op.M * op.top_k;
    return 4096 + slots * op.I * 4;
}

template <int KIND>
static cudaError_t launch_moe_kind(const dg_moe& op, void* ws, cudaStream_t s) {
    int* ids = static_cast<int*>(ws);                              // [256]
    float* wts = reinterpret_cast<float*>(ids + 256);              // [256]
    float* h = reinterpret_cast<float*>(static_cast<char*>(ws) + 4096);
    void* a1[] = {const_cast<dg_moe*>(&op), &ids, &wts};
    cudaError_t e = launch_pdl((const void*)k_moe_route<KIND == DG_LINEAR_BF16>, dim3(op.M), dim3(256), 0, s, a1);
    if (e != cudaSuccess) return e;
    void* a2[] = {const_cast<dg_moe*>(&op), &ids, &h};
    e = launch_pdl((const void*)k_moe_up<KIND>, dim3((op.I + 7) / 8, op.M * op.top_k), dim3(256), 0, s, a2);
    if (e != cudaSuccess) return e;
    void* a3[] = {const_cast<dg_moe*>(&op), &ids, &wts, &h};
    return launch_pdl((const void*)k_moe_down<KIND>, dim3((op.K + 7) / 8, op.M), dim3(256), 0, s, a3);
}

cudaError_t launch_moe(const dg_moe& op, void* ws, cudaStream_t s) {
    switch (op.kind) {
        case DG_LINEAR_F16: return launch_moe_kind<DG_LINEAR_F16>(op, ws, s);
        case DG_LINEAR_BF16: return launch_moe_kind<DG_LINEAR_BF16>(op, ws, s);
        default: return launch_moe_kind<DG_LINEAR_W4A16>(op, ws, s);
    }
}

}  // namespace dg
