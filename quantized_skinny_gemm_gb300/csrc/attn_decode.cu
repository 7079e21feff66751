// Attention of a step's new tokens over the paged key-value cache.
//
// The cost is the cache: 4 * head_dim bytes per visible position and key /
// value head, read once, against 4 * head_dim flops per query row, so up to a
// few dozen rows per key / value head (query heads of the group x new tokens)
// the kernel is bound by HBM as long as the rows share each key they read.
// Rows therefore form 16-row tiles of mma.sync (m16n8k16, fp32 accumulators);
// one stage of a warp is 16 keys (32 of up to 64 dims) and their values, copied
// into the warp's own ring of shared memory by cp.async (16 bytes a lane: any
// page size, stride and head size), so warps never wait for one another while
// they stream.
//
// Work split.  The visible positions of one (sequence, key / value head, row
// group) are a unit of blocks of kBlockKeys positions.  All blocks of the call,
// counted on the device from the lengths, are cut into one equal contiguous
// range per CTA; a unit that lies in one CTA's range is finished there, one
// that was cut leaves fp32 parts (maximum, sum, output) in the workspace that
// k_attn_join adds in CTA order.  So ragged batches and single long sequences
// load every SM alike, and no sum depends on timing.
//
// Softmax is one pass: each warp keeps the running maximum m and sum l of its
// own positions and rescales its output only when m has grown by more than
// 2^8 since (weights then stay below 256); differences of scores are turned to
// units of log2(e) inside the exponent.  A weight meets the values as two 16-bit numbers
// (split_pair), at half as many matrix instructions again: 0.4 % on the long
// cache below, 4 to 5 % on the others, 19 % where 64 rows share a key.
//
// Measured: 200001 positions of 8 x 128 bf16, 32 heads: 127 us, 6.4 TB/s of the
// copy's 6.8; 16 sequences of up to 8191, 12 heads on 2: 11.5 us; one of 100: 5.6
// us, one launch where the table holds 128 positions at most, else two (in a graph
// 5.1 and, in a table of 4096, 5.9); 8 tokens
// of 8 sequences on windows of 4096, 32 heads on 8 of 64: 33 us, bound by the
// latency of a few stages per warp and of the join.
#include "attn_common.cuh"

namespace dg {

template <int DP, int RT>
struct AttnShape {
    // 16-key pieces of a stage: two where they are small, for the bookkeeping of a
    // stage (64 dims, with weights of one 16-bit number: 31 us on the windows above
    // and 60 on 12 sequences of up to 84056 positions; stages of 16 keys with 3 CTAs
    // per SM 42 and 85)
    static constexpr int kSub = DP <= 64 && RT < 4 ? 2 : 1;
    static constexpr int kKeys = 16 * kSub;
    static constexpr int kPitch = DP * 2;                   // bytes; see piece()
    static constexpr int kStage = 2 * kKeys * kPitch;       // keys, then values
    static constexpr int kCtas = DP <= 192 ? 2 : 1;  // per SM
    static constexpr int kStages = RT == 4 ? 5 : DP <= 128 ? 3 : DP <= 192 ? 2 : 3;
    static constexpr int kRing = kStages * kStage;
    static constexpr int kRows = RT * 16;
    static constexpr int kQ = kRows * kPitch;
    static constexpr size_t kSmem = (size_t)kAttnWarps * kRing + kQ + 2 * kAttnWarps * kRows * 4;
    static constexpr int kPart = part_floats(kRows, DP);
    // Byte of 16-byte piece c of row r: the pieces of 128 bytes change places by
    // the row's low bits, so that eight rows' same piece lie in different banks.
    __device__ static constexpr int piece(int r, int c) { return r * kPitch + ((c ^ (r & 7)) << 4); }
    // Value group d (8 floats) of row r of a warp's output, in place of stages.
    __device__ static constexpr int out_at(int r, int d) { return r * DP + ((d ^ (r & 3)) << 3); }
    static_assert(kRows * DP * 4 <= (kStages - 1) * kStage, "a warp's output leaves a stage free");
    static_assert(kCtas * (kSmem + 2048) <= 228 * 1024, "an SM holds its CTAs");
};

template <bool BF16, int DP, int RT>
__global__ void __launch_bounds__(kAttnThreads, AttnShape<DP, RT>::kCtas) k_attn(const AttnParams p) {
    using S = AttnShape<DP, RT>;
    extern __shared__ __align__(128) unsigned char smem[];
    const dg_attn& op = p.op;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = op.kv.head_dim, G = op.heads / op.kv.kv_heads;
    const int heads = op.kv.kv_heads * p.groups;   // units per sequence
    unsigned char* ring = smem + warp * S::kRing;
    const uint32_t ring_a = (uint32_t)__cvta_generic_to_shared(ring);
    unsigned char* qs = smem + kAttnWarps * S::kRing;
    const uint32_t qs_a = (uint32_t)__cvta_generic_to_shared(qs);
    float* sm_m = reinterpret_cast<float*>(qs + S::kQ);
    float* sm_l = sm_m + kAttnWarps * S::kRows;

    griddep_launch_dependents();
    griddep_wait();

    __shared__ RangeScan scan;
    const CtaRange range = find_range(op, heads, scan);
    const long long begin = range.begin, end = range.end;
    int b = range.b;
    long long seq_at = range.seq_at;   // first block of sequence b
    if (begin >= end) return;

    // e^(scale q.k) = 2^(c2 (q'.k)) with c2 > 0: the sign, and a scale of zero, go into
    // q'.  A weight's exponent is c2 times the difference to the maximum, not the
    // difference of two products: past scores of 2^24 those are rounded by whole
    // numbers, and a strongest key of weight 2^64 overflows.  (Parts are joined by
    // products: there the greatest one's weight is 1 whatever the rounding.)
    const float c2 = op.scale == 0.f ? 1.f : fabsf(op.scale) * kLog2e;
    const float sign = op.scale > 0.f ? 1.f : op.scale < 0.f ? -1.f : 0.f;
    const uint32_t sign2 = pair_16<BF16>(sign, sign);
    const float grow = fminf(8.f / c2, FLT_MAX);   // finite: the first maximum is always taken
    const int g = lane >> 2, t4 = lane & 3;

    // ---- the range's part of one unit after another ---------------------------------------
    struct Segment {
        int b, hk, row0;   // sequence, key / value head, first row
        int kb, ke, nb;    // blocks [kb, ke) of nb
        Span sp;
        int key0, lim, n;  // this warp's n stages: kKeys keys from key0 on, then every
                           // kStep further, up to lim
    } sg;
    constexpr int kKeys = S::kKeys, kStep = kAttnWarps * kKeys, kStages = S::kStages;
    auto enter = [&](long long blk, bool first) {
        sg.sp = span_of(op, b);
        sg.nb = blocks_of(sg.sp);
        while (blk >= seq_at + (long long)sg.nb * heads) {
            seq_at += (long long)sg.nb * heads;
            sg.sp = span_of(op, ++b);
            sg.nb = blocks_of(sg.sp);
        }
        const int unit = quotient(blk - seq_at, sg.nb);
        sg.b = b;
        sg.kb = (int)(blk - seq_at - (long long)unit * sg.nb);
        sg.ke = (int)min((long long)sg.nb, sg.kb + (end - blk));
        sg.hk = unit / p.groups;
        sg.row0 = (unit - sg.hk * p.groups) * S::kRows;
        sg.key0 = sg.kb * kBlockKeys + warp * kKeys;
        sg.lim = sg.ke == sg.nb ? sg.sp.count() : sg.ke * kBlockKeys;   // nb * kBlockKeys may be 2^31
        sg.n = sg.key0 < sg.lim ? (int)((unsigned)(sg.lim - sg.key0 + kStep - 1) / kStep) : 0;
        if (sg.kb == 0 && tid == 0 && p.info)
            p.info[(long long)b * heads + unit] = unit_parts(range, blk, sg.nb, sg.ke, first);
    };
    // Position and cache offset (elements; -1: nothing there) of key `lane` (lane
    // mod kKeys) of stage i.
    auto locate = [&](int i, int& pos, long long& off) {
        const unsigned c = (unsigned)sg.key0 + (unsigned)i * kStep + (lane & (kKeys - 1));
        pos = INT_MAX;
        off = -1;
        if (i < sg.n && c < (unsigned)sg.lim) {
            const int j = sg.sp.position((int)c);
            int slot = 0;
            const int page = sg.sp.seen(j) ? page_slot(op.kv, p.page_size, sg.b, j, slot) : -1;
            if (page >= 0) {
                pos = j;
                off = page * op.kv.page_stride + slot * op.kv.token_stride + sg.hk * op.kv.head_stride;
            }
        }
    };
    // Stage i lies in ring place (i - 1) mod kStages, so that the first one's is
    // not in the way of the last segment's output.
    auto place = [](int i) { return (i + kStages - 1) % kStages; };
    auto issue = [&](int i, long long off) {
        if (i < sg.n) {
            const uint32_t dst = ring_a + place(i) * S::kStage;
            constexpr int kChunks = DP / 8;
            // keys in a row in one page: addresses without exchanges
            const long long o0 = __shfl_sync(0xffffffffu, off, 0);
            const bool run = off >= 0 && off == o0 + (lane & (kKeys - 1)) * op.kv.token_stride;
            if (32 % kChunks == 0 && __all_sync(0xffffffffu, run)) {
                constexpr int kRows = 32 % kChunks == 0 ? 32 / kChunks : 1;   // rows of an instruction
                const int row = lane / kChunks, ch = lane % kChunks;
                const bool in = ch * 8 < D;   // dims past the head's read as zero
                const long long at = o0 + row * op.kv.token_stride + (in ? ch * 8 : 0);
                const uint16_t* k = static_cast<const uint16_t*>(op.kv.k) + at;
                const uint16_t* v = static_cast<const uint16_t*>(op.kv.v) + at;
                const long long step = kRows * op.kv.token_stride;
#pragma unroll
                for (int it = 0; it < kKeys / kRows; ++it) {
                    const uint32_t d = dst + S::piece(it * kRows + row, ch);
                    cp_async16(d, k, in);
                    cp_async16(d + kKeys * S::kPitch, v, in);
                    k += step;
                    v += step;
                }
            } else {
#pragma unroll
                for (int it = 0; it < kKeys * kChunks / 32; ++it) {
                    const int idx = it * 32 + lane, row = idx / kChunks, ch = idx % kChunks;
                    const long long o = __shfl_sync(0xffffffffu, off, row);
                    const bool in = o >= 0 && ch * 8 < D;
                    const long long at = in ? o + ch * 8 : 0;
                    const uint32_t d = dst + S::piece(row, ch);
                    cp_async16(d, static_cast<const uint16_t*>(op.kv.k) + at, in);
                    cp_async16(d + kKeys * S::kPitch, static_cast<const uint16_t*>(op.kv.v) + at, in);
                }
            }
        }
        cp_commit();
    };
    // q rows of the unit, zero past the last and past the head's dims
    constexpr int kQv = (S::kRows * (DP / 8) + kAttnThreads - 1) / kAttnThreads;
    uint4 qv[kQv];
    auto load_q = [&] {
#pragma unroll
        for (int x = 0; x < kQv; ++x) {
            const int i = x * kAttnThreads + tid, r = i / (DP / 8), ch = i % (DP / 8), row = sg.row0 + r;
            qv[x] = make_uint4(0, 0, 0, 0);
            if (r < S::kRows && row < p.rows && ch * 8 < D) {
                const int tok = row / G;
                qv[x] = __ldcg(reinterpret_cast<const uint4*>(
                    static_cast<const uint16_t*>(op.q) + ((long long)sg.b * op.q_len + tok) * op.q_stride +
                    (long long)(sg.hk * G + row - tok * G) * D + ch * 8));
            }
        }
    };
    auto store_q = [&] {
#pragma unroll
        for (int x = 0; x < kQv; ++x) {
            const int i = x * kAttnThreads + tid, r = i / (DP / 8), ch = i % (DP / 8);
            if (r >= S::kRows) continue;
            const uint4 v = qv[x];   // a product, so that zero times infinity is NaN
            *reinterpret_cast<uint4*>(qs + S::piece(r, ch)) =
                make_uint4(mul_16<BF16>(v.x, sign2), mul_16<BF16>(v.y, sign2), mul_16<BF16>(v.z, sign2),
                           mul_16<BF16>(v.w, sign2));
        }
    };

    int pos[kStages];              // positions of the stages in flight, by stage mod kStages
    long long offs[kStages];
    int pos_next;
    long long off_next;
    long long blk = begin;
    enter(blk, true);
    load_q();
#pragma unroll
    for (int i = 0; i < kStages; ++i) locate(i, pos[i], offs[i]);
    issue(0, offs[0]);
    for (bool first_segment = true;; first_segment = false) {
#pragma unroll
        for (int i = 1; i < kStages - 1; ++i) issue(i, offs[i]);
        pos_next = pos[kStages - 1];
        off_next = offs[kStages - 1];
        store_q();
        __syncthreads();
        const Span sp = sg.sp;
        const int row0 = sg.row0, n = sg.n, last = sp.first + op.q_len - 1;

        float o[RT][DP / 8][4], m[RT][2], l[RT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int d = 0; d < DP / 8; ++d) o[r][d][0] = o[r][d][1] = o[r][d][2] = o[r][d][3] = 0.f;
            m[r][0] = m[r][1] = -INFINITY;
            l[r][0] = l[r][1] = 0.f;
        }
        // q stays in registers where they suffice, else it is read again for every stage
        constexpr bool kKeepQ = RT == 1 || RT * DP <= 128;
        uint32_t qf[kKeepQ ? RT : 1][kKeepQ ? DP / 16 : 1][4];
        // ldmatrix: this lane's row and first piece; piece 2 k further is 32 k bytes on,
        // xor-ed inside 128 bytes
        const uint32_t qa = qs_a + S::piece((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
        auto on = [](uint32_t at, int k) { return (at ^ (k * 32 & 127)) + (k * 32 & ~127); };
        if constexpr (kKeepQ) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) ldsm4(qf[r][k], on(qa, k) + r * 16 * S::kPitch);
        }

#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            cp_wait<kStages - 2>();
            __syncwarp();
            const int slot = place(i);
            const uint32_t ka = ring_a + slot * S::kStage, va = ka + kKeys * S::kPitch;
            int my_pos = pos[0];
#pragma unroll
            for (int q = 1; q < kStages; ++q)
                if (i % kStages == q) my_pos = pos[q];
            // the place that the last stage left is free: refill it
            const int ni = i + kStages - 1;
#pragma unroll
            for (int q = 0; q < kStages; ++q)
                if (ni % kStages == q) pos[q] = pos_next;
            issue(ni, off_next);
            locate(ni + 1, pos_next, off_next);

            // scores of the stage's keys, 8 to a block
            constexpr int kBlk = 2 * S::kSub;
            float s[RT][kBlk][4];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int j = 0; j < kBlk; ++j) s[r][j][0] = s[r][j][1] = s[r][j][2] = s[r][j][3] = 0.f;
            const uint32_t kl = ka + S::piece((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
                uint32_t kf[S::kSub][4];
#pragma unroll
                for (int u = 0; u < S::kSub; ++u) ldsm4(kf[u], on(kl, k) + u * 16 * S::kPitch);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    uint32_t qr[4];
                    if (!kKeepQ) ldsm4(qr, on(qa, k) + r * 16 * S::kPitch);
                    const uint32_t(&a)[4] = kKeepQ ? qf[kKeepQ ? r : 0][kKeepQ ? k : 0] : qr;
#pragma unroll
                    for (int u = 0; u < S::kSub; ++u) {
                        mma16816<BF16>(s[r][2 * u], a, kf[u][0], kf[u][1]);
                        mma16816<BF16>(s[r][2 * u + 1], a, kf[u][2], kf[u][3]);
                    }
                }
            }
            // masks, where some row does not see some key of the stage
            const bool all = my_pos <= sp.first &&
                             (!op.window || last - my_pos < op.window || my_pos < op.sinks);
            unsigned poison = 0;   // keys whose values are not finite
            if (!__all_sync(0xffffffffu, all)) {
#pragma unroll
                for (int j = 0; j < kBlk; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int kp = __shfl_sync(0xffffffffu, my_pos, j * 8 + t4 * 2 + e);
#pragma unroll
                        for (int r = 0; r < RT; ++r)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int pr = sp.first + (row0 + r * 16 + g + h * 8) / G;
                                const bool see = kp <= pr && (!op.window || pr - kp < op.window ||
                                                              kp < op.sinks);
                                if (!see) s[r][j][2 * h + e] = -INFINITY;
                            }
                    }
                if (op.q_len > 1) {
                    // a value that only some rows see must not meet the others' zero
                    // weights if it is not finite: 32 / kKeys lanes look at each key
                    constexpr int kPer = 32 / kKeys, kBytes = DP * 2 / kPer;
                    bool bad = false;
                    const unsigned char* vr = ring + slot * S::kStage +
                                              (kKeys + (lane & (kKeys - 1))) * S::kPitch + lane / kKeys * kBytes;
                    constexpr uint32_t kExp = BF16 ? 0x7F80u : 0x7C00u;
#pragma unroll 4
                    for (int q = 0; q < kBytes / 16; ++q) {
                        const uint4 v = *reinterpret_cast<const uint4*>(vr + q * 16);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            bad = bad || (w[x] & kExp) == kExp || ((w[x] >> 16) & kExp) == kExp;
                    }
                    poison = __ballot_sync(0xffffffffu, bad);
                    if (kPer == 2) poison = (poison | poison >> 16) & 0xFFFFu;
                }
            }

            // running maximum, weights, rescaling
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                float nm[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v = fmaxf(s[r][0][2 * h], s[r][0][2 * h + 1]);
#pragma unroll
                    for (int j = 1; j < kBlk; ++j) v = fmaxf(v, fmaxf(s[r][j][2 * h], s[r][j][2 * h + 1]));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                    nm[h] = fmaxf(m[r][h], v);
                }
                if (__any_sync(0xffffffffu, nm[0] > m[r][0] + grow || nm[1] > m[r][1] + grow)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float f = nm[h] == m[r][h] ? 1.f : exp2_fast((m[r][h] - nm[h]) * c2);
                        m[r][h] = nm[h];
                        l[r][h] *= f;
#pragma unroll
                        for (int d = 0; d < DP / 8; ++d) {
                            o[r][d][2 * h] *= f;
                            o[r][d][2 * h + 1] *= f;
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float shift = m[r][h] == -INFINITY ? 0.f : -m[r][h];
#pragma unroll
                    for (int j = 0; j < kBlk; ++j) {
                        const float2 d = fma2(make_float2(s[r][j][2 * h], s[r][j][2 * h + 1]), make_float2(1.f, 1.f),
                                              make_float2(shift, shift));
                        const float2 z = fma2(d, make_float2(c2, c2), make_float2(kLift<BF16>, kLift<BF16>));
                        const float a = exp2_fast(z.x), c = exp2_fast(z.y);
                        l[r][h] += a + c;
                        s[r][j][2 * h] = a;
                        s[r][j][2 * h + 1] = c;
                    }
                }
            }
            if (poison) {
                unsigned char* vb = ring + slot * S::kStage + kKeys * S::kPitch;
#pragma unroll 1
                for (int k = 0; k < kKeys; ++k) {
                    if (!((poison >> k) & 1u)) continue;
                    const int kp = __shfl_sync(0xffffffffu, my_pos, k);
                    const int src = (lane & ~3) | ((k & 7) >> 1);
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float w = 0.f;
#pragma unroll
                            for (int j = 0; j < kBlk; ++j) {
                                const float w0 = __shfl_sync(0xffffffffu, s[r][j][2 * h], src);
                                const float w1 = __shfl_sync(0xffffffffu, s[r][j][2 * h + 1], src);
                                if (j == k >> 3) w = (k & 1) ? w1 : w0;
                            }
                            const int pr = sp.first + (row0 + r * 16 + g + h * 8) / G;
                            const bool see = kp <= pr && (!op.window || pr - kp < op.window ||
                                                          kp < op.sinks);
                            if (see) {
#pragma unroll
                                for (int d = 0; d < DP / 8; ++d) {
                                    const float2 v = pair_f32<BF16>(*reinterpret_cast<const uint32_t*>(
                                        vb + S::piece(k, d) + t4 * 4));
                                    o[r][d][2 * h] = fmaf(w, v.x, o[r][d][2 * h]);
                                    o[r][d][2 * h + 1] = fmaf(w, v.y, o[r][d][2 * h + 1]);
                                }
                            }
                        }
                    __syncwarp();
                    for (int q = lane; q < DP / 8; q += 32)
                        *reinterpret_cast<uint4*>(vb + k * S::kPitch + q * 16) = make_uint4(0, 0, 0, 0);
                    __syncwarp();
                }
            }

            // output += weights x values
            const uint32_t vl = va + S::piece((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
#pragma unroll
            for (int u = 0; u < S::kSub; ++u) {
                uint32_t hi[RT][4], lo[RT][4];
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        split_pair<BF16>(s[r][2 * u + (x >> 1)][2 * (x & 1)], s[r][2 * u + (x >> 1)][2 * (x & 1) + 1],
                                         hi[r][x], lo[r][x]);
#pragma unroll
                for (int d = 0; d < DP / 16; ++d) {
                    uint32_t vf[4];
                    ldsm4_t(vf, on(vl, d) + u * 16 * S::kPitch);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        mma16816<BF16>(o[r][2 * d], hi[r], vf[0], vf[1]);
                        mma16816<BF16>(o[r][2 * d + 1], hi[r], vf[2], vf[3]);
                        mma16816<BF16>(o[r][2 * d], lo[r], vf[0], vf[1]);
                        mma16816<BF16>(o[r][2 * d + 1], lo[r], vf[2], vf[3]);
                    }
                }
            }
        }
        cp_wait<0>();
        __syncwarp();

        // the next segment's first copies start before this one's output is written
        const int cur_b = sg.b, hk = sg.hk;
        const bool whole = sg.kb == 0 && sg.ke == sg.nb;
        blk += sg.ke - sg.kb;
        const bool more = blk < end;
        if (more) {
            enter(blk, false);
            load_q();
#pragma unroll
            for (int i = 0; i < kStages; ++i) locate(i, pos[i], offs[i]);
            issue(0, offs[0]);
        }

        // ---- the four warps' parts, through shared memory ---------------------------------
        float* wo = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[r][h] += __shfl_xor_sync(0xffffffffu, l[r][h], 1);
                l[r][h] += __shfl_xor_sync(0xffffffffu, l[r][h], 2);
                const int row = r * 16 + g + h * 8;
                if (t4 == 0) {
                    sm_m[warp * S::kRows + row] = m[r][h] * c2;
                    sm_l[warp * S::kRows + row] = l[r][h];
                }
#pragma unroll
                for (int d = 0; d < DP / 8; ++d)
                    *reinterpret_cast<float2*>(wo + S::out_at(row, d) + t4 * 2) =
                        make_float2(o[r][d][2 * h], o[r][d][2 * h + 1]);
            }
        }
        __syncthreads();
        float* part = p.part + ((size_t)blockIdx.x * 2 + (first_segment ? 0 : 1)) * S::kPart;
        for (int i = tid; i < S::kRows * (DP / 8); i += kAttnThreads) {
            const int r = i / (DP / 8), d = i % (DP / 8) * 8, row = row0 + r;
            if (row >= p.rows || d >= D) continue;
            float top = -INFINITY, sum = 0.f, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, sm_m[w * S::kRows + r]);
            const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float f = exp2_fast(sm_m[w * S::kRows + r] - base);
                sum = fmaf(f, sm_l[w * S::kRows + r], sum);
                const float4* src = reinterpret_cast<const float4*>(
                    reinterpret_cast<const float*>(smem + w * S::kRing) + S::out_at(r, d >> 3));
                const float4 x = src[0], y = src[1];
                v[0] = fmaf(f, x.x, v[0]), v[1] = fmaf(f, x.y, v[1]);
                v[2] = fmaf(f, x.z, v[2]), v[3] = fmaf(f, x.w, v[3]);
                v[4] = fmaf(f, y.x, v[4]), v[5] = fmaf(f, y.y, v[5]);
                v[6] = fmaf(f, y.z, v[6]), v[7] = fmaf(f, y.w, v[7]);
            }
            if (whole) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
                for (int x = 0; x < 8; ++x) v[x] *= inv;
                const int tok = row / G, h = hk * G + row - tok * G;
                const long long t = (long long)cur_b * op.q_len + tok;
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(op.out) + t * op.out_stride +
                                          (long long)h * D + d) = pack8<BF16>(v);
                if (d == 0 && op.lse)
                    op.lse[t * op.heads + h] = lse_of<BF16>(top, sum);
            } else {
                if (d == 0) {
                    part[r] = top;
                    part[S::kRows + r] = sum;
                }
                float4* dst = reinterpret_cast<float4*>(part + 2 * S::kRows + r * DP + d);
                dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                dst[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
        if (!more) return;
        __syncthreads();
    }
}

// Row tiles of a CTA: as many as share its keys with 128 output registers.
static int attn_dp(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : D <= 192 ? 192 : 256; }
static int attn_tiles(const dg_attn& op) {
    const int rows = op.q_len * (op.heads / op.kv.kv_heads), dp = attn_dp(op.kv.head_dim);
    const int most = dp <= 64 ? 4 : dp <= 128 ? 2 : 1, want = (rows + 15) / 16;
    return want >= most ? most : want == 3 ? 4 : want;
}

size_t attn_ws_bytes(const dg_attn& op) {
    const int tiles = attn_tiles(op), dp = attn_dp(op.kv.head_dim);
    const int rows = op.q_len * (op.heads / op.kv.kv_heads), groups = (rows + tiles * 16 - 1) / (tiles * 16);
    if (never_split(op)) return 16;
    const long long ctas = max_blocks(op, groups) < kAttnMaxCtas ? max_blocks(op, groups) : kAttnMaxCtas;
    return info_bytes(op, groups) + (size_t)ctas * 2 * tiles * 16 * (dp + 2) * 4;
}

template <bool BF16, int DP, int RT>
static cudaError_t launch_attn_t(const dg_attn& op, void* ws, cudaStream_t s) {
    using S = AttnShape<DP, RT>;
    AttnParams p;
    p.op = op;
    p.rows = op.q_len * (op.heads / op.kv.kv_heads);
    p.groups = (p.rows + S::kRows - 1) / S::kRows;
    p.info = never_split(op) ? nullptr : static_cast<int2*>(ws);
    p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + info_bytes(op, p.groups));
    p.page_size = fast_div((uint32_t)op.kv.page_size);
    p.out_factor = 1.f;
    const void* fn = (const void*)k_attn<BF16, DP, RT>;
    cudaError_t e = tc::smem_attr_once(fn, S::kSmem);
    if (e != cudaSuccess) return e;
    const long long blocks = max_blocks(op, p.groups);
    int grid = sm_count() * S::kCtas;
    if (grid > kAttnMaxCtas) grid = kAttnMaxCtas;
    if (grid > blocks) grid = (int)blocks;
    void* args[] = {&p};
    e = launch_pdl(fn, dim3(grid), dim3(kAttnThreads), S::kSmem, s, args);
    if (e != cudaSuccess || never_split(op)) return e;
    return launch_join<BF16, DP, S::kRows, BF16>(p, grid, s);
}

template <bool BF16>
static cudaError_t launch_attn_b(const dg_attn& op, void* ws, cudaStream_t s) {
    const int rt = attn_tiles(op);
    switch (attn_dp(op.kv.head_dim)) {
        case 64:
            return rt == 1   ? launch_attn_t<BF16, 64, 1>(op, ws, s)
                   : rt == 2 ? launch_attn_t<BF16, 64, 2>(op, ws, s)
                             : launch_attn_t<BF16, 64, 4>(op, ws, s);
        case 128:
            return rt == 1 ? launch_attn_t<BF16, 128, 1>(op, ws, s)
                           : launch_attn_t<BF16, 128, 2>(op, ws, s);
        case 192: return launch_attn_t<BF16, 192, 1>(op, ws, s);
        default: return launch_attn_t<BF16, 256, 1>(op, ws, s);
    }
}

cudaError_t launch_attn(const dg_attn& op, void* ws, cudaStream_t s) {
    return op.kv.type == DG_BF16 ? launch_attn_b<true>(op, ws, s) : launch_attn_b<false>(op, ws, s);
}

}  // namespace dg
