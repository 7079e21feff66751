// Attention of a step's new tokens over a paged cache held in 4 bits.
//
// The split into ranges of blocks, the running softmax and the join are those of the
// 16-bit cache (attn_common.cuh).  What differs is what a stage costs: 4.5 bits a value
// instead of 16, so that unpacking and the matrix instruction's feeding weigh as much as
// the bytes.
//
//  - A code is 3 bits and a sign, an e4m3 scale 4 bits: their product is exact in fp16.
//    One LOP3 turns a pair of codes into 1024 + (c + 8), or 1024 + 16 (c + 8) for the upper
//    nibbles, and one HFMA2 with (s', -1032 s') or (s' / 16, -72 s') gives c s' itself, s' = s /
//    16 so that no step leaves fp16 (the 16 goes into the score's and the output's factor).
//  - Keys and values are the matrix instruction's 16-row operand A (keys x dims for the
//    scores, dims x keys for the output), the query rows its 8 columns, so that 8 rows a
//    key head waste nothing where 16-row tiles of rows would leave half.  Both products
//    run in fp16: bf16 queries are scaled by a power of two per row, so nothing of them is lost that an
//    fp32 score would keep.
//  - Any order of the dims inside a product is as good as another: a lane takes 8 (DP = 64) or 16
//    consecutive bytes of a key and unpacks what it loaded, q is laid out to match; of the values
//    a lane takes 8 or 16 dims of four keys, and byte permutes pair up
//    two keys' nibbles.  No ldmatrix, no exchange but movmatrix for the weights.
//  - Weights meet the values as two fp16 numbers, as in the 16-bit kernel.
//  - A score is checked against the running maximum by each lane for its own keys; lanes
//    exchange only when that has grown by 2^8.
//
// Measured: 200001 positions of 8 x 128, 32 heads, bf16: 69 us with the join, 3.3 TB/s; 50000: 26;
// 16 sequences of 1..8191, 2 x 128: 12; 100 positions: 5.3.  Long calls fill no unit: 370
// instructions for 16 keys of 128 dims, of which 64 LOP3, 64 HFMA2, 64 PRMT and shifts and 24
// matrix instructions, in chains that leave two warps a scheduler half of the issue slots (ALU 40 %, tensor pipe 26 %, DRAM
// 44 %); 8, 12 or 16 warps an SM take the same time.  Short ones are bound by the chain length -> page -> key -> sum, and by
// the join.  Several tokens (four row tiles: 251 registers at 64 dims; 255 and 60 bytes of spills at 128): 8 tokens of 8
// sequences on windows of 4096, 32 heads on 8 of 64: 27.5 us, 31 % of the issue slots, four or five stages a warp.
#include "attn_common.cuh"

namespace dg {

template <int DP, int RT>
struct Attn4Shape {
    static constexpr int kKeys = 32;                                 // of a stage
    static constexpr int kWide = DP / 128, kHalf = DP % 128 / 64;    // parts of 128 and of 64 dims
    static constexpr int kPitch = DP == 192 ? 128 : DP / 2;          // bytes of a key's codes
    static constexpr int kScales = DP / 16;
    static constexpr int kCodes = kKeys * kPitch;
    static constexpr int kStage = 2 * (kCodes + kKeys * kScales) + kKeys * 4;   // codes (k, v), scales (k, v), positions
    static constexpr int kPos = kStage - kKeys * 4;
    static constexpr int kRows = RT * 8;
    static constexpr int kOut = kRows * DP * 4;                      // a warp's output, in place of stages
    static constexpr int kNeed = (kOut + kStage - 1) / kStage + 1;
    static constexpr int kLeast = DP <= 128 ? 3 : 2;
    static constexpr int kStages = kNeed < kLeast ? kLeast : kNeed;
    static constexpr int kRing = kStages * kStage;
    static constexpr int kKeyWords = 4 * kWide + 2 * kHalf;          // words (8 dims) of a lane, of a key
    static constexpr int kValWords = 2 * kWide + kHalf;              // of a value
    static constexpr int kQ = RT * kKeyWords * 512;
    static constexpr size_t kSmem = (size_t)kAttnWarps * kRing + kQ + (2 * kAttnWarps + 1) * kRows * 4;
    // Two CTAs an SM, whose 255 registers leave the compiler room to interleave the unpacking with
    // the products.  (One row tile of 128 dims, bf16: three CTAs of 168 registers 66 us for 200001 positions
    // and 32 for 50000, four of 128 registers 70 and 33, these 68 and 26.)
    static constexpr int kFit = 228 * 1024 / (kSmem + 2048), kWish = 2;
    static constexpr int kCtas = kFit < kWish ? kFit : kWish;
    static constexpr int kPart = part_floats(kRows, DP);
    // Byte of 16-byte piece c of row r; eight rows on it is 8 kPitch more.  Pieces change places inside 128 bytes, so that what a
    // phase of the reads below takes lies in different banks: 8 lanes 16 bytes of two
    // neighbouring keys, 16 lanes 8 bytes (or 32 lanes 4 bytes) of every second value row.
    __device__ static constexpr int piece(int r, int c) {
        if (kPitch == 128) return r * 128 + ((c ^ ((r & 6) ^ ((r & 1) << 2))) << 4);
        if (kPitch == 64) return (r >> 1) * 128 + ((((r & 1) * 4 + c) ^ (((r >> 1) & 3) << 1)) << 4);
        return (r >> 2) * 128 + ((((r & 3) * 2 + c) ^ (((r >> 2) & 1) << 1)) << 4);
    }
    __device__ static constexpr int out_at(int r, int d) { return r * DP + ((d ^ ((r >> 1) & 3)) << 3); }
    static_assert(kOut <= (kStages - 1) * kStage, "a warp's output leaves a stage free");
    static_assert(kCtas >= 1 && kSmem <= 227 * 1024, "an SM holds its CTAs");
};

struct Attn4Params {
    AttnParams a;                 // a.op: the same masks and outputs; its k and v are not read
    const uint8_t *k, *k_scale;
    int64_t to_v, to_v_scale;     // bytes from a key's codes and scales to its value's
    uint32_t page_stride, token_stride, head_stride;                     // of codes, in 8 bytes
    uint32_t scale_page_stride, scale_token_stride, scale_head_stride;   // bytes
    float c2;                     // |scale| k_factor log2(e) 16; 0 for a scale of zero
    int wide;                     // code rows in pieces of 16 bytes, not 8
    int runs;                     // and sixteen keys of a stage lie in one page
    int scale_piece;              // bytes that scales are copied by: 16, 8, 4; 1: by ordinary loads
};

__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b) { return h2_as_u32(__hmul2(u32_as_h2(a), u32_as_h2(b))); }

// Two scales of fp16 (as pairs with the codes) and what unpacking needs of them.
struct Scales {
    uint32_t lo, lo_off, hi, hi_off;   // s', -1032 s', s' / 16, -72 s'
    __device__ __forceinline__ explicit Scales(uint32_t e4m3x2) {
        uint32_t s;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s) : "h"((uint16_t)e4m3x2));
        lo = h2mul(s, 0x2C002C00u);       // 2^-4
        hi = h2mul(s, 0x1C001C00u);       // 2^-8
        lo_off = h2mul(s, 0xD408D408u);   // -64.5
        hi_off = h2mul(s, 0xC480C480u);   // -4.5
    }
};
__device__ __forceinline__ uint32_t h2fma(uint32_t a, uint32_t b, uint32_t c) {
    return h2_as_u32(__hfma2(u32_as_h2(a), u32_as_h2(b), u32_as_h2(c)));
}
// The codes in bits 0-3 and 16-19 (lower), 4-7 and 20-23 (upper) of w, times their scales.
__device__ __forceinline__ uint32_t lower(uint32_t w, const Scales& s) {
    return h2fma(and_xor(w, 0x000F000Fu, 0x64086408u), s.lo, s.lo_off);
}
__device__ __forceinline__ uint32_t upper(uint32_t w, const Scales& s) {
    return h2fma(and_xor(w, 0x00F000F0u, 0x64806480u), s.hi, s.hi_off);
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void cp_async_n(uint32_t dst, const void* src, int bytes, bool fetch) {
    const int n = fetch ? bytes : 0;
    if (bytes == 16)
        cp_async16(dst, src, fetch);
    else if (bytes == 8)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

template <bool BF16, int DP, int RT>
__global__ void __launch_bounds__(kAttnThreads, Attn4Shape<DP, RT>::kCtas) k_attn4(const Attn4Params p) {
    using S = Attn4Shape<DP, RT>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ RangeScan scan;
    const dg_attn& op = p.a.op;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = op.kv.head_dim, G = op.heads / op.kv.kv_heads;
    const int heads = op.kv.kv_heads * p.a.groups;   // units per sequence
    unsigned char* ring = smem + warp * S::kRing;
    const uint32_t ring_a = (uint32_t)__cvta_generic_to_shared(ring);
    unsigned char* qs = smem + kAttnWarps * S::kRing;
    float* sm_m = reinterpret_cast<float*>(qs + S::kQ);
    float* sm_l = sm_m + kAttnWarps * S::kRows;
    float* sm_c = sm_l + kAttnWarps * S::kRows;   // a row's factor of its scores

    griddep_launch_dependents();
    griddep_wait();

    const CtaRange range = find_range(op, heads, scan);
    const long long begin = range.begin, end = range.end;
    int b = range.b;
    long long seq_at = range.seq_at;   // first block of sequence b
    if (begin >= end) return;

    const int g = lane >> 2, t4 = lane & 3;
    // ---- the range's part of one unit after another ---------------------------------------
    struct Segment {
        int b, hk, row0;   // sequence, key / value head, first row
        int kb, ke, nb;    // blocks [kb, ke) of nb
        Span sp;
        int key0, lim, n;  // this warp's n stages: kKeys keys from key0 on, then every
                           // kStep further, up to lim
        const uint8_t *k, *ks;   // codes and scales of the head's keys
        const uint8_t* k_row;    // this lane's piece of its row of the first ones
    } sg;
    auto times = [](int a, uint32_t b) { return (long long)((unsigned long long)(unsigned)a * b); };
    constexpr int kKeys = S::kKeys, kStep = kAttnWarps * kKeys, kStages = S::kStages;
    const int row_bytes = D / 2, scale_bytes = D / 16;
    constexpr int kChunks16 = DP / 32;                    // 16-byte pieces of a row
    constexpr bool kEven = 32 % kChunks16 == 0;           // a warp's pieces are whole rows
    constexpr int kAtOnce = kEven ? 32 / kChunks16 : 1;   // rows
    const int my_row = lane / kChunks16, my_piece = lane % kChunks16;
    const int my_byte = my_piece * 16 < row_bytes ? my_piece * 16 : 0;
    const uint32_t my_place = S::piece(my_row, my_piece);
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
        sg.hk = unit / p.a.groups;
        sg.row0 = (unit - sg.hk * p.a.groups) * S::kRows;
        sg.key0 = sg.kb * kBlockKeys + warp * kKeys;
        sg.lim = sg.ke == sg.nb ? sg.sp.count() : sg.ke * kBlockKeys;   // nb * kBlockKeys may be 2^31
        sg.n = sg.key0 < sg.lim ? (int)((unsigned)(sg.lim - sg.key0 + kStep - 1) / kStep) : 0;
        sg.k = p.k + 8 * times(sg.hk, p.head_stride);
        sg.ks = p.k_scale + times(sg.hk, p.scale_head_stride);
        sg.k_row = sg.k + times(my_row, 8 * p.token_stride) + my_byte;
        if (sg.kb == 0 && tid == 0 && p.a.info)
            p.a.info[(long long)b * heads + unit] = unit_parts(range, blk, sg.nb, sg.ke, first);
    };
    // Position, code offset and scale offset (bytes from the head's base; -1: nothing there) of
    // position c of the segment's walk.
    auto find = [&](unsigned c, int& pos, long long& off, long long& soff) {
        pos = INT_MAX;
        off = -1;
        soff = 0;
        if (c < (unsigned)sg.lim) {
            const int j = sg.sp.position((int)c);
            int slot = 0;
            const int page = page_slot(op.kv, p.a.page_size, sg.b, j, slot);
            if (page >= 0) {
                pos = j;
                off = 8 * (times(page, p.page_stride) + times(slot, p.token_stride));
                soff = times(page, p.scale_page_stride) + times(slot, p.scale_token_stride);
            }
        }
    };
    // Where sixteen positions in a row lie in one page (p.runs), the lanes find the next sixteen stages'
    // halves at once, 32 places, and a stage takes its two from them; else each lane finds its
    // key of the next stage.
    int pos_at;
    long long off_at, soff_at;
    auto locate = [&](int i) {
        if (p.runs) {
            if (i % 16 == 0)
                find((unsigned)sg.key0 + (unsigned)(i + (lane >> 1)) * kStep + (lane & 1) * 16, pos_at, off_at, soff_at);
        } else {
            find(i < sg.n ? (unsigned)sg.key0 + (unsigned)i * kStep + lane : UINT_MAX, pos_at, off_at, soff_at);
            if (pos_at != INT_MAX && !sg.sp.seen(pos_at)) {
                pos_at = INT_MAX;
                off_at = -1;
            }
        }
    };
    auto place = [](int i) { return (i + kStages - 1) % kStages; };
    // the byte of a row's piece, `rows` (a multiple of kAtOnce) further
    auto piece_on = [](uint32_t at, int rows) {
        return rows % 8 == 0 ? at + rows * S::kPitch : (at + rows * S::kPitch) ^ 64;   // kPitch 128, 4 rows
    };
    auto issue = [&](int i) {
        if (i < sg.n) {
            const uint32_t dst = ring_a + place(i) * S::kStage;
            int pos = pos_at;
            long long off = off_at, soff = soff_at;
            if (p.runs) {
                const int from = (i % 16) * 2 + (lane >> 4);
                pos = __shfl_sync(0xffffffffu, pos_at, from);
                soff = __shfl_sync(0xffffffffu, soff_at, from) + times(lane & 15, p.scale_token_stride);
                const unsigned c = (unsigned)sg.key0 + (unsigned)i * kStep + lane;
                if (pos != INT_MAX) pos += lane & 15;
                if (!(c < (unsigned)sg.lim && sg.sp.seen(pos))) pos = INT_MAX;
            }
            const bool there = pos != INT_MAX;
            *reinterpret_cast<int*>(ring + place(i) * S::kStage + S::kPos + lane * 4) = pos;
            if (kEven && p.runs) {
                // addresses without an exchange for each row: a half's sixteen rows exist where its page
                // does (else page 0's stand in for them), whether or not they are copied
                const unsigned have = __ballot_sync(0xffffffffu, there);
                const bool all = have == 0xffffffffu && D == DP;
                const long long step = (long long)(8 * kAtOnce) * p.token_stride;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const long long o = max(__shfl_sync(0xffffffffu, off_at, (i % 16) * 2 + half), 0ll);
                    const uint8_t *k = sg.k_row + o, *v = k + p.to_v;
#pragma unroll
                    for (int it = 0; it < 16 / kAtOnce; ++it) {
                        const uint32_t d = dst + piece_on(my_place, half * 16 + it * kAtOnce);
                        if (all) {
                            cp_async16(d, k);
                            cp_async16(d + S::kCodes, v);
                        } else {
                            const bool in = my_piece * 16 < row_bytes && (have >> (half * 16 + it * kAtOnce + my_row)) & 1u;
                            cp_async16(d, k, in);
                            cp_async16(d + S::kCodes, v, in);
                        }
                        k += step;
                        v += step;
                    }
                }
            } else if (p.wide) {
                if (p.runs) {
                    off = __shfl_sync(0xffffffffu, off_at, (i % 16) * 2 + (lane >> 4));
                    off = there ? off + times(lane & 15, 8 * p.token_stride) : -1;
                }
                constexpr int kChunks = DP / 32;   // 16-byte pieces of a row
#pragma unroll
                for (int it = 0; it < kChunks; ++it) {
                    const int idx = it * 32 + lane, row = idx / kChunks, ch = idx % kChunks;
                    const long long o = __shfl_sync(0xffffffffu, off, row);
                    const bool in = o >= 0 && ch * 16 < row_bytes;
                    const long long at = in ? o + ch * 16 : 0;
                    const uint32_t d = dst + S::piece(row, ch);
                    cp_async16(d, sg.k + at, in);
                    cp_async16(d + S::kCodes, sg.k + p.to_v + at, in);
                }
            } else {
                constexpr int kChunks = DP / 16;   // 8-byte ones
#pragma unroll 2
                for (int it = 0; it < kChunks; ++it) {
                    const int idx = it * 32 + lane, row = idx / kChunks, ch = idx % kChunks;
                    const long long o = __shfl_sync(0xffffffffu, off, row);
                    const bool in = o >= 0 && ch * 8 < row_bytes;
                    const long long at = in ? o + ch * 8 : 0;
                    const uint32_t d = dst + S::piece(row, ch >> 1) + (ch & 1) * 8;
                    cp_async_n(d, sg.k + at, 8, in);
                    cp_async_n(d + S::kCodes, sg.k + p.to_v + at, 8, in);
                }
            }
            // this lane's key: its scales
            const uint32_t d = dst + 2 * S::kCodes + lane * S::kScales;
            const uint8_t *ks = sg.ks + (there ? soff : 0), *vs = ks + p.to_v_scale;
            constexpr bool kOnce = S::kScales == 4 || S::kScales == 8 || S::kScales == 16;
            if (kOnce && p.scale_piece == S::kScales) {
                cp_async_n(d, ks, S::kScales, there);
                cp_async_n(d + kKeys * S::kScales, vs, S::kScales, there);
            } else if (p.scale_piece > 1) {
                const int step = p.scale_piece;
#pragma unroll 1
                for (int at = 0; at < S::kScales; at += step) {
                    const bool in = there && at < scale_bytes;
                    const int from = in ? at : 0;
                    cp_async_n(d + at, ks + from, step, in);
                    cp_async_n(d + kKeys * S::kScales + at, vs + from, step, in);
                }
            } else {
                // all loads before the first store
                uint32_t* to = reinterpret_cast<uint32_t*>(ring + place(i) * S::kStage + 2 * S::kCodes + lane * S::kScales);
                uint32_t kw[S::kScales / 4], vw[S::kScales / 4];
#pragma unroll
                for (int w = 0; w < S::kScales / 4; ++w) {
                    kw[w] = vw[w] = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (there && w * 4 + e < scale_bytes) {
                            kw[w] |= (uint32_t)__ldcg(ks + w * 4 + e) << (8 * e);
                            vw[w] |= (uint32_t)__ldcg(vs + w * 4 + e) << (8 * e);
                        }
                }
#pragma unroll
                for (int w = 0; w < S::kScales / 4; ++w) {
                    to[w] = kw[w];
                    to[kKeys * S::kScales / 4 + w] = vw[w];
                }
            }
        }
        cp_commit();
    };
    // q as the matrix instruction's operand B: for tile r, the pairs of dims (a + e, b + e), e < 4, that
    // the lane unpacks together (unit w), in row r * 8 + g.  bf16 rows are scaled to 2^14..2^15.
    // A warp takes tiles warp, warp + 4, ..
    auto stage_q = [&] {
        const float sign = op.scale > 0.f ? 1.f : op.scale < 0.f ? -1.f : 0.f;
        for (int r = warp; r < RT; r += kAttnWarps) {
            const int row = sg.row0 + r * 8 + g, tok = row / G;
            const bool have = row < p.a.rows;
            const uint16_t* q = static_cast<const uint16_t*>(op.q) +
                                ((long long)sg.b * op.q_len + (have ? tok : 0)) * op.q_stride +
                                (long long)(sg.hk * G + (have ? row - tok * G : 0)) * D;
            auto load = [&](int w) {
                const bool wide = w < 4 * S::kWide;
                const int a = wide ? (w >> 2) * 128 + t4 * 32 + (w & 3) * 4
                                   : S::kWide * 128 + t4 * 16 + (w - 4 * S::kWide) * 4, b = a + (wide ? 16 : 8);
                uint2 x = make_uint2(0, 0), y = x;
                if (have && a < D) x = __ldcg(reinterpret_cast<const uint2*>(q + a));
                if (have && b < D) y = __ldcg(reinterpret_cast<const uint2*>(q + b));
                return make_uint4(x.x, x.y, y.x, y.y);
            };
            float up = 1.f, c2 = p.c2;
            if (BF16) {
                float top = 0.f;
#pragma unroll
                for (int w = 0; w < S::kKeyWords; ++w) {
                    float f[8];
                    unpack8<true>(load(w), f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (fabsf(f[e]) <= FLT_MAX) top = fmaxf(top, fabsf(f[e]));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^(14 - exponent of top), inside fp32's normal numbers
                const int e = top > 0.f ? max(-126, min(126, 141 - (int)(__float_as_uint(top) >> 23))) : 0;
                up = __uint_as_float((uint32_t)(127 + e) << 23);
                c2 *= __uint_as_float((uint32_t)(127 - e) << 23);
            }
            c2 = p.c2 == 0.f ? 1.f : fminf(fmaxf(c2, FLT_MIN), FLT_MAX);
            if (t4 == 0) sm_c[r * 8 + g] = c2;
#pragma unroll
            for (int w = 0; w < S::kKeyWords; ++w) {
                float f[8];
                unpack8<BF16>(load(w), f);
                const float k = sign * up;
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = pair_16<false>(f[e] * k, f[e + 4] * k);
                *reinterpret_cast<uint4*>(qs + (r * S::kKeyWords + w) * 512 + lane * 16) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    };

    long long blk = begin;
    enter(blk, true);
    auto start = [&](int from, int to) {   // the first stages, one after the other
#pragma unroll
        for (int i = 0; i < kStages; ++i) {
            if (i < from || i >= to) continue;
            locate(i);
            if (i < kStages - 1) issue(i);
        }
    };
    start(0, 1);
    for (bool first_segment = true;; first_segment = false) {
        start(1, kStages);
        stage_q();
        __syncthreads();
        const Span sp = sg.sp;
        const int row0 = sg.row0, n = sg.n, last = sp.first + op.q_len - 1;

        // output: word u of a lane, its dims 2 x and 2 x + 1, rows 2 t4 and 2 t4 + 1 of a tile
        float o[RT][S::kValWords][4][4], m[RT][2], shift[RT][2], l[RT][2], c2[RT][2], grow[RT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int u = 0; u < S::kValWords; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[r][u][x][0] = o[r][u][x][1] = o[r][u][x][2] = o[r][u][x][3] = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                m[r][h] = -INFINITY;
                shift[r][h] = 0.f;   // -m, or 0 while m is -infinity
                l[r][h] = 0.f;
                c2[r][h] = sm_c[r * 8 + 2 * t4 + h];
                grow[r][h] = fminf(8.f / c2[r][h], FLT_MAX);   // finite: the first maximum is always taken
            }
        }

        // this lane's places in a stage: keys g, g + 8, ..; values 2 t4 and 2 t4 + 1, + 8, ..
        const int key_at = S::piece(g, S::kWide ? t4 : t4 >> 1) + (S::kWide ? 0 : (t4 & 1) * 8);
        const int val_at = S::piece(2 * t4, S::kWide ? g >> 1 : g >> 2) + (S::kWide ? (g & 1) * 8 : (g & 3) * 4);
        const int val_at1 = S::piece(2 * t4 + 1, S::kWide ? g >> 1 : g >> 2) + (S::kWide ? (g & 1) * 8 : (g & 3) * 4);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            cp_wait<kStages - 2>();
            __syncwarp();
            const int slot = place(i);
            unsigned char* stage = ring + slot * S::kStage;
            unsigned char* ks = stage + 2 * S::kCodes;      // scales of the keys, then of the values
            unsigned char* vs = ks + kKeys * S::kScales;
            const int my_pos = *reinterpret_cast<const int*>(stage + S::kPos + lane * 4);
            // the place that the last stage left is free: refill it
            const int ni = i + kStages - 1;
            issue(ni);
            locate(ni + 1);

            const bool all = my_pos <= sp.first &&
                             (!op.window || last - my_pos < op.window || my_pos < op.sinks);
            const bool whole_stage = __all_sync(0xffffffffu, all);
            auto sees = [&](int kp, int r, int h) {   // row 2 t4 + h of tile r
                const int pr = sp.first + (row0 + r * 8 + 2 * t4 + h) / G;
                return kp <= pr && (!op.window || pr - kp < op.window || kp < op.sinks);
            };
#pragma unroll(RT == 1 ? 2 : 1)
            for (int sub = 0; sub < 2; ++sub) {
                // ---- scores of 16 keys: rows g and g + 8 of operand A ---------------------------
                float s[RT][4];
#pragma unroll
                for (int r = 0; r < RT; ++r) s[r][0] = s[r][1] = s[r][2] = s[r][3] = 0.f;
                float s_odd[4] = {0.f, 0.f, 0.f, 0.f};   // of one tile: two chains of products
                const int k0 = sub * 16 + g, k1 = k0 + 8;
                // words a and b of two keys: nibble e of both side by side
                auto score_words = [&](uint32_t a0, uint32_t b0, uint32_t a1, uint32_t b1, const Scales& s0,
                                       const Scales& s1, int unit) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t pick = y ? 0x7632u : 0x5410u;
                        const uint32_t x0 = __byte_perm(a0, b0, pick), x1 = __byte_perm(a1, b1, pick);
                        const uint32_t f0[4] = {lower(x0, s0), lower(x1, s1), upper(x0, s0), upper(x1, s1)};
                        const uint32_t f1[4] = {lower(x0 >> 8, s0), lower(x1 >> 8, s1), upper(x0 >> 8, s0),
                                                upper(x1 >> 8, s1)};
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            const uint4 q = *reinterpret_cast<const uint4*>(
                                qs + (r * S::kKeyWords + unit + y) * 512 + lane * 16);
                            mma16816<false>(s[r], f0, q.x, q.y);
                            if constexpr (RT == 1) mma16816<false>(s_odd, f1, q.z, q.w);
                            else mma16816<false>(s[r], f1, q.z, q.w);
                        }
                    }
                };
#pragma unroll
                for (int h = 0; h < S::kWide; ++h) {
                    // (64 bytes on, inside 128, is another piece's bit 2)
                    const unsigned char* at = stage + (key_at ^ (h * 64)) + sub * 16 * S::kPitch;
                    const uint4 x = *reinterpret_cast<const uint4*>(at);
                    const uint4 y = *reinterpret_cast<const uint4*>(at + 8 * S::kPitch);
                    const Scales s0(*reinterpret_cast<const uint16_t*>(ks + k0 * S::kScales + h * 8 + t4 * 2));
                    const Scales s1(*reinterpret_cast<const uint16_t*>(ks + k1 * S::kScales + h * 8 + t4 * 2));
                    score_words(x.x, x.z, y.x, y.z, s0, s1, h * 4);
                    score_words(x.y, x.w, y.y, y.w, s0, s1, h * 4 + 2);
                }
                if constexpr (S::kHalf) {
                    constexpr int base = S::kWide * 4;   // piece of the last 64 dims
                    const unsigned char* at =
                        stage + (S::kWide ? S::piece(g, base + (t4 >> 1)) + (t4 & 1) * 8 : key_at) + sub * 16 * S::kPitch;
                    const uint2 x = *reinterpret_cast<const uint2*>(at);
                    const uint2 y = *reinterpret_cast<const uint2*>(at + 8 * S::kPitch);
                    const uint32_t e0 = ks[k0 * S::kScales + S::kWide * 8 + t4], e1 = ks[k1 * S::kScales + S::kWide * 8 + t4];
                    score_words(x.x, x.y, y.x, y.y, Scales(e0 | e0 << 8), Scales(e1 | e1 << 8), S::kWide * 4);
                }
                if constexpr (RT == 1) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[0][x] += s_odd[x];
                }
                // ---- masks, where some row does not see some key of the stage -----------------
                if (!whole_stage) {
                    const int p0 = __shfl_sync(0xffffffffu, my_pos, k0), p1 = __shfl_sync(0xffffffffu, my_pos, k1);
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!sees(p0, r, h)) s[r][h] = -INFINITY;
                            if (!sees(p1, r, h)) s[r][2 + h] = -INFINITY;
                        }
                    if (op.q_len > 1) {
                        // a value of NaN that only some rows see: it goes straight to
                        // their outputs, and the matrix instruction meets a zero
#pragma unroll
                        for (int u = 0; u < S::kValWords; ++u) {
                            const int at = u < 2 * S::kWide ? (u >> 1) * 8 + g : S::kWide * 8 + (g >> 1);
                            unsigned bad = 0;
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                bad |= (unsigned)((vs[(sub * 16 + k) * S::kScales + at] & 0x7F) == 0x7F) << k;
                            if (!__any_sync(0xffffffffu, bad)) continue;
#pragma unroll 1
                            for (int k = 0; k < 16; ++k) {
                                const int kp = __shfl_sync(0xffffffffu, my_pos, sub * 16 + k);
                                if (!((bad >> k) & 1u)) continue;
#pragma unroll
                                for (int r = 0; r < RT; ++r)
#pragma unroll
                                    for (int h = 0; h < 2; ++h)
                                        if (sees(kp, r, h))
#pragma unroll
                                            for (int x = 0; x < 4; ++x)
                                                o[r][u][x][h] = o[r][u][x][2 + h] = __uint_as_float(0x7fffffffu);
                            }
                            // (words of a scale that two lanes or two words share are all seen before any is cleared)
                        }
                        __syncwarp();
                        for (int x = lane; x < 16 * S::kScales; x += 32) {
                            unsigned char* at = vs + sub * 16 * S::kScales + x;
                            if ((*at & 0x7F) == 0x7F) *at = 0;
                        }
                        __syncwarp();
                    }
                }
                // ---- weights -----------------------------------------------------------------
                uint32_t hi[RT][2], lo[RT][2];
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    float nm[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) nm[h] = fmaxf(s[r][h], s[r][2 + h]);
                    if (__any_sync(0xffffffffu, nm[0] > m[r][0] + grow[r][0] || nm[1] > m[r][1] + grow[r][1])) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float v = nm[h];
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                            v = fmaxf(v, m[r][h]);
                            const float f = v == m[r][h] ? 1.f : exp2_fast((m[r][h] - v) * c2[r][h]);
                            m[r][h] = v;
                            shift[r][h] = v == -INFINITY ? 0.f : -v;
                            l[r][h] *= f;
#pragma unroll
                            for (int u = 0; u < S::kValWords; ++u)
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    o[r][u][x][h] *= f;
                                    o[r][u][x][2 + h] *= f;
                                }
                        }
                    }
                    const float2 one = make_float2(1.f, 1.f), lift = make_float2(kLift<false>, kLift<false>);
                    const float2 cc = make_float2(c2[r][0], c2[r][1]), off = make_float2(shift[r][0], shift[r][1]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {   // key g + 8 x, rows 2 t4 and 2 t4 + 1
                        const float2 d = fma2(make_float2(s[r][2 * x], s[r][2 * x + 1]), one, off);
                        const float2 z = fma2(d, cc, lift);
                        const float2 w = make_float2(exp2_fast(z.x), exp2_fast(z.y));
                        const float2 sum = fma2(w, one, make_float2(l[r][0], l[r][1]));
                        l[r][0] = sum.x;
                        l[r][1] = sum.y;
                        split_pair<false>(w.x, w.y, hi[r][x], lo[r][x]);   // [key][row], operand B is [row][key]
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        hi[r][x] = movmatrix(hi[r][x]);
                        lo[r][x] = movmatrix(lo[r][x]);
                    }
                }
                // ---- output += values x weights: keys 2 t4, 2 t4 + 1 and the same + 8 -----------
                const unsigned char* vals = stage + S::kCodes;
                const int v0 = sub * 16 + 2 * t4;
                auto add = [&](int u, uint32_t wa, uint32_t wb, uint32_t wc, uint32_t wd, const Scales& s0,
                               const Scales& s1) {
                    // two keys' nibbles of the same dims: dims 0..3, then 4..7
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t pick = y ? 0x7632u : 0x5410u;
                        const uint32_t x0 = __byte_perm(wa, wb, pick), x1 = __byte_perm(wc, wd, pick);
#pragma unroll
                        for (int z = 0; z < 2; ++z) {   // dims 4 y + 2 z, + 1
                            const uint32_t e0 = z ? x0 >> 8 : x0, e1 = z ? x1 >> 8 : x1;
                            const uint32_t a[4] = {lower(e0, s0), upper(e0, s0), lower(e1, s1), upper(e1, s1)};
#pragma unroll
                            for (int r = 0; r < RT; ++r) {
                                mma16816<false>(o[r][u][2 * y + z], a, hi[r][0], hi[r][1]);
                                mma16816<false>(o[r][u][2 * y + z], a, lo[r][0], lo[r][1]);
                            }
                        }
                    }
                };
                auto scale_of = [&](int key, int at) { return (uint32_t)vs[key * S::kScales + at]; };
#pragma unroll
                for (int h = 0; h < S::kWide; ++h) {
                    uint2 w[4];
                    uint32_t e[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int key = v0 + (x & 1) + (x >> 1) * 8;
                        w[x] = *reinterpret_cast<const uint2*>(vals + ((x & 1 ? val_at1 : val_at) ^ (h * 64)) +
                                                               (sub * 16 + (x >> 1) * 8) * S::kPitch);
                        e[x] = scale_of(key, h * 8 + g);
                    }
                    const Scales s0(e[0] | e[1] << 8), s1(e[2] | e[3] << 8);
                    add(2 * h, w[0].x, w[1].x, w[2].x, w[3].x, s0, s1);
                    add(2 * h + 1, w[0].y, w[1].y, w[2].y, w[3].y, s0, s1);
                }
                if constexpr (S::kHalf) {
                    uint32_t w[4], e[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int key = v0 + (x & 1) + (x >> 1) * 8;
                        const int at = S::kWide ? S::piece(2 * t4 + (x & 1), S::kWide * 4 + (g >> 2)) + (g & 3) * 4
                                                : x & 1 ? val_at1 : val_at;
                        w[x] = *reinterpret_cast<const uint32_t*>(vals + at + (sub * 16 + (x >> 1) * 8) * S::kPitch);
                        e[x] = scale_of(key, S::kWide * 8 + (g >> 1));
                    }
                    add(2 * S::kWide, w[0], w[1], w[2], w[3], Scales(e[0] | e[1] << 8), Scales(e[2] | e[3] << 8));
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
            start(0, 1);
        }

        // ---- the four warps' parts, through shared memory ---------------------------------
        float* wo = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[r][h] += __shfl_xor_sync(0xffffffffu, l[r][h], 4);
                l[r][h] += __shfl_xor_sync(0xffffffffu, l[r][h], 8);
                l[r][h] += __shfl_xor_sync(0xffffffffu, l[r][h], 16);
                const int row = r * 8 + 2 * t4 + h;
                if (g == 0) {
                    sm_m[warp * S::kRows + row] = m[r][h] * c2[r][h];
                    sm_l[warp * S::kRows + row] = l[r][h];
                }
#pragma unroll
                for (int u = 0; u < S::kValWords; ++u) {
                    const int d = u < 2 * S::kWide ? (u >> 1) * 128 + g * 16 + (u & 1) * 8 : S::kWide * 128 + g * 8;
                    float4* to = reinterpret_cast<float4*>(wo + S::out_at(row, d >> 3));
                    to[0] = make_float4(o[r][u][0][h], o[r][u][0][2 + h], o[r][u][1][h], o[r][u][1][2 + h]);
                    to[1] = make_float4(o[r][u][2][h], o[r][u][2][2 + h], o[r][u][3][h], o[r][u][3][2 + h]);
                }
            }
        __syncthreads();
        float* part = p.a.part + ((size_t)blockIdx.x * 2 + (first_segment ? 0 : 1)) * S::kPart;
        for (int i = tid; i < S::kRows * (DP / 8); i += kAttnThreads) {
            const int r = i / (DP / 8), d = i % (DP / 8) * 8, row = row0 + r;
            if (row >= p.a.rows || d >= D) continue;
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
                // (the factor last: its product with the sum or with the sum's reciprocal might leave fp32's range)
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
                for (int x = 0; x < 8; ++x) v[x] = v[x] * inv * p.a.out_factor;
                const int tok = row / G, h = hk * G + row - tok * G;
                const long long t = (long long)cur_b * op.q_len + tok;
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(op.out) + t * op.out_stride +
                                          (long long)h * D + d) = pack8<BF16>(v);
                if (d == 0 && op.lse)
                    op.lse[t * op.heads + h] = lse_of<false>(top, sum);
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
static int attn4_tiles(const dg_attn4& op) {
    const int rows = op.q_len * (op.heads / op.kv.kv_heads), D = op.kv.head_dim, want = (rows + 7) / 8;
    const int most = D <= 128 ? 4 : 2;
    return want >= most ? most : want == 3 ? 4 : want;
}
static int attn4_dp(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : D <= 192 ? 192 : 256; }

// The op's masks and outputs as those of the 16-bit attention.
static dg_attn as_attn(const dg_attn4& op) {
    dg_attn a = {};
    a.kv.type = op.kv.type;
    a.kv.batch = op.kv.batch;
    a.kv.kv_heads = op.kv.kv_heads;
    a.kv.head_dim = op.kv.head_dim;
    a.kv.page_size = op.kv.page_size;
    a.kv.num_pages = op.kv.num_pages;
    a.kv.max_pages = op.kv.max_pages;
    a.kv.page_stride = op.kv.page_stride;
    a.kv.token_stride = op.kv.token_stride;
    a.kv.head_stride = op.kv.head_stride;
    a.kv.block_table = op.kv.block_table;
    a.kv.table_stride = op.kv.table_stride;
    a.kv.seq_lens = op.kv.seq_lens;
    a.q_len = op.q_len;
    a.heads = op.heads;
    a.window = op.window;
    a.sinks = op.sinks;
    a.scale = op.scale;
    a.q = op.q;
    a.out = op.out;
    a.lse = op.lse;
    a.q_stride = op.q_stride;
    a.out_stride = op.out_stride;
    return a;
}

size_t attn4_ws_bytes(const dg_attn4& op) {
    const dg_attn a = as_attn(op);
    if (never_split(a)) return 16;
    const int tiles = attn4_tiles(op), rows = op.q_len * (op.heads / op.kv.kv_heads);
    const int groups = (rows + tiles * 8 - 1) / (tiles * 8);
    const long long ctas = std::min<long long>(max_blocks(a, groups), kAttnMaxCtas);
    return info_bytes(a, groups) + (size_t)ctas * 2 * part_floats(tiles * 8, attn4_dp(op.kv.head_dim)) * 4;
}

template <bool BF16, int DP, int RT>
static cudaError_t launch_attn4_t(const dg_attn4& op, void* ws, cudaStream_t s) {
    using S = Attn4Shape<DP, RT>;
    Attn4Params p;
    p.a.op = as_attn(op);
    p.a.rows = op.q_len * (op.heads / op.kv.kv_heads);
    p.a.groups = (p.a.rows + S::kRows - 1) / S::kRows;
    p.a.info = never_split(p.a.op) ? nullptr : static_cast<int2*>(ws);
    p.a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + info_bytes(p.a.op, p.a.groups));
    p.a.page_size = fast_div((uint32_t)op.kv.page_size);
    p.k = op.kv.k;
    p.k_scale = op.kv.k_scale;
    p.to_v = (int64_t)((intptr_t)op.kv.v - (intptr_t)op.kv.k);
    p.to_v_scale = (int64_t)((intptr_t)op.kv.v_scale - (intptr_t)op.kv.k_scale);
    p.page_stride = (uint32_t)(op.kv.page_stride / 8);
    p.token_stride = (uint32_t)(op.kv.token_stride / 8);
    p.head_stride = (uint32_t)(op.kv.head_stride / 8);
    p.scale_page_stride = (uint32_t)op.kv.scale_page_stride;
    p.scale_token_stride = (uint32_t)op.kv.scale_token_stride;
    p.scale_head_stride = (uint32_t)op.kv.scale_head_stride;
    p.c2 = op.scale == 0.f ? 0.f : fmaxf(fabsf(op.scale) * kLog2e * 16.f * op.kv.k_factor, FLT_MIN);
    p.a.out_factor = 16.f * op.kv.v_factor;
    const uintptr_t rows = (uintptr_t)op.kv.k | (uintptr_t)op.kv.v | (uintptr_t)op.kv.page_stride |
                           (uintptr_t)op.kv.token_stride | (uintptr_t)op.kv.head_stride;
    p.wide = rows % 16 == 0 && op.kv.head_dim % 32 == 0;
    p.runs = p.wide && op.kv.page_size % 16 == 0;
    const uintptr_t scales = (uintptr_t)op.kv.k_scale | (uintptr_t)op.kv.v_scale | (uintptr_t)op.kv.scale_page_stride |
                             (uintptr_t)op.kv.scale_token_stride | (uintptr_t)op.kv.scale_head_stride |
                             (uintptr_t)(op.kv.head_dim / 16) | (uintptr_t)S::kScales;
    p.scale_piece = scales % 16 == 0 ? 16 : scales % 8 == 0 ? 8 : scales % 4 == 0 ? 4 : 1;
    const void* fn = (const void*)k_attn4<BF16, DP, RT>;
    cudaError_t e = tc::smem_attr_once(fn, S::kSmem);
    if (e != cudaSuccess) return e;
    const long long blocks = max_blocks(p.a.op, p.a.groups);
    int grid = sm_count() * S::kCtas;
    if (grid > kAttnMaxCtas) grid = kAttnMaxCtas;
    if (grid > blocks) grid = (int)blocks;
    void* args[] = {&p};
    e = launch_pdl(fn, dim3(grid), dim3(kAttnThreads), S::kSmem, s, args);
    if (e != cudaSuccess || never_split(p.a.op)) return e;
    return launch_join<BF16, DP, S::kRows, false>(p.a, grid, s);
}

template <bool BF16, int DP>
static cudaError_t launch_attn4_d(const dg_attn4& op, void* ws, cudaStream_t s) {
    const int rt = attn4_tiles(op);
    if constexpr (DP <= 128)
        if (rt == 4) return launch_attn4_t<BF16, DP, 4>(op, ws, s);
    return rt == 1 ? launch_attn4_t<BF16, DP, 1>(op, ws, s) : launch_attn4_t<BF16, DP, 2>(op, ws, s);
}

template <bool BF16>
static cudaError_t launch_attn4_b(const dg_attn4& op, void* ws, cudaStream_t s) {
    switch (attn4_dp(op.kv.head_dim)) {
        case 64: return launch_attn4_d<BF16, 64>(op, ws, s);
        case 128: return launch_attn4_d<BF16, 128>(op, ws, s);
        case 192: return launch_attn4_d<BF16, 192>(op, ws, s);
        default: return launch_attn4_d<BF16, 256>(op, ws, s);
    }
}

cudaError_t launch_attn4(const dg_attn4& op, void* ws, cudaStream_t s) {
    return op.kv.type == DG_BF16 ? launch_attn4_b<true>(op, ws, s) : launch_attn4_b<false>(op, ws, s);
}

}  // namespace dg
