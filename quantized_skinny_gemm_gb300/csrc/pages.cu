// Pages and slots for the tokens of a step, from the sequences' lengths.
//
// Three running sums over the sequences say everything: of the tokens asked for
// (where a sequence's tokens lie in the map, and whether they fit it), of the pages
// that the fitting ones need beyond those held (who is served, and which pages of the
// queue are whose), and of the pages given back.  One CTA takes the sums and leaves a
// record for each sequence; then each token, page taken and page given back finds its
// sequence by a search over the records and is written by a thread of its own.
//
// Bound by latency: small calls are one CTA that keeps the records in shared memory and
// writes everything itself (64 sequences, a token each: 3.7 us); others two launches, the sums by
// one CTA and the rest by many (3000 sequences, 2.1 million places: 18.5 us, 4 of them the bytes, about 6 the
// sums, the rest search -> table -> store, at 56 % of the issue slots).
#include <climits>

#include "elem.cuh"

namespace dg {

constexpr int kPlanThreads = 1024;
constexpr int kPlanItems = 4;            // sequences of a thread in a round of the large form
constexpr int kAtOnce = 4;              // entries of a thread under way
constexpr int kPlanSmallBatch = 1024, kPlanSmallTokens = 16384;

struct PlanTotals {
    int first, count, taken, given;
};
struct PlanParams {
    dg_page_plan op;
    FastDiv page;
    PlanTotals* totals;   // large form: workspace
    int4* rec;            // [batch + 1]
};

// A sequence's record: x its first token in the map, y its first page of those taken,
// z its first page of those given back, w its length, or ~length where it is not
// served.  Sums past 2^31 - 1 stay there.
__device__ __forceinline__ int sat(long long v) { return v > INT_MAX ? INT_MAX : (int)v; }

// Inclusive sums over the CTA's threads, and their totals.
struct Pair {
    long long a, b;
};
__device__ __forceinline__ Pair block_scan(Pair v, Pair* warps, Pair& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, v.a, o), b = __shfl_up_sync(0xffffffffu, v.b, o);
        if (lane >= o) {
            v.a += a;
            v.b += b;
        }
    }
    __syncthreads();   // the last call's sums have been read
    if (lane == 31) warps[warp] = v;
    __syncthreads();
    Pair w = lane < n ? warps[lane] : Pair{0, 0};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, w.a, o), b = __shfl_up_sync(0xffffffffu, w.b, o);
        if (lane >= o) {
            w.a += a;
            w.b += b;
        }
    }
    total = {__shfl_sync(0xffffffffu, w.a, 31), __shfl_sync(0xffffffffu, w.b, 31)};
    const Pair before = {__shfl_sync(0xffffffffu, w.a, max(warp - 1, 0)),
                         __shfl_sync(0xffffffffu, w.b, max(warp - 1, 0))};
    if (warp) {
        v.a += before.a;
        v.b += before.b;
    }
    return v;
}

// Pages of 0 <= tokens < 2^31, without a division and its many instructions (of 64 bits, 12 a thread in the sums:
// 3000 sequences and 2.1 million places 24 us, this way 21.5).
__device__ __forceinline__ int pages_of(int tokens, FastDiv page) { return tokens > 0 ? (tokens - 1) / page + 1 : 0; }

// All running sums, by one CTA.  rec may be shared memory.
template <int ITEMS>
__device__ void plan_sums(const PlanParams& p, int4* rec, PlanTotals& out) {
    __shared__ Pair warps[32];
    __shared__ int most;
    const dg_page_plan& op = p.op;
    const int B = op.batch, N = op.pool_size;
    int first = op.pool_state[0] % N;
    if (first < 0) first += N;
    const int count = min(max(op.pool_state[1], 0), N);
    if (threadIdx.x == 0) most = 0;
    __syncthreads();
    Pair carry = {0, 0}, asked = {0, 0};   // tokens and pages given back; pages asked for
    int taken = 0;
    for (int b0 = 0; b0 < B; b0 += blockDim.x * ITEMS) {
        const int mine = b0 + threadIdx.x * ITEMS;
        int len[ITEMS], want[ITEMS], back[ITEMS];
        int more[ITEMS];
        Pair sum = {0, 0};
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int b = mine + i;
            len[i] = want[i] = back[i] = 0;
            if (b < B) {
                const int n = op.new_lens ? op.new_lens[b] : op.new_len;
                len[i] = max(op.lens[b], 0);
                want[i] = n;
                if (n < 0) back[i] = min(pages_of(len[i], p.page), op.max_pages);
            }
            sum.a += max(want[i], 0);
            sum.b += back[i];
        }
        Pair total;
        Pair at = block_scan(sum, warps, total);
        at = {carry.a + at.a - sum.a, carry.b + at.b - sum.b};
        carry = {carry.a + total.a, carry.b + total.b};
        Pair need = {0, 0};
        long long end = at.a;
        bool fits[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int w = max(want[i], 0);
            end += w;
            const long long grown = (long long)len[i] + w;
            const int pages = pages_of((int)min(grown, (long long)INT_MAX), p.page);
            fits[i] = mine + i < B && want[i] >= 0 && pages <= op.max_pages && grown <= INT_MAX &&
                      (!op.slots || end <= op.max_tokens);
            more[i] = fits[i] ? pages - pages_of(len[i], p.page) : 0;
            need.a += more[i];
        }
        Pair all;
        Pair pg = block_scan(need, warps, all);
        long long upto = asked.a + pg.a - need.a;
        asked.a += all.a;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int b = mine + i;
            if (b >= B) break;
            const long long from = upto;
            upto += more[i];
            const bool served = fits[i] && (more[i] == 0 || upto <= count);
            if (served && more[i]) taken = (int)upto;
            rec[b] = make_int4(sat(at.a), sat(from), sat(at.b), served ? len[i] : ~len[i]);
            if (op.starts) op.starts[b] = sat(at.a);
            op.lens_out[b] = want[i] < 0 ? 0 : served ? len[i] + want[i] : op.lens[b];
            at.a += max(want[i], 0);
            at.b += back[i];
        }
    }
    if (taken) atomicMax(&most, taken);
    __syncthreads();
    out.first = first;
    out.count = count;
    out.taken = most;
    out.given = (int)min(carry.b, (long long)N - count);   // the queue holds no more
    if (threadIdx.x == 0) {
        rec[B] = make_int4(sat(carry.a), INT_MAX, INT_MAX, 0);
        if (op.starts) op.starts[B] = sat(carry.a);
        op.pool_state_out[0] = (int)(((long long)first + out.taken) % N);
        op.pool_state_out[1] = count - out.taken + out.given;
    }
}

// The last record whose field F is at most v, from record lo on.
template <int F>
__device__ __forceinline__ int find(const int4* rec, int B, int v, int lo = 0) {
    int hi = B;   // rec[lo] <= v < rec[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        const int x = F == 0 ? rec[mid].x : F == 1 ? rec[mid].y : rec[mid].z;
        if (x <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Tokens, pages taken and pages given back, by all threads of the launch.  A warp takes runs of
// up to 256 tokens and looks for the sequences of the run's first and last one, 32 records a step;
// a lane then searches between these for its first token's sequence and mostly stays there.  Four
// tokens of a lane are under way at once.  (2.1 million places of 3000 sequences, the whole call: 18 us; 21.5
// with a lane's own search over all records and one token after the other, 22 and 20 with one of the two.)
template <bool ALONE>   // the launch is one CTA
__device__ __forceinline__ void plan_fill(const PlanParams& p, const int4* rec, const PlanTotals& t, unsigned id,
                                          unsigned threads) {
    const dg_page_plan& op = p.op;
    const int N = op.pool_size;
    auto queue = [&](int i) {
        const long long at = (long long)t.first + i;   // below 2 N
        return (int)(at < N ? at : at - N);
    };
    const int tokens = min(rec[op.batch].x, op.max_tokens);
    if (op.slots) {
        const int run = (int)min(256ll, max(32ll, ((long long)op.max_tokens + threads - 1) / threads * 32));   // of a warp
        for (long long i0 = (long long)(id >> 5) * run; i0 < op.max_tokens; i0 += (long long)(threads >> 5) * run) {
            int b = -1, last = -1;   // the sequence of the last token, and the first token behind it
            int4 r = make_int4(0, 0, 0, 0);
            // the sequences of the run's first and last token, by the warp: 32 places a step
            int b0 = 0, b1 = op.batch;   // rec[b0].x <= first, rec[b1].x > last
            if (!ALONE && i0 < tokens) {
                const int v = (int)i0, w = (int)min(i0 + run, (long long)tokens) - 1;
                int hi = op.batch, lo = 0;
                while (hi - b0 > 1 || b1 - lo > 1) {
                    const int s0 = (hi - b0 + 31) >> 5, s1 = (b1 - lo + 31) >> 5;
                    const int a0 = b0 + (int)(id & 31) * s0, a1 = lo + (int)(id & 31) * s1;
                    const unsigned m0 = __ballot_sync(0xffffffffu, a0 < hi && rec[min(a0, hi)].x <= v);
                    const unsigned m1 = __ballot_sync(0xffffffffu, a1 < b1 && rec[min(a1, b1)].x <= w);
                    b0 += (31 - __clz(m0)) * s0;
                    hi = min(hi, b0 + s0);
                    lo += (31 - __clz(m1)) * s1;
                    b1 = min(b1, lo + s1);
                }
            }
            for (int k = id & 31; k < run; k += 32 * kAtOnce) {
                int page[kAtOnce], pos[kAtOnce], in[kAtOnce];
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    const long long i = i0 + k + 32 * j;
                    page[j] = pos[j] = -1;
                    in[j] = 0;
                    if (k + 32 * j >= run || i >= tokens) continue;
                    if (i >= last) {
                        b = find<0>(rec, ALONE ? op.batch : b1, (int)i, max(b, b0));
                        r = rec[b];
                        last = rec[b + 1].x;
                    }
                    if (r.w < 0) continue;
                    pos[j] = r.w + ((int)i - r.x);
                    const int at = pos[j] / p.page, held = pages_of(r.w, p.page);
                    in[j] = pos[j] - at * op.page_size;
                    page[j] = at < held ? op.block_table[(long long)b * op.table_stride + at]
                                        : op.pool[queue(r.y + at - held)];
                }
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    const long long i = i0 + k + 32 * j;
                    if (k + 32 * j >= run || i >= op.max_tokens) continue;
                    op.slots[i] = page[j] >= 0 ? (long long)page[j] * op.page_size + in[j] : -1;
                    if (op.positions) op.positions[i] = pos[j];
                }
            }
        }
    }
    for (long long i = id; i < t.taken; i += threads) {
        const int b = find<1>(rec, op.batch, (int)i);
        const int4 r = rec[b];
        op.block_table[(long long)b * op.table_stride + pages_of(r.w, p.page) + ((int)i - r.y)] =
            op.pool[queue((int)i)];
    }
    if constexpr (!ALONE) {
        for (long long i = id; i < t.given; i += threads) {
            const int b = find<2>(rec, op.batch, (int)i);
            op.pool[queue(t.count + (int)i)] =
                op.block_table[(long long)b * op.table_stride + ((int)i - rec[b].z)];
        }
        return;
    }
    // One CTA: runs of a warp here too, four entries of a lane at once (64 sequences of 4096 tokens that end, pages
    // of 16: 25 us, with a search for each entry 58).
    const int run = (int)min(256ll, max(32ll, ((long long)t.given + threads - 1) / threads * 32));
    for (long long i0 = (long long)(id >> 5) * run; i0 < t.given; i0 += (long long)(threads >> 5) * run) {
        int b = -1, first = 0, last = -1;
        for (int k = id & 31; k < run; k += 32 * kAtOnce) {
            int page[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const long long i = i0 + k + 32 * j;
                if (k + 32 * j >= run || i >= t.given) continue;
                if (i >= last) {
                    b = find<2>(rec, op.batch, (int)i, max(b, 0));
                    first = rec[b].z;
                    last = rec[b + 1].z;
                }
                page[j] = op.block_table[(long long)b * op.table_stride + ((int)i - first)];
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const long long i = i0 + k + 32 * j;
                if (k + 32 * j < run && i < t.given) op.pool[queue(t.count + (int)i)] = page[j];
            }
        }
    }
}

__global__ void __launch_bounds__(kPlanThreads) k_plan_small(const PlanParams p) {
    __shared__ int4 rec[kPlanSmallBatch + 1];
    griddep_launch_dependents();
    griddep_wait();
    PlanTotals t;
    plan_sums<1>(p, rec, t);
    __syncthreads();
    plan_fill<true>(p, rec, t, threadIdx.x, blockDim.x);
}

__global__ void __launch_bounds__(kPlanThreads) k_plan_sums(const PlanParams p) {
    griddep_launch_dependents();
    griddep_wait();
    PlanTotals t;
    plan_sums<kPlanItems>(p, p.rec, t);
    if (threadIdx.x == 0) *p.totals = t;
}

__global__ void __launch_bounds__(256) k_plan_fill(const PlanParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const PlanTotals t = *p.totals;
    plan_fill<false>(p, p.rec, t, blockIdx.x * blockDim.x + threadIdx.x, gridDim.x * blockDim.x);
}

// One CTA against two launches, us: 64 sequences with a map of 64 places 3.4 and 7.5, of 4096 7.2 and 8.0, of 16384 12.6
// and 8.0, of 65536 36 and 7.8; 1024 sequences with 1024 places 5.9 and 8.5, with 16384 21 and 9.8.  So the forms cross
// between 4096 and 8192 places.  Pages that move have no part in the rule, nor in the second launch's size: 64
// sequences of 131072 tokens that end without a map take 704 and 979, of 4096 25 and 41.
static bool plan_small(const dg_page_plan& op) {
    return op.batch <= kPlanSmallBatch && op.max_tokens <= kPlanSmallTokens;
}

size_t plan_ws_bytes(const dg_page_plan& op) {
    return plan_small(op) ? 0 : sizeof(PlanTotals) + ((size_t)op.batch + 1) * sizeof(int4);
}

cudaError_t launch_plan(const dg_page_plan& op, void* ws, cudaStream_t s) {
    PlanParams p{op, fast_div((uint32_t)op.page_size), static_cast<PlanTotals*>(ws),
                 reinterpret_cast<int4*>(static_cast<char*>(ws) + sizeof(PlanTotals))};
    void* args[] = {&p};
    if (plan_small(op)) {
        const int work = op.batch > op.max_tokens ? op.batch : op.max_tokens;
        const int threads = work <= 128 ? 128 : work <= 256 ? 256 : kPlanThreads;
        return launch_pdl((const void*)k_plan_small, dim3(1),
                          dim3(op.batch > threads ? kPlanThreads : threads), 0, s, args);
    }
    const cudaError_t e = launch_pdl((const void*)k_plan_sums, dim3(1), dim3(kPlanThreads), 0, s, args);
    if (e != cudaSuccess) return e;
    const long long want = ((long long)op.max_tokens + 4ll * op.batch + 255) / 256, most = sm_count() * 8ll;
    return launch_pdl((const void*)k_plan_fill, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, s, args);
}

}  // namespace dg
