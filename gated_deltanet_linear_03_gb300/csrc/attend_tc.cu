// gdn_attend for many query rows per key/value head (prompts and pieces of prompts): tcgen05.
//
// The mathematics is attend.cu's: x_j = s_j log2 e + log2 V_b, weights w_j = 2^{x_j - M}, o = sum w_j v_j / sum_b
// (1 / V_b) sum_{j in b} w_j.  An item is (sequence, key/value head, NQ * 128 query rows), a row being a head of the
// group at a token, so all heads of a group share every loaded and converted tile.  A unit is 64 tokens of an item.
// attend_plan_kernel lists the items and cuts their units into equal runs, one per CTA (one CTA per SM); an item
// that crosses CTAs is joined by attend_join_kernel.
//
// Warps of a CTA, each following the same run of units through mbarriers:
//   softmax (4 NQ)  thread = row.  Load the query rows, scale each exactly by a power of two, and put them into TMEM
//                   as the fp16 A operand of the score products; per unit read 64 scores, keep maximum and sum in
//                   registers, write the fp16 weights over the scores in TMEM as the A operand of the output
//                   products; rescale O in TMEM only when a weight would pass 2^15, the most that fp16 holds, so that
//                   few units pay a second pass or one over O; store the outputs.
//   loaders (8)     codes from global memory to registers (a unit ahead), turned to fp16 exactly, into 128B-swizzled
//                   shared-memory tiles: the same layout serves K (K-major B) and V (MN-major B).
//   MMA (1)         S = Q K^T of the next unit before O += W V of this one, so the tensor pipe works while the
//                   softmax does.
//   scales (1)      the unit's four block scales, their logarithms and reciprocals.
// Queries and weights as TMEM operands leave shared memory to K and V: per unit 2 x 64 x D x 2 bytes written by the
// loaders and read once by the MMAs.
// Bound by the tensor pipe (4 D FLOP a row and token).
#include "attend.cuh"

namespace gdn {
namespace {

using namespace attend;
using namespace sm100;

constexpr int kTile = 64;
constexpr int kStages = 3;
constexpr int kScaleSlots = 4;
constexpr int kLoaderWarps = 8;

template <int D>
struct Tc {
    static constexpr int NQ = D == 256 ? 1 : 2;              // 128-row tiles of a CTA
    static constexpr int ROWS = 128 * NQ;
    static constexpr int SB = NQ * (D + D / 2 + 128) <= 512 ? 2 : 1;   // score buffers of a tile
    static constexpr int O = 0, Q = NQ * D, S = NQ * (D + D / 2);      // TMEM columns
    static constexpr int CS = 2 / NQ;                        // softmax threads a row, each on 64 / CS of a unit's tokens
    static constexpr int SOFTMAX_WARPS = 8;
    static constexpr int WARPS = SOFTMAX_WARPS + kLoaderWarps + 4;     // the last four: MMA, scales, two idle
    static constexpr int THREADS = 32 * WARPS;
    // Registers a thread: at launch (the most that WARPS warps can have, a multiple of 8), then per role.  The roles'
    // shares stay within what the CTA was launched with: 640 x 96 = 256 x 136 + 256 x 72 + 128 x 64.
    static constexpr int REGS_LAUNCH = 96, REGS_SOFTMAX = 136, REGS_LOADER = 72, REGS_OTHER = 64;
    static_assert(32 * (SOFTMAX_WARPS * REGS_SOFTMAX + kLoaderWarps * REGS_LOADER + 4 * REGS_OTHER) <= THREADS * REGS_LAUNCH, "registers");
    static constexpr int TILE_BYTES = kTile * D * 2;
};

template <int D>
struct __align__(1024) TcSmem {
    uint8_t k[kStages][Tc<D>::TILE_BYTES];
    uint8_t v[kStages][Tc<D>::TILE_BYTES];
    float scale[kScaleSlots][12];        // K scales, log2 of V scales, reciprocals of V scales
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t s_full[Tc<D>::NQ][2], p_full[Tc<D>::NQ][2], pv_done[Tc<D>::NQ], q_full[Tc<D>::NQ];
    uint64_t sc_full[kScaleSlots], sc_empty[kScaleSlots], drain;
    float row_scale[Tc<D>::ROWS];                  // the power of two taken out of each query row
    // what the two warps of a row tell each other: maxima, sums, and whether a weight would be too large
    float pair[Tc<D>::CS][128], pair_sum[Tc<D>::CS][128];
    int over[2][Tc<D>::CS][4];
    uint64_t pair_bar[4];
    uint32_t tmem;
    int abort;
};

// Where a run begins: unit j of an item, and that unit's number in the whole call.
struct RunStart {
    int item, j;
    long long unit;
};

// Workspace of a call: the merge entries, the runs' starts, the item list, the parts.
struct TcPlan {
    MergeMeta *meta;       // [ctas]
    RunStart *start;       // [ctas + 1]
    long long *per;        // cost of a run
    int4 *items;           // (sequence, head, row tile, units)
    float *parts;
    int ctas;
};

__host__ __device__ inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int kPlanThreads = 1024;
// What an item costs beside its units, in units: its queries' way into TMEM, the pipeline's fill, its outputs.
constexpr int kItemCost = 4;

// Exclusive prefix of v over the CTA, and the sum.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T &sum, T *part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) part[warp] = x;
    __syncthreads();
    T before = 0;
    sum = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) {
        if (w < warp) before += part[w];
        sum += part[w];
    }
    return before + x - v;
}

// One CTA lists the items (sequence-major, heads inside, row tiles inside) and finds where every run begins.  Each thread
// takes consecutive items, so one scan over the threads gives all positions; the sequences' first items are scanned
// before, a batch of sequences at a time.
template <int ROWS>
__global__ void __launch_bounds__(kPlanThreads) attend_plan_kernel(const __grid_constant__ AttendProblem p,
                                                                   const __grid_constant__ TcPlan plan) {
    __shared__ int part[kPlanThreads / 32];
    __shared__ long long part_cost[kPlanThreads / 32];
    __shared__ int first[kPlanThreads + 1];       // first item of each sequence of the batch
    __shared__ Sequence seqs[kPlanThreads];
    const int tid = threadIdx.x, group = p.hq / p.pool.hkv;
    grid_launch_dependents();
    int items = 0;
    for (int n0 = 0; n0 < p.n_seqs; n0 += kPlanThreads) {
        const int n = n0 + tid, batch = min(kPlanThreads, p.n_seqs - n0);
        Sequence s{};
        if (n < p.n_seqs) {
            s = load_sequence(p, n);
            const int a = __ldg(p.cu + n), b = __ldg(p.cu + n + 1), c = __ldg(p.kv_lens + n);
            if (b - a > p.max_q_len || c > p.max_kv_len || c < 0 || b > p.total || a < 0 || b < a) raise_error(p.err, kErrInternal);
        }
        seqs[tid] = s;
        int sum;
        first[tid] = block_scan(row_tiles<ROWS>(s.qlen, group) * p.pool.hkv, sum, part);
        if (tid == 0) first[batch] = sum;
        __syncthreads();
        for (int k = tid; k < sum; k += kPlanThreads) {
            int lo = 0;
            for (int hi = batch; hi - lo > 1;) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= k) lo = mid;
                else hi = mid;
            }
            const int mts = row_tiles<ROWS>(seqs[lo].qlen, group), h = (k - first[lo]) / mts, mt = k - first[lo] - h * mts;
            plan.items[items + k] = make_int4(n0 + lo, h, mt, make_item<ROWS, kTile>(p, seqs[lo], group, mt).tiles);
        }
        items += sum;
        __syncthreads();
    }
    const int each = (items + kPlanThreads - 1) / kPlanThreads, i0 = min(tid * each, items), i1 = min(i0 + each, items);
    long long mine = 0, total;
    for (int i = i0; i < i1; ++i) mine += plan.items[i].w + kItemCost;
    long long at = block_scan(mine, total, part_cost);
    const long long per = max((total + plan.ctas - 1) / plan.ctas, 1LL);
    if (tid == 0) plan.per[0] = per;
    long long c = (at + per - 1) / per;           // the first run that begins at or after this thread's items
    for (int i = i0; i < i1; ++i) {
        const int w = plan.items[i].w + kItemCost;
        // a run that would begin inside an item's fixed cost begins at its first unit
        for (; c < plan.ctas && c * per < at + w; ++c) {
            const int j = max(0, (int)(c * per - at) - kItemCost);
            plan.start[c] = {i, j, at - (long long)i * kItemCost + j};
        }
        at += w;
    }
    for (long long r = (total + per - 1) / per + tid; r <= plan.ctas; r += kPlanThreads) plan.start[r] = {0, 0, total - (long long)items * kItemCost};
}

// The run of one CTA, unit by unit; every role keeps its own.
template <int ROWS>
struct Walk {
    const AttendProblem &p;
    const TcPlan &plan;
    int group, item, j, tiles, n, h, mt;
    Sequence s;
    Item it;
    __device__ __forceinline__ Walk(const AttendProblem &p_, const TcPlan &plan_, int group_) : p(p_), plan(plan_), group(group_) {
        const RunStart st = plan.start[blockIdx.x];
        item = st.item;
        load();
        j = st.j;
    }
    __device__ __forceinline__ void load() {
        const int4 d = plan.items[item];
        n = d.x;
        h = d.y;
        mt = d.z;
        tiles = d.w;
        s = load_sequence(p, n);
        it = make_item<ROWS, kTile>(p, s, group, mt);
        j = 0;
    }
    __device__ __forceinline__ int token() const { return it.token(j, kTile); }
    __device__ __forceinline__ bool last() const { return j == tiles - 1; }
    // to the next unit (which the run must hold)
    __device__ __forceinline__ void next() {
        if (++j == tiles) {
            ++item;
            load();
        }
    }
};

template <int D, int FMT>
__global__ void __launch_bounds__(Tc<D>::THREADS, 1) attend_tc_kernel(const __grid_constant__ AttendProblem p,
                                                                     const __grid_constant__ TcPlan plan) {
    using L = Tc<D>;
    constexpr int NQ = L::NQ, SB = L::SB, ROWS = L::ROWS;
    extern __shared__ uint8_t raw[];
    TcSmem<D> &sm = *reinterpret_cast<TcSmem<D> *>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int group = p.hq / p.pool.hkv, cta = blockIdx.x;

    if (warp == 0) tmem_alloc(&sm.tmem, 512);
    if (tid == 32) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sm.k_full[i], kLoaderWarps);
            mbar_init(&sm.v_full[i], kLoaderWarps);
            mbar_init(&sm.k_empty[i], 1);
            mbar_init(&sm.v_empty[i], 1);
        }
        for (int q = 0; q < NQ; ++q) {
            for (int b = 0; b < 2; ++b) {
                mbar_init(&sm.s_full[q][b], 1);
                mbar_init(&sm.p_full[q][b], 4 * L::CS);
            }
            mbar_init(&sm.pv_done[q], 1);
            mbar_init(&sm.q_full[q], 4 * L::CS);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&sm.sc_full[i], 1);
            mbar_init(&sm.sc_empty[i], L::SOFTMAX_WARPS);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&sm.pair_bar[i], 2);
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    grid_dependency_wait();
    grid_launch_dependents();
    const long long per = plan.per[0];
    const int units = (int)(plan.start[cta + 1].unit - plan.start[cta].unit);

    // A bounded wait: when it runs out, or another thread's has, every role leaves its loop.
    volatile int *abort = &sm.abort;
    auto wait_one = [&](uint64_t *bar, int phase) -> bool {
        if (mbar_try_wait(bar, (uint32_t)phase & 1)) return true;
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(bar, (uint32_t)phase & 1)) {
            if (*abort) return false;
            if (global_timer_ns() - t0 > kWaitTimeoutNs) {
                *abort = 1;
                raise_error(p.err, kErrTimeout);
                return false;
            }
        }
        return true;
    };
    // ... by all lanes of a warp, with one answer: what follows may be warp-wide.
    auto wait = [&](uint64_t *bar, int phase) -> bool { return __all_sync(0xffffffffu, wait_one(bar, phase)); };

    if (warp < L::SOFTMAX_WARPS) {
        set_max_registers_up<L::REGS_SOFTMAX>();
        // ------------------------------------------------------------------------------------------ softmax
        constexpr int CS = L::CS, NC = 64 / CS;                          // tokens of a thread's share of a unit
        const int q = CS == 2 ? 0 : warp / 4, part_of = CS == 2 ? warp / 4 : 0, quadrant = warp & 3;
        const int row = 32 * quadrant + lane;                            // of the 128-row tile
        const uint32_t quad = tmem + ((uint32_t)quadrant << 21);         // its lanes
        const uint32_t o_at = quad + L::O + q * D, q_at = quad + L::Q + q * (D / 2), s_at = quad + L::S + q * SB * 64;
        // The two warps that share rows meet at an mbarrier, so that this wait is bounded like the others.
        int pair_phase = 0;
        auto come = [&]() {
            __syncwarp();
            if (CS == 2 && lane == 0) mbar_arrive(&sm.pair_bar[quadrant]);
        };
        auto meet = [&]() -> bool { return CS == 1 || wait(&sm.pair_bar[quadrant], pair_phase++); };   // after come()
        MergeMeta mm;
        mm.last = -1;
        if (units > 0) {
            Walk<ROWS> w(p, plan, group);
            bool ok = true;
            int buf = 0, buf_phase = 0, slot = 0, slot_phase = 0;
            for (int u = 0; ok && u < units;) {
                // ---- a segment: the query rows
                const bool begun = w.j == 0;
                const int seg_slot = u == 0 ? 0 : 1;
                const int grow = w.mt * ROWS + q * 128 + row, i = grow / group;
                const bool valid = i < w.s.qlen;
                const int pos = w.s.kvlen - w.s.qlen + i;
                const size_t out_row = ((size_t)(w.s.q0 + (valid ? i : 0)) * p.hq + w.h * group + grow % group) * D;
                // 4 lanes to a row, 16 bytes each, 8 rows at a time: rows 16 half + 8 k + lane / 4 of the warp's 32.  The
                // first pass finds the rows' scales, the second (from L1) converts: fewer registers than holding them.
#pragma unroll 1
                for (int half = CS == 2 ? part_of : 0; half < (CS == 2 ? part_of + 1 : 2); ++half) {
                    const uint4 *src[2];
                    float down[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int r = 32 * quadrant + 16 * half + 8 * k + lane / 4, gr = w.mt * ROWS + q * 128 + r;
                        const int i = gr / group;
                        src[k] = i < w.s.qlen
                                     ? reinterpret_cast<const uint4 *>(p.q + ((size_t)(w.s.q0 + i) * p.hq + w.h * group + gr % group) * D) + lane % 4
                                     : nullptr;
                        uint32_t big = 0;
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) big = max(big, amax_bits(src[k] ? __ldg(src[k] + 4 * c) : make_uint4(0, 0, 0, 0)));
                        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
                        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
                        float up;
                        power_of_two_scale(big, down[k], up);
                        if (p.sm_scale < 0.f) down[k] = -down[k];     // the row factor stays >= 0
                        if (lane % 4 == 0) sm.row_scale[q * 128 + r] = up;
                    }
#pragma unroll 2
                    for (int c = 0; c < D / 64; ++c) {
                        uint32_t x[16];
#pragma unroll
                        for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint4 z = src[k] ? __ldg(src[k] + 4 * (2 * c + i2)) : make_uint4(0, 0, 0, 0);
                                x[8 * i2 + 2 * k] = bf16x2_to_f16x2(z.x, down[k]);
                                x[8 * i2 + 2 * k + 1] = bf16x2_to_f16x2(z.y, down[k]);
                                x[8 * i2 + 4 + 2 * k] = bf16x2_to_f16x2(z.z, down[k]);
                                x[8 * i2 + 4 + 2 * k + 1] = bf16x2_to_f16x2(z.w, down[k]);
                            }
                        tmem_st_16x32(q_at + ((uint32_t)(16 * half) << 16) + 32 * c, x);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                come();
                if (!(ok = meet())) break;
                if (lane == 0) mbar_arrive(&sm.q_full[q]);
                const float rs = sm.row_scale[q * 128 + row] * fabsf(p.sm_scale) * 1.4426950408889634f;
                float m = -INFINITY, l = 0.f;
                bool ends;
                for (bool first = true;; first = false) {
                    // ---- one unit
                    const uint32_t s_tm = s_at + buf * 64;
                    const int tok0 = w.token() + part_of * NC;
                    ends = w.last();
                    if (!(ok = wait(&sm.sc_full[slot], slot_phase))) break;
                    if (!(ok = wait(&sm.s_full[q][buf], buf_phase))) break;
                    tc_fence_after();
                    const bool all_seen = w.it.all_seen(tok0, tok0 + NC, p.window, p.sinks);
                    float f[NC / 16], lv[NC / 16];
                    // In the common pass the weights are formed at once with the maximum that the rows have, while the unit's
                    // own maxima are found: only where one is above it by more than 2^15 (or the row saw nothing so far) the maximum is
                    // raised, O scaled, and the pass done again.  Raised maxima then leave weights of at most 1, and they
                    // never pass 2^15, which fp16 holds.
                    bool raise = first;
                    for (;;) {
                        float s[NC];
                        if constexpr (CS == 2) tmem_ld32(s_tm + part_of * 32, s);
                        else tmem_ld32x2(s_tm, s_tm + 32, s, s + 32);
#pragma unroll
                        for (int b = 0; b < NC / 16; ++b) {
                            f[b] = rs * sm.scale[slot][part_of * (NC / 16) + b];
                            lv[b] = sm.scale[slot][4 + part_of * (NC / 16) + b];
                        }
                        if (!all_seen) {
#pragma unroll
                            for (int c = 0; c < NC; ++c)
                                s[c] = sees(pos, tok0 + c, p.window, p.sinks) ? fmaf(s[c], f[c / 16], lv[c / 16]) : -INFINITY;
#pragma unroll
                            for (int b = 0; b < NC / 16; ++b) f[b] = 1.f, lv[b] = 0.f;
                        }
                        const bool raised = raise;
                        if (raise) {
                            float top = -INFINITY;
#pragma unroll
                            for (int b = 0; b < NC / 16; ++b) {
                                float x[4];
#pragma unroll
                                for (int c = 0; c < 4; ++c) x[c] = fmaxf(fmaxf(s[16 * b + c], s[16 * b + 4 + c]), fmaxf(s[16 * b + 8 + c], s[16 * b + 12 + c]));
                                top = fmaxf(top, fmaf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), f[b], lv[b]));
                            }
                            if (CS == 2) {
                                sm.pair[part_of][row] = top;
                                come();
                                if (!(ok = meet())) break;
                                top = fmaxf(top, sm.pair[CS - 1 - part_of][row]);
                            }
                            if (first) {
                                m = top;
                            } else {
                                if (!(ok = wait(&sm.pv_done[q], u - 1))) break;
                                tc_fence_after();
                                const float to = fmaxf(m, top), c = m == to ? 1.f : exp2f(m - to);
                                m = to;
                                l *= c;
#pragma unroll 1
                                for (int k = part_of; k < D / 32; k += CS) {
                                    float o[32];
                                    tmem_ld32(o_at + 32 * k, o);
                                    uint32_t x[32];
#pragma unroll
                                    for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(o[e] * c);
                                    tmem_st32(o_at + 32 * k, x);
                                }
                                tmem_st_wait();
                            }
                        }
                        const float base = m == -INFINITY ? 0.f : m;
                        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int b = 0; b < NC / 16; ++b) {
                            const float off = lv[b] - base;
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                fma2(s[16 * b + 2 * c], s[16 * b + 2 * c + 1], f[b], off);
                                top[c & 1] = fmaxf(top[c & 1], fmaxf(s[16 * b + 2 * c], s[16 * b + 2 * c + 1]));
                            }
                        }
                        bool over = !raised && __any_sync(0xffffffffu, fmaxf(top[0], top[1]) > (m == -INFINITY ? m : 15.f));
                        if (CS == 2 && !raised) {
                            if (lane == 0) sm.over[pair_phase & 1][part_of][quadrant] = over;
                            come();
                        }
                        uint32_t x[NC / 2];
                        float add = 0.f;
#pragma unroll
                        for (int b = 0; b < NC / 16; ++b) {
                            float sum[2] = {0.f, 0.f};
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const float e0 = exp2_fast(s[16 * b + 2 * c]), e1 = exp2_fast(s[16 * b + 2 * c + 1]);
                                add2(sum[0], sum[1], e0, e1);
                                const __half2 hh = __floats2half2_rn(e0, e1);
                                x[8 * b + c] = *reinterpret_cast<const uint32_t *>(&hh);
                            }
                            sum[0] += sum[1];
                            // a block that no row sees may have any scale
                            if (sum[0] != 0.f) add = fmaf(sum[0], sm.scale[slot][8 + part_of * (NC / 16) + b], add);
                        }
                        if (CS == 2 && !raised) {
                            const int turn = pair_phase & 1;
                            if (!(ok = meet())) break;   // both have read their scores too, so weights may overwrite them
                            over |= sm.over[turn][CS - 1 - part_of][quadrant];
                        }
                        if (over) {
                            raise = true;
                            continue;
                        }
                        l += add;
                        if constexpr (CS == 2) tmem_st16(s_tm + part_of * 16, x);
                        else tmem_st32(s_tm, x);
                        break;
                    }
                    if (!ok) break;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.sc_empty[slot]);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.p_full[q][buf]);
                    if (++buf == SB) buf = 0, buf_phase ^= 1;
                    if (++slot == kScaleSlots) slot = 0, slot_phase ^= 1;
                    ++u;
                    if (ends || u == units) break;
                    w.next();
                }
                if (!ok) break;
                // ---- the segment's end
                if (!(ok = wait(&sm.pv_done[q], u - 1))) break;
                tc_fence_after();
                if (CS == 2) {
                    sm.pair_sum[part_of][row] = l;
                    come();
                    if (!(ok = meet())) break;
                    l += sm.pair_sum[CS - 1 - part_of][row];
                }
                const bool whole = begun && ends;
                float *part = plan.parts + (size_t)(2 * cta + seg_slot) * (ROWS * D + 2 * ROWS) + (size_t)(q * 128 + row) * D;
                const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
#pragma unroll 1
                for (int k = part_of; k < D / 32; k += CS) {
                    float o[32];
                    tmem_ld32(o_at + 32 * k, o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] *= inv;
                    if (valid && whole) {
                        store_row<32>(p, out_row + 32 * k, o);
                    } else if (valid) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4 *>(part + 32 * k + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                    __syncwarp();   // the next load is warp-wide
                }
                if (!whole && part_of == 0) {
                    float *ml = plan.parts + (size_t)(2 * cta + seg_slot) * (ROWS * D + 2 * ROWS) + ROWS * D;
                    ml[q * 128 + row] = m;
                    ml[ROWS + q * 128 + row] = l;
                }
                tc_fence_before();
                if (begun && !ends) {
                    const long long left = (long long)w.tiles - 1 - w.j;
                    mm.first = cta;
                    mm.slot = seg_slot;
                    mm.last = cta + (int)((left + per - 1) / per);
                    mm.n = w.n;
                    mm.h = w.h;
                    mm.mt = w.mt;
                }
                if (u < units) w.next();
            }
        }
        if (tid == 0) plan.meta[cta] = mm;
    } else if (warp < L::SOFTMAX_WARPS + kLoaderWarps) {
        set_max_registers_down<L::REGS_LOADER>();
        // ------------------------------------------------------------------------------------------ loaders
        const int lw = warp - L::SOFTMAX_WARPS;                        // rows 8 lw .. 8 lw + 7 of a tile
        // 4 lanes take the 64 codes of a column chunk of one row.  The 8 lanes that store together hold rows that
        // differ in the two low bits, so that their pieces fall on different banks in both tiles' orders.
        const int r = 8 * lw + ((lane >> 4) << 2) + ((((lane >> 2) & 1) * 3) ^ ((lane >> 3) & 1)), c16 = lane & 3;
        const uint32_t v_lo = sw128_offset(r, 16 * c16), v_hi = sw128_offset(r, 16 * c16 + 8);
        // K's columns stand in the order in which a query row's 32-element pieces enter TMEM: components 8 t + 0..3
        // at 4 t, components 8 t + 4..7 at 16 + 4 t (t = 0..3)
        const uint32_t k_lo = sw128_offset(r, 32 * (c16 >> 1) + 8 * (c16 & 1)), k_hi = sw128_offset(r, 32 * (c16 >> 1) + 16 + 8 * (c16 & 1));
        if (units > 0) {
            Walk<ROWS> w(p, plan, group);
            uint4 kr[D / 64], vr[D / 64];
            int page = -1, in_page = 0, head = 0;   // of this thread's row in the unit that `w` is at; -1: no such token
            auto look_up = [&]() {
                const int tok = w.token() + r;
                head = w.h;
                page = -1;
                if (tok >= w.s.kvlen) return;
                const int at = p.pool.page_of(tok);
                in_page = tok - at * p.pool.page_size;
                page = __ldg(p.pool.table + (size_t)w.n * p.pool.max_pages + at);
                if ((unsigned)page >= (unsigned)p.pool.n_pages) page = -2;
            };
            auto row_offset = [&]() -> long long {                     // byte offset of that row, or -1
                if (page == -2) raise_error(p.err, kErrInternal);
                return page < 0 ? -1 : ((long long)(page * p.pool.hkv + head) * p.pool.page_size + in_page) * D + 16 * c16;
            };
            auto fetch = [&](const uint8_t *pages, long long off, uint4 (&x)[D / 64]) {
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    x[c] = off >= 0 ? __ldg(reinterpret_cast<const uint4 *>(pages + off + 64 * c)) : make_uint4(0, 0, 0, 0);
            };
            auto put = [&](uint8_t *tile, const uint4 (&x)[D / 64], uint32_t lo, uint32_t hi, bool keys) {
                const uint32_t at = smem_u32(tile);
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t y[8];
                    codes_to_f16x2<FMT>(x[c].x, y[0], y[1]);
                    codes_to_f16x2<FMT>(keys ? x[c].z : x[c].y, y[2], y[3]);
                    codes_to_f16x2<FMT>(keys ? x[c].y : x[c].z, y[4], y[5]);
                    codes_to_f16x2<FMT>(x[c].w, y[6], y[7]);
                    const uint32_t a = at + c * (kTile * 128);
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a + lo), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a + hi), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7]) : "memory");
                }
                fence_proxy_async_smem();
                __syncwarp();
            };
            // codes are a unit ahead of their conversion, the table's entry another unit ahead
            look_up();
            long long off = row_offset();
            fetch(p.k_pages, off, kr);
            fetch(p.v_pages, off, vr);
            if (units > 1) {
                w.next();
                look_up();
            }
            for (int u = 0; u < units; ++u) {
                const int st = u % kStages, ph = u / kStages;
                off = row_offset();
                if (u + 2 < units) {
                    w.next();
                    look_up();
                }
                if (!wait(&sm.k_empty[st], ph + 1)) break;
                put(sm.k[st], kr, k_lo, k_hi, true);
                if (lane == 0) mbar_arrive(&sm.k_full[st]);
                if (u + 1 < units) fetch(p.k_pages, off, kr);
                if (!wait(&sm.v_empty[st], ph + 1)) break;
                put(sm.v[st], vr, v_lo, v_hi, false);
                if (lane == 0) mbar_arrive(&sm.v_full[st]);
                if (u + 1 < units) fetch(p.v_pages, off, vr);
            }
        }
    } else {
        set_max_registers_down<L::REGS_OTHER>();
        const int role = warp - L::SOFTMAX_WARPS - kLoaderWarps;
        // ------------------------------------------------------------------------------------------ MMA
        if (role == 0 && units > 0 && elect_one()) {
            // Only the ends of the items matter here: units left of this one, the next one's read ahead.
            int item = plan.start[cta].item, left = plan.items[item].w - plan.start[cta].j, next_left = 0;
            if (left < units) next_left = plan.items[item + 1].w;
            constexpr uint32_t id_s = idesc_f16_f32(128, kTile, false, false), id_o = idesc_f16_f32(128, D, false, true);
            const uint64_t kd0 = smem_desc(smem_u32(sm.k[0]), 16, 1024, kLayoutSwizzle128B);
            const uint64_t vd0 = smem_desc(smem_u32(sm.v[0]), kTile * 128, 1024, kLayoutSwizzle128B);
            constexpr uint32_t kStep = L::TILE_BYTES >> 4;
            auto scores = [&](int q, int stage, int buf) {     // S = Q K^T
                const uint64_t kd = kd0 + stage * kStep;
                const uint32_t d = tmem + L::S + (q * SB + buf) * 64, a = tmem + L::Q + q * (D / 2);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) mma_tmem_a(d, a + 8 * k, kd + ((k >> 2) * (kTile * 128) >> 4) + 2 * (k & 3), id_s, k > 0);
                mma_commit(&sm.s_full[q][buf]);
            };
            auto outputs = [&](int q, int stage, int buf, bool first) {   // O += W V
                const uint64_t vd = vd0 + stage * kStep;
                const uint32_t a = tmem + L::S + (q * SB + buf) * 64;
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k) mma_tmem_a(tmem + L::O + q * D, a + 8 * k, vd + 128 * k, id_o, !(first && k == 0));
                mma_commit(&sm.pv_done[q]);
            };
            int st = 0, ph = 0, buf = 0, buf_phase = 0, seg = 0;   // of unit u
            bool first = true;
            for (int u = 0; u < units; ++u) {
                if (first) {
                    bool ok = true;
                    for (int q = 0; q < NQ; ++q) ok = ok && wait_one(&sm.q_full[q], seg);
                    if (!ok || !wait_one(&sm.k_full[st], ph)) break;
                    tc_fence_after();
                    for (int q = 0; q < NQ; ++q) scores(q, st, buf);
                    mma_commit(&sm.k_empty[st]);
                }
                const bool ends = left == 1 || u == units - 1;
                const int nst = st + 1 == kStages ? 0 : st + 1, nph = nst == 0 ? ph ^ 1 : ph;
                const int nbuf = SB == 2 ? buf ^ 1 : 0, nbuf_phase = nbuf == 0 ? buf_phase ^ 1 : buf_phase;
                if (!ends) {
                    if (!wait_one(&sm.k_full[nst], nph)) break;
                    tc_fence_after();
                    if (SB == 2) {
                        for (int q = 0; q < NQ; ++q) scores(q, nst, nbuf);
                        mma_commit(&sm.k_empty[nst]);
                    }
                }
                if (!wait_one(&sm.v_full[st], ph)) break;
                bool ok = true;
                for (int q = 0; q < NQ; ++q) {
                    if (!(ok = wait_one(&sm.p_full[q][buf], buf_phase))) break;
                    tc_fence_after();
                    outputs(q, st, buf, first);
                    if (SB == 1 && !ends) scores(q, nst, nbuf);
                }
                if (!ok) break;
                mma_commit(&sm.v_empty[st]);
                if (SB == 1 && !ends) mma_commit(&sm.k_empty[nst]);
                st = nst;
                ph = nph;
                buf = nbuf;
                buf_phase = nbuf_phase;
                first = ends;
                if (--left == 0) {
                    ++seg;
                    ++item;
                    left = next_left;
                    if (u + 1 + left < units) next_left = plan.items[item + 1].w;
                }
            }
            // every MMA has finished before the tensor memory is given back
            mma_commit(&sm.drain);
            if (!mbar_wait(&sm.drain, 0)) raise_error(p.err, kErrTimeout);
        }
        // ------------------------------------------------------------------------------------------ scales
        if (role == 1 && units > 0) {
            Walk<ROWS> w(p, plan, group);
            // lanes 0..3 hold the unit's K scales, 4..7 its V scales: read a unit ahead, the table another one
            const float *scales = lane < 4 ? p.k_scales : p.v_scales;
            int page = -1, block = 0, head = 0;
            auto look_up = [&]() {
                const int tok = w.token() + (lane & 3) * kKvBlock;
                head = w.h;
                page = -1;
                if (lane >= 8 || tok >= w.s.kvlen) return;
                const int at = p.pool.page_of(tok);
                block = (tok - at * p.pool.page_size) / kKvBlock;
                page = __ldg(p.pool.table + (size_t)w.n * p.pool.max_pages + at);
            };
            auto fetch = [&]() {
                return (unsigned)page < (unsigned)p.pool.n_pages
                           ? __ldg(scales + ((size_t)page * p.pool.hkv + head) * (p.pool.page_size / kKvBlock) + block)
                           : 0.f;
            };
            look_up();
            float x = fetch();
            if (units > 1) {
                w.next();
                look_up();
            }
            for (int u = 0; u < units; ++u) {
                const int slot = u % kScaleSlots;
                const float next = u + 1 < units ? fetch() : 0.f;
                if (u + 2 < units) {
                    w.next();
                    look_up();
                }
                if (!wait(&sm.sc_empty[slot], u / kScaleSlots + 1)) break;
                if (lane < 4) {
                    sm.scale[slot][lane] = x;
                } else if (lane < 8) {
                    if (x == 0.f) x = kAmaxFloor;
                    sm.scale[slot][lane] = log2f(x);
                    sm.scale[slot][lane + 4] = 1.f / x;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.sc_full[slot]);
                x = next;
            }
        }
    }
    __syncthreads();
    if (warp == 0) {
        tmem_relinquish();
        tmem_dealloc(tmem, 512);
    }
}

struct TcSizes {
    long long items;
    int ctas;
    size_t start, per, list, parts, bytes;
};

// Workspace layout; `sms` bounds the CTAs (the size is asked for with the largest).
TcSizes tc_sizes(int n_seqs, int total, int hq, int hkv, int d, int sms) {
    TcSizes z;
    const int rows = d == 256 ? 128 : 256;
    z.items = hkv * (((long long)total * (hq / hkv) + rows - 1) / rows + n_seqs);
    z.ctas = min(sms, kMaxTcCtas);
    z.start = round256(kMaxTcCtas * sizeof(MergeMeta));
    z.per = z.start + round256((kMaxTcCtas + 1) * sizeof(RunStart));
    z.list = z.per + 256;
    z.parts = z.list + round256((size_t)z.items * sizeof(int4));
    z.bytes = z.parts + (size_t)2 * z.ctas * (rows * d + 2 * rows) * sizeof(float);
    return z;
}

template <int D, int FMT>
cudaError_t launch_tc(const AttendProblem &p) {
    using L = Tc<D>;
    const TcSizes z = tc_sizes(p.n_seqs, p.total, p.hq, p.pool.hkv, D, multiprocessor_count());
    uint8_t *ws = static_cast<uint8_t *>(p.workspace);
    TcPlan plan{};
    plan.meta = reinterpret_cast<MergeMeta *>(ws);
    plan.start = reinterpret_cast<RunStart *>(ws + z.start);
    plan.per = reinterpret_cast<long long *>(ws + z.per);
    plan.items = reinterpret_cast<int4 *>(ws + z.list);
    plan.parts = reinterpret_cast<float *>(ws + z.parts);
    plan.ctas = z.ctas;
    constexpr size_t smem = sizeof(TcSmem<D>) + 1024;
    static std::atomic<bool> ready[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(attend_tc_kernel<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) ready[dev].store(true, std::memory_order_relaxed);
    }
    attend_plan_kernel<L::ROWS><<<1, kPlanThreads, 0, p.stream>>>(p, plan);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_after(p.stream, dim3((unsigned)z.ctas), L::THREADS, smem, attend_tc_kernel<D, FMT>, p, plan)) != cudaSuccess) return e;
    return launch_after(p.stream, dim3((unsigned)z.ctas, L::ROWS / 8), 256, 0, attend_join_kernel<D, L::ROWS>, p,
                        static_cast<const MergeMeta *>(plan.meta), static_cast<const float *>(plan.parts));
}

}  // namespace

size_t attend_tc_workspace_bytes(int n_seqs, int total, int hq, int hkv, int d) {
    return tc_sizes(n_seqs, total, hq, hkv, d, attend::kMaxTcCtas).bytes;
}

cudaError_t launch_attend_tc(const AttendProblem &p) {
    const bool e4m3 = p.format == GDN_KV_E4M3;
    switch (p.d) {
        case 64: return e4m3 ? launch_tc<64, GDN_KV_E4M3>(p) : launch_tc<64, GDN_KV_INT8>(p);
        case 128: return e4m3 ? launch_tc<128, GDN_KV_E4M3>(p) : launch_tc<128, GDN_KV_INT8>(p);
        default: return e4m3 ? launch_tc<256, GDN_KV_E4M3>(p) : launch_tc<256, GDN_KV_INT8>(p);
    }
}

}  // namespace gdn
