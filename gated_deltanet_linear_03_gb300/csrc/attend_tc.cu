// gdn_attend for many query rows per key/value head (prompts and pieces of prompts): tcgen05.
//
// The mathematics is attend.cu's: x_j = s_j log2 e + log2 V_b, weights w_j = 2^{x_j - M}, o = sum w_j v_j / sum_b
// (1 / V_b) sum_{j in b} w_j.  An item is (sequence, key/value head, NQ * 128 query rows), a row being a head of the
// group at a token, so all heads of a group share every loaded and converted tile.  A unit is 64 tokens of an item.
// attend_plan_kernel lists the items and cuts their units into equal runs, one per CTA (one CTA per SM); an item
// that crosses CTAs is joined by attend_join_kernel.
//
// Warps of a CTA, each following the same run of units through mbarriers (28 warps, 896 threads):
//   softmax (8 NQ)  a warp has 16 rows, 4 lanes to a row.  It brings their queries, scaled exactly by a power of two, into
//                   TMEM (d = 128: shared memory) as the fp16 A operand of the score products; per unit it reads the rows' 64 scores, forms the
//                   weights in one pass with the rows' present reference M and writes them as fp16 over the scores, where
//                   they are the A operand of the output products.  Only where a score is above M by more than 15 (2^15
//                   is the most that fp16 holds) M is raised, O scaled in TMEM, and the pass done again.  So the
//                   common pass needs no exchange beyond the warp, and no reduction over a row until the item's end.
//                   At an item's end it writes its rows' outputs, or their part for the join.
//   look-up (1)     table entries, rows in the pool and block scales of eight units at a time, a lane to a block of 16 tokens.
//   loaders (8, 16) codes from global memory to registers, turned to fp16 exactly, into 128B-swizzled shared-memory tiles:
//                   the same layout serves K (K-major B) and V (MN-major B).
//   MMA (2)         one issues S = Q K^T, as far ahead as there are score buffers, one O += W V.
// Queries and weights as TMEM operands leave shared memory to K and V: per unit 2 x 64 x D x 2 bytes written by the
// loaders and read NQ times by the MMAs.
//
// Floor: the tensor pipe, 4 D FLOP a row and token (1024 cycles a unit at d = 256).  Measured at d = 256, 16 heads over 2:
// 8192-token prompt 439 us, 0.66 of a library product's rate; 509 tokens behind 16384 119 us, 0.60; d = 128: 8192 tokens of
// 16 heads over 2 254 us, 0.57, ragged prompts of 100 to 5000 tokens of 32 over 8 207 us, 0.44; of d = 64 171 us, 0.27 (its
// exponentials are as many as at d = 128, its products half).  What bounds a unit is the way
// of its scores from product to product (commit, TMEM to registers, weights, back, commit) with two score buffers a tile, which is
// all that TMEM holds; the softmax and loader warps issue in more than half of the cycles and share them with that way, and the
// tiles' writes and the products' reads together take most of shared memory's bandwidth.  An item's ends (queries in, pipeline
// full, outputs out) cost some 7 units' time, which short prompts pay most often.
// Tried and slower: weights in buffers of their own, so that the next score product may start when the scores are in
// registers; two sets of softmax warps on alternate units; one warp that issues both products in a fixed order.
#include "attend.cuh"

namespace gdn {
namespace {

using namespace attend;
using namespace sm100;

constexpr int kTile = 64;
constexpr int kSlots = 32, kSlotGroup = 8;   // what the look-up warp leaves of a unit: a ring of slots, filled eight at a time

template <int D>
struct Tc {
    // 128-row tiles of a CTA, which share its K and V.  At d = 256 TMEM holds one; below, two are faster than one: ragged prompts
    // of d = 128 207 us against 285, of d = 64 172 against 251.
    static constexpr int NQ = D == 256 ? 1 : 2;
    static constexpr int ROWS = 128 * NQ;
    // Queries in shared memory instead of TMEM at d = 128: a score product then takes 1.5 times as long, but there is room for a
    // second score buffer a tile (8192-token prompt 276 us against 315, ragged prompts 226 / 249; at d = 256, four buffers instead
    // of two, 493 / 441; at d = 64, as many as without, 177 / 173 for ragged prompts).
    static constexpr bool QS = D == 128;
    // TMEM columns: O fp32, Q two fp16 a column, then SB buffers a tile of 64 scores, over which the weights are written.
    static constexpr int O = 0, Q = NQ * D, S = NQ * (QS ? D : D + D / 2), SB = (512 - S) / (64 * NQ);
    static_assert(SB >= 1 && S + NQ * SB * 64 <= 512, "tensor memory");
    // Stages of K and V tiles in shared memory.  What they leave is L1 cache, through which queries and codes come: at d = 256
    // three stages leave next to none (8192-token prompt 468 us with three, 441 with two; of d = 128 276 / 272).
    static constexpr int STAGES = 2;
    static constexpr int LG = D == 256 ? 2 : 1;              // groups of 8 loader warps, which take the tiles in turn
    static constexpr int SOFTMAX_WARPS = 8 * NQ, LOADER_WARPS = 8 * LG;
    static constexpr int WARPS = SOFTMAX_WARPS + LOADER_WARPS + 4;     // the last four: MMA, MMA, look-up, idle
    static constexpr int THREADS = 32 * WARPS;               // 896
    // Registers a thread: at launch (the most that 28 warps can have, a multiple of 8), then per role.  The roles' shares
    // stay within what the CTA was launched with: 896 x 72 = 256 x 104 + 512 x 56 + 128 x 72 = 512 x 88 + 256 x 48 + 128 x 56.
    static constexpr int REGS_LAUNCH = 72, REGS_SOFTMAX = NQ == 1 ? 104 : 88, REGS_LOADER = NQ == 1 ? 56 : 48, REGS_OTHER = NQ == 1 ? 72 : 56;
    static_assert(32 * (SOFTMAX_WARPS * REGS_SOFTMAX + LOADER_WARPS * REGS_LOADER + 4 * REGS_OTHER) <= THREADS * REGS_LAUNCH, "registers");
    static constexpr int TILE_BYTES = kTile * D * 2, CHUNK = kTile * 128;   // CHUNK: 64 columns
    static constexpr int Q_BYTES = QS ? 128 * D * 2 : 0, Q_CHUNK = 128 * 128;   // of a tile's queries
};

template <int D>
struct __align__(1024) TcSmem {
    static constexpr int NQ = Tc<D>::NQ, STAGES = Tc<D>::STAGES;
    uint8_t k[STAGES][Tc<D>::TILE_BYTES];
    uint8_t v[STAGES][Tc<D>::TILE_BYTES];
    uint8_t q[NQ * Tc<D>::Q_BYTES + 1024 * !Tc<D>::QS];   // (never empty)
    float scale[kSlots][12];             // of a unit's 4 blocks: K scales, log2 of V scales, reciprocals of V scales
    int2 block[kSlots][4];               // and their first rows in the pool (-1: none), and how many tokens they hold
    uint64_t slots_full[kSlots / kSlotGroup], slots_free[kSlots / kSlotGroup];
    uint64_t k_full[STAGES], k_empty[STAGES], v_full[STAGES], v_empty[STAGES];
    uint64_t s_full[NQ * Tc<D>::SB], p_full[NQ * Tc<D>::SB], p_free[NQ * Tc<D>::SB], q_full[NQ], drain[2];
    uint32_t tmem;
    int abort;
};

// Where a run begins: unit j of an item, and that unit's number in the whole call.
struct RunStart {
    int item, j;
    long long unit;
};

// An item as its units' roles see it, worked out once: (sequence, key/value head, row tile) and its units, the sequence,
// and the tokens that its rows see (an Item's fields).
struct __align__(16) TcItem {
    int n, h, mt, tiles, q0, qlen, kvlen, lo_pos, hi_pos, near_tiles, far_tile, unused;
};

// Workspace of a call: the merge entries, the runs' starts, the item list, the parts.
struct TcPlan {
    MergeMeta *meta;       // [ctas]
    RunStart *start;       // [ctas + 1]
    long long *per;        // cost of a run
    TcItem *items;
    float *parts;
    int ctas;
    int max_items;         // that the list has room for: all that sequences in order within `total` rows can have
};

__host__ __device__ inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int kPlanThreads = 1024;
// What an item costs beside its units, in units: its queries' way in, the pipeline's fill, its outputs.  (8192-token prompt of
// d = 256 491 us with 5, 441 with 7, 442 with 8; ragged prompts of d = 128 227 us with 4, 207 with 6, 211 with 8, of d = 64 174
// with 4, 172 with 5, 176 with 7.)
template <int D>
__host__ __device__ constexpr int item_cost() { return D == 256 ? 7 : D == 128 ? 6 : 5; }

// Exclusive prefix of v over the CTA, and the sum.
__device__ __forceinline__ long long block_scan(long long v, long long &sum, long long *part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) part[warp] = x;
    __syncthreads();
    long long before = 0;
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
template <int ROWS, int ITEM_COST>
__global__ void __launch_bounds__(kPlanThreads) attend_plan_kernel(const __grid_constant__ AttendProblem p, const __grid_constant__ TcPlan plan) {
    __shared__ long long part[kPlanThreads / 32];
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
        // (in 64 bits: sequences out of order may hold the call's rows many times over; what is too many is cut, and recorded)
        const long long room = plan.max_items - items;
        long long all;
        first[tid] = (int)min(block_scan((long long)row_tiles<ROWS>(s.qlen, group) * p.pool.hkv, all, part), room);
        const int sum = (int)min(all, room);
        if (tid == 0) first[batch] = sum;
        __syncthreads();
        if (tid == 0 && all > room) raise_error(p.err, kErrInternal);
        for (int k = tid; k < sum; k += kPlanThreads) {
            int lo = 0;
            for (int hi = batch; hi - lo > 1;) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= k) lo = mid;
                else hi = mid;
            }
            const int mts = row_tiles<ROWS>(seqs[lo].qlen, group), h = (k - first[lo]) / mts, mt = k - first[lo] - h * mts;
            const Sequence q = seqs[lo];
            const Item it = make_item<ROWS, kTile>(p, q, group, mt);
            plan.items[items + k] = {n0 + lo, h, mt, it.tiles, q.q0, q.qlen, q.kvlen, it.lo_pos, it.hi_pos, it.near_tiles, it.far_tile, 0};
        }
        items += sum;
        __syncthreads();
    }
    const int each = (items + kPlanThreads - 1) / kPlanThreads, i0 = min(tid * each, items), i1 = min(i0 + each, items);
    long long mine = 0, total;
    for (int i = i0; i < i1; ++i) mine += plan.items[i].tiles + ITEM_COST;
    long long at = block_scan(mine, total, part);
    const long long per = max((total + plan.ctas - 1) / plan.ctas, 1LL);
    if (tid == 0) plan.per[0] = per;
    long long c = (at + per - 1) / per;           // the first run that begins at or after this thread's items
    for (int i = i0; i < i1; ++i) {
        const int w = plan.items[i].tiles + ITEM_COST;
        // a run that would begin inside an item's fixed cost begins at its first unit
        for (; c < plan.ctas && c * per < at + w; ++c) {
            const int j = max(0, (int)(c * per - at) - ITEM_COST);
            plan.start[c] = {i, j, at - (long long)i * ITEM_COST + j};
        }
        at += w;
    }
    for (long long r = (total + per - 1) / per + tid; r <= plan.ctas; r += kPlanThreads) plan.start[r] = {0, 0, total - (long long)items * ITEM_COST};
}

// M of a row that has seen no token yet: so low that the weight of any token against it is infinite, however small its score.
// (Under a window a row may see its first token in a later unit than its item's first row.)
constexpr float kNoReference = -3.4028235e38f;

// A word with its n lowest bits set (none below 0, all above 63).
__device__ __forceinline__ unsigned long long low_bits(int n) { return n <= 0 ? 0ull : n > 63 ? ~0ull : (1ull << n) - 1; }

template <bool V>
struct Flag {
    static constexpr bool value = V;
};

template <int AT>
__device__ __forceinline__ void store_shared(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0 + %5], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w), "n"(AT) : "memory");
}

// A loader thread's codes of a unit's tile as fp16, from piece N (16 codes) on: the first and the last 8 of K's order, or of V's.
template <int D, int FMT, bool KEYS, int N = 0>
__device__ __forceinline__ void put_codes(uint32_t lo, uint32_t hi, const uint4 (&x)[D / 64]) {
    const uint4 z = x[N];
    uint32_t y[8];
    codes_to_f16x2<FMT>(z.x, y[0], y[1]);
    codes_to_f16x2<FMT>(KEYS ? z.z : z.y, y[2], y[3]);
    codes_to_f16x2<FMT>(KEYS ? z.y : z.z, y[4], y[5]);
    codes_to_f16x2<FMT>(z.w, y[6], y[7]);
    store_shared<N * Tc<D>::CHUNK>(lo, y[0], y[1], y[2], y[3]);
    store_shared<N * Tc<D>::CHUNK>(hi, y[4], y[5], y[6], y[7]);
    if constexpr (N + 1 < D / 64) put_codes<D, FMT, KEYS, N + 1>(lo, hi, x);
}

// 4 x 4 words of 4 neighbouring lanes, lane t's word i becoming lane i's word t.
__device__ __forceinline__ void transpose4(uint32_t (&y)[4], int t) {
#pragma unroll
    for (int s = 1; s <= 2; s <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & s) continue;
            const uint32_t r = __shfl_xor_sync(0xffffffffu, t & s ? y[i] : y[i + s], s);
            if (t & s) y[i] = r;
            else y[i + s] = r;
        }
}

// The first token of unit j of an item with these fields.
__device__ __forceinline__ int first_token(int near_tiles, int far_tile, int j) { return (j < near_tiles ? j : far_tile + j - near_tiles) * kTile; }

template <int D, int FMT>
__global__ void __launch_bounds__(Tc<D>::THREADS, 1) attend_tc_kernel(const __grid_constant__ AttendProblem p,
                                                                     const __grid_constant__ TcPlan plan) {
    using L = Tc<D>;
    constexpr int NQ = L::NQ, SB = L::SB, STAGES = L::STAGES, ROWS = L::ROWS;
    extern __shared__ uint8_t raw[];
    TcSmem<D> &sm = *reinterpret_cast<TcSmem<D> *>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int group = p.hq / p.pool.hkv, cta = blockIdx.x;

    if (warp == 0) tmem_alloc(&sm.tmem, 512);
    if (tid == 32) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&sm.k_full[i], 8);
            mbar_init(&sm.v_full[i], 8);
            mbar_init(&sm.k_empty[i], 1);
            mbar_init(&sm.v_empty[i], 1);
        }
        for (int q = 0; q < NQ; ++q) mbar_init(&sm.q_full[q], 8);
        for (int b = 0; b < NQ * SB; ++b) {
            mbar_init(&sm.s_full[b], 2);
            mbar_init(&sm.p_full[b], 8);
            mbar_init(&sm.p_free[b], 1);
        }
        for (int i = 0; i < kSlots / kSlotGroup; ++i) {
            mbar_init(&sm.slots_full[i], 1);
            mbar_init(&sm.slots_free[i], 1);
        }
        mbar_init(&sm.drain[0], 1);
        mbar_init(&sm.drain[1], 1);
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

    // Waits are bounded.  One that runs out sets a flag with which every later wait returns at once and which becomes the
    // call's error at the end; no warp leaves its loop.
    auto poll = [&](uint64_t *bar, int phase) { mbar_poll(bar, (uint32_t)phase & 1, &sm.abort); };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };

    if (warp < L::SOFTMAX_WARPS) {
        set_max_registers<L::REGS_SOFTMAX, L::REGS_LAUNCH>();
        // ------------------------------------------------------------------------------------------ softmax
        const int q = NQ == 2 ? warp / 8 : 0, quadrant = warp & 3, half = (warp >> 2) & 1, g = lane >> 2, t = lane & 3;
        const int row0 = 128 * q + 32 * quadrant + 16 * half + g;        // this lane's rows: row0 and row0 + 8
        const uint32_t quad = tmem + ((uint32_t)quadrant << 21), part16 = quad + ((uint32_t)(16 * half) << 16);   // lanes
        const uint32_t o_cols = L::O + q * D, q_at = part16 + L::Q + q * (D / 2);
        const uint32_t q_tile = smem_u32(sm.q) + q * L::Q_BYTES;
        auto wait = [&](uint64_t *bar, int phase) {
            poll(bar, phase);
            __syncwarp();
        };
        if (tid == 0) plan.meta[cta].last = -1;
        if (units > 0) {
            int item = plan.start[cta].item, j = plan.start[cta].j;      // the item, and its unit that is next
            // unit u's score buffer, and which use of it that is
            auto buffer = [&](int u) { return q * SB + u % SB; };
            auto use = [&](int u) { return u / SB; };
            // An item's queries, 4 lanes to a row, 16 bytes each.  Their lines are brought into L2 while the item before writes
            // its outputs.  Up to d = 128 a lane holds its pieces over both passes, which find the rows' scales and convert; at
            // d = 256 that many registers spill (8192-token prompt 592 us against 560), and the second pass reads L1.
            constexpr bool kHold = D <= 128;
            constexpr int HELD = kHold ? D / 32 : 1;
            const uint4 *src[2] = {nullptr, nullptr};
            auto ask = [&](const TcItem &it) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int gr = it.mt * ROWS + row0 + 8 * k, i = gr / group;
                    src[k] = i < it.qlen
                                 ? reinterpret_cast<const uint4 *>(p.q + ((size_t)(it.q0 + i) * p.hq + it.h * group + gr % group) * D) + t
                                 : nullptr;
                    if (src[k] && t < D / 64) prefetch_l2(src[k] + 7 * t);      // its lines, a lane each
                }
            };
            ask(plan.items[item]);
            for (int u = 0, seg = 0; u < units; ++seg) {
                // ---- a segment: units of one item
                // (few of the item's fields stay in registers over its units; at its end they are read again)
                const int u_first = u, j_first = j;
                int u_end, seen_to, hi_pos, near_tiles, far_tile;
                float rs[2];
                int pos[2];
                {
                    const TcItem it = plan.items[item];
                    u_end = min(units, u + it.tiles - j);
                    seen_to = it.lo_pos + 2 - kTile;                 // units that begin before are in no row's future
                    hi_pos = it.hi_pos;
                    near_tiles = it.near_tiles;
                    far_tile = it.far_tile;
                    float down[2];
                    uint4 raw[2][HELD];
                    auto piece = [&](int k, int c) { return src[k] ? __ldg(src[k] + 4 * c) : make_uint4(0, 0, 0, 0); };
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int c = 0; c < HELD; ++c)
                            if (kHold) raw[k][c] = piece(k, c);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        pos[k] = it.kvlen - it.qlen + (it.mt * ROWS + row0 + 8 * k) / group;
                        uint32_t big = 0;
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) big = max(big, amax_bits(kHold ? raw[k][c % HELD] : piece(k, c)));
                        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
                        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
                        float up;
                        power_of_two_scale(big, down[k], up);
                        if (p.sm_scale < 0.f) down[k] = -down[k];     // the row factor stays >= 0
                        rs[k] = up * fabsf(p.sm_scale) * 1.4426950408889634f;
                    }
#pragma unroll kHold ? D / 64 : 2
                    for (int c = 0; c < D / 64; ++c) {
                        uint32_t x[16];
#pragma unroll
                        for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint4 z = kHold ? raw[k][(2 * c + i2) % HELD] : piece(k, 2 * c + i2);
                                x[8 * i2 + 2 * k] = bf16x2_to_f16x2(z.x, down[k]);
                                x[8 * i2 + 2 * k + 1] = bf16x2_to_f16x2(z.y, down[k]);
                                x[8 * i2 + 4 + 2 * k] = bf16x2_to_f16x2(z.z, down[k]);
                                x[8 * i2 + 4 + 2 * k + 1] = bf16x2_to_f16x2(z.w, down[k]);
                            }
                        if (L::QS) {
                            // a row's 64 columns c, in their own order: pieces 4 i2 + t of 8
#pragma unroll
                            for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const uint32_t at = q_tile + c * L::Q_CHUNK + sw128_offset((row0 & 127) + 8 * k, 32 * i2 + 8 * t);
                                    store_shared<0>(at, x[8 * i2 + 2 * k], x[8 * i2 + 2 * k + 1], x[8 * i2 + 4 + 2 * k], x[8 * i2 + 4 + 2 * k + 1]);
                                }
                        } else {
                            tmem_st_16x32(q_at + 32 * c, x);
                        }
                    }
                    if (L::QS) fence_proxy_async_smem();
                    else tmem_st_wait();
                }
                if (u_end < units) prefetch_l1(plan.items + item + 1);
                tc_fence_before();
                arrive(&sm.q_full[q]);              // also: this warp has read its part of the item before
                float m[2] = {kNoReference, kNoReference}, l[2] = {0.f, 0.f};
                bool raise = true;                  // the item's first unit sets M
                for (; u < u_end; ++u, ++j) {
                    // ---- one unit
                    const int buf = buffer(u);
                    const uint32_t s_tm = part16 + L::S + 64 * buf;
                    const int tok0 = first_token(near_tiles, far_tile, j);
                    const bool all_seen = tok0 < seen_to && (p.window == 0 || tok0 > hi_pos - p.window || tok0 + kTile <= p.sinks);
                    const float *scale = sm.scale[u % kSlots];
                    wait(&sm.s_full[buf], use(u));
                    const float4 ks = *reinterpret_cast<const float4 *>(scale), lv = *reinterpret_cast<const float4 *>(scale + 4);
                    const float ksc[4] = {ks.x, ks.y, ks.z, ks.w}, lvs[4] = {lv.x, lv.y, lv.z, lv.w};
                    tc_fence_after();
                    // scores of row k at tokens 8 i + 2 t, + 1: s[4 i + 2 k], + 1
                    float s[32];
                    tmem_ld_16x64(s_tm, s);
                    if (!all_seen) {
                        // a score that the row does not see becomes -infinity
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            unsigned long long seen = low_bits(pos[k] - tok0 + 1);
                            if (p.window != 0) seen &= ~low_bits(pos[k] - min(p.window, max(pos[k], 0) + 1) - tok0 + 1) | low_bits(p.sinks - tok0);
                            seen >>= 2 * t;
#pragma unroll
                            for (int i = 0; i < 8; ++i)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (!(seen >> (8 * i + e) & 1)) s[4 * i + 2 * k + e] = -INFINITY;
                        }
                    }
                    const bool first = raise;
                    for (;;) {
                        if (raise) {
                            float top[2] = {-INFINITY, -INFINITY}, c[2];
#pragma unroll
                            for (int b = 0; b < 4; ++b)
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const float *x = s + 8 * b + 2 * k;
                                    const float y = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[4], x[5]));
                                    top[k] = fmaxf(top[k], y == -INFINITY ? y : fmaf(y, rs[k] * ksc[b], lvs[b]));
                                }
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 1));
                                top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 2));
                                const float to = fmaxf(m[k], top[k]);
                                c[k] = m[k] == to ? 1.f : exp2f(m[k] - to);
                                m[k] = to;
                                l[k] *= c[k];
                            }
                            if (!first) {
                                wait(&sm.p_free[buffer(u - 1)], use(u - 1));     // the output product of the unit before
                                tc_fence_after();
#pragma unroll 1
                                for (int k = 0; k < D / 32; ++k) {
                                    float o[16];
                                    tmem_ld_16x32(part16 + o_cols + 32 * k, o);
                                    uint32_t x[16];
#pragma unroll
                                    for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(o[e] * c[(e >> 1) & 1]);
                                    tmem_st_16x32(part16 + o_cols + 32 * k, x);
                                }
                                tmem_st_wait();
                            }
                        }
                        uint32_t x[16];      // of 8 tokens i: row 0, row 1
                        float sum[2][4];     // of row k's four blocks
                        auto weigh = [&](auto masked) {
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
#pragma unroll
                                for (int b = 0; b < 4; ++b) {
                                    const float f = rs[k] * ksc[b], off = lvs[b] - m[k];
                                    float part[2];
#pragma unroll
                                    for (int i = 0; i < 2; ++i) {
                                        const float s0 = s[8 * b + 4 * i + 2 * k], s1 = s[8 * b + 4 * i + 2 * k + 1];
                                        float e0 = s0, e1 = s1;
                                        fma2(e0, e1, f, off);
                                        e0 = exp2_fast(e0);
                                        e1 = exp2_fast(e1);
                                        if (masked.value) {     // whatever the block's scales are
                                            if (s0 == -INFINITY) e0 = 0.f;
                                            if (s1 == -INFINITY) e1 = 0.f;
                                        }
                                        if (i == 0) part[0] = e0, part[1] = e1;
                                        else add2(part[0], part[1], e0, e1);
                                        const __half2 hh = __floats2half2_rn(e0, e1);
                                        x[2 * (2 * b + i) + k] = *reinterpret_cast<const uint32_t *>(&hh);
                                    }
                                    sum[k][b] = part[0] + part[1];
                                }
                            }
                        };
                        if (all_seen) weigh(Flag<false>());
                        else weigh(Flag<true>());
                        const float4 rvv = *reinterpret_cast<const float4 *>(scale + 8);
                        float add[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) add[k] = (sum[k][0] + sum[k][1]) + (sum[k][2] + sum[k][3]);
                        // a weight above 2^15 makes its sum so too, and so does any token that a row without M sees
                        if (!raise && __any_sync(0xffffffffu, add[0] > 32768.f || add[1] > 32768.f)) {
                            raise = true;
                            continue;
                        }
                        raise = false;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (all_seen) {
                                l[k] += sum[k][0] * rvv.x + sum[k][1] * rvv.y + sum[k][2] * rvv.z + sum[k][3] * rvv.w;
                            } else {
                                if (sum[k][0] != 0.f) l[k] = fmaf(sum[k][0], rvv.x, l[k]);
                                if (sum[k][1] != 0.f) l[k] = fmaf(sum[k][1], rvv.y, l[k]);
                                if (sum[k][2] != 0.f) l[k] = fmaf(sum[k][2], rvv.z, l[k]);
                                if (sum[k][3] != 0.f) l[k] = fmaf(sum[k][3], rvv.w, l[k]);
                            }
                        }
                        tmem_st_16x32b(s_tm, x);
                        break;
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    arrive(&sm.p_full[buf]);
                }
                // ---- the segment's end.  The next item's queries are on their way while this one's outputs are written.
                int out_row[2];                     // token and head, -1: none
                bool whole;
                const bool more = u < units;
                TcItem next;
                {
                    const TcItem it = plan.items[item];
                    if (more) next = plan.items[item + 1];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int grow = it.mt * ROWS + row0 + 8 * k, i = grow / group;
                        out_row[k] = i < it.qlen ? (it.q0 + i) * p.hq + it.h * group + grow % group : -1;
                    }
                    whole = j_first == 0 && j == it.tiles;
                    if (tid == 0 && j_first == 0 && !whole)
                        plan.meta[cta] = {cta, u_first == 0 ? 0 : 1, cta + (int)(((long long)it.tiles - j + per - 1) / per), it.n, it.h, it.mt};
                }
                if (more) {
                    ++item;
                    j = 0;
                    ask(next);
                }
                float inv[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
                    l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
                    inv[k] = whole ? (l[k] == 0.f ? 0.f : 1.f / l[k]) : 1.f;
                }
                // The last output product (a barrier for all units in turn would not do here: it may be two phases behind, which
                // looks like one ahead)
                wait(&sm.p_free[buffer(u_end - 1)], use(u_end - 1));
                tc_fence_after();
                float *part = plan.parts + (size_t)(2 * cta + (u_first == 0 ? 0 : 1)) * (ROWS * D + 2 * ROWS);
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[16];            // columns c + 8 i + 2 t, + 1 of row k: o[4 i + 2 k], + 1
                    tmem_ld_16x32(part16 + o_cols + c, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] *= inv[(e >> 1) & 1];
                    // the 4 lanes of a row exchange, so that each holds 4 (8) neighbouring columns and 16 bytes leave at a time
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (whole && !p.out_f32) {
                            uint32_t y[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const __nv_bfloat162 b = __floats2bfloat162_rn(o[4 * i + 2 * k], o[4 * i + 2 * k + 1]);
                                y[i] = *reinterpret_cast<const uint32_t *>(&b);
                            }
                            transpose4(y, t);
                            if (out_row[k] >= 0)
                                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + (size_t)out_row[k] * D + c + 8 * t) = make_uint4(y[0], y[1], y[2], y[3]);
                            continue;
                        }
                        float *to = whole ? static_cast<float *>(p.out) + (size_t)max(out_row[k], 0) * D : part + (size_t)(row0 + 8 * k) * D;
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            const float *a = o + 4 * i + 2 * k, *b = a + 4;
                            const bool odd = t & 1;
                            const float r0 = __shfl_xor_sync(0xffffffffu, odd ? a[0] : b[0], 1), r1 = __shfl_xor_sync(0xffffffffu, odd ? a[1] : b[1], 1);
                            const float4 y = odd ? make_float4(r0, r1, b[0], b[1]) : make_float4(a[0], a[1], r0, r1);
                            if (out_row[k] >= 0) *reinterpret_cast<float4 *>(to + c + 8 * (i + (t & 1)) + 4 * (t >> 1)) = y;
                        }
                    }
                    __syncwarp();   // the next load is warp-wide
                }
                if (!whole && t == 0) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        part[ROWS * D + row0 + 8 * k] = m[k];
                        part[ROWS * D + ROWS + row0 + 8 * k] = l[k];
                    }
                }
                tc_fence_before();
            }
        }
    } else if (warp < L::SOFTMAX_WARPS + L::LOADER_WARPS) {
        set_max_registers<L::REGS_LOADER, L::REGS_LAUNCH>();
        // ------------------------------------------------------------------------------------------ loaders
        // At d = 256 two groups of 8 warps take the units in turn, so that two units' codes are on their way at a time: their
        // latency is longer than one unit's products (8192-token prompt 457 us against 546 with one group).  With two tiles of
        // rows the softmax warps take the registers.  The codes go through L1 (read past it: 457 against 440), because each
        // request takes half of a row's lines.
        constexpr int CH = D / 64;
        const int lg = (warp - L::SOFTMAX_WARPS) / 8, lw = (warp - L::SOFTMAX_WARPS) % 8;   // rows 8 lw .. 8 lw + 7 of every unit
        // 4 lanes take the 64 codes of a column chunk of one row.  The 8 lanes that store together hold rows that
        // differ in the two low bits, so that their pieces fall on different banks in both tiles' orders.
        const int r = 8 * lw + ((lane >> 4) << 2) + ((((lane >> 2) & 1) * 3) ^ ((lane >> 3) & 1)), c16 = lane & 3;
        const uint32_t v_lo = sw128_offset(r, 16 * c16), v_hi = sw128_offset(r, 16 * c16 + 8);
        // K's columns stand in the order in which a query row's 32-element pieces enter TMEM: components 8 t + 0..3
        // at 4 t, components 8 t + 4..7 at 16 + 4 t (t = 0..3); with queries in shared memory, in their own
        const uint32_t k_lo = L::QS ? v_lo : sw128_offset(r, 32 * (c16 >> 1) + 8 * (c16 & 1)),
                       k_hi = L::QS ? v_hi : sw128_offset(r, 32 * (c16 >> 1) + 16 + 8 * (c16 & 1));
        auto wait = [&](uint64_t *bar, int phase) {
            poll(bar, phase);
            __syncwarp();
        };
        const int in_block = r % kKvBlock;
        const unsigned pool_rows = (unsigned)(p.pool.n_pages * p.pool.hkv * p.pool.page_size);
        for (int u = lg; u < units; u += L::LG) {
            // the unit's codes are asked for; they are on their way while its place is waited for
            const int st = u % STAGES, ph = u / STAGES + 1;
            if (u % kSlotGroup < L::LG) wait(&sm.slots_full[u / kSlotGroup % (kSlots / kSlotGroup)], u / kSlots);
            const int2 block = sm.block[u % kSlots][lw / 2];
            // (a slot that the look-up gave up on holds anything: rows outside the pool are not read either)
            const bool there = in_block < block.y && (unsigned)(block.x + in_block) < pool_rows;
            const size_t at = (size_t)(there ? block.x + in_block : 0) * D + 16 * c16;
            uint4 kr[CH], vr[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) kr[c] = __ldg(reinterpret_cast<const uint4 *>(p.k_pages + at + 64 * c));
#pragma unroll
            for (int c = 0; c < CH; ++c) vr[c] = __ldg(reinterpret_cast<const uint4 *>(p.v_pages + at + 64 * c));
            wait(&sm.k_empty[st], ph);
            if (!there) {       // rows that do not exist become zeros
#pragma unroll
                for (int c = 0; c < CH; ++c) kr[c] = vr[c] = make_uint4(0, 0, 0, 0);
            }
            put_codes<D, FMT, !L::QS>(smem_u32(sm.k[st]) + k_lo, smem_u32(sm.k[st]) + k_hi, kr);
            fence_proxy_async_smem();
            arrive(&sm.k_full[st]);
            wait(&sm.v_empty[st], ph);
            put_codes<D, FMT, false>(smem_u32(sm.v[st]) + v_lo, smem_u32(sm.v[st]) + v_hi, vr);
            fence_proxy_async_smem();
            arrive(&sm.v_full[st]);
        }
    } else {
        set_max_registers<L::REGS_OTHER, L::REGS_LAUNCH>();
        const int role = warp - L::SOFTMAX_WARPS - L::LOADER_WARPS;
        // ------------------------------------------------------------------------------------------ MMA
        // Two warps, each with one thread that issues: the issue of an MMA blocks while the few before it run, so one
        // thread for both products leaves the tensor pipe idle during each of its waits.  Of the items only their ends
        // matter here: units left of this one, the next one's read ahead.
        if (role < 2 && units > 0 && elect_one()) {
            int item = plan.start[cta].item, left = plan.items[item].tiles - plan.start[cta].j, next_left = 0;
            if (left < units) next_left = plan.items[item + 1].tiles;
            int st = 0, ph = 0, seg = 0;            // of unit u: its tiles' stage
            int buf = 0, buf_phase = 0;             // its score buffer
            bool first = true;
            for (int u = 0; u < units; ++u) {
                const bool ends = left == 1;
                if (role == 0) {
                    // S = Q K^T.  A buffer is free once the output product has read the weights that took its place.
                    poll(&sm.k_full[st], ph);
                    constexpr uint32_t id = idesc_f16_f32(128, kTile, false, false);
                    const uint64_t kd = smem_desc(smem_u32(sm.k[0]), 16, 1024, kLayoutSwizzle128B) +
                                        (st * L::TILE_BYTES >> 4);
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        if (first) poll(&sm.q_full[q], seg);
                        poll(&sm.p_free[q * SB + buf], buf_phase ^ 1);
                        tc_fence_after();
                        const uint32_t d = tmem + L::S + 64 * (q * SB + buf), a = tmem + L::Q + q * (D / 2);
                        const uint64_t qd = smem_desc(smem_u32(sm.q) + q * L::Q_BYTES, 16, 1024, kLayoutSwizzle128B);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint64_t kk = kd + ((k >> 2) * L::CHUNK >> 4) + 2 * (k & 3);
                            if (L::QS) mma_f16(d, qd + ((k >> 2) * L::Q_CHUNK >> 4) + 2 * (k & 3), kk, id, k > 0);
                            else mma_tmem_a(d, a + 8 * k, kk, id, k > 0);
                        }
                        mma_commit(&sm.s_full[q * SB + buf]);
                        mbar_arrive(&sm.s_full[q * SB + buf]);   // the block scales, which this thread has waited for, are visible too
                    }
                    mma_commit(&sm.k_empty[st]);
                } else {
                    // O += W V, from 0 at an item's first unit in this run
                    poll(&sm.v_full[st], ph);
                    constexpr uint32_t id = idesc_f16_f32(128, D, false, true);
                    const uint64_t vd = smem_desc(smem_u32(sm.v[0]), L::CHUNK, 1024, kLayoutSwizzle128B) +
                                        (st * L::TILE_BYTES >> 4);
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        poll(&sm.p_full[q * SB + buf], buf_phase);
                        tc_fence_after();
                        const uint32_t a = tmem + L::S + 64 * (q * SB + buf);
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k) mma_tmem_a(tmem + L::O + q * D, a + 8 * k, vd + 128 * k, id, !(first && k == 0));
                        mma_commit(&sm.p_free[q * SB + buf]);
                    }
                    mma_commit(&sm.v_empty[st]);
                    // the softmax warps have read the slots of all units up to this one
                    if (u % kSlotGroup == kSlotGroup - 1) mbar_arrive(&sm.slots_free[u / kSlotGroup % (kSlots / kSlotGroup)]);
                }
                if (++st == STAGES) st = 0, ph ^= 1;
                if (++buf == SB) buf = 0, buf_phase ^= 1;
                first = ends;
                --left;
                if (ends) {
                    ++seg;
                    ++item;
                    left = next_left;
                    if (u + 1 + left < units) next_left = plan.items[item + 1].tiles;
                }
            }
            // every MMA has finished before the tensor memory is given back
            mma_commit(&sm.drain[role]);
            poll(&sm.drain[role], 0);
        } else if (role == 2 && units > 0) {
            // -------------------------------------------------------------------------------------- look-up
            // Eight units at a time, a lane to a block of 16 tokens: its place in the pool and its scales.
            const int b = lane & 3;
            const RunStart start = plan.start[cta];
            int item = start.item, j = start.j;
            TcItem it = plan.items[item];
            bool bad = false;                       // an entry outside the pool
            j += lane >> 2;
            for (int g = 0; g * kSlotGroup < units; ++g, j += kSlotGroup) {
                const int u = g * kSlotGroup + (lane >> 2);
                int2 block = make_int2(-1, 0);
                float ks = 0.f, vs = 0.f;
                if (u < units) {
                    while (j >= it.tiles) {
                        j -= it.tiles;
                        it = plan.items[++item];
                    }
                    const int tok = first_token(it.near_tiles, it.far_tile, j) + kKvBlock * b;
                    if (tok < it.kvlen && in_sight(it.lo_pos, it.hi_pos, tok, tok + kKvBlock, p.window, p.sinks)) {
                        const int at = p.pool.page_of(tok), entry = __ldg(p.pool.table + (size_t)it.n * p.pool.max_pages + at);
                        if ((unsigned)entry < (unsigned)p.pool.n_pages) {
                            block = make_int2((entry * p.pool.hkv + it.h) * p.pool.page_size + tok - at * p.pool.page_size, min(it.kvlen - tok, kKvBlock));
                            ks = __ldg(p.k_scales + block.x / kKvBlock);
                            vs = __ldg(p.v_scales + block.x / kKvBlock);
                        } else {
                            bad = true;
                        }
                    }
                }
                if (vs == 0.f) vs = kAmaxFloor;
                if (u >= kSlots) poll(&sm.slots_free[g % (kSlots / kSlotGroup)], g / (kSlots / kSlotGroup) - 1);
                float *scale = sm.scale[u % kSlots] + b;
                scale[0] = ks;
                scale[4] = log2f(vs);
                scale[8] = 1.f / vs;
                sm.block[u % kSlots][b] = block;
                arrive(&sm.slots_full[g % (kSlots / kSlotGroup)]);
            }
            if (bad) raise_error(p.err, kErrInternal);
        }
    }
    __syncthreads();
    if (tid == 0 && sm.abort) raise_error(p.err, kErrTimeout);
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
    const int rows = d == 256 ? Tc<256>::ROWS : Tc<128>::ROWS;
    z.items = hkv * (((long long)total * (hq / hkv) + rows - 1) / rows + n_seqs);
    z.ctas = min(sms, kMaxTcCtas);
    z.start = round256(kMaxTcCtas * sizeof(MergeMeta));
    z.per = z.start + round256((kMaxTcCtas + 1) * sizeof(RunStart));
    z.list = z.per + 256;
    z.parts = z.list + round256((size_t)z.items * sizeof(TcItem));
    z.bytes = z.parts + (size_t)2 * z.ctas * (rows * d + 2 * rows) * sizeof(float);
    return z;
}

template <int D, int FMT>
cudaError_t launch_tc(const AttendProblem &p) {
    const TcSizes z = tc_sizes(p.n_seqs, p.total, p.hq, p.pool.hkv, D, multiprocessor_count());
    uint8_t *ws = static_cast<uint8_t *>(p.workspace);
    TcPlan plan{};
    plan.meta = reinterpret_cast<MergeMeta *>(ws);
    plan.start = reinterpret_cast<RunStart *>(ws + z.start);
    plan.per = reinterpret_cast<long long *>(ws + z.per);
    plan.items = reinterpret_cast<TcItem *>(ws + z.list);
    plan.parts = reinterpret_cast<float *>(ws + z.parts);
    plan.ctas = z.ctas;
    plan.max_items = (int)min(z.items, 2147483647LL);
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
    using L = Tc<D>;
    attend_plan_kernel<L::ROWS, item_cost<D>()><<<1, kPlanThreads, 0, p.stream>>>(p, plan);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_after(p.stream, dim3((unsigned)z.ctas), Tc<D>::THREADS, smem, attend_tc_kernel<D, FMT>, p, plan)) != cudaSuccess) return e;
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
