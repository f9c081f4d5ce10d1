// 4-bit products for many rows, on tcgen05: y[m, n] = sum_i W[n, i] x[m, i] with W = scale * code + offset.
//
// The weights are the product's first operand, 128 rows of W a CTA, and up to 256 rows of x its second: D[n, m] in TMEM.  Codes come by
// TMA, 128 rows of 256 inputs a stage; 8 or 16 warps turn them into fp16 and write them into TMEM as the first operand's next 64 inputs,
// a row a thread; x lies in shared memory.  So a weight is unpacked once for all rows of x of its CTA, and never goes through
// shared memory as a number.
//
// Both operands are fp16, each row scaled by a power of two, and nothing of a weight is lost:
//     W = scale (code - 8) + (offset + 8 scale),
// of which the first part has 8 + 3 significant bits, as many as a half, and the second is the same for all inputs of a group: it
// meets the group's sum of x.  These sums and second parts are two halves each (22 bits), so that a group is four inputs more:
//     (hi, hi, lo, lo) of the second part by (hi, lo, hi, lo) of the sum,  16 groups to a block of 64 inputs.
// Without offsets the second part is zero and the blocks are not there; with them they are 1/16 or 1/32 of the work.
//   x    the row's largest magnitude goes to [2^14, 2^15).  A bf16 number keeps all its bits down to 2^-32 of that.  A first kernel
//        does this, puts each 8 inputs in the order 0 4 1 5 2 6 3 7, in which a code word's pairs come out, and adds the groups' means
//        (a sum would leave fp16; the second parts are multiplied by the group's size instead).
//   W    by the row's largest 15 |scale| + |offset| at the CTA's inputs, which goes to [2^-2, 2^-1): first parts are exact for scales down to
//        2^-15 of that, below lose 2^-22 of it at most.  A code c in bits 4 to 7 of a half is c 2^-20 (a subnormal, which the
//        arithmetic takes as any other number), so a shift, an AND and one fused product-sum with (scale 2^20, -8 scale) make two
//        weights.  Codes taken from bits 0 to 3 as well save two shifts in four pairs, but leave 2^-18 (131071 x 2048, 33 rows, with
//        caches flushed: 76 us instead of 77); codes under the exponent of 1024 leave 2^-24 (84).
// Sums are fp32, in TMEM, where an addition cuts what does not fit: with 2048 inputs 6e-4 of the bf16 outputs are not the nearest to the
// exact ones, twice as many as by sums that round.  The powers of two are undone at the end.
//
// CTAs of a cluster share the inputs of one tile and join through distributed shared memory, in a fixed order.
//
// Bound by the products for many rows (with x as second operand of N rows a product of 16 inputs takes N / 2 + 11 cycles, at least 41), by
// a CTA's beginning and end for few: launch, scales and first codes 3 us, last barrier, join and outputs 3 us.  Measured on a GB300:
// 4096 x 4096 without offsets, 33 rows 11.0 us, 128 rows 13.8, 512 rows 23.8 (720 TFLOP/s), with offsets in groups of 64 13.2, 16.1 and 29.7;
// with offsets 131071 x 2048, 33 rows 71 us, 100 rows 84 (640); gated 2 x 6000 x 2048, 509 rows, 30.5 us (820 TFLOP/s; tensor pipe 0.46 active
// over the whole time).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "layer_ops.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kRowsA = 128;               // weight rows of a CTA
constexpr int kBlockIn = 64;              // inputs that a thread unpacks at once: 32 columns of TMEM
constexpr int kChunkIn = 256;             // inputs of a stage of codes
constexpr int kCodeBytes = kRowsA * kChunkIn / 2;
constexpr int kMaxStages = 4, kMaxSlots = 4;
constexpr int kPerGroup = 4, kBlockGroups = kBlockIn / kPerGroup;      // inputs that a group's offset stands for; groups of a block of them

// A step is what one wait of the thread that issues the products is for.  Its instructions between two products, a few dozen in a
// row, take longer than a product with few columns: with one matrix a step is two blocks, which two groups of four unpacking warps
// share; of two matrices each has its group of warps, its own issuing warp, and steps of one block.  What a warp does for a step
// takes 1000 cycles, most of them waits (a barrier that is found complete 250, the store to TMEM 150).  16 warps take turns, those of
// each of the two slots theirs; 8 are enough where two CTAs are on an SM.
template <bool GATED, int WARPS>
struct Tc {
    static constexpr int MATS = GATED ? 2 : 1, BLOCKS = GATED ? 1 : 2, STEP = BLOCKS * kBlockIn;
    static constexpr int GROUPS = WARPS / 4, TURNS = WARPS / 8, PARTS = GROUPS / MATS;
    static constexpr int THREADS = 32 * (WARPS + 4);      // one warp each for TMA of codes and of x, one or two for the products
};

struct TcPlan {
    int ntok, m_tiles, row_tiles, cluster;
    int slice;                            // chunks of inputs of one CTA
    bool pair;                            // two CTAs an SM
    int slot_bits;                        // 2^slot_bits steps of weights are in TMEM
    int code_stages, x_stages, tmem_cols; // (columns: the sums, and the slots, 64 each)
};

struct TcBars {
    uint64_t code_full[kMaxStages], code_empty[kMaxStages], x_full[kMaxStages], x_empty[kMaxStages], a_full[2][kMaxSlots], a_empty[2][kMaxSlots], done;
    uint32_t tmem;
    int abort;
    float2 undo[256];                     // of each row of x: the two halves of 2^-exponent
    float tops[4][kRowsA];                // largest() of a weight row's parts
};

// 32 lanes x 32 columns of 32 bits, a lane a thread, and the wait for them.
__device__ __forceinline__ void tmem_st_row(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
                 "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n tcgen05.wait::st.sync.aligned;\n" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
                 "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
                 "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
                 "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
                 : "memory");
}

__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

__device__ __forceinline__ uint32_t f16_twice(float v) {
    const __half2 h = __float2half2_rn(v);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }      // -126 .. 127

// A wait of a whole warp in which one lane asks: 256 lanes that ask keep the shared-memory pipe from the threads that issue (a
// poll that finds its phase complete then took those 230 cycles).
__device__ __forceinline__ void warp_poll(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (threadIdx.x % 32 == 0) mbar_poll(bar, parity, abort);
    __syncwarp();
}
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}

// 16 bytes of a matrix's scales or offsets; what would lie behind the last of them is zero.
__device__ __forceinline__ uint4 eight(const __nv_bfloat16 *all, size_t at, size_t total) {
    if (at + 8 <= total) return *reinterpret_cast<const uint4 *>(all + at);
    uint32_t v[4] = {};
    for (int e = 0; at + e < total; ++e) v[e / 2] |= (uint32_t)__bfloat16_as_ushort(all[at + e]) << 16 * (e % 2);
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// Sixteen of them from `at` on, in pairs, by aligned reads: a lane's lie in a line of their own, so that every read costs a warp 32
// (759 x 7808, 122 groups, 122 rows: 17.0 us by reads of two, 15.1).  `aligned`: at is a multiple of 8 in every lane, which
// saves the shifts (131071 x 2048, 3 rows: 68.6 us with them, 65.9).
__device__ __forceinline__ void sixteen(const __nv_bfloat16 *all, size_t at, size_t total, bool aligned, uint32_t (&v)[8]) {
    if (aligned) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint4 u = at + 8 * q < total ? *reinterpret_cast<const uint4 *>(all + at + 8 * q) : make_uint4(0, 0, 0, 0);
            v[4 * q] = u.x, v[4 * q + 1] = u.y, v[4 * q + 2] = u.z, v[4 * q + 3] = u.w;
        }
        return;
    }
    const int before = at % 8;
    uint32_t w[12];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        const uint4 u = q < 2 || before ? eight(all, at - before + 8 * q, total) : make_uint4(0, 0, 0, 0);
        w[4 * q] = u.x, w[4 * q + 1] = u.y, w[4 * q + 2] = u.z, w[4 * q + 3] = u.w;
    }
#pragma unroll
    for (int i = 0; i < 10; ++i) w[i] = before & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 9; ++i) w[i] = before & 2 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = before & 1 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
}

// The largest 15/16 |scale| + 1/16 |offset| of `groups` groups (which is finite where they are), by aligned reads: eight numbers may begin before them or end behind them.
template <bool OFFSETS>
__device__ __forceinline__ float largest(const Q4Matrix &w, size_t first, int groups, size_t total) {
    float top = 0.f;
    const int before = first % 8, end = before + groups;
    for (int i = 0; i < end; i += 32) {                  // reads of four pieces are in flight together
        uint4 vs[4], vo[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const bool there = i + 8 * q < end;
            const size_t at = first - before + i + 8 * q;
            vs[q] = vo[q] = make_uint4(0, 0, 0, 0);
            if (there) vs[q] = eight(w.scales, at, total);
            if (OFFSETS && there) vo[q] = eight(w.offsets, at, total);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float fs[8], fo[8];
            unpack8(vs[q], fs);
            unpack8(vo[q], fo);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = 0.9375f * fabsf(fs[e]) + 0.0625f * fabsf(fo[e]);
                if ((unsigned)(i + 8 * q + e - before) < (unsigned)groups) top = fmaxf(top, v);
            }
        }
    }
    return top;
}

template <bool GATED, bool OFFSETS, int WARPS>
__global__ void __launch_bounds__(Tc<GATED, WARPS>::THREADS, WARPS == 8 ? 2 : 1)
q4_tc_kernel(const __grid_constant__ Q4Problem p, const __grid_constant__ TcPlan l, const __grid_constant__ CUtensorMap code_map,
             const __grid_constant__ CUtensorMap up_map, const __grid_constant__ CUtensorMap x_map, const int *x_exponents,
             unsigned int *err) {
    using T = Tc<GATED, WARPS>;
    constexpr int MATS = T::MATS;
    extern __shared__ unsigned char raw[];
    __shared__ TcBars sm;
    unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    unsigned char *codes = base, *xs = base + (size_t)l.code_stages * MATS * kCodeBytes;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int rank = l.cluster > 1 ? (int)cluster_ctarank() : 0, unit = blockIdx.x / l.cluster;
    const int row0 = unit / l.m_tiles * kRowsA, m0 = unit % l.m_tiles * l.ntok;
    const int chunk0 = rank * l.slice, k0 = chunk0 * kChunkIn;
    const int blocks = min(l.slice * (kChunkIn / kBlockIn), (p.k - k0) / kBlockIn);                          // at least one
    const int chunks = (blocks + 3) / 4;
    // groups of these inputs; the blocks of their second parts, which come first, while the codes are on their way
    const int groups = p.k / p.group, group0 = k0 / p.group, group_end = group0 + blocks * kBlockIn / p.group;
    const int extra = OFFSETS ? (group_end - group0 + kBlockGroups - 1) / kBlockGroups : 0;
    const int extra_steps = (extra + T::BLOCKS - 1) / T::BLOCKS, steps = extra_steps + (blocks + T::BLOCKS - 1) / T::BLOCKS;
    const auto blocks_of = [&](int t) { return min(T::BLOCKS, t < extra_steps ? extra - t * T::BLOCKS : blocks - (t - extra_steps) * T::BLOCKS); };
    const int x_block = l.ntok * 128;                   // bytes of a block of x
    const int last_slot = (1 << l.slot_bits) - 1;
    constexpr int SLOT_COLS = 64;                       // two blocks, of one matrix or of each of two
    const int r = tid & 127;
    const size_t row = min(row0 + r, p.n_out - 1);

    const auto load_codes = [&](int c, int s) {
        mbar_arrive_expect_tx(&sm.code_full[s], MATS * kCodeBytes);
        unsigned char *to = codes + (size_t)s * MATS * kCodeBytes;
        tma_load_2d(to, &code_map, &sm.code_full[s], (k0 + c * kChunkIn) / 2, row0);
        if (GATED) tma_load_2d(to + kCodeBytes, &up_map, &sm.code_full[s], (k0 + c * kChunkIn) / 2, row0);
    };
    const auto load_x = [&](int t, int s) {
        const int n = blocks_of(t), at = t < extra_steps ? p.k + kPerGroup * group0 + t * T::STEP : k0 + (t - extra_steps) * T::STEP;
        mbar_arrive_expect_tx(&sm.x_full[s], n * x_block);
        for (int i = 0; i < n; ++i)                     // (the map counts bytes; a CTA's first group is even)
            tma_load_2d(xs + (size_t)(s * T::BLOCKS + i) * x_block, &x_map, &sm.x_full[s], 2 * (at + i * kBlockIn), m0);
    };

    // The first loads are on their way before the scales have been looked over
    if (warp == WARPS) {
        if (elect_one()) {
            for (int i = 0; i < kMaxStages; ++i) {
                mbar_init(&sm.code_full[i], 1);
                mbar_init(&sm.code_empty[i], WARPS);
            }
            fence_mbar_init();
            for (int c = 0; c < min(l.code_stages, chunks); ++c) load_codes(c, c);
        }
    } else if (warp == WARPS + 1) {
        if (elect_one()) {
            for (int i = 0; i < kMaxStages; ++i) {
                mbar_init(&sm.x_full[i], 1);
                mbar_init(&sm.x_empty[i], MATS);
            }
            fence_mbar_init();
            grid_dependency_wait();                     // the kernel before this one scales x
            for (int t = 0; t < min(l.x_stages, steps); ++t) load_x(t, t);
        }
    } else if (warp == WARPS + 2) {
        tmem_alloc(&sm.tmem, l.tmem_cols);
        tmem_relinquish();                              // another CTA may be on this SM, which allocates as well
    } else if (warp == WARPS + 3 && elect_one()) {
        for (int i = 0; i < 2; ++i)
            for (int k = 0; k < kMaxSlots; ++k) {
                mbar_init(&sm.a_full[i][k], GATED ? 4 : 8);
                mbar_init(&sm.a_empty[i][k], 1);
            }
        mbar_init(&sm.done, MATS);
        sm.abort = 0;
        fence_mbar_init();
    }
    if (warp < WARPS) {                         // each group of warps a part of what this CTA needs of one matrix's groups
        const int each = (group_end - group0 + T::PARTS - 1) / T::PARTS;
        const int m = warp / 4 / T::PARTS, g0 = min(group0 + warp / 4 % T::PARTS * each, group_end);
        sm.tops[warp / 4][r] = largest<OFFSETS>(m ? p.up : p.w, row * groups + g0, min(each, group_end - g0), (size_t)p.n_out * groups);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int exponent[MATS];                         // of this thread's weight rows, at this CTA's inputs: W is scaled by 2^-exponent
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
        float top = sm.tops[m * T::PARTS][r];
#pragma unroll
        for (int i = 1; i < T::PARTS; ++i) top = fmaxf(top, sm.tops[m * T::PARTS + i][r]);
        // 2^e <= top < 2^(e + 1), a sixteenth, goes to [2^-6, 2^-5); nothing, or what is not finite, stays
        const int e = (int)(__float_as_uint(top) >> 23) - 127;
        exponent[m] = top > 0.f && e < 128 ? e + 6 : 0;
    }
    const uint32_t tmem = sm.tmem, a_cols = tmem + MATS * l.ntok;
    volatile int *abort = &sm.abort;

    if (warp == WARPS) {
        if (elect_one()) {
            int s = 0, phase = 0;
            for (int c = l.code_stages; c < chunks; ++c) {
                mbar_poll(&sm.code_empty[s], phase, abort);
                if (*abort) break;
                load_codes(c, s);
                if (++s == l.code_stages) s = 0, phase ^= 1;
            }
        }
    } else if (warp == WARPS + 1) {
        if (elect_one()) {
            int s = 0, phase = 0;
            for (int t = l.x_stages; t < steps; ++t) {
                mbar_poll(&sm.x_empty[s], phase, abort);
                if (*abort) break;
                load_x(t, s);
                if (++s == l.x_stages) s = 0, phase ^= 1;
            }
        }
    } else if (warp > WARPS) {
        const int which = warp - WARPS - 2;
        if (which < MATS && elect_one()) {
            const uint32_t id = idesc_f16_f32(kRowsA, l.ntok, false, false), d = tmem + which * l.ntok, a = a_cols + 32 * which;
            const uint64_t first = smem_desc(smem_u32(xs), 16, 1024, kLayoutSwizzle128B);
            int s = 0, phase = 0;
            uint64_t xd = first;
            bool x_here = false, a_here = false;    // asked for a step ahead: the answer takes 200 cycles
            for (int t = 0; t < steps; ++t) {
                const int slot = t & last_slot;
                if (!x_here) mbar_poll(&sm.x_full[s], phase, abort);
                if (!a_here) mbar_poll(&sm.a_full[which][slot], (t >> l.slot_bits) & 1, abort);
                if (*abort) break;
                tc_fence_after();
                const int next = s + 1 == l.x_stages ? 0 : s + 1;
                if (t + 1 < steps) {
                    x_here = mbar_test_wait(&sm.x_full[next], next ? phase : phase ^ 1);
                    a_here = mbar_test_wait(&sm.a_full[which][(t + 1) & last_slot], ((t + 1) >> l.slot_bits) & 1);
                }
                const uint32_t as = a + SLOT_COLS * slot;
                if (t == 0) mma_tmem_a(d, as, xd, id, 0);
                else mma_tmem_a(d, as, xd, id, 1);
#pragma unroll
                for (int i = 1; i < 4; ++i) mma_tmem_a(d, as + 8 * i, xd + 2 * i, id, 1);
                if (T::BLOCKS == 2 && blocks_of(t) == 2) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma_tmem_a(d, as + 32 + 8 * i, xd + (x_block >> 4) + 2 * i, id, 1);
                }
                mma_commit(&sm.a_empty[which][slot]);
                mma_commit(&sm.x_empty[s]);
                xd += T::BLOCKS * (x_block >> 4);
                if ((s = next) == 0) phase ^= 1, xd = first;
            }
            mma_commit(&sm.done);
        }
    } else {
        // Unpacking: two groups of four warps take a step's two blocks, or each one of the two matrices
        const int half = warp / 4 % 2, turn = warp / 8, mine = GATED ? half : 0, f = exponent[mine];
        const int count = kChunkIn / p.group;
        const bool vector = groups % count == 0;
        const uint32_t to = a_cols + ((uint32_t)(warp % 4) << 21) + 32 * half;        // this warp's lanes of TMEM
        const Q4Matrix &w = mine ? p.up : p.w;
        const float f0 = power_of_two(-f / 2), f1 = power_of_two(-f - -f / 2);
        bool gone = false;
        // Weights of a step go to its slot once the products have read what was there
        const auto give = [&](int t, const uint32_t (&v)[32]) {
            const int slot = t & last_slot;
            if (t > last_slot) {
                warp_poll(&sm.a_empty[mine][slot], ((t >> l.slot_bits) - 1) & 1, abort);
                tc_fence_after();
            }
            if (gone = __any_sync(0xffffffffu, *abort)) return;
            tmem_st_row(to + SLOT_COLS * slot, v);         // (a block beyond the last is not multiplied)
            tc_fence_before();
            warp_arrive(&sm.a_full[mine][slot]);
        };
        int wanted = 0;                         // of a chunk's scales, for this warp's blocks
#pragma unroll
        for (int i = 0; i < 4 / T::BLOCKS; ++i)
            if (T::TURNS == 1 || (extra_steps + i) % 2 == turn) wanted |= 1 << (T::BLOCKS * i + (GATED ? 0 : half)) * count / 4;
        ChunkScales next = chunk_scales<OFFSETS>(w, row, groups, chunk0 * count, count, vector, wanted);
        if constexpr (OFFSETS) {
            for (int t = T::TURNS > 1 ? turn : 0; t < extra_steps && !gone; t += T::TURNS) {
                const int first = group0 + (T::BLOCKS * t + (GATED ? 0 : half)) * kBlockGroups;
                uint32_t scales[kBlockGroups / 2], offsets[kBlockGroups / 2];
                const bool aligned = groups % 8 == 0 && group0 % 8 == 0;
                sixteen(w.scales, row * groups + first, (size_t)p.n_out * groups, aligned, scales);
                sixteen(w.offsets, row * groups + first, (size_t)p.n_out * groups, aligned, offsets);
                uint32_t v[32];
#pragma unroll
                for (int q = 0; q < kBlockGroups; ++q) {
                    const bool there = first + q < group_end;
                    const float sc = (q % 2 ? bf16_hi(scales[q / 2]) : bf16_lo(scales[q / 2])) * f0 * f1;
                    const float of = (q % 2 ? bf16_hi(offsets[q / 2]) : bf16_lo(offsets[q / 2])) * f0 * f1;
                    const float both = there ? fmaf(8.f, sc, of) * (float)p.group : 0.f, hi = __half2float(__float2half_rn(both));
                    v[2 * q] = f16_twice(hi);
                    v[2 * q + 1] = f16_twice(both - hi);
                }
                give(t, v);
            }
        }
        int s = 0, phase = 0;
        for (int c = 0; c < chunks && !gone; ++c) {
            const ChunkScales cur = next;
            if (c + 1 < chunks) next = chunk_scales<OFFSETS>(w, row, groups, (chunk0 + c + 1) * count, count, vector, wanted);
            warp_poll(&sm.code_full[s], phase, abort);
            const unsigned char *line = codes + (size_t)(s * MATS + mine) * kCodeBytes + r * 128;
#pragma unroll
            for (int i = 0; i < 4 / T::BLOCKS; ++i) {
                const int t = extra_steps + 4 / T::BLOCKS * c + i, j = T::BLOCKS * i + (GATED ? 0 : half);
                if (T::TURNS > 1 && t % 2 != turn) continue;
                if (t >= steps) break;
                uint32_t v[32];
                {
                    const float sc = nth_bf16(cur.s, count == 4 ? j : j / 2) * f0 * f1;
                    const uint32_t s0 = f16_twice(sc * 1048576.f), o2 = f16_twice(-8.f * sc);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 q = *reinterpret_cast<const uint4 *>(line + (((2 * j + h) ^ (r & 7)) << 4));
                        const uint32_t words[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t a = words[e];
                            constexpr uint32_t CODES = 0x00f000f0u;
                            v[16 * h + 4 * e] = fma_f16x2(a << 4 & CODES, s0, o2);
                            v[16 * h + 4 * e + 1] = fma_f16x2(a & CODES, s0, o2);
                            v[16 * h + 4 * e + 2] = fma_f16x2(a >> 4 & CODES, s0, o2);
                            v[16 * h + 4 * e + 3] = fma_f16x2(a >> 8 & CODES, s0, o2);
                        }
                    }
                }
                give(t, v);
                if (gone) break;
            }
            if (!gone) warp_arrive(&sm.code_empty[s]);
            if (++s == l.code_stages) s = 0, phase ^= 1;
        }
        grid_dependency_wait();
        for (int m = tid; m < l.ntok; m += 32 * WARPS) {
            // (the kernel before this one writes them while this one runs: no read-only load, none that may move before the wait)
            const int e = m0 + m < p.rows ? -*const_cast<const volatile int *>(x_exponents + m0 + m) : 0;
            sm.undo[m] = make_float2(power_of_two(e / 2), power_of_two(e - e / 2));
        }
        asm volatile("barrier.sync 1, %0;" ::"n"(32 * WARPS) : "memory");
        warp_poll(&sm.done, 0, abort);
        tc_fence_after();
    }

    // Outputs.  Groups of four warps take eight columns (rows of x) in turn
    __syncwarp();
    const bool good = !__any_sync(0xffffffffu, *abort);
    const int n = row0 + r, m_end = min(l.ntok, p.rows - m0);
    const uint32_t lanes = (uint32_t)(warp % 4) << 21;
    const float2 undo0 = make_float2(power_of_two(exponent[0] / 2), power_of_two(exponent[0] - exponent[0] / 2));
    const int e1 = exponent[MATS - 1];
    const float2 undo1 = make_float2(power_of_two(e1 / 2), power_of_two(e1 - e1 / 2));
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + (size_t)m0 * p.n_out + n;
    // the halves of a power have its sign, so that nothing overflows in between that does not in the end
    const auto undone = [&](int m, float v, const float2 &of_row) {
        const float2 u = sm.undo[m];
        return v * (of_row.x * u.x) * (of_row.y * u.y);
    };
    const auto write = [&](int m, float y, float z) {
        if constexpr (GATED) y = ffn_act_fast(y, p.gelu) * z;
        if (n < p.n_out) out[(size_t)m * p.n_out] = __float2bfloat16_rn(y);
    };
    float *part = reinterpret_cast<float *>(base);            // [matrix][column][row]: the pipeline is done with this memory
    if (warp < WARPS && good) {
        for (int col = 8 * (warp / 4); col < l.ntok; col += 8 * T::GROUPS) {
            float y[8], z[8];
            tmem_ld8x2(tmem + col + lanes, tmem + (MATS - 1) * l.ntok + col + lanes, y, z);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int m = col + i;
                if (m >= m_end) continue;
                const float v = undone(m, y[i], undo0), w = GATED ? undone(m, z[i], undo1) : 0.f;
                if (l.cluster > 1) {
                    part[m * kRowsA + r] = v;
                    if (GATED) part[(l.ntok + m) * kRowsA + r] = w;
                } else {
                    write(m, v, w);
                }
            }
        }
    }
    if (l.cluster > 1) {
        cluster_sync();
        if (warp < WARPS && good) {
            for (int col = T::GROUPS * rank + warp / 4; col < m_end; col += T::GROUPS * l.cluster) {
                float ys[8] = {}, zs[8] = {}, y = 0.f, z = 0.f;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    if (q >= l.cluster) continue;
                    ys[q] = ld_dsmem_f32(part + col * kRowsA + r, q);
                    if (GATED) zs[q] = ld_dsmem_f32(part + (l.ntok + col) * kRowsA + r, q);
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) y += ys[q], z += zs[q];
                write(col, y, z);
            }
        }
        cluster_sync();                            // a CTA's sums are read before it is gone
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && sm.abort) raise_error(err, kErrTimeout);
    if (warp == WARPS + 2) tmem_dealloc(tmem, l.tmem_cols);
}

// Rows of x in fp16, scaled by 2^exponent, each 8 inputs in the order 0 4 1 5 2 6 3 7, and, where `means` is set, behind them two halves
// twice for the mean of every group.  A CTA a row: its 256 threads hold 8192 inputs; of longer rows they read the rest again.
constexpr int kScaleThreads = 256, kHeld = 4;
__global__ void __launch_bounds__(kScaleThreads) scale_rows_kernel(const __grid_constant__ Q4Problem p, __half *__restrict__ out, int pitch, bool means,
                                                                   int *__restrict__ exponents) {
    __shared__ uint32_t tops[kScaleThreads / 32];
    grid_launch_dependents();
    const int m = blockIdx.x, tid = threadIdx.x, n = p.k / 8;
    const uint4 *x = reinterpret_cast<const uint4 *>(p.x + (long long)m * p.x_stride);
    uint4 held[kHeld];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        held[i] = make_uint4(0, 0, 0, 0);
        if (tid + kScaleThreads * i < n) held[i] = x[tid + kScaleThreads * i];
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) top = max(top, amax_bits(held[i]));
    for (int i = tid + kScaleThreads * kHeld; i < n; i += kScaleThreads) top = max(top, amax_bits(x[i]));
    top = __reduce_max_sync(0xffffffffu, top);
    if (tid % 32 == 0) tops[tid / 32] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kScaleThreads / 32; ++i) top = max(top, tops[i]);
    // the largest goes to [2^14, 2^15); a row of zeros, or with what is not finite, stays as it is
    const int e = (int)(top >> 23) - 127, s = top != 0 && e < 128 ? 14 - e : 0;
    const float f0 = power_of_two(s / 2), f1 = power_of_two(s - s / 2);
    if (tid == 0) exponents[m] = s;
    uint4 *to = reinterpret_cast<uint4 *>(out + (size_t)m * pitch);
    uint2 *mean_to = reinterpret_cast<uint2 *>(out + (size_t)m * pitch + p.k);
    const int lanes = p.group / 8;                       // that have a group's inputs: 8 or 16, neighbours
    const auto write = [&](int i, const uint4 &v) {      // (a whole warp, whose threads beyond the row have zeros)
        float f[8];
        unpack8(v, f);
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = f[k] * f0 * f1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __half2 v = __floats2half2_rn(f[k], f[k + 4]);
            h[k] = *reinterpret_cast<const uint32_t *>(&v);
        }
        if (i < n) to[i] = make_uint4(h[0], h[1], h[2], h[3]);
        if (!means) return;
        float sum = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
        for (int o = 1; o < lanes; o *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        sum *= lanes == 8 ? 1.f / 64 : 1.f / 128;
        const __half hi = __float2half_rn(sum);
        const __half2 both = __halves2half2(hi, __float2half_rn(sum - __half2float(hi)));
        const uint32_t w = *reinterpret_cast<const uint32_t *>(&both);
        if (i < n && i % lanes == 0) mean_to[i / lanes] = make_uint2(w, w);
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) write(tid + kScaleThreads * i, held[i]);
    for (int first = kScaleThreads * kHeld; first < n; first += kScaleThreads)
        write(first + tid, first + tid < n ? x[first + tid] : make_uint4(0, 0, 0, 0));
}

int round_up(int a, int b) { return (a + b - 1) / b * b; }

size_t tc_shared(const TcPlan &l, int mats) {
    const size_t pipeline = (size_t)l.code_stages * mats * kCodeBytes + (size_t)l.x_stages * (mats == 2 ? 1 : 2) * l.ntok * 128;
    return 1024 + pipeline;
}

constexpr size_t kTcShared = 227 * 1024 - sizeof(TcBars) - 64, kTcSharedOfTwo = 112 * 1024 - sizeof(TcBars) - 64;

// Stages of codes and x for this much shared memory, as many as there is room for; false: not even two of each.
bool fit_stages(TcPlan &l, int mats, size_t room) {
    l.code_stages = mats == 2 ? 3 : 4;
    l.x_stages = kMaxStages;
    while (tc_shared(l, mats) > room && l.x_stages > 2) --l.x_stages;
    while (tc_shared(l, mats) > room && l.code_stages > 2) --l.code_stages;
    return tc_shared(l, mats) <= room;
}

// Clusters of 2, 4 or 8 CTAs with an SM each that are on the GPU at once.  They lie within the GPU's processing clusters of SMs, some of
// whose SMs are left over: those of 8 do not fit 19 times (759 x 7808, 122 rows, 26.1 us with 18 of them, 15.1 with fewer).
int clusters_at_once(int size) {
    static std::atomic<int> known[kMaxDevices][9];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    if (dev < kMaxDevices && (n = known[dev][size].load(std::memory_order_relaxed)) > 0) return n;
    const auto fn = q4_tc_kernel<false, false, 16>;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(Tc<false, 16>::THREADS);
    cfg.dynamicSmemBytes = kTcShared;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcShared) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = max(1, multiprocessor_count() / size - 3);
    }
    if (dev < kMaxDevices) known[dev][size].store(n, std::memory_order_relaxed);
    return n;
}

// The division that should be done first: waves of CTAs times a CTA's blocks, each as long as the product's or the unpacking's
// part of it takes (cycles), and what a CTA takes besides.  Two CTAs on an SM take 1.35 times as long as one (97 to 71 us for 131071 x
// 2048 and 33 rows of x), or as long as both their products.
//
// CTAs of a cluster, and those that need more than half of TMEM, have an SM's shared memory for themselves: no CTA of a cluster
// ever waits for columns of TMEM that are held by a CTA which in turn waits for another of that cluster.
TcPlan plan_tc(int rows, int n_out, int k, int group, bool offsets, bool gated) {
    const int mats = gated ? 2 : 1, most = gated ? 192 : 256, sms = multiprocessor_count();
    const int chunks = (k + kChunkIn - 1) / kChunkIn, fewest = (rows + most - 1) / most;
    TcPlan best{};
    double least = 1e300;
    for (int tiles = fewest; tiles <= (rows + 15) / 16 && tiles <= fewest + 4; ++tiles) {
        for (int cluster = 1; cluster <= 8 && cluster <= chunks; cluster *= 2) {
            TcPlan l{};
            l.ntok = round_up((rows + tiles - 1) / tiles, 16);
            l.m_tiles = (rows + l.ntok - 1) / l.ntok;
            l.row_tiles = (n_out + kRowsA - 1) / kRowsA;
            l.cluster = cluster;
            l.slice = (chunks + cluster - 1) / cluster;
            if ((long)l.slice * (cluster - 1) >= chunks) continue;            // every CTA has inputs
            if (cluster > 1 && 1024 + (size_t)mats * l.ntok * kRowsA * 4 > kTcShared) continue;       // (what they join)
            const auto columns = [&](int bits) {
                int c = 32;
                while (c < mats * l.ntok + (64 << bits)) c *= 2;
                return c;
            };
            l.slot_bits = 1;
            l.tmem_cols = columns(1);
            const double ctas = (double)l.row_tiles * l.m_tiles * cluster;
            l.pair = cluster == 1 && ctas > sms && l.tmem_cols <= 256 && fit_stages(l, mats, kTcSharedOfTwo);
            if (!l.pair && !fit_stages(l, mats, kTcShared)) continue;
            if (!l.pair && columns(2) <= 512) l.slot_bits = 2, l.tmem_cols = columns(2);
            const int blocks = 4 * l.slice + (offsets ? (l.slice * kChunkIn / group + kBlockGroups - 1) / kBlockGroups : 0);
            const double products = blocks * mats * (2.0 * l.ntok + 44), rest = 9000 + 30.0 * l.ntok * mats + (cluster > 1 ? 2000 : 0);
            const double one = max(products, blocks * mats * 250.0) + rest;
            const double time = l.pair ? ceil(ctas / (2 * sms)) * max(1.35 * one, 2 * products + rest)
                                       : ceil(ctas / (cluster > 1 ? cluster * clusters_at_once(cluster) : sms)) * one;
            if (time < least) least = time, best = l;
        }
    }
    return best;
}

template <bool GATED, bool OFFSETS, int WARPS>
cudaError_t launch_tc(const Q4Problem &p, const TcPlan &l, const CUtensorMap &codes, const CUtensorMap &up, const CUtensorMap &x,
                      const int *exponents) {
    const auto fn = q4_tc_kernel<GATED, OFFSETS, WARPS>;
    const size_t smem = l.pair ? tc_shared(l, GATED ? 2 : 1) : kTcShared;
    static std::atomic<bool> ready[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcShared);
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) ready[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long)l.row_tiles * l.m_tiles * l.cluster));
    cfg.blockDim = dim3(Tc<GATED, WARPS>::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = p.stream;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = l.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = l.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fn, p, l, codes, up, x, exponents, error_word());
}

size_t exponent_bytes(int rows) { return ((size_t)rows * 4 + 255) / 256 * 256; }

}  // namespace

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        cudaDriverEntryPointQueryResult q;
        void *f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        return nullptr;
    }();
    return fn;
}

bool box_map(CUtensorMap *m, const void *at, uint64_t rows, uint64_t row_bytes, uint64_t pitch, uint32_t box_bytes, uint32_t box_rows,
             bool swizzled) {
    const auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {row_bytes, rows}, strides[1] = {pitch};
    const cuuint32_t box[2] = {box_bytes, box_rows}, es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(at), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool byte_map(CUtensorMap *m, const void *at, uint64_t rows, uint64_t row_bytes, uint64_t pitch, uint32_t box_rows) {
    return box_map(m, at, rows, row_bytes, pitch, 128, box_rows, true);
}

// A row of x as halves, with its groups' means.
static int row_pitch(int k, int group) { return k + (kPerGroup * (k / group) + 7) / 8 * 8; }

size_t q4_tc_workspace_bytes(int rows, int k, int group) { return exponent_bytes(rows) + (size_t)rows * row_pitch(k, group) * 2; }

cudaError_t launch_q4_tc(const Q4Problem &p) {
    int *exponents = static_cast<int *>(p.workspace);
    __half *x16 = reinterpret_cast<__half *>(static_cast<uint8_t *>(p.workspace) + exponent_bytes(p.rows));
    const bool offsets = p.w.offsets != nullptr;
    const int pitch = row_pitch(p.k, p.group), used = offsets ? p.k + kPerGroup * (p.k / p.group) : p.k;
    const TcPlan l = plan_tc(p.rows, p.n_out, p.k, p.group, offsets, p.gated);
    CUtensorMap codes, up, x;
    if (!byte_map(&codes, p.w.codes, p.n_out, p.k / 2, p.k / 2, kRowsA) || !byte_map(&x, x16, p.rows, 2 * (uint64_t)used, 2 * (uint64_t)pitch, l.ntok))
        return cudaErrorInvalidValue;
    if (!p.gated) up = codes;
    else if (!byte_map(&up, p.up.codes, p.n_out, p.k / 2, p.k / 2, kRowsA)) return cudaErrorInvalidValue;
    scale_rows_kernel<<<(unsigned)p.rows, kScaleThreads, 0, p.stream>>>(p, x16, pitch, offsets, exponents);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    using Fn = cudaError_t (*)(const Q4Problem &, const TcPlan &, const CUtensorMap &, const CUtensorMap &, const CUtensorMap &, const int *);
    static const Fn fns[2][2][2] = {{{launch_tc<false, false, 16>, launch_tc<false, false, 8>}, {launch_tc<false, true, 16>, launch_tc<false, true, 8>}},
                                    {{launch_tc<true, false, 16>, launch_tc<true, false, 8>}, {launch_tc<true, true, 16>, launch_tc<true, true, 8>}}};
    return fns[p.gated][offsets][l.pair](p, l, codes, up, x, exponents);
}

}  // namespace gdn
