// gdn_attend for few query rows per key/value head (decode, drafted tokens): split over the cache.
//
// With query row r at position p_r, codes k_j, v_j and the scales K_b, V_b of token j's block b,
//     s_j = (q.k_j) K_b sm_scale,   o = sum_j e^{s_j} V_b v_j / sum_j e^{s_j}    over the tokens that p_r sees.
// V_b is folded into the exponent, x_j = (s_j log2 e) + log2 V_b: the weights w_j = 2^{x_j - M} multiply bare
// codes, are at most 1 for a running maximum M of x (so they fit fp16 whatever the scales are), and
// sum_j e^{s_j} = 2^M sum_b (1 / V_b) sum_{j in b} w_j.
//
// Work.  A unit is 64 tokens of one item, an item is (sequence, key/value head, 16 query rows: the group's heads
// of consecutive tokens).  All units of the call form one line; CTA c of G takes units [c per, (c + 1) per), so
// ragged batches balance by themselves and one long sequence spreads over the whole GPU.  Lengths are read on
// the device, so a captured graph follows them.  A CTA writes finished items to `out`; of an item that crosses
// CTAs each writes (O, M, l) to the workspace and attend_merge_kernel joins them.
//
// A CTA has a producer warp and four compute warps.  The producer looks pages up a unit ahead and brings K and V
// rows (codes) and block scales through a ring of shared-memory stages with cp.async.  Of a unit, compute warp w
// forms the 16 x 16 scores of tokens 16 w .. 16 w + 15 (one scale block) with mma.m16n8k16 on codes turned to
// fp16 exactly; the warps exchange row maxima and weights through shared memory; warp w then accumulates columns
// [w D/4, (w + 1) D/4) of O over all 64 tokens.  Splitting O by columns keeps it at D/8 registers a thread.
// Bound by memory: the codes are read once for all heads of a group.
#include "attend.cuh"

namespace gdn {
namespace {

using namespace attend;

constexpr int kRows = 16;        // query rows of an item
constexpr int kTile = 64;        // tokens of a unit
constexpr int kCompute = 128;    // threads of the compute warps
constexpr int kThreads = kCompute + 32;

template <int D>
__host__ __device__ constexpr int stages() { return D == 256 ? 3 : D == 128 ? 4 : 6; }
template <int D>
__host__ __device__ constexpr int ctas_per_sm() { return D == 256 ? 2 : D == 128 ? 3 : 4; }

template <int D>
struct __align__(128) Smem {
    uint8_t k[stages<D>()][kTile * D];
    uint8_t v[stages<D>()][kTile * D];
    __half p[kRows * kTile];               // weights, 16-byte pieces swizzled by row
    float scale[stages<D>()][8];           // K scales of the unit's four blocks, then V scales
    float red[4][kRows];                   // row maxima (then sums) of the four warps
    uint64_t full[stages<D>()], empty[stages<D>()];
    int abort;
    long long scan[4];
    int start_seq;
    long long start_off;
};

// Byte offset of 16-byte piece u of row r in a stage.  The piece index is permuted by the row so that the two
// access patterns (scores: 8 lanes read 4 pieces of 2 neighbouring rows; outputs: 16 lanes read 2 pieces of 4
// even, or 4 odd, rows) touch each bank once.
template <int D>
__device__ __forceinline__ uint32_t piece(int r, int u) {
    if (D == 64) return (uint32_t)((r >> 1) * 128 + ((((r & 1) << 2) | (u ^ ((r >> 1) & 3))) << 4));
    const int f = (((r >> 1) & 3) << 1) ^ ((r & 1) << 2);
    return (uint32_t)(r * D + ((u ^ f) << 4));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Arrive on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sm100::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// The compute warps' barrier.  None of them leaves the unit loop early (a wait that runs out only sets a flag).
__device__ __forceinline__ void sync_compute() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kCompute) : "memory"); }

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Fragments of V for one 8-token half of a k-step: rows r and r + 1 of the stage, the columns 8 (or 4, 2)
// * g .. of warp w's quarter.  b[i] = (code at row r, code at row r + 1) of column i as an fp16 pair.
template <int D, int FMT>
__device__ __forceinline__ void value_columns(uint32_t base, int r, int w, int g, uint32_t (&b)[D / 32]) {
    const int col = w * (D / 4) + g * (D / 32);   // first column byte
    const uint32_t a0 = base + piece<D>(r, col >> 4) + (col & 15), a1 = base + piece<D>(r + 1, col >> 4) + (col & 15);
    if constexpr (D == 64) {
        uint16_t x, y;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(a0) : "memory");
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(y) : "r"(a1) : "memory");
        codes_to_f16x2<FMT>(__byte_perm(x, y, 0x5140), b[0], b[1]);
    } else {
        uint32_t x[D / 128], y[D / 128];
        if constexpr (D == 128) {
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x[0]) : "r"(a0) : "memory");
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(y[0]) : "r"(a1) : "memory");
        } else {
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(a0) : "memory");
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(y[0]), "=r"(y[1]) : "r"(a1) : "memory");
        }
#pragma unroll
        for (int i = 0; i < D / 128; ++i) {
            codes_to_f16x2<FMT>(__byte_perm(x[i], y[i], 0x5140), b[4 * i], b[4 * i + 1]);
            codes_to_f16x2<FMT>(__byte_perm(x[i], y[i], 0x7362), b[4 * i + 2], b[4 * i + 3]);
        }
    }
}

// Where a unit line is read: the item (n, h, mt), its tile j of `tiles`, and the sequence's lengths.
struct Cursor {
    int n, h, mt, j;
    Sequence s;
    Item it;
};

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<D>()) attend_split_kernel(const __grid_constant__ AttendProblem p,
                                                                                  const __grid_constant__ SplitPlan plan) {
    constexpr int S = stages<D>(), KI = D / 64, NT = D / 32;
    extern __shared__ __align__(128) uint8_t raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int group = p.hq / p.pool.hkv, cta = blockIdx.x;
    sm100::grid_launch_dependents();

    // ---- this CTA's units: a scan over the sequences' costs
    if (tid == kCompute) {
        for (int i = 0; i < S; ++i) {
            sm100::mbar_init(&sm.full[i], 32);
            sm100::mbar_init(&sm.empty[i], 4);
        }
        sm.abort = 0;
        sm100::fence_mbar_init();
    }
    const int chunk = (p.n_seqs + kCompute - 1) / kCompute;
    const int s_lo = tid < kCompute ? min(tid * chunk, p.n_seqs) : p.n_seqs, s_hi = min(s_lo + chunk, p.n_seqs);
    long long mine = 0;
    for (int n = s_lo; n < s_hi; ++n) mine += sequence_cost<kRows, kTile>(p, load_sequence(p, n), group);
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    if (lane == 31 && warp < 4) sm.scan[warp] = upto;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < warp) upto += sm.scan[w];
        total += sm.scan[w];
    }
    const long long per = max((total + gridDim.x - 1) / gridDim.x, (long long)plan.min_units);
    const long long start = cta * per, stop = min(total, start + per);
    if (tid == 0 && !plan.meta_by_item) plan.meta[cta].last = -1;
    if (tid == 0) report_lengths(p, cta);
    if (start >= stop) return;
    if (start >= upto - mine && start < upto) {
        long long off = start - (upto - mine);
        for (int n = s_lo; n < s_hi; ++n) {
            const long long c = sequence_cost<kRows, kTile>(p, load_sequence(p, n), group);
            if (off < c) {
                sm.start_seq = n;
                sm.start_off = off;
                break;
            }
            off -= c;
        }
    }
    __syncthreads();

    Cursor cc;   // the unit being computed
    cc.n = sm.start_seq;
    cc.s = load_sequence(p, cc.n);
    {
        const int mts = row_tiles<kRows>(cc.s.qlen, group);
        long long off = sm.start_off;
        const long long head_cost = sequence_cost<kRows, kTile>(p, cc.s, group) / p.pool.hkv;
        cc.h = (int)(off / head_cost);
        off -= cc.h * head_cost;
        for (cc.mt = 0; cc.mt < mts; ++cc.mt) {
            cc.it = make_item<kRows, kTile>(p, cc.s, group, cc.mt);
            if (off < cc.it.tiles) break;
            off -= cc.it.tiles;
        }
        cc.j = (int)off;
    }
    auto advance = [&](Cursor &c) {
        if (++c.j < c.it.tiles) return;
        c.j = 0;
        if (++c.mt >= row_tiles<kRows>(c.s.qlen, group)) {
            c.mt = 0;
            if (++c.h == p.pool.hkv) {
                c.h = 0;
                do {
                    if (++c.n == p.n_seqs) return;   // past the last unit
                    c.s = load_sequence(p, c.n);
                } while (c.s.qlen == 0);
            }
        }
        c.it = make_item<kRows, kTile>(p, c.s, group, c.mt);
    };
    // A bounded wait; when it runs out the error is recorded and every later wait returns at once.
    volatile int *abort = &sm.abort;
    auto wait = [&](uint64_t *bar, int phase) {
        if (sm100::mbar_try_wait(bar, (uint32_t)phase & 1)) return;
        const uint64_t t0 = sm100::global_timer_ns();
        while (!sm100::mbar_try_wait(bar, (uint32_t)phase & 1)) {
            if (*abort) return;
            if (sm100::global_timer_ns() - t0 > sm100::kWaitTimeoutNs) {
                *abort = 1;
                raise_error(p.err, kErrTimeout);
                return;
            }
        }
    };
    const int units = (int)(stop - start);

    if (warp == 4) {
        // ---- the producer: lane b (mod 4) holds the pool row where block b of a unit begins, -1 for none
        auto look_up = [&]() -> int {
            const int tok = cc.it.token(cc.j, kTile) + (lane & 3) * kKvBlock;
            if (tok >= cc.s.kvlen) return -1;
            const int at = p.pool.page_of(tok), page = __ldg(p.pool.table + (size_t)cc.n * p.pool.max_pages + at);
            if ((unsigned)page < (unsigned)p.pool.n_pages) return (page * p.pool.hkv + cc.h) * p.pool.page_size + tok - at * p.pool.page_size;
            raise_error(p.err, kErrInternal);
            return -1;
        };
        constexpr int UPR = D / 16, RPI = 32 / UPR;      // pieces a row, rows a warp-wide copy
        const int u = lane % UPR, r0 = lane / UPR;
        int row = look_up(), kept = cc.s.kvlen - cc.it.token(cc.j, kTile);   // tokens of the unit that exist
        int stage = 0, phase = 1;
        for (int unit = 0; unit < units; ++unit) {
            int next_row = -1, next_kept = 0;
            if (unit + 1 < units) {
                advance(cc);
                next_row = look_up();
                next_kept = cc.s.kvlen - cc.it.token(cc.j, kTile);
            }
            wait(&sm.empty[stage], phase);
            if (*abort) break;
            if (lane < 8) {
                const float *sc = lane < 4 ? p.k_scales : p.v_scales;
                cp_async4(sm100::smem_u32(&sm.scale[stage][lane]), row >= 0 ? sc + row / kKvBlock : sc, row >= 0 ? 4 : 0);
            }
            const uint32_t ks = sm100::smem_u32(sm.k[stage]), vs = sm100::smem_u32(sm.v[stage]);
#pragma unroll
            for (int b = 0; b < kTile / kKvBlock; ++b) {
                const int base = __shfl_sync(0xffffffffu, row, b);
                const size_t off = base >= 0 ? (size_t)base * D + r0 * D + u * 16 : 0;
#pragma unroll
                for (int i = 0; i < kKvBlock / RPI; ++i) {
                    const int r = b * kKvBlock + i * RPI + r0;
                    const int bytes = base >= 0 && r < kept ? 16 : 0;        // rows that do not exist become zeros
                    const size_t at = bytes ? off + i * RPI * D : 0;
                    cp_async16(ks + piece<D>(r, u), p.k_pages + at, bytes);
                    cp_async16(vs + piece<D>(r, u), p.v_pages + at, bytes);
                }
            }
            cp_async_arrive(&sm.full[stage]);
            if (++stage == S) stage = 0, phase ^= 1;
            row = next_row;
            kept = next_kept;
        }
        cp_async_wait_all();
        return;
    }

    uint32_t qf[KI][4][4];      // queries in fp16: rows g and g + 8, component order as the codes are read
    float acc[NT][4];           // O: rows g, g + 8 of this warp's columns
    float m[2], l[2], rs[2];    // running maximum, this thread's part of the sum, row scale (log2 units per product)
    int pos[2];
    bool begun = false;         // the segment starts its item
    int seg_unit = 0;           // first unit of the segment

    int stage = 0, phase = 0;
    for (int unit = 0; unit < units; ++unit) {
        if (unit == 0 || cc.j == 0) {   // a new item: queries to registers
            begun = cc.j == 0;
            seg_unit = unit;
            const int first_row = cc.mt * kRows;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = first_row + g + 8 * r, i = row / group;
                const bool ok = i < cc.s.qlen;
                pos[r] = cc.s.kvlen - cc.s.qlen + i;
                m[r] = -INFINITY;
                l[r] = 0.f;
                const __nv_bfloat16 *src = p.q + ((size_t)(cc.s.q0 + (ok ? i : 0)) * p.hq + cc.h * group + row % group) * D + 16 * t;
                uint4 w[KI][2];
                uint32_t big = 0;
#pragma unroll
                for (int k = 0; k < KI; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        w[k][e] = ok ? __ldg(reinterpret_cast<const uint4 *>(src + 64 * k) + e) : make_uint4(0, 0, 0, 0);
                        big = max(big, amax_bits(w[k][e]));
                    }
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
                float down, up;
                power_of_two_scale(big, down, up);
                rs[r] = p.sm_scale * 1.4426950408889634f * up;
#pragma unroll
                for (int k = 0; k < KI; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t x[4] = {w[k][e].x, w[k][e].y, w[k][e].z, w[k][e].w};
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            qf[k][2 * e + f / 2][(f & 1) * 2 + r] = bf16x2_to_f16x2(x[f], down);
                    }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
        }

        wait(&sm.full[stage], phase);
        __syncwarp();

        // ---- scores of this warp's 16 tokens
        const int tok0 = cc.it.token(cc.j, kTile) + warp * kKvBlock;
        float sc[2][2][4] = {};
        const uint32_t kbase = sm100::smem_u32(sm.k[stage]);
#pragma unroll
        for (int k = 0; k < KI; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t w[4];
                lds128(kbase + piece<D>(warp * kKvBlock + 8 * j + g, 4 * k + t), w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t b0, b1;
                    codes_to_f16x2<FMT>(w[e], b0, b1);
                    mma_f16(sc[j][e & 1], qf[k][e], b0, b1);
                }
            }
        const float kscale = sm.scale[stage][warp];
        float vscale = sm.scale[stage][4 + warp];
        if (vscale == 0.f) vscale = kAmaxFloor;
        const float lv = log2f(vscale), rv = 1.f / vscale;
        const bool all_seen = cc.it.all_seen(tok0, tok0 + kKvBlock, p.window, p.sinks);
        float x[2][2][2];   // [row][n-tile][column]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float f = rs[r] * kscale;
            float big = -INFINITY;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float y = fmaf(sc[j][0][2 * r + e] + sc[j][1][2 * r + e], f, lv);
                    if (!all_seen && !sees(pos[r], tok0 + 8 * j + 2 * t + e, p.window, p.sinks)) y = -INFINITY;
                    x[r][j][e] = y;
                    big = fmaxf(big, y);
                }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            if (t == 0) sm.red[warp][g + 8 * r] = big;
        }
        sync_compute();
        // ---- weights
        float corr[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = g + 8 * r;
            const float big = fmaxf(fmaxf(fmaxf(sm.red[0][row], sm.red[1][row]), fmaxf(sm.red[2][row], sm.red[3][row])), m[r]);
            const float safe = big == -INFINITY ? 0.f : big;
            corr[r] = exp2f(m[r] - safe);
            m[r] = big;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float a = exp2f(x[r][j][0] - safe), b = exp2f(x[r][j][1] - safe);
                sum += a + b;
                // fp16 weights: at most 1, 2^-11 relative error each, far below the bf16 rounding of the output
                const __half2 h = __floats2half2_rn(a, b);
                const int u = (2 * warp + j) ^ (row & 7);
                *reinterpret_cast<__half2 *>(reinterpret_cast<uint8_t *>(sm.p) + row * 128 + u * 16 + 4 * t) = h;
            }
            l[r] = l[r] * corr[r] + (sum == 0.f ? 0.f : sum * rv);   // a block that the row does not see may have any scale
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            acc[i][0] *= corr[0]; acc[i][1] *= corr[0];
            acc[i][2] *= corr[1]; acc[i][3] *= corr[1];
        }
        sync_compute();
        // ---- outputs: this warp's columns over all 64 tokens
        const uint32_t vbase = sm100::smem_u32(sm.v[stage]), pbase = sm100::smem_u32(sm.p);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            uint32_t a[4];
            {
                const int row = lane & 15, u = (2 * b + (lane >> 4)) ^ (row & 7);
                asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                             : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                             : "r"(pbase + row * 128 + u * 16)
                             : "memory");
            }
            uint32_t b0[NT], b1[NT];
            value_columns<D, FMT>(vbase, b * 16 + 2 * t, warp, g, b0);
            value_columns<D, FMT>(vbase, b * 16 + 2 * t + 8, warp, g, b1);
#pragma unroll
            for (int i = 0; i < NT; ++i) mma_f16(acc[i], a, b0[i], b1[i]);
        }
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&sm.empty[stage]);
        if (++stage == S) stage = 0, phase ^= 1;

        // ---- the segment's end: finish the item, or hand its part to the merge
        const bool ends = cc.j == cc.it.tiles - 1;
        if (ends || unit == units - 1) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                if (t == 0) sm.red[warp][g + 8 * r] = l[r];   // every warp has read the maxima
            }
            sync_compute();
            const bool whole = begun && ends;
            const int slot = 2 * cta + (seg_unit == 0 ? 0 : 1);
            float *part = plan.parts + (size_t)slot * (kRows * D + 2 * kRows);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = g + 8 * r, grow = cc.mt * kRows + row, i = grow / group;
                const float sum = (sm.red[0][row] + sm.red[1][row]) + (sm.red[2][row] + sm.red[3][row]);
                if (i >= cc.s.qlen) continue;
                const int col = warp * (D / 4) + 2 * NT * t;
                float y[2 * NT];
                const float f = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
#pragma unroll
                for (int k = 0; k < NT; ++k) {
                    y[k] = acc[k][2 * r] * f;
                    y[NT + k] = acc[k][2 * r + 1] * f;
                }
                if (whole) {
                    store_row<2 * NT>(p, ((size_t)(cc.s.q0 + i) * p.hq + cc.h * group + grow % group) * D + col, y);
                } else {
                    float *o = part + row * D + col;
#pragma unroll
                    for (int k = 0; k < 2 * NT; k += 4) *reinterpret_cast<float4 *>(o + k) = make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
                    if (warp == 0 && t == 0) {
                        part[kRows * D + row] = m[r];
                        part[kRows * D + kRows + row] = sum;
                    }
                }
            }
            if (begun && tid == 0 && (plan.meta_by_item || !ends)) {
                // units left of the item after this CTA decide how many CTAs carry it
                const long long left = (long long)cc.it.tiles - 1 - cc.j;
                MergeMeta mm;
                mm.first = cta;
                mm.slot = seg_unit == 0 ? 0 : 1;
                mm.last = ends ? -1 : cta + (int)((left + per - 1) / per);
                mm.n = cc.n;
                mm.h = cc.h;
                mm.mt = cc.mt;
                plan.meta[plan.meta_by_item ? (cc.n * p.pool.hkv + cc.h) * plan.mt_max + cc.mt : cta] = mm;
            }
            sync_compute();   // red is free again
        }
        advance(cc);
    }
}

constexpr int kMergeThreads = 256;

// Joins the parts of one item's row, 64 columns a CTA: o = sum_i 2^{M_i - M} O_i / sum_i 2^{M_i - M} l_i.  16 lanes
// hold the columns and 16 groups of them share the parts, so that all of an item's parts are asked for at once.
template <int D, int ROWS>
__global__ void __launch_bounds__(kMergeThreads) attend_merge_kernel(const __grid_constant__ AttendProblem p,
                                                                     const __grid_constant__ SplitPlan plan) {
    constexpr int LANES = 16, GROUPS = kMergeThreads / LANES;
    __shared__ float weight[kMaxSplitCtas];
    __shared__ float red[2][kMergeThreads / 32];
    __shared__ float4 sum[GROUPS][LANES];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = blockIdx.y;
    const int group = p.hq / p.pool.hkv;
    sm100::grid_dependency_wait();
    if (plan.meta_by_item) {   // items that no CTA visited have no entry
        const int per_seq = p.pool.hkv * plan.mt_max, n = blockIdx.x / per_seq;
        if (blockIdx.x % plan.mt_max >= row_tiles<ROWS>(load_sequence(p, n).qlen, group)) return;
    }
    const MergeMeta mm = plan.meta[blockIdx.x];
    if (mm.last < 0) return;
    const Sequence s = load_sequence(p, mm.n);
    const int grow = mm.mt * ROWS + row, i = grow / group;
    if (i >= s.qlen) return;
    const size_t stride = ROWS * D + 2 * ROWS;
    const int count = mm.last - mm.first + 1;
    auto part = [&](int k) { return plan.parts + (size_t)(2 * (mm.first + k) + (k == 0 ? mm.slot : 0)) * stride; };

    const int col = blockIdx.z * 64 + 4 * (tid % LANES), grp = tid / LANES;
    constexpr int HELD = 8;   // parts of a thread that are asked for before the weights are known
    float4 held[HELD];
#pragma unroll
    for (int k = 0; k < HELD; ++k)
        if (grp + k * GROUPS < count) held[k] = *reinterpret_cast<const float4 *>(part(grp + k * GROUPS) + row * D + col);

    float big = -INFINITY;
    for (int k = tid; k < count; k += kMergeThreads) {
        const float x = part(k)[ROWS * D + row];
        weight[k] = x;
        big = fmaxf(big, x);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    if (lane == 0) red[0][warp] = big;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w) big = fmaxf(big, red[0][w]);
    const float safe = big == -INFINITY ? 0.f : big;
    float l = 0.f;
    for (int k = tid; k < count; k += kMergeThreads) {
        const float w = exp2f(weight[k] - safe);
        weight[k] = w;
        l += w * part(k)[ROWS * D + ROWS + row];
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) red[1][warp] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w) l += red[1][w];

    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4 &o, float w) {
        a.x += w * o.x; a.y += w * o.y; a.z += w * o.z; a.w += w * o.w;
    };
#pragma unroll
    for (int k = 0; k < HELD; ++k)
        if (grp + k * GROUPS < count) add(held[k], weight[grp + k * GROUPS]);
    for (int k = grp + HELD * GROUPS; k < count; k += GROUPS)
        add(*reinterpret_cast<const float4 *>(part(k) + row * D + col), weight[k]);
    sum[grp][tid % LANES] = a;
    __syncthreads();
    if (grp != 0) return;
#pragma unroll
    for (int k = 1; k < GROUPS; ++k) add(sum[k][tid], 1.f);
    const float f = l == 0.f ? 0.f : 1.f / l;
    const float y[4] = {a.x * f, a.y * f, a.z * f, a.w * f};
    store_row<4>(p, ((size_t)(s.q0 + i) * p.hq + mm.h * group + grow % group) * D + col, y);
}

long long unit_bound(int n_seqs, int hq, int hkv, int max_q_len, int max_kv_len) {
    const long long mts = row_tiles<kRows>(max_q_len, hq / hkv);
    const long long tiles = max_kv_len > 0 ? (max_kv_len + kTile - 1) / kTile : 1;
    return n_seqs * (long long)hkv * mts * tiles;
}

template <int D, int FMT>
cudaError_t launch_split(const AttendProblem &p) {
    const int group = p.hq / p.pool.hkv;
    const long long bound = unit_bound(p.n_seqs, p.hq, p.pool.hkv, p.max_q_len, p.max_kv_len);
    const long long fit = (long long)multiprocessor_count() * ctas_per_sm<D>();
    const int ctas = (int)min(bound, min(fit, (long long)kMaxSplitCtas));
    SplitPlan plan{};
    plan.mt_max = row_tiles<kRows>(p.max_q_len, group);
    plan.min_units = 1;
    const long long items = (long long)p.n_seqs * p.pool.hkv * plan.mt_max;
    plan.meta_by_item = items <= ctas;
    plan.meta = static_cast<MergeMeta *>(p.workspace);
    plan.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(p.workspace) + kMetaBytes);

    static std::atomic<bool> ready[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(attend_split_kernel<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Smem<D>));
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) ready[dev].store(true, std::memory_order_relaxed);
    }
    attend_split_kernel<D, FMT><<<ctas, kThreads, sizeof(Smem<D>), p.stream>>>(p, plan);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (ctas == 1 || bound == items) return cudaSuccess;   // no item crosses CTAs
    return launch_after(p.stream, dim3((unsigned)(plan.meta_by_item ? items : ctas), (unsigned)min(kRows, p.max_q_len * group), D / 64), kMergeThreads, 0,
                        attend_merge_kernel<D, kRows>, p, plan);
}

// The tensor-core kernel (attend_tc.cu) for more query rows than four of this kernel's items.
bool use_tensor_kernel(int group, int max_q_len) { return (long long)group * max_q_len > 64; }

}  // namespace

size_t attend_workspace_bytes(int n_seqs, int total, int hq, int hkv, int d, int max_q_len, int max_kv_len) {
    if (n_seqs == 0 || total == 0) return 0;
    if (use_tensor_kernel(hq / hkv, max_q_len)) return attend_tc_workspace_bytes(n_seqs, total, hq, hkv, d);
    const long long slots = 2 * min(unit_bound(n_seqs, hq, hkv, max_q_len, max_kv_len), (long long)kMaxSplitCtas);
    return kMetaBytes + (size_t)slots * (kRows * d + 2 * kRows) * sizeof(float);
}

cudaError_t launch_attend(const AttendProblem &p) {
    if (use_tensor_kernel(p.hq / p.pool.hkv, p.max_q_len)) return launch_attend_tc(p);
    const bool e4m3 = p.format == GDN_KV_E4M3;
    switch (p.d) {
        case 64: return e4m3 ? launch_split<64, GDN_KV_E4M3>(p) : launch_split<64, GDN_KV_INT8>(p);
        case 128: return e4m3 ? launch_split<128, GDN_KV_E4M3>(p) : launch_split<128, GDN_KV_INT8>(p);
        default: return e4m3 ? launch_split<256, GDN_KV_E4M3>(p) : launch_split<256, GDN_KV_INT8>(p);
    }
}

}  // namespace gdn
