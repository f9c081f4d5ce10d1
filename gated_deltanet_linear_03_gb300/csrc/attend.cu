// gdn_attend for few query rows per key/value head (decode, drafted tokens): split over the cache.
//
// With query row r at position p_r, codes k_j, v_j and the scales K_b, V_b of token j's block b,
//     s_j = (q.k_j) K_b sm_scale,   o = sum_j e^{s_j} V_b v_j / sum_j e^{s_j}    over the tokens that p_r sees.
// V_b is folded into the exponent, x_j = (s_j log2 e) + log2 V_b: the weights w_j = 2^{x_j - M} multiply bare
// codes, are at most 1 for a running maximum M of x (so they fit fp16 whatever the scales are), and
// sum_j e^{s_j} = 2^M sum_b (1 / V_b) sum_{j in b} w_j.
//
// Work.  A unit is 64 tokens of one item, an item is (sequence, key/value head, 8 NR query rows: the group's heads
// of consecutive tokens; NR = 1 where no sequence has more than 8 rows, else 2).  All units of the call form one line;
// CTA c of G takes units [c per, (c + 1) per), so ragged batches balance by themselves and one long sequence spreads over the whole GPU.  Lengths are read on
// the device, so a captured graph follows them.  A CTA writes finished items to `out`; of an item that crosses
// CTAs each writes (O, M, l) to the workspace and attend_merge_kernel joins them.
//
// A CTA has a producer warp and four compute warps.  The producer looks pages up and reads block scales a unit ahead
// and brings the blocks' codes through a ring of shared-memory stages by TMA, a box of 16 rows for each block.  Of a unit, compute warp w
// forms the scores of tokens 16 w .. 16 w + 15 (one scale block) with mma.m16n8k16 on codes turned to fp16 exactly,
// as S^T = K Q^T: the 16 tokens are the instruction's rows and 8 query rows its columns, so that a group of 8 heads
// fills it.  The warps exchange maxima and weights through shared memory; warp w then accumulates columns
// [w D/4, (w + 1) D/4) of O^T = V^T W^T over all 64 tokens, D/16 registers a thread and 8 rows.
// Bound by memory: the codes are read once for all heads of a group.  128 K tokens of 2 heads of d = 256, 134 MB: 30 us, and
// 4 for the merge, 0.58 of a copy's rate together; 64 sequences of 256 to 8192 tokens
// and 8 heads of d = 128, 300 MB: 63 us, 0.70.  The kernel's own
// DRAM rate is 0.58 to 0.65 of the peak, issue slots 44 to 57 % busy: what is missing is the start (lengths, table, first codes:
// three latencies one after another, some 4 us) and the end (CTAs that finish between 22 and 26 us, parts, merge).
#include <cudaTypedefs.h>

#include "attend.cuh"

namespace gdn {
namespace {

using namespace attend;

constexpr int kTile = 64;        // tokens of a unit
constexpr int kCompute = 128;    // threads of the compute warps
constexpr int kThreads = kCompute + 32;

// Stages and CTAs of an SM: 128 to 192 KB of codes in flight, as many CTAs as the registers allow (their chains of
// short steps hide one another: 64 sequences of d = 128 63 us with 4, 67 with 3, 69 with 5).  Below d = 256 a stage less leaves
// L1 to the table and the scales: 128 K tokens of d = 128 22.6 us against 24.0, of d = 64 21.8 / 23.8; 64 sequences 63.3 / 62.7, 55 / 55.
template <int D, int NR>
__host__ __device__ constexpr int ctas_per_sm() { return D == 256 ? (NR == 1 ? 3 : 2) : D == 128 ? (NR == 1 ? 4 : 3) : (NR == 1 ? 6 : 4); }
template <int D, int NR>
__host__ __device__ constexpr int stages() { return (D == 256 ? 196608 : 163840) / (ctas_per_sm<D, NR>() * 2 * kTile * D); }

template <int D, int NR>
struct __align__(1024) Smem {
    static constexpr int S = stages<D, NR>(), kRows = 8 * NR;
    uint8_t k[S][kTile * D];
    uint8_t v[S][kTile * D];
    __half p[kRows * kTile];               // weights, 16-byte pieces swizzled by row
    float scale[S][8];                     // K scales of the unit's four blocks, then V scales
    float red[4][kRows];                   // row maxima (then sums) of the four warps
    uint64_t full[S], empty[S];
    int abort;
    int scan[4];
    int start_seq;
    int start_off;
};

// Byte offset of 16-byte piece u of row r in a stage, as TMA's swizzle places it: boxes of 16 rows and 128 bytes, one
// after another for each block, pieces exchanged by the row's low bits (at d = 64 boxes of 64-byte rows, by row pairs).
template <int D>
__device__ __forceinline__ uint32_t piece(int r, int u) {
    if (D == 64) return (uint32_t)(r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
    return (uint32_t)(((r >> 4) * (D / 128) + (u >> 3)) * 2048 + (r & 15) * 128 + (((u & 7) ^ (r & 7)) << 4));
}

// The row of an 8-row group that takes place k in the matrix instructions.  Rows of neighbouring places differ in bit
// 2 and the even (odd) places hold one row of each pair, so that with the swizzle above the lanes that read together
// (scores: 4 pieces of places 2 a, 2 a + 1; outputs: 2 pieces of the four even, or odd, places) touch each bank once.
__device__ __forceinline__ int row_at(int k) { return (0x37156240 >> (4 * k)) & 7; }

// The compute warps' barrier.  None of them leaves the unit loop early (a wait that runs out only sets a flag).
__device__ __forceinline__ void sync_compute() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kCompute) : "memory"); }

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Fragments of V for one 8-token half of a k-step: rows r and s of the stage, the columns 8 (or 4, 2) * g .. of warp
// w's quarter.  b[i] = (code at row r, code at row s) of column i as an fp16 pair.
template <int D, int FMT>
__device__ __forceinline__ void value_columns(uint32_t base, int r, int s, int w, int g, uint32_t (&b)[D / 32]) {
    const int col = w * (D / 4) + g * (D / 32);   // first column byte
    const uint32_t a0 = base + piece<D>(r, col >> 4) + (col & 15), a1 = base + piece<D>(s, col >> 4) + (col & 15);
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

template <int D, int FMT, int NR>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<D, NR>()) attend_split_kernel(const __grid_constant__ AttendProblem p,
                                                                                      const __grid_constant__ SplitPlan plan,
                                                                                      const __grid_constant__ CUtensorMap k_map,
                                                                                      const __grid_constant__ CUtensorMap v_map) {
    constexpr int S = stages<D, NR>(), KI = D / 64, NT = D / 32, kRows = 8 * NR;
    extern __shared__ uint8_t raw[];
    Smem<D, NR> &sm = *reinterpret_cast<Smem<D, NR> *>(raw + ((1024u - (sm100::smem_u32(raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int group = p.hq / p.pool.hkv, cta = blockIdx.x;
    sm100::grid_launch_dependents();

    // ---- this CTA's units: a scan over the sequences' costs
    if (tid == kCompute) {
        sm100::tma_prefetch_desc(&k_map);
        sm100::tma_prefetch_desc(&v_map);
        for (int i = 0; i < S; ++i) {
            sm100::mbar_init(&sm.full[i], 1);
            sm100::mbar_init(&sm.empty[i], 4);
        }
        sm.abort = 0;
        sm100::fence_mbar_init();
        sm100::tma_prefetch_desc(&k_map);
        sm100::tma_prefetch_desc(&v_map);
    }
    const int chunk = (p.n_seqs + kCompute - 1) / kCompute;
    const int s_lo = tid < kCompute ? min(tid * chunk, p.n_seqs) : p.n_seqs, s_hi = min(s_lo + chunk, p.n_seqs);
    int mine = 0;                                     // the host has checked that all units fit 31 bits
    for (int n = s_lo; n < s_hi; ++n) mine += sequence_cost<kRows, kTile>(p, load_sequence(p, n), group);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    if (lane == 31 && warp < 4) sm.scan[warp] = upto;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < warp) upto += sm.scan[w];
        total += sm.scan[w];
    }
    const int per = max((int)(((unsigned)total + gridDim.x - 1) / gridDim.x), 1);
    const int start = (int)min((long long)cta * per, (long long)total), stop = min(total - start, per) + start;
    if (tid == 0 && !plan.meta_by_item) plan.meta[cta].last = -1;
    if (tid == 0) report_lengths(p, cta);
    if (start >= stop) return;
    if (start >= upto - mine && start < upto) {
        int off = start - (upto - mine);
        for (int n = s_lo; n < s_hi; ++n) {
            const int c = sequence_cost<kRows, kTile>(p, load_sequence(p, n), group);
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
        int off = sm.start_off;
        const int head_cost = sequence_cost<kRows, kTile>(p, cc.s, group) / p.pool.hkv;
        cc.h = off / head_cost;
        off -= cc.h * head_cost;
        for (cc.mt = 0; cc.mt < mts; ++cc.mt) {
            cc.it = make_item<kRows, kTile>(p, cc.s, group, cc.mt);
            if (off < cc.it.tiles) break;
            off -= cc.it.tiles;
        }
        cc.j = off;
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
    // A bounded wait; when it runs out a flag is set with which every later wait returns at once and which becomes the
    // call's error at the end.
    volatile int *abort = &sm.abort;
    auto wait = [&](uint64_t *bar, int phase) { sm100::mbar_poll(bar, (uint32_t)phase & 1, abort); };
    const int units = stop - start;

    if (warp == 4) {
        // ---- the producer: of lanes 0..7, lane b holds K's block b of a unit and lane 4 + b V's: the pool row where it
        // begins, -1 where there is none
        bool exists;
        int entry, in_page, head;
        auto look_up = [&]() {      // asks for the table's entry, which is looked at when the unit's turn comes
            const int tok = cc.it.token(cc.j, kTile) + (lane & 3) * kKvBlock;
            exists = lane < 8 && tok < cc.s.kvlen && in_sight(cc.it.lo_pos, cc.it.hi_pos, tok, tok + kKvBlock, p.window, p.sinks);
            if (!exists) return;
            const int at = p.pool.page_of(tok);
            entry = __ldg(p.pool.table + (size_t)cc.n * p.pool.max_pages + at);
            in_page = tok - at * p.pool.page_size;
            head = cc.h;
        };
        auto pool_row = [&]() -> int {
            if (!exists) return -1;
            if ((unsigned)entry < (unsigned)p.pool.n_pages) return (entry * p.pool.hkv + head) * p.pool.page_size + in_page;
            raise_error(p.err, kErrInternal);
            return -1;
        };
        auto scale_of = [&](int row) -> float { return row >= 0 ? __ldg((lane < 4 ? p.k_scales : p.v_scales) + row / kKvBlock) : 0.f; };
        const CUtensorMap *map = lane < 4 ? &k_map : &v_map;
        const int no_row = p.pool.n_pages * p.pool.hkv * p.pool.page_size;      // past the pool's last: the load fills zeros in
        look_up();
        int row = pool_row(), stage = 0, phase = 1, issued = 0;
        float scale = scale_of(row);
        if (units > 1) {
            advance(cc);
            look_up();
        }
        for (int unit = 0; unit < units; ++unit) {
            wait(&sm.empty[stage], phase);
            __syncwarp();
            if (*abort) break;
            if (lane < 8) {
                uint8_t *dst = (lane < 4 ? sm.k[stage] : sm.v[stage]) + (lane & 3) * (kKvBlock * D);
#pragma unroll
                for (int x = 0; x < D; x += 128) sm100::tma_load_2d(dst + x * kKvBlock, map, &sm.full[stage], x, row >= 0 ? row : no_row);
            }
            // the next unit's rows and scales, and the table's entries of the one after it, while this one's codes come
            const int next_row = unit + 1 < units ? pool_row() : -1;
            const float next_scale = scale_of(next_row);
            if (unit + 2 < units) {
                advance(cc);
                look_up();
            }
            if (lane < 8) sm.scale[stage][lane] = scale;
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive_expect_tx(&sm.full[stage], 2 * kTile * D);
            if (++stage == S) stage = 0, phase ^= 1;
            row = next_row;
            scale = next_scale;
            ++issued;
        }
        // every copy is waited for by the compute warps; where they have given up, here
        if (*abort) {
            for (int k = max(0, issued - S); k < issued; ++k) sm100::mbar_wait(&sm.full[k % S], (uint32_t)(k / S) & 1);
            raise_error(p.err, kErrTimeout);
        }
        return;
    }

    uint32_t qf[NR][KI][4][2];  // queries in fp16: row 8 r + g, component order as the codes are read
    float acc[NR][NT / 2][4];   // O^T: this warp's columns NT g .. NT g + NT - 1 of rows 8 r + 2 t and + 1
    float m[NR][2], l[NR][2];   // those rows' running maximum, and this thread's part of their sum
    float rs[NR][2];            // and their scale, log2 units per product
    int pos[NR][2];
    bool begun = false;         // the segment starts its item
    int seg_unit = 0;           // first unit of the segment

    int stage = 0, phase = 0;
    for (int unit = 0; unit < units; ++unit) {
        if (unit == 0 || cc.j == 0) {   // a new item: queries to registers
            begun = cc.j == 0;
            seg_unit = unit;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const int row = cc.mt * kRows + 8 * r + g, i = row / group;
                const bool ok = i < cc.s.qlen;
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
#pragma unroll
                for (int k = 0; k < KI; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t x[4] = {w[k][e].x, w[k][e].y, w[k][e].z, w[k][e].w};
#pragma unroll
                        for (int f = 0; f < 4; ++f) qf[r][k][2 * e + f / 2][f & 1] = bf16x2_to_f16x2(x[f], down);
                    }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    // row 8 r + 2 t + c is loaded by the lanes of g = 2 t + c
                    rs[r][c] = p.sm_scale * 1.4426950408889634f * __shfl_sync(0xffffffffu, up, 4 * (2 * t + c));
                    pos[r][c] = cc.s.kvlen - cc.s.qlen + (cc.mt * kRows + 8 * r + 2 * t + c) / group;
                    m[r][c] = -INFINITY;
                    l[r][c] = 0.f;
                }
#pragma unroll
                for (int i2 = 0; i2 < NT / 2; ++i2)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[r][i2][e] = 0.f;
            }
        }

        wait(&sm.full[stage], phase);
        __syncwarp();

        // ---- scores of this warp's 16 tokens: places g and g + 8 of the block against every query row
        const int tok0 = cc.it.token(cc.j, kTile) + warp * kKvBlock;
        float sc[NR][2][4] = {};
        const uint32_t kbase = sm100::smem_u32(sm.k[stage]);
#pragma unroll
        for (int k = 0; k < KI; ++k) {
            uint32_t w0[4], w1[4];
            lds128(kbase + piece<D>(warp * kKvBlock + row_at(g), 4 * k + t), w0);
            lds128(kbase + piece<D>(warp * kKvBlock + 8 + row_at(g), 4 * k + t), w1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t a[4];
                codes_to_f16x2<FMT>(w0[e], a[0], a[2]);
                codes_to_f16x2<FMT>(w1[e], a[1], a[3]);
#pragma unroll
                for (int r = 0; r < NR; ++r) mma_f16(sc[r][e & 1], a, qf[r][k][e][0], qf[r][k][e][1]);
            }
        }
        const float kscale = sm.scale[stage][warp];
        float vscale = sm.scale[stage][4 + warp];
        if (vscale == 0.f) vscale = kAmaxFloor;
        const float lv = log2f(vscale), rv = 1.f / vscale;
        const bool all_seen = cc.it.all_seen(tok0, tok0 + kKvBlock, p.window, p.sinks);
        float x[NR][2][2];   // [8 rows][token g, g + 8][row 2 t, 2 t + 1]
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float f = rs[r][c] * kscale;
                float big = -INFINITY;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float y = fmaf(sc[r][0][2 * j + c] + sc[r][1][2 * j + c], f, lv);
                    if (!all_seen && !sees(pos[r][c], tok0 + 8 * j + row_at(g), p.window, p.sinks)) y = -INFINITY;
                    x[r][j][c] = y;
                    big = fmaxf(big, y);
                }
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 4));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 8));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 16));
                if (g == 0) sm.red[warp][8 * r + 2 * t + c] = big;
            }
        // V rows of the last block that lie past the sequence's end, whatever they hold, are cleared: their weights are 0, and 0
        // times a code is not 0 for a code that is NaN.  (Keys there only make scores that the mask replaces.)
        const bool tail = tok0 < cc.s.kvlen && tok0 + kKvBlock > cc.s.kvlen;
        if (tail) {
            for (int i = lane; i < kKvBlock * (D / 16); i += 32)
                if (tok0 + i / (D / 16) >= cc.s.kvlen)
                    *reinterpret_cast<uint4 *>(sm.v[stage] + piece<D>(warp * kKvBlock + i / (D / 16), i % (D / 16))) = make_uint4(0, 0, 0, 0);
            sm100::fence_proxy_async_smem();   // before the stage is filled by TMA again
        }
        sync_compute();
        // ---- weights
        const uint32_t pbase = sm100::smem_u32(sm.p);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float e[2][2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = 8 * r + 2 * t + c;
                const float big = fmaxf(fmaxf(fmaxf(sm.red[0][row], sm.red[1][row]), fmaxf(sm.red[2][row], sm.red[3][row])), m[r][c]);
                const float safe = big == -INFINITY ? 0.f : big;
                const float corr = exp2f(m[r][c] - safe);
                m[r][c] = big;
                e[0][c] = exp2_fast(x[r][0][c] - safe);
                e[1][c] = exp2_fast(x[r][1][c] - safe);
                const float sum = e[0][c] + e[1][c];
                l[r][c] = l[r][c] * corr + (sum == 0.f ? 0.f : sum * rv);   // a block that the row does not see may have any scale
#pragma unroll
                for (int i = 0; i < NT / 2; ++i) {
                    acc[r][i][c] *= corr;
                    acc[r][i][2 + c] *= corr;
                }
            }
            // fp16 weights: at most 1, with an error of 2^-11 of themselves or 2^-25, whichever is larger, far below the bf16
            // rounding of the output.  They are stored transposed, as 64 tokens of each row.
            const __half2 h0 = __floats2half2_rn(e[0][0], e[0][1]), h1 = __floats2half2_rn(e[1][0], e[1][1]);
            const int row = 8 * r + (lane & 7), u = (2 * warp + ((lane >> 3) & 1)) ^ (lane & 7);
            asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(pbase + row * 128 + u * 16),
                         "r"(*reinterpret_cast<const uint32_t *>(&h0)), "r"(*reinterpret_cast<const uint32_t *>(&h1))
                         : "memory");
        }
        sync_compute();
        // ---- outputs: this warp's columns over all 64 tokens
        const uint32_t vbase = sm100::smem_u32(sm.v[stage]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t wt[NR][4];     // weights of 32 tokens: the two registers of two k-steps
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const int row = 8 * r + (lane & 7), u = (4 * half + (lane >> 3)) ^ (lane & 7);
                asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                             : "=r"(wt[r][0]), "=r"(wt[r][1]), "=r"(wt[r][2]), "=r"(wt[r][3])
                             : "r"(pbase + row * 128 + u * 16)
                             : "memory");
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t v0[NT], v1[NT];
                const int r0 = (2 * half + b) * 16 + row_at(2 * t), r1 = (2 * half + b) * 16 + row_at(2 * t + 1);
                value_columns<D, FMT>(vbase, r0, r1, warp, g, v0);
                value_columns<D, FMT>(vbase, r0 + 8, r1 + 8, warp, g, v1);
#pragma unroll
                for (int i = 0; i < NT / 2; ++i) {
                    const uint32_t a[4] = {v0[2 * i], v0[2 * i + 1], v1[2 * i], v1[2 * i + 1]};
#pragma unroll
                    for (int r = 0; r < NR; ++r) mma_f16(acc[r][i], a, wt[r][2 * b], wt[r][2 * b + 1]);
                }
            }
        }
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&sm.empty[stage]);
        if (++stage == S) stage = 0, phase ^= 1;

        // ---- the segment's end: finish the item, or hand its part to the merge
        const bool ends = cc.j == cc.it.tiles - 1;
        if (ends || unit == units - 1) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    l[r][c] += __shfl_xor_sync(0xffffffffu, l[r][c], 4);
                    l[r][c] += __shfl_xor_sync(0xffffffffu, l[r][c], 8);
                    l[r][c] += __shfl_xor_sync(0xffffffffu, l[r][c], 16);
                    if (g == 0) sm.red[warp][8 * r + 2 * t + c] = l[r][c];   // every warp has read the maxima
                }
            sync_compute();
            const bool whole = begun && ends;
            const int slot = 2 * cta + (seg_unit == 0 ? 0 : 1);
            float *part = plan.parts + (size_t)slot * (kRows * D + 2 * kRows);
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int row = 8 * r + 2 * t + c, grow = cc.mt * kRows + row, i = grow / group;
                    const float sum = (sm.red[0][row] + sm.red[1][row]) + (sm.red[2][row] + sm.red[3][row]);
                    if (i >= cc.s.qlen) continue;
                    const int col = warp * (D / 4) + NT * g;
                    float y[NT];
                    const float f = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
#pragma unroll
                    for (int k = 0; k < NT / 2; ++k) {
                        y[2 * k] = acc[r][k][c] * f;
                        y[2 * k + 1] = acc[r][k][2 + c] * f;
                    }
                    if (whole) {
                        store_row<NT>(p, ((size_t)(cc.s.q0 + i) * p.hq + cc.h * group + grow % group) * D + col, y);
                    } else {
                        float *o = part + row * D + col;
#pragma unroll
                        for (int k = 0; k < NT; k += 2) *reinterpret_cast<float2 *>(o + k) = make_float2(y[k], y[k + 1]);
                        if (warp == 0 && g == 0) {
                            part[kRows * D + row] = m[r][c];
                            part[kRows * D + kRows + row] = sum;
                        }
                    }
                }
            if (begun && tid == 0 && (plan.meta_by_item || !ends)) {
                // units left of the item after this CTA decide how many CTAs carry it
                const int left = cc.it.tiles - 1 - cc.j;
                MergeMeta mm;
                mm.first = cta;
                mm.slot = seg_unit == 0 ? 0 : 1;
                mm.last = ends ? -1 : cta + (left - 1) / per + 1;
                mm.n = cc.n;
                mm.h = cc.h;
                mm.mt = cc.mt;
                plan.meta[plan.meta_by_item ? (cc.n * p.pool.hkv + cc.h) * plan.mt_max + cc.mt : cta] = mm;
            }
            sync_compute();   // red is free again
        }
        advance(cc);
    }
    if (tid == 0 && *abort) raise_error(p.err, kErrTimeout);
}

constexpr int kMergeThreads = 256;

// Joins the parts of one item's row, 64 columns a CTA: o = sum_i 2^{M_i - M} O_i / sum_i 2^{M_i - M} l_i.  16 lanes
// hold the columns and 16 groups of them share the parts, so that all of an item's parts are asked for at once.
template <int D, int ROWS>
__global__ void __launch_bounds__(kMergeThreads) attend_merge_kernel(const __grid_constant__ AttendProblem p,
                                                                     const __grid_constant__ SplitPlan plan) {
    constexpr int LANES = 16, GROUPS = kMergeThreads / LANES;
    __shared__ float weight[kMaxSplitCtas], part_l[kMaxSplitCtas];
    __shared__ float red[2][kMergeThreads / 32];
    __shared__ float4 sum[GROUPS][LANES];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = blockIdx.y;
    const int group = p.hq / p.pool.hkv;
    // An item's sequence is read before the split kernel has ended; items that no CTA visited have no entry.  Their CTAs wait too:
    // a grid whose CTAs all had left would let the stream's next kernel start while the split kernel still reads its lengths.
    // (Two waits, because the lengths are read behind a single one: one token behind 131072 34.7 us instead of 34.0.)
    const Sequence s = load_sequence(p, blockIdx.x / (p.pool.hkv * plan.mt_max));
    if ((int)(blockIdx.x % plan.mt_max) >= row_tiles<ROWS>(s.qlen, group)) {
        sm100::grid_dependency_wait();
        return;
    }
    sm100::grid_dependency_wait();
    const MergeMeta mm = plan.meta[blockIdx.x];
    if (mm.last < 0) return;
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
        const float x = part(k)[ROWS * D + row], y = part(k)[ROWS * D + ROWS + row];
        weight[k] = x;
        part_l[k] = y;
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
        l += w * part_l[k];
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

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
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

// The pool as rows of d bytes, read in boxes of one block (and at most 128 bytes of its rows).
bool pool_map(CUtensorMap *m, const uint8_t *pages, const KvPool &pool, int d) {
    const auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)pool.n_pages * pool.hkv * pool.page_size}, strides[1] = {(cuuint64_t)d};
    const cuuint32_t box[2] = {(cuuint32_t)min(d, 128), kKvBlock}, es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(pages), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query rows of an item: 8 where no sequence has more (a head group's single tokens), else 16, of which half would idle there
// (8 rows: 2 heads x 32768 tokens of d = 256 16.5 us as 8, 21 us as 16; 16 x 8 heads x 8192 tokens of d = 128 62 / 79 us).
int item_rows(int group, int max_q_len) { return (long long)group * max_q_len <= 8 ? 8 : 16; }

long long unit_bound(int n_seqs, int hq, int hkv, int max_q_len, int max_kv_len) {
    const int group = hq / hkv, rows = item_rows(group, max_q_len);
    const long long mts = ((long long)max_q_len * group + rows - 1) / rows;
    const long long tiles = max_kv_len > 0 ? (max_kv_len + kTile - 1) / kTile : 1;
    return (long long)min((double)n_seqs * hkv * mts * tiles, 4e18);   // far above what is accepted, and no overflow
}

template <int D, int FMT, int NR>
cudaError_t launch_split(const AttendProblem &p) {
    const int group = p.hq / p.pool.hkv;
    const long long bound = unit_bound(p.n_seqs, p.hq, p.pool.hkv, p.max_q_len, p.max_kv_len);
    const long long fit = (long long)multiprocessor_count() * ctas_per_sm<D, NR>();
    SplitPlan plan{};
    plan.mt_max = row_tiles<8 * NR>(p.max_q_len, group);
    const long long items = (long long)p.n_seqs * p.pool.hkv * plan.mt_max;
    const int ctas = (int)min(bound, min(fit, (long long)kMaxSplitCtas));
    // Few items: the merge goes by item, with a CTA for each piece of its rows.  Otherwise by the CTAs that items cross, one CTA
    // for 8 rows.  Measured for 16 heads over 2 of d = 256, us by item / by CTA: 2 items of 5 units 8.8 / 10.1, of 64 units 9.5 / 24,
    // of 2048 35 / 88, 16 items of 128 units 23 / 29, 32 items 35 / 37, 48 of 64 31.6 / 30.5, 64 of 64 38.5 / 35.5, 96 of 64 54 / 45,
    // 200 items of 32 68 / 46; of d = 128, 32 items of 64 units 14.6 / 16.5, 48 19.1 / 20.8, 64 21.1 / 22.5, 96 28.7 / 28.9, 192 46.6 /
    // 43.6; of d = 64, 48 items of 64 units 16.5 / 18.2, 64 20.6 / 22.5, 96 26.4 / 25.8: at 48 no head size loses more than 4 %.
    plan.meta_by_item = items <= 48;
    plan.meta = static_cast<MergeMeta *>(p.workspace);
    plan.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(p.workspace) + kMetaBytes);

    constexpr size_t smem = sizeof(Smem<D, NR>) + 1024;
    static std::atomic<bool> ready[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(attend_split_kernel<D, FMT, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) ready[dev].store(true, std::memory_order_relaxed);
    }
    CUtensorMap k_map, v_map;
    if (!pool_map(&k_map, p.k_pages, p.pool, D) || !pool_map(&v_map, p.v_pages, p.pool, D)) return cudaErrorInvalidValue;
    attend_split_kernel<D, FMT, NR><<<ctas, kThreads, smem, p.stream>>>(p, plan, k_map, v_map);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (ctas == 1 || bound == items) return cudaSuccess;   // no item crosses CTAs
    if (plan.meta_by_item)
        return launch_after(p.stream, dim3((unsigned)items, (unsigned)min(8 * NR, p.max_q_len * group), D / 64), kMergeThreads, 0,
                            attend_merge_kernel<D, 8 * NR>, p, plan);
    return launch_after(p.stream, dim3((unsigned)ctas, NR), 256, 0, attend_join_kernel<D, 8 * NR>, p,
                        static_cast<const MergeMeta *>(plan.meta), static_cast<const float *>(plan.parts));
}

template <int D, int FMT>
cudaError_t launch_split(const AttendProblem &p) {
    return item_rows(p.hq / p.pool.hkv, p.max_q_len) == 8 ? launch_split<D, FMT, 1>(p) : launch_split<D, FMT, 2>(p);
}

// The tensor-core kernel (attend_tc.cu) reads the cache once for 128 (d = 256) or 256 query rows, this one for 16, but it
// has a planning launch, a longer pipeline to fill and larger parts to join.  By query rows of a key/value head and, where these
// are few, by this kernel's units of work.  Measured, us here / there (sequences x heads x tokens):
//   d = 256:  1 x 2 x 2048   128 rows 19 / 28   256 rows 28 / 31       1 x 2 x 8192  128 rows 32 / 40  256 rows 52 / 34
//             1 x 2 x 32768   48 rows 39 / 46    64 rows 46 / 48       4 x 2 x 8192   32 rows 34 / 31   64 rows 53 / 34
//   d = 128:  1 x 8 x 2048    64 rows 20 / 21   128 rows 28 / 22       4 x 8 x 8192   32 rows 51 / 58   64 rows 77 / 58
//             1 x 8 x 32768   32 rows 46 / 60    48 rows 63 / 61      16 x 8 x 8192   32 rows 144 / 180 48 rows 209 / 181
//   d = 64:   1 x 1 x 2048   128 rows 11 / 20   256 rows 15 / 22       4 x 1 x 8192   64 rows 17 / 22  128 rows 25 / 23
//             1 x 1 x 32768  128 rows 24 / 37   256 rows 39 / 39      16 x 1 x 8192   32 rows 24 / 28   48 rows 33 / 28
// `tokens` bounds what a row sees.
bool use_tensor_kernel(int n_seqs, int hq, int hkv, int d, int max_q_len, int tokens) {
    const long long rows = (long long)(hq / hkv) * max_q_len, units = unit_bound(n_seqs, hq, hkv, max_q_len, tokens);
    if (d == 256) return rows > 256 || (rows > 16 && units >= 4000);
    if (d == 128) return rows > 64 || (rows > 32 && units >= 4000);
    return rows > 256 || (rows > 32 && units >= 6000);
}

bool use_tensor_kernel(const AttendProblem &p) {
    const long long tokens = p.window == 0 ? p.max_kv_len : min((long long)p.max_kv_len, (long long)p.window + p.sinks + p.max_q_len);
    return use_tensor_kernel(p.n_seqs, p.hq, p.pool.hkv, p.d, p.max_q_len, (int)tokens);
}

}  // namespace

size_t attend_workspace_bytes(int n_seqs, int total, int hq, int hkv, int d, int max_q_len, int max_kv_len) {
    if (n_seqs == 0 || total == 0) return 0;
    // whichever kernels a call of these bounds may take: with a window it may be the one for fewer tokens
    size_t need = 0;
    if (use_tensor_kernel(n_seqs, hq, hkv, d, max_q_len, max_kv_len)) need = attend_tc_workspace_bytes(n_seqs, total, hq, hkv, d);
    if (use_tensor_kernel(n_seqs, hq, hkv, d, max_q_len, 1)) return need;
    const int rows = item_rows(hq / hkv, max_q_len);
    const long long slots = 2 * min(unit_bound(n_seqs, hq, hkv, max_q_len, max_kv_len), (long long)kMaxSplitCtas);
    return max(need, kMetaBytes + (size_t)slots * (rows * d + 2 * rows) * sizeof(float));
}

bool attend_supported(int n_seqs, int hq, int hkv, int d, int max_q_len, int max_kv_len) {
    return use_tensor_kernel(n_seqs, hq, hkv, d, max_q_len, max_kv_len) || unit_bound(n_seqs, hq, hkv, max_q_len, max_kv_len) < 2147483647LL;
}

cudaError_t launch_attend(const AttendProblem &p) {
    if (use_tensor_kernel(p)) return launch_attend_tc(p);
    const bool e4m3 = p.format == GDN_KV_E4M3;
    switch (p.d) {
        case 64: return e4m3 ? launch_split<64, GDN_KV_E4M3>(p) : launch_split<64, GDN_KV_INT8>(p);
        case 128: return e4m3 ? launch_split<128, GDN_KV_E4M3>(p) : launch_split<128, GDN_KV_INT8>(p);
        default: return e4m3 ? launch_split<256, GDN_KV_E4M3>(p) : launch_split<256, GDN_KV_INT8>(p);
    }
}

}  // namespace gdn
