// 4-bit products with one or two rows of x: bound by reading the codes, 0.5625 bytes a weight with scales and offsets of 64 inputs.
//
// A warp reads 512 inputs of a weight row at once, 8 bytes a lane: 256 bytes in a row.  Lane 4 g + t has inputs 16 (4 g + t) ..
// + 15, so the four lanes of g have the 64 inputs of one group.  The tensor cores sum a group's products over its lanes and keep
// the groups apart: in mma.sync (16 x 8 x 16) row g of the first operand is group g of one weight row, row g + 8 that of another,
// and column g of the second operand is x at the inputs of group g, which lane (g, t) holds in registers for all the rows that
// come.  Of the product the diagonal is wanted, D[g][g] and D[g + 8][g]; the rest is thrown away, which costs nothing: with one row
// of x all but one of a product's eight columns would be empty anyhow.  So no operand goes through shared memory, a weight costs
// about 1.5 instructions, and scale and offset meet each group's sum in one lane of its four.
//
// Codes are halves almost as they lie in a word: a code in bits 4 to 7 of a half is c 2^-20, so a word's four pairs (i, i + 4) cost
// four ANDs and three shifts.  The tensor cores multiply such subnormals exactly, but line up a product by its exponents as if it
// began with a one, so that up to 6 of a sum's last bits are lost: no more than fp32 sums of another order differ by (12352 x 2048: of
// the bf16 outputs 1.6e-4 are not the nearest to the exact ones, with fp32 outputs rounded as many; codes in bits 0 to 3 as
// well save two shifts, but lose 10 bits: 1.9e-3).  For fp32 outputs each pair is put under the exponent of 1024, which is taken off
// again: c and 16 c as normal numbers.  x goes to fp16, its row scaled by a power of two to [2^14, 2^15), which keeps all bits of a
// bf16 number down to 2^-28 of the row's largest (some down to 2^-36), for fp32 outputs with every other pair divided by 16; it is
// put into the pairs' order once.
//
// Measured (device times, weights from memory): 131071 x 2048 with offsets, one row, bf16 outputs 32.4 us, 4.7 TB/s, 0.69 of the copy
// rate (29.8 with codes in bits 0 to 3); fp32 outputs 39.3 us, where the subtractions make the issue slots (0.63 busy) the limit.
// 12352 x 2048 7.6 us, gated 2 x 5632 x 2048 7.1: launch, the first loads' latency, and 1544 turns of 8 rows on 608 schedulers; the bytes alone are 2 us.
#include "layer_ops.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kSlice = 512;                // inputs that a warp reads at once
template <int M>
constexpr int kSlicesOf = M == 1 ? 4 : 2;  // that it holds x for, in registers
constexpr int kRows = 8;                   // weight rows of a warp's turn (4 of either matrix)

__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_next(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }      // -126 .. 127

// What a code of one is in the sums of products.  Codes as normal numbers get it with the scale: a sum of 64 of x's scaled numbers
// times codes, 2^25 at most, by a scale would leave fp32 where scales are large.
template <bool EXACT>
constexpr float kCodeUnit = EXACT ? 0x1p-24f : 0x1p-20f;

// Two codes of a word, of which MASK leaves their bits.
template <bool EXACT>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t mask) {
    if (!EXACT) return w & mask;
    uint32_t r;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w & mask | 0x64006400u), "r"(0x64006400u));
    return r;
}

// What a warp reads of its rows at one slice comes by TMA into its own ring, kDeep slices ahead: no registers wait for memory, and a
// row's place in a stage is a constant.  Scales come the same way where the rows of scales can be a tensor's (a multiple of
// 16 bytes), else through registers, a slice ahead.
constexpr int kDeep = 3;
template <int MATS>
struct Stage {                             // each box begins on a 128-byte boundary
    uint2 code[kRows][32];                 // by lane
    __nv_bfloat16 scale[MATS][8][8], offset[MATS][8][8];
};

struct Scales {
    uint32_t scale[kRows], offset[kRows];  // (bf16 in the low half: as 16-bit numbers they would be packed in between)
};

struct VecMaps {
    CUtensorMap codes[2], scales[2], offsets[2];      // of the matrix, or of both
};

template <int M, bool GATED, bool OFFSETS, bool SCALE_TMA, bool EXACT>
__global__ void __launch_bounds__(kThreads, 2)
q4_vec_kernel(const __grid_constant__ Q4Problem p, const __grid_constant__ VecMaps maps, int kw, int each, unsigned int *err) {
    constexpr int OUT = GATED ? kRows / 2 : kRows;                     // outputs of a turn
    constexpr int kSlices = kSlicesOf<M>;
    extern __shared__ __align__(128) unsigned char raw[];
    __shared__ float part[2][kWarps][kRows * M];
    __shared__ uint64_t full[kWarps][kDeep];
    __shared__ int gave_up;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int ks = warp % kw, together = kWarps / kw;                  // the warp's part of the inputs; turns of a CTA at once
    const int groups = p.k / p.group, shift = p.group == 128 ? 1 : 0;
    const int step = gridDim.x * together, turns = (p.n_out + OUT - 1) / OUT;
    // Warps on their own take turns that are gridDim.x apart, so that all SMs get as many, but for one (2 x 5632 x 2048 7.6 -> 6.6 us).
    // Warps that meet go through the same number of turns, of which the last may be beyond the matrix
    int turn = kw > 1 ? blockIdx.x * together + warp / kw : blockIdx.x + gridDim.x * warp;
    const int rounds = kw > 1 ? (turns + step - 1) / step : turn < turns ? (turns - turn + step - 1) / step : 0;
    const int slice0 = ks * each, slices = rounds ? min(each, (p.k + kSlice - 1) / kSlice - slice0) : 0;

    constexpr int MATS = GATED ? 2 : 1;
    Stage<MATS> *ring = reinterpret_cast<Stage<MATS> *>(raw) + warp * kDeep;
    volatile int *abort = &gave_up;
    const int total = rounds * max(slices, 0);
    int buffer = 0;
    if (lane == 0) {
        for (int i = 0; i < kDeep; ++i) mbar_init(&full[warp][i], 1);
        if (warp == 0) gave_up = 0;
        fence_mbar_init();
    }
    __syncthreads();
    // the next slice to ask for
    int ask_turn = turn, ask_slice = 0, asked = 0;
    auto ask = [&](int place) {
        if (asked++ < total && elect_one()) {
            Stage<MATS> &to = ring[place];
            const int col = (slice0 + ask_slice) * kSlice, row = ask_turn * OUT, group = (col / 64 >> shift) & ~7;
            uint64_t *bar = &full[warp][place];
            mbar_arrive_expect_tx(bar, kRows * (kSlice / 2 + (SCALE_TMA ? OFFSETS ? 32 : 16 : 0)));
#pragma unroll
            for (int m = 0; m < MATS; ++m) {                      // (the maps count bytes)
                tma_load_2d(to.code[m * OUT], &maps.codes[m], bar, col / 2, row);
                if (SCALE_TMA) {
                    tma_load_2d(to.scale[m], &maps.scales[m], bar, 2 * group, row);
                    if (OFFSETS) tma_load_2d(to.offset[m], &maps.offsets[m], bar, 2 * group, row);
                }
            }
        }
        if (++ask_slice == slices) ask_slice = 0, ask_turn += step;
    };
    for (int i = 0; i < kDeep; ++i) ask(i);
    // x at this lane's inputs as halves in the order of the codes' pairs, and its sum over the lane's group, both scaled
    constexpr float ODD = EXACT ? 0.0625f : 1.f;            // pairs 1 and 3 of normal numbers are 16 times their codes
    uint32_t x[M][kSlices][8];
    float xsum[M][kSlices];
    int exponent[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        uint4 v[kSlices][2];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kSlices; ++i) {
            const int at = (slice0 + i) * kSlice + 16 * lane;
            v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
            if (i < slices && at < p.k) {
                const uint4 *from = reinterpret_cast<const uint4 *>(p.x + m * p.x_stride + at);
                v[i][0] = from[0];
                v[i][1] = from[1];
            }
            top = max(top, max(amax_bits(v[i][0]), amax_bits(v[i][1])));
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (kw > 1) {
            __shared__ uint32_t tops[kWarps];
            if (m > 0) __syncthreads();
            if (lane == 0) tops[warp] = top;
            __syncthreads();
            for (int q = 0; q < kw; ++q) top = max(top, tops[q]);        // (the other parts of the row: warps 0 .. kw - 1 have all)
        }
        // the largest goes to [2^14, 2^15); a row of zeros, or with what is not finite, stays as it is
        const int e = (int)(top >> 23) - 127;
        exponent[m] = top != 0 && e < 128 ? 14 - e : 0;
        const float f0 = power_of_two(exponent[m] / 2), f1 = power_of_two(exponent[m] - exponent[m] / 2);
#pragma unroll
        for (int i = 0; i < kSlices; ++i) {
            float sum = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float f[8];
                unpack8(v[i][h], f);
#pragma unroll
                for (int q = 0; q < 8; ++q) f[q] = f[q] * f0 * f1;
                sum += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
                x[m][i][4 * h] = f16_pair(f[0], f[4]);
                x[m][i][4 * h + 1] = f16_pair(f[1] * ODD, f[5] * ODD);
                x[m][i][4 * h + 2] = f16_pair(f[2], f[6]);
                x[m][i][4 * h + 3] = f16_pair(f[3] * ODD, f[7] * ODD);
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            xsum[m][i] = sum * kCodeUnit<EXACT>;
        }
    }

    const auto scales_of = [&](Scales &q, int at_turn, int i) {
        const int group = min((slice0 + i) * kSlice + 16 * lane, p.k - 16) / 64 >> shift;          // (inputs beyond the last meet zeros of x)
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const Q4Matrix &w = r >= OUT ? p.up : p.w;
            const size_t from = (size_t)min(at_turn * OUT + r % OUT, p.n_out - 1) * groups + group;
            q.scale[r] = __ldg(reinterpret_cast<const unsigned short *>(w.scales) + from);
            if (OFFSETS) q.offset[r] = __ldg(reinterpret_cast<const unsigned short *>(w.offsets) + from);
        }
    };
    Scales ahead;
    if (!SCALE_TMA && slices > 0) scales_of(ahead, turn, 0);
    int place = 0, phase = 0;
    bool gone = false;
    for (int round = 0; round < rounds; ++round, turn += step) {
        float acc[kRows][M];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int m = 0; m < M; ++m) acc[r][m] = 0.f;
#pragma unroll
        for (int i = 0; i < kSlices; ++i) {
            if (i >= slices || gone) break;
            Scales cur;
            if (!SCALE_TMA) {
                cur = ahead;
                if (i + 1 < slices) scales_of(ahead, turn, i + 1);
                else if (round + 1 < rounds) scales_of(ahead, turn + step, 0);
            }
            mbar_poll(&full[warp][place], phase, abort);
            if (gone = __any_sync(0xffffffffu, *abort)) break;
            const Stage<MATS> &stage = ring[place];
            const int mine = (((slice0 + i) * (kSlice / 64) >> shift) & 7) + (g >> shift);
#pragma unroll
            for (int r = 0; r < kRows; r += 2) {
                const int r1 = GATED ? r / 2 : r, r2 = GATED ? r1 + OUT : r + 1;         // a pair: two rows, or one of either matrix
                const uint2 qa = stage.code[r1][lane], qb = stage.code[r2][lane];
                float d[M][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t a = h ? qa.y : qa.x, b = h ? qb.y : qb.x;
                    const uint32_t a8 = a >> 8, b8 = b >> 8;
                    constexpr uint32_t HI = 0x00f000f0u, LO = EXACT ? 0x000f000fu : HI;
                    const uint32_t a0 = EXACT ? a : a << 4, b0 = EXACT ? b : b << 4, a4 = EXACT ? a8 : a >> 4, b4 = EXACT ? b8 : b >> 4;
                    const uint32_t v[8] = {code_pair<EXACT>(a0, LO), code_pair<EXACT>(b0, LO), code_pair<EXACT>(a, HI), code_pair<EXACT>(b, HI),
                                           code_pair<EXACT>(a4, LO), code_pair<EXACT>(b4, LO), code_pair<EXACT>(a8, HI), code_pair<EXACT>(b8, HI)};
#pragma unroll
                    for (int m = 0; m < M; ++m) {
                        const uint32_t *xm = &x[m][i][4 * h];
                        if (h == 0) mma_first(d[m], v[0], v[1], v[2], v[3], xm[0], xm[1]);
                        else mma_next(d[m], v[0], v[1], v[2], v[3], xm[0], xm[1]);
                        mma_next(d[m], v[4], v[5], v[6], v[7], xm[2], xm[3]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = e ? r2 : r1;
                    const float s = SCALE_TMA ? __bfloat162float(stage.scale[row / OUT][row % OUT][mine]) : bf16_lo(cur.scale[row]);
                    const float o = !OFFSETS ? -8.f * s : SCALE_TMA ? __bfloat162float(stage.offset[row / OUT][row % OUT][mine]) : bf16_lo(cur.offset[row]);
#pragma unroll
                    for (int m = 0; m < M; ++m) {
                        const float v = g & 1 ? d[m][2 * e + 1] : d[m][2 * e];
                        acc[r + e][m] = fmaf(EXACT ? s * kCodeUnit<EXACT> : s, v, fmaf(o, xsum[m][i], acc[r + e][m]));
                    }
                }
            }
            __syncwarp();                  // the stage has been read by all
            ask(place);
            if (++place == kDeep) place = 0, phase ^= 1;
        }
        // Over the groups: of each group's four lanes one has the diagonal's sum.  Rows 0 .. 3 end in lanes with bit 16 clear, and
        // so on by halves, so that 8 rows take 7 exchanges and the two over t's bits
        float v[M];
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float a[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) a[r] = t == g >> 1 ? acc[r][m] : 0.f;
#pragma unroll
            for (int n = kRows / 2, o = 16; n >= 1; n /= 2, o /= 2) {
                const bool up = lane & o;
#pragma unroll
                for (int r = 0; r < n; ++r) {
                    const float give = up ? a[r] : a[r + n], keep = up ? a[r + n] : a[r];
                    a[r] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
            }
            v[m] = a[0];
            v[m] += __shfl_xor_sync(0xffffffffu, v[m], 1);
            v[m] += __shfl_xor_sync(0xffffffffu, v[m], 2);
        }
        const int r = g;                                    // lane bits 16, 8, 4 are the row's bits 4, 2, 1
        if (kw > 1) {
            // the other parts of the inputs; two buffers in turn, so that one barrier a turn is enough
            if (t == 0) {
#pragma unroll
                for (int m = 0; m < M; ++m) part[buffer][warp][r * M + m] = v[m];
            }
            __syncthreads();
            if (ks == 0) {
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    v[m] = 0.f;
                    for (int q = 0; q < kw; ++q) v[m] += part[buffer][warp + q][r * M + m];
                }
            }
            buffer ^= 1;
            if (ks != 0) continue;
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
            // the scalings undone, by halves of one sign, so that nothing overflows in between that does not in the end
            const int e = (EXACT ? 24 : 20) - exponent[m];
            float y = v[m] * power_of_two(e / 2) * power_of_two(e - e / 2);
            int n = turn * OUT + r;
            if constexpr (GATED) {
                const float z = __shfl_xor_sync(0xffffffffu, y, 4);          // rows 2 i and 2 i + 1: gate and up of output i
                y = ffn_act(y, p.gelu) * z;
                n = turn * OUT + r / 2;
            }
            if (t != 0 || n >= p.n_out || (GATED && r % 2)) continue;
            const size_t to = (size_t)m * p.n_out + n;
            if (p.out_f32) static_cast<float *>(p.out)[to] = y;
            else static_cast<__nv_bfloat16 *>(p.out)[to] = __float2bfloat16_rn(y);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && gave_up) raise_error(err, kErrTimeout);
}

bool scale_tensors(const Q4Problem &p) { return p.k / p.group % 8 == 0; }

// [rows, entries] of bf16, read in boxes of 8 entries.
bool scale_map(CUtensorMap *m, const void *at, uint64_t rows, uint64_t entries, uint32_t box_rows) {
    return box_map(m, at, rows, 2 * entries, 2 * entries, 16, box_rows, false);
}

template <int M, bool GATED>
cudaError_t launch(const Q4Problem &p) {
    int kw = 1;
    const int slices = (p.k + kSlice - 1) / kSlice;
    while (kw * kSlicesOf<M> < slices) kw *= 2;
    // More warps to a row's inputs where the outputs would leave half of the SMs idle (1000 x 2048: 5.2 us with a warp a row, 3.75 with
    // 4; 1000 x 8192: 5.6 with 4, 4.4 with 8; 12352 x 2048, which fills them: 7.3 with one, 8.0 with 2)
    constexpr int OUT = GATED ? kRows / 2 : kRows;
    const long turns = ((long)p.n_out + OUT - 1) / OUT;
    while (kw < kWarps && kw < slices && turns * kw * 2 <= (long)kWarps * multiprocessor_count()) kw *= 2;
    const int each = (slices + kw - 1) / kw;
    const bool tensors = scale_tensors(p);
    VecMaps maps{};
    for (int m = 0; m < (GATED ? 2 : 1); ++m) {
        const Q4Matrix &w = m ? p.up : p.w;
        if (!box_map(&maps.codes[m], w.codes, p.n_out, p.k / 2, p.k / 2, kSlice / 2, OUT, false)) return cudaErrorInvalidValue;
        if (!tensors) continue;
        if (!scale_map(&maps.scales[m], w.scales, p.n_out, p.k / p.group, OUT)) return cudaErrorInvalidValue;
        if (w.offsets && !scale_map(&maps.offsets[m], w.offsets, p.n_out, p.k / p.group, OUT)) return cudaErrorInvalidValue;
    }
    using Fn = void (*)(const Q4Problem, const VecMaps, int, int, unsigned int *);
    static const Fn fns[2][2][2] = {{{q4_vec_kernel<M, GATED, false, false, false>, q4_vec_kernel<M, GATED, false, false, true>},
                                     {q4_vec_kernel<M, GATED, false, true, false>, q4_vec_kernel<M, GATED, false, true, true>}},
                                    {{q4_vec_kernel<M, GATED, true, false, false>, q4_vec_kernel<M, GATED, true, false, true>},
                                     {q4_vec_kernel<M, GATED, true, true, false>, q4_vec_kernel<M, GATED, true, true, true>}}};
    const int offsets = p.w.offsets != nullptr, exact = p.out_f32;
    const Fn fn = fns[offsets][tensors][exact];
    constexpr int smem = kWarps * kDeep * (int)sizeof(Stage<GATED ? 2 : 1>);
    static std::atomic<bool> ready[kMaxDevices][2][2][2];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !ready[dev][offsets][tensors][exact].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) ready[dev][offsets][tensors][exact].store(true, std::memory_order_relaxed);
    }
    const long ctas = kw > 1 ? (turns * kw + kWarps - 1) / kWarps : turns;
    fn<<<(unsigned)min(ctas, 2L * multiprocessor_count()), kThreads, smem, p.stream>>>(p, maps, kw, each, error_word());
    return cudaGetLastError();
}

}  // namespace

bool q4_vec_takes(int rows, int k) { return rows <= 2 && k <= kWarps * kSlice * (rows == 1 ? kSlicesOf<1> : kSlicesOf<2>); }

cudaError_t launch_q4_vec(const Q4Problem &p) {
    if (p.rows == 1) return p.gated ? launch<1, true>(p) : launch<1, false>(p);
    return p.gated ? launch<2, true>(p) : launch<2, false>(p);
}

}  // namespace gdn
