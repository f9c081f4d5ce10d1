// gdn_q4_linear and gdn_q4_gated: products of activations with weights of 4 bits,
//     y[m, n] = sum_G ( s[n, G] sum_{i in G} c[n, i] x[m, i]  +  o[n, G] sum_{i in G} x[m, i] ),
// G over groups of 64 or 128 inputs; o = -8 s where the matrix has no offsets.  This is the kernel for small products and for fp32
// outputs; one or two rows go to q4_vec.cu, large products to q4_tc.cu.
//
// The inner sums go to the tensor cores (mma.sync, 16 weight rows by 8 rows of x by 16 inputs): a code is an integer below 16,
// exact in bf16, so the products are exact and the sums fp32, and scale and offset meet them once a group instead of once a
// weight.
//
// Codes and x come by TMA, stages of 16 w weight rows (w = 1, 2, 4 or 8) and all rows of x by 256 inputs, which one thread asks for
// several stages ahead, across tiles: what reads memory is never waiting for what computes.  Eight warps compute, w along the rows by
// 8 / w along the inputs; a ninth asks; a tenth sums x over blocks of 64 inputs.  Partial sums meet in shared memory in a fixed order; where there are few tiles, those of up to 8
// CTAs of a cluster that share a tile's inputs (608 x 7424, 31 rows, fp32: 25.7 to 9.9 us).
//
// Bound by latencies, of barriers above all (a wait that finds its phase complete takes some 250 cycles, and a stage has three), not by
// the codes: 12352 x 2048 with 3 rows 12.7 us, 1.1 TB/s; with 16 and fp32 outputs 15.4.  fp32 outputs of many rows, which have to keep
// groups apart, pay for every 32 rows again: 4096 x 4096 with 33 rows 21 us, 512 rows 109 (158 TFLOP/s); 131071 x 2048 with 33 rows 220.
//
// A fragment's order of inputs is free as long as both operands keep it: lane (g, t) takes inputs 16 t .. 16 t + 15 of a block of 64,
// for weight rows g and g + 8 (of two matrices, rows g of each) and for row g of x: 8 bytes of codes and 32 bytes of x in a row.
#include "layer_ops.cuh"
#include "sm100.cuh"

namespace gdn {

namespace {

using namespace sm100;

constexpr int kWarps = 8, kThreads = 32 * (kWarps + 2);
constexpr int kChunkIn = 256;
constexpr int kMaxStages = 6;

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The products enter their sums as 2^-10 of themselves, so that a group's sum of codes times x (below 2^10 of x's largest) and its sum
// of x stay in range for every x; the outputs get it back.
constexpr float kShrunk = 0x1p-10f, kGrown = 0x1p10f;

// The eight codes of a word as four bf16 pairs of neighbours, times 2^-10.  Under the exponent of 2^-3 a code is 2^-3 + c 2^-10 exactly.
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t (&v)[4]) {
    const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
    const uint32_t lo = __byte_perm(even, odd, 0x5140), hi = __byte_perm(even, odd, 0x7362);
    v[0] = __byte_perm(lo, 0x3e3e3e3eu, 0x4140);
    v[1] = __byte_perm(lo, 0x3e3e3e3eu, 0x4342);
    v[2] = __byte_perm(hi, 0x3e3e3e3eu, 0x4140);
    v[3] = __byte_perm(hi, 0x3e3e3e3eu, 0x4342);
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("sub.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(v[i]), "r"(0x3e003e00u));
}

struct FewPlan {
    int w, m_blocks, row_tiles, stages;
    int cluster, slice;                   // CTAs that share a tile's inputs (then each has one tile), and a CTA's chunks of them
    int codes_bytes;                      // of a stage
};

struct FewBars {
    uint64_t full[kMaxStages], summed[kMaxStages], empty[kMaxStages], joined[2];
    int abort;
};

template <int NT, int FIT, bool GATED, bool OFFSETS>
__global__ void __launch_bounds__(kThreads, FIT)
q4_few_kernel(const __grid_constant__ Q4Problem p, const __grid_constant__ FewPlan l, const __grid_constant__ CUtensorMap code_map,
              const __grid_constant__ CUtensorMap up_map, const __grid_constant__ CUtensorMap x_map, unsigned int *err) {
    constexpr int COLS = 8 * NT, X_BOX = COLS * 128, X_BYTES = 4 * X_BOX;
    extern __shared__ unsigned char raw[];
    __shared__ FewBars sm;
    unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int stage_bytes = l.codes_bytes + X_BYTES;
    float *sums = reinterpret_cast<float *>(base + (size_t)l.stages * stage_bytes);      // [stage][4][COLS]
    float *part = sums + l.stages * 4 * COLS;                                            // [2][8 / w][COLS][16 w + 4]
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int w = l.w, kw = kWarps / w, rows = 16 * w, out_rows = GATED ? rows / 2 : rows;
    const int units = l.row_tiles * l.m_blocks, rank = l.cluster > 1 ? (int)cluster_ctarank() : 0;
    const int first = blockIdx.x / l.cluster, step = gridDim.x / l.cluster;
    const int c0 = rank * l.slice, c1 = min(c0 + l.slice, (p.k + kChunkIn - 1) / kChunkIn);
    volatile int *abort = &sm.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < l.stages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.summed[i], 1);
            mbar_init(&sm.empty[i], kWarps + 1);
        }
        mbar_init(&sm.joined[0], kWarps);
        mbar_init(&sm.joined[1], kWarps);
        sm.abort = 0;
        fence_mbar_init();
    }
    __syncthreads();

    // Output i of a tile, neighbours for neighbouring threads: where its sums are in a part, and its end
    const int stride = rows + 4;
    const auto place = [&](int i) {
        const int r = i & (out_rows - 1);
        return i / out_rows * stride + (GATED ? r / 8 * 16 + r % 8 : r);
    };
    const auto write = [&](int n0, int m0, int i, float y, float z) {
        const int n = n0 + (i & (out_rows - 1)), m = m0 + i / out_rows;
        y *= kGrown, z *= kGrown;
        if (GATED) y = ffn_act(y, p.gelu) * z;
        if (n >= p.n_out) return;
        const size_t to = (size_t)m * p.n_out + n;
        if (p.out_f32) static_cast<float *>(p.out)[to] = y;
        else static_cast<__nv_bfloat16 *>(p.out)[to] = __float2bfloat16_rn(y);
    };

    int s = 0, phase = 0;
    const auto advance = [&] { if (++s == l.stages) s = 0, phase ^= 1; };
    if (warp == kWarps) {
        if (elect_one()) {
            for (int u = first; u < units && !*abort; u += step) {
                const int n0 = u / l.m_blocks * out_rows, m0 = u % l.m_blocks * COLS;
                for (int c = c0; c < c1; ++c) {
                    mbar_poll(&sm.empty[s], phase ^ 1, abort);
                    if (*abort) break;
                    unsigned char *to = base + (size_t)s * stage_bytes;
                    mbar_arrive_expect_tx(&sm.full[s], stage_bytes);
                    tma_load_2d(to, &code_map, &sm.full[s], c * (kChunkIn / 2), n0);
                    if (GATED) tma_load_2d(to + l.codes_bytes / 2, &up_map, &sm.full[s], c * (kChunkIn / 2), n0);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        tma_load_2d(to + l.codes_bytes + j * X_BOX, &x_map, &sm.full[s], 2 * (c * kChunkIn + 64 * j), m0);    // (the map counts bytes)
                    advance();
                }
            }
        }
    } else if (warp == kWarps + 1) {
        // sums of x over blocks of 64 inputs: a lane a block of a row, the four blocks at different banks
        const int j = lane % 4;
        bool gone = false;
        for (int u = first; u < units && !gone; u += step)
            for (int c = c0; c < c1; ++c) {
                mbar_poll(&sm.full[s], phase, abort);
                if (gone = __any_sync(0xffffffffu, *abort)) break;
                const unsigned char *x = base + (size_t)s * stage_bytes + l.codes_bytes + j * X_BOX;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int m = lane / 4 + 8 * i;
                    float sum = 0.f;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        float f[8];
                        unpack8(*reinterpret_cast<const uint4 *>(x + m * 128 + ((((q + 2 * j) & 7) ^ (m & 7)) << 4)), f);
                        float a = f[0] * kShrunk, b = f[1] * kShrunk;
#pragma unroll
                        for (int e = 2; e < 8; e += 2) a = fmaf(f[e], kShrunk, a), b = fmaf(f[e + 1], kShrunk, b);
                        sum += a + b;
                    }
                    sums[(s * 4 + j) * COLS + m] = sum;
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sm.summed[s]);
                    mbar_arrive(&sm.empty[s]);
                }
                advance();
            }
    } else {
        const int g = lane / 4, t = lane % 4, rg = warp % w, ks = warp / w;
        const int groups = p.k / p.group, count = kChunkIn / p.group;
        const bool vector = groups % count == 0;
        const Q4Matrix &second = GATED ? p.up : p.w;
        // where this lane's codes are in a stage: rows g and g + 8 of its 16, or row g of its 8 of either matrix
        const int line0 = (GATED ? 8 * rg + g : 16 * rg + g) * 128, line1 = GATED ? l.codes_bytes / 2 + line0 : line0 + 8 * 128;
        size_t r0 = 0, r1 = 0;
        ChunkScales next0, next1;
        const auto ask = [&](int u, int c) {      // the scales of unit u's chunk c (a row beyond the matrix repeats its last one)
            if (c == c0) {
                const int n = u / l.m_blocks * out_rows + (GATED ? 8 : 16) * rg + g;
                r0 = min(n, p.n_out - 1);
                r1 = GATED ? r0 : min(n + 8, p.n_out - 1);
            }
            next0 = chunk_scales<OFFSETS>(p.w, r0, groups, c * count, count, vector);
            next1 = chunk_scales<OFFSETS>(second, r1, groups, c * count, count, vector);
        };
        int buffer = 0, joins = 0;
        bool gone = false;
        if (first < units) ask(first, c0);
        for (int u = first; u < units && !gone; u += step) {
            float acc[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
            for (int c = c0; c < c1; ++c) {
                const ChunkScales cur0 = next0, cur1 = next1;
                if (c + 1 < c1) ask(u, c + 1);
                else if (u + step < units) ask(u + step, c0);
                mbar_poll(&sm.full[s], phase, abort);
                mbar_poll(&sm.summed[s], phase, abort);
                if (gone = __any_sync(0xffffffffu, *abort)) break;
                const unsigned char *stage = base + (size_t)s * stage_bytes;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (((4 * c + j) & (kw - 1)) != ks) continue;
                    const int at = (((2 * j + t / 2) ^ g) << 4) + 8 * (t & 1);
                    const uint2 q0 = *reinterpret_cast<const uint2 *>(stage + line0 + at), q1 = *reinterpret_cast<const uint2 *>(stage + line1 + at);
                    uint32_t v0[4], v1[4], a[4][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        code_pairs(h ? q0.y : q0.x, v0);
                        code_pairs(h ? q1.y : q1.x, v1);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            a[2 * h + i][0] = v0[2 * i];
                            a[2 * h + i][1] = v1[2 * i];
                            a[2 * h + i][2] = v0[2 * i + 1];
                            a[2 * h + i][3] = v1[2 * i + 1];
                        }
                    }
                    const int which = count == 4 ? j : j / 2;
                    const float s0 = nth_bf16(cur0.s, which), s1 = nth_bf16(cur1.s, which);
                    const float o0 = OFFSETS ? nth_bf16(cur0.o, which) : -8.f * s0, o1 = OFFSETS ? nth_bf16(cur1.o, which) : -8.f * s1;
                    const unsigned char *x = stage + l.codes_bytes + j * X_BOX + g * 128;
                    const float *xsum = sums + (s * 4 + j) * COLS + 2 * t;
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const uint4 b0 = *reinterpret_cast<const uint4 *>(x + i * 1024 + (((2 * t) ^ g) << 4));
                        const uint4 b1 = *reinterpret_cast<const uint4 *>(x + i * 1024 + (((2 * t + 1) ^ g) << 4));
                        float d[4] = {0.f, 0.f, 0.f, 0.f};
                        mma_16816(d, a[0], b0.x, b0.y);
                        mma_16816(d, a[1], b0.z, b0.w);
                        mma_16816(d, a[2], b1.x, b1.y);
                        mma_16816(d, a[3], b1.z, b1.w);
                        const float2 xs = *reinterpret_cast<const float2 *>(xsum + 8 * i);
                        acc[i][0] = fmaf(s0, d[0], fmaf(o0, xs.x, acc[i][0]));
                        acc[i][1] = fmaf(s0, d[1], fmaf(o0, xs.y, acc[i][1]));
                        acc[i][2] = fmaf(s1, d[2], fmaf(o1, xs.x, acc[i][2]));
                        acc[i][3] = fmaf(s1, d[3], fmaf(o1, xs.y, acc[i][3]));
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.empty[s]);
                advance();
            }
            if (gone) break;
            // The warps' sums meet.  Two buffers in turn: whoever writes one again has waited for all of the other, whose writers had
            // read this one
            float *mine = part + (size_t)buffer * kw * COLS * stride;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mine[(ks * COLS + 8 * i + 2 * t + (e & 1)) * stride + 16 * rg + g + (e & 2) * 4] = acc[i][e];
            if (l.cluster > 1) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.joined[buffer]);
            mbar_poll(&sm.joined[buffer], joins >> 1 & 1, abort);
            if (gone = __any_sync(0xffffffffu, *abort)) break;
            ++joins;
            const int n0 = u / l.m_blocks * out_rows, m0 = u % l.m_blocks * COLS, m_rows = min(COLS, p.rows - m0);
            for (int i = threadIdx.x; i < out_rows * m_rows; i += 32 * kWarps) {
                const float *at = mine + place(i);
                float y = 0.f, z = 0.f;
                for (int k = 0; k < kw; ++k) {
                    y += at[k * COLS * stride];
                    if (GATED) z += at[k * COLS * stride + 8];
                }
                write(n0, m0, i, y, z);
            }
            buffer ^= 1;
        }
    }
    if (l.cluster > 1) {
        __syncwarp();
        cluster_sync();
        if (warp < kWarps && !*abort) {
            const int n0 = first / l.m_blocks * out_rows, m0 = first % l.m_blocks * COLS, m_rows = min(COLS, p.rows - m0);
            for (int i = threadIdx.x + 32 * kWarps * rank; i < out_rows * m_rows; i += 32 * kWarps * l.cluster) {
                const float *at = part + place(i);
                float y = 0.f, z = 0.f;
                for (int k = 0; k < kw; ++k) {
                    float ys[8], zs[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        ys[q] = q < l.cluster ? ld_dsmem_f32(at + k * COLS * stride, q) : 0.f;
                        if (GATED) zs[q] = q < l.cluster ? ld_dsmem_f32(at + k * COLS * stride + 8, q) : 0.f;
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        y += ys[q];
                        if (GATED) z += zs[q];
                    }
                }
                write(n0, m0, i, y, z);
            }
        }
        cluster_sync();                    // a CTA's sums are read before it is gone
    }
    __syncthreads();
    if (threadIdx.x == 0 && sm.abort) raise_error(err, kErrTimeout);
}

size_t few_shared(int cols, const FewPlan &l) {
    const size_t stage = l.codes_bytes + (size_t)cols * 512;
    return 1024 + l.stages * (stage + 16 * cols) + (size_t)2 * (kWarps / l.w) * cols * (16 * l.w + 4) * 4;
}

template <int NT, int FIT, bool GATED>
cudaError_t launch(const Q4Problem &p) {
    constexpr int COLS = 8 * NT;
    const int sms = multiprocessor_count();
    FewPlan l{};
    l.m_blocks = (p.rows + COLS - 1) / COLS;
    // Rows of a tile, and CTAs that share its inputs where that fills the GPU: as few rounds as possible of tiles that cost their rows
    // and a little, for each chunk of inputs.  A join costs as much as four such units.
    const int chunks = (p.k + kChunkIn - 1) / kChunkIn;
    double least = 1e300;
    for (int w = 8; w >= 1; w /= 2) {
        const long tiles = (p.n_out + (GATED ? 8 : 16) * w - 1) / ((GATED ? 8 : 16) * w);
        for (int cluster = 1; cluster <= 8 && cluster <= chunks; cluster *= 2) {
            const int slice = (chunks + cluster - 1) / cluster;
            const double ctas = (double)tiles * l.m_blocks * cluster;
            if (cluster > 1 && (ctas > 0.85 * sms * FIT || (long)slice * (cluster - 1) >= chunks)) continue;
            const double cost = ceil(ctas / (sms * FIT)) * (w + 0.7) * slice + (cluster > 1 ? 4 : 0);
            if (cost < least) least = cost, l.w = w, l.row_tiles = (int)tiles, l.cluster = cluster, l.slice = slice;
        }
    }
    l.codes_bytes = 16 * l.w * 128;
    constexpr size_t kShared = (FIT == 2 ? 112 : 226) * 1024 - sizeof(FewBars);
    l.stages = kMaxStages;
    while (l.stages > 2 && few_shared(COLS, l) > kShared) --l.stages;
    const int box_rows = (GATED ? 8 : 16) * l.w;
    CUtensorMap codes, up, x;
    if (!byte_map(&codes, p.w.codes, p.n_out, p.k / 2, p.k / 2, box_rows) || !byte_map(&x, p.x, p.rows, 2 * (uint64_t)p.k, 2 * p.x_stride, COLS))
        return cudaErrorInvalidValue;
    if (!GATED) up = codes;
    else if (!byte_map(&up, p.up.codes, p.n_out, p.k / 2, p.k / 2, box_rows)) return cudaErrorInvalidValue;

    using Fn = void (*)(const Q4Problem, const FewPlan, const CUtensorMap, const CUtensorMap, const CUtensorMap, unsigned int *);
    const int offsets = p.w.offsets != nullptr;
    const Fn fn = offsets ? q4_few_kernel<NT, FIT, GATED, true> : q4_few_kernel<NT, FIT, GATED, false>;
    static std::atomic<bool> ready[kMaxDevices][2];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !ready[dev][offsets].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kShared);
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) ready[dev][offsets].store(true, std::memory_order_relaxed);
    }
    const long units = (long)l.row_tiles * l.m_blocks;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(l.cluster > 1 ? units * l.cluster : min(units, (long)sms * FIT)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = few_shared(COLS, l);
    cfg.stream = p.stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = l.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = l.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, p, l, codes, up, x, error_word());
}

// A CTA takes 8, 16 or 32 rows of x.  With 32 rows two CTAs fit on an SM at 96 registers a thread instead of 168, which pays where there
// is work for them: 4096 x 4096, 512 rows, 109 us instead of 154, 15540 x 3968, 143 rows, 155 instead of 176; but 12352 x 1344, 59 rows, 38.8
// instead of 36.3, and 4096 x 4096, 24 rows, 12.5 and 12.3.
template <bool GATED>
cudaError_t by_rows(const Q4Problem &p) {
    if (p.rows > 16) return (long)p.rows * p.n_out >= 1l << 20 ? launch<4, 2, GATED>(p) : launch<4, 1, GATED>(p);
    if (p.rows > 8) return launch<2, 2, GATED>(p);
    return launch<1, 2, GATED>(p);
}

}  // namespace

// bf16 outputs: the kernel that multiplies on tcgen05, or the one above for small products.  The one above unpacks for every 8 to 32
// rows; the other takes 7 us for nothing.  With offsets in groups of 64:
//     n_out x k        above                     on tcgen05
//     300 x 512        3, 16 rows  3.9,  4.2 us   7.7,  8.0 us
//     1000 x 8192                  7.7,  9.4     12.0, 12.4
//     4096 x 4096                  8.0,  9.5     12.0, 12.6
//     12000 x 4096                17.8, 22.8     24.7, 24.9
//     12352 x 2048                12.7, 15.3     14.1, 14.3
//     131071 x 2048               73.7, 95.2     66.0, 67.0
//     2 x 14000 x 2048            25.9, 30.5     20.5, 21.1
//     400 x 512        100 rows    5.9            8.3
//     200 x 512        500 rows    6.7           10.2
//     266 x 8192       67 rows    10.0           13.1
//     1208 x 1984      318 rows   33.3           13.7
//     1000 x 2048      64 rows    12.9           10.2
static bool on_tcgen05(int rows, int n_out, int k, int matrices, int out_f32) {
    if (rows <= 2 || out_f32) return false;
    if (rows <= 16) return (double)n_out * matrices * k >= (rows > 8 ? 20e6 : 50e6);
    return (long)rows * n_out >= (k < 1536 ? 1l << 17 : 3l << 13) || (k >= 1536 && n_out > 512);
}

// (of either call, that with one matrix and that with two)
size_t q4_workspace_bytes(int rows, int n_out, int k, int group, int out_f32) {
    return on_tcgen05(rows, n_out, k, 2, out_f32) ? q4_tc_workspace_bytes(rows, k, group) : 0;
}

cudaError_t launch_q4(const Q4Problem &p) {
    if (q4_vec_takes(p.rows, p.k)) return launch_q4_vec(p);
    if (on_tcgen05(p.rows, p.n_out, p.k, p.gated ? 2 : 1, p.out_f32)) return launch_q4_tc(p);
    return p.gated ? by_rows<true>(p) : by_rows<false>(p);
}

}  // namespace gdn
