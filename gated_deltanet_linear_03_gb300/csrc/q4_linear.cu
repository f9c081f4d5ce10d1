// gdn_q4_linear and gdn_q4_gated: products of activations with weights of 4 bits,
//     y[m, n] = sum_G ( s[n, G] sum_{i in G} c[n, i] x[m, i]  +  o[n, G] sum_{i in G} x[m, i] ),
// G over groups of 64 or 128 inputs; o = -8 s where the matrix has no offsets.
//
// The inner sums go to the tensor cores (mma.sync, 16 weight rows by 8 rows of x by 16 inputs): a code is an integer below 16,
// exact in bf16, so the products are exact and the sums fp32, and scale and offset meet them once a group instead of once a
// weight.  Few rows are bound by reading the codes, where this takes the fewest instructions a weight; a matrix
// instruction of the tcgen05 kind would have to be fed from shared memory or TMEM, by the same registers.
//
// A fragment's order of inputs is free as long as both operands keep it.  Lane (g, t) of a warp reads the 16 codes
// 16 t .. 16 t + 15 of a block of 64 inputs for weight rows g and g + 8: 8 bytes each, whole 32-byte sectors of a row, as they
// lie in memory.  A code word's pairs (i, i + 4) come out of one AND/OR each, and x lies in shared memory with each 8 inputs in
// the order 0 4 1 5 2 6 3 7, so a lane's x is 32 consecutive bytes.
//
// The 8 warps of a CTA are WN along the rows (16 each) by 8 / WN along the inputs; CTAs of a cluster share the inputs further, and
// each CTA keeps its slice of x in shared memory for all the tiles of rows that it comes to.  Partial sums meet in shared
// memory, across a cluster through distributed shared memory: the order of the sum is fixed.
#include "layer_ops.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kBlock = 64;            // inputs of one step of a warp
constexpr int kAhead = 4;             // blocks whose codes are asked for at once

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes i and i + 4 (i = SHIFT / 4) of a word as a bf16 pair: under the exponent of 128 a code is 128 + c exactly.
template <int SHIFT>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    const uint32_t biased = ((w >> SHIFT) & 0x000f000fu) | 0x43004300u;
    uint32_t r;
    asm("sub.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(biased), "r"(0x43004300u));
    return r;
}

__device__ __forceinline__ float bf16_value(__nv_bfloat16 v) { return __bfloat162float(v); }

struct Q4Launch {
    int slice;                // inputs of one CTA, a multiple of the group
    int cluster;              // CTAs that share the inputs
    int row_tiles, m_blocks;
};

// What a warp reads for kAhead blocks: codes of two rows, their scales and offsets.
template <bool OFFSETS>
struct Piece {
    uint2 code[kAhead][2];
    __nv_bfloat16 scale[kAhead][2], offset[OFFSETS ? kAhead : 1][2];
};

template <int NT, int WN, bool GATED, bool OFFSETS>
__global__ void __launch_bounds__(kThreads, NT <= 2 ? 2 : 1) q4_kernel(const __grid_constant__ Q4Problem p, const Q4Launch l) {
    constexpr int WK = kWarps / WN, COLS = 8 * NT, ROWS = 16 * WN, OUT_ROWS = GATED ? ROWS / 2 : ROWS;
    extern __shared__ __align__(16) unsigned char smem[];
    const int rank = l.cluster > 1 ? (int)sm100::cluster_ctarank() : 0;
    const int k0 = rank * l.slice, slice = min(l.slice, p.k - k0), blocks = slice / kBlock;     // (the last slice may be shorter)
    const int x_row = l.slice * 2 + 16;                      // bytes; the 16 keep lanes of different rows on different banks
    float *sums = reinterpret_cast<float *>(smem);           // [slice / 64][COLS]
    unsigned char *xs = smem + (size_t)(l.slice / kBlock) * COLS * 4;
    float *part = reinterpret_cast<float *>(xs + (size_t)COLS * x_row);     // [WK][ROWS][COLS]
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int wn = warp / WK, wk = warp % WK;
    const int work = blockIdx.x / l.cluster, workers = gridDim.x / l.cluster;
    const int m0 = (work % l.m_blocks) * COLS, m_rows = min(COLS, p.rows - m0);

    // this CTA's slice of x, and its sums over blocks of 64: 8 lanes a block
    {
        const int pieces = slice / 8;
        for (int i = threadIdx.x; i < COLS * pieces; i += kThreads) {     // pieces is a multiple of 8: 8 lanes stay together
            const int m = i / pieces, c = i % pieces;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (m < m_rows) v = *reinterpret_cast<const uint4 *>(p.x + (long long)(m0 + m) * p.x_stride + k0 + 8 * c);
            float f[8];
            unpack8(v, f);
            float s = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
            const unsigned live = __activemask();
#pragma unroll
            for (int o = 4; o >= 1; o >>= 1) s += __shfl_xor_sync(live, s, o);
            if (c % 8 == 0) sums[(c / 8) * COLS + m] = s;
            uint4 q;
            q.x = __byte_perm(v.x, v.z, 0x5410);        // 0 4
            q.y = __byte_perm(v.x, v.z, 0x7632);        // 1 5
            q.z = __byte_perm(v.y, v.w, 0x5410);        // 2 6
            q.w = __byte_perm(v.y, v.w, 0x7632);        // 3 7
            *reinterpret_cast<uint4 *>(xs + (size_t)m * x_row + 16 * c) = q;
        }
    }
    __syncthreads();

    const int per = (blocks + WK - 1) / WK, b_lo = min(wk * per, blocks), b_hi = min(b_lo + per, blocks);
    const int groups = p.k / p.group, shift = p.group == 128 ? 1 : 0;
    const unsigned char *x_lane = xs + (size_t)g * x_row + 32 * t;
    const int step = workers / l.m_blocks;
    for (int tile = work / l.m_blocks; tile < l.row_tiles; tile += step) {
        // this lane's two weight rows (a row beyond the matrix repeats its last one, and is not written)
        const int n0 = tile * OUT_ROWS + wn * (GATED ? 8 : 16) + g;
        const int r0 = min(n0, p.n_out - 1), r1 = GATED ? r0 : min(n0 + 8, p.n_out - 1);
        const Q4Matrix &second = GATED ? p.up : p.w;
        const uint8_t *code0 = p.w.codes + (size_t)r0 * (p.k / 2) + k0 / 2 + 8 * t;
        const uint8_t *code1 = second.codes + (size_t)r1 * (p.k / 2) + k0 / 2 + 8 * t;
        const size_t at0 = (size_t)r0 * groups + (k0 / kBlock >> shift), at1 = (size_t)r1 * groups + (k0 / kBlock >> shift);
        float acc[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;

        auto load = [&](Piece<OFFSETS> &q, int b) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int at = min(b + i, b_hi - 1);
                q.code[i][0] = __ldg(reinterpret_cast<const uint2 *>(code0 + (size_t)at * 32));
                q.code[i][1] = __ldg(reinterpret_cast<const uint2 *>(code1 + (size_t)at * 32));
                q.scale[i][0] = p.w.scales[at0 + (at >> shift)];
                q.scale[i][1] = second.scales[at1 + (at >> shift)];
                if constexpr (OFFSETS) {
                    q.offset[i][0] = p.w.offsets[at0 + (at >> shift)];
                    q.offset[i][1] = second.offsets[at1 + (at >> shift)];
                }
            }
        };
        Piece<OFFSETS> next;
        if (b_lo < b_hi) load(next, b_lo);
        for (int b = b_lo; b < b_hi; b += kAhead) {
            const Piece<OFFSETS> cur = next;
            if (b + kAhead < b_hi) load(next, b + kAhead);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (b + i >= b_hi) break;
                uint32_t a[4][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t w0 = h ? cur.code[i][0].y : cur.code[i][0].x, w1 = h ? cur.code[i][1].y : cur.code[i][1].x;
                    a[2 * h][0] = code_pair<0>(w0);
                    a[2 * h][1] = code_pair<0>(w1);
                    a[2 * h][2] = code_pair<4>(w0);
                    a[2 * h][3] = code_pair<4>(w1);
                    a[2 * h + 1][0] = code_pair<8>(w0);
                    a[2 * h + 1][1] = code_pair<8>(w1);
                    a[2 * h + 1][2] = code_pair<12>(w0);
                    a[2 * h + 1][3] = code_pair<12>(w1);
                }
                const float s0 = bf16_value(cur.scale[i][0]), s1 = bf16_value(cur.scale[i][1]);
                const float o0 = OFFSETS ? bf16_value(cur.offset[OFFSETS ? i : 0][0]) : -8.f * s0;
                const float o1 = OFFSETS ? bf16_value(cur.offset[OFFSETS ? i : 0][1]) : -8.f * s1;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint4 *xb = reinterpret_cast<const uint4 *>(x_lane + (size_t)(8 * j) * x_row + (size_t)(b + i) * 128);
                    const uint4 u = xb[0], v = xb[1];
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_16816(d, a[0], u.x, u.y);
                    mma_16816(d, a[1], u.z, u.w);
                    mma_16816(d, a[2], v.x, v.y);
                    mma_16816(d, a[3], v.z, v.w);
                    const float2 xsum = *reinterpret_cast<const float2 *>(sums + (b + i) * COLS + 8 * j + 2 * t);
                    acc[j][0] = fmaf(s0, d[0], fmaf(o0, xsum.x, acc[j][0]));
                    acc[j][1] = fmaf(s0, d[1], fmaf(o0, xsum.y, acc[j][1]));
                    acc[j][2] = fmaf(s1, d[2], fmaf(o1, xsum.x, acc[j][2]));
                    acc[j][3] = fmaf(s1, d[3], fmaf(o1, xsum.y, acc[j][3]));
                }
            }
        }
        // partial sums of [WK][rows][columns], joined in the same order every time
        float *mine = part + ((size_t)wk * ROWS + wn * 16) * COLS;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            *reinterpret_cast<float2 *>(mine + g * COLS + 8 * j + 2 * t) = make_float2(acc[j][0], acc[j][1]);
            *reinterpret_cast<float2 *>(mine + (g + 8) * COLS + 8 * j + 2 * t) = make_float2(acc[j][2], acc[j][3]);
        }
        if (l.cluster > 1) sm100::cluster_sync();
        else __syncthreads();
        const int elements = OUT_ROWS * m_rows, share = (elements + l.cluster - 1) / l.cluster;
        for (int i = rank * share + threadIdx.x; i < min((rank + 1) * share, elements); i += kThreads) {
            const int r = i % OUT_ROWS, m = i / OUT_ROWS;            // neighbours write neighbouring outputs
            const int row = GATED ? r / 8 * 16 + r % 8 : r;
            float y = 0.f, z = 0.f;
            for (int q = 0; q < l.cluster; ++q)
#pragma unroll
                for (int w = 0; w < WK; ++w) {
                    const float *from = part + ((size_t)w * ROWS + row) * COLS + m;
                    y += l.cluster > 1 ? sm100::ld_dsmem_f32(from, q) : *from;
                    if constexpr (GATED) z += l.cluster > 1 ? sm100::ld_dsmem_f32(from + 8 * COLS, q) : from[8 * COLS];
                }
            if constexpr (GATED) y = ffn_act(y, p.gelu) * z;
            const int n = tile * OUT_ROWS + r;
            if (n >= p.n_out) continue;
            const size_t at = (size_t)(m0 + m) * p.n_out + n;
            if (p.out_f32) static_cast<float *>(p.out)[at] = y;
            else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(y);
        }
        if (l.cluster > 1) sm100::cluster_sync();      // the sums are read before they are overwritten, or their CTA is gone
        else __syncthreads();
    }
}

constexpr int kMaxCluster = 8;
constexpr size_t kMaxShared = 220 * 1024;

// Inputs of a CTA are a multiple of 128: of either group, and whole lines of a weight row.
int units_of(int k) { return (k + 127) / 128; }

template <int NT, int WN>
size_t shared_bytes(int k, int cluster) {
    constexpr int COLS = 8 * NT;
    const size_t slice = (size_t)(units_of(k) + cluster - 1) / cluster * 128;
    return slice / kBlock * COLS * 4 + COLS * (slice * 2 + 16) + (size_t)(kWarps / WN) * 16 * WN * COLS * 4;
}

template <int NT, int WN, bool GATED>
cudaError_t launch(const Q4Problem &p) {
    constexpr int COLS = 8 * NT, ROWS = 16 * WN, OUT_ROWS = GATED ? ROWS / 2 : ROWS;
    Q4Launch l;
    l.row_tiles = (p.n_out + OUT_ROWS - 1) / OUT_ROWS;
    l.m_blocks = (p.rows + COLS - 1) / COLS;
    const int sms = multiprocessor_count();
    // CTAs of a cluster: enough that x fits into shared memory, and that there is a CTA for every SM
    const int units = units_of(p.k);
    l.cluster = 1;
    while (l.cluster < kMaxCluster && (shared_bytes<NT, WN>(p.k, l.cluster) > 100 * 1024 || (long)l.row_tiles * l.m_blocks * l.cluster < sms) &&
           units >= 4 * l.cluster) l.cluster *= 2;
    while ((units + l.cluster - 1) / l.cluster * (l.cluster - 1) >= units) l.cluster /= 2;     // every CTA has inputs
    l.slice = (units + l.cluster - 1) / l.cluster * 128;
    const size_t smem = shared_bytes<NT, WN>(p.k, l.cluster);
    using Fn = void (*)(const Q4Problem, const Q4Launch);
    const Fn fn = p.w.offsets ? (Fn)q4_kernel<NT, WN, GATED, true> : (Fn)q4_kernel<NT, WN, GATED, false>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int fit = smem <= 100 * 1024 && NT <= 2 ? 2 : 1;
    // clusters that stay: as many as fit, the same number of tiles each as far as that goes
    long workers = (long)sms * fit / l.cluster / l.m_blocks;
    if (workers < 1) workers = 1;
    const long rounds = (l.row_tiles + workers - 1) / workers;
    workers = (l.row_tiles + rounds - 1) / rounds;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(workers * l.m_blocks * l.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = p.stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = l.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = l.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, p, l);
}

// A CTA takes 8, 16, 32 or 64 rows of x, as many as there are and as its shared memory holds of them.
template <int NT, int WN>
bool fits(const Q4Problem &p) { return shared_bytes<NT, WN>(p.k, kMaxCluster) <= kMaxShared; }

template <bool GATED>
cudaError_t by_rows(const Q4Problem &p) {
    if (p.rows > 32 && fits<8, 8>(p)) return launch<8, 8, GATED>(p);
    if (p.rows > 16 && fits<4, 4>(p)) return launch<4, 4, GATED>(p);
    if (p.rows > 8 && fits<2, 2>(p)) return launch<2, 2, GATED>(p);
    return launch<1, 1, GATED>(p);
}

}  // namespace

// Many rows and bf16 outputs: the kernel that multiplies on tcgen05, whose weights are rounded to fp16.
static bool many_rows(int rows, int out_f32) { return rows > 16 && !out_f32; }

size_t q4_workspace_bytes(int rows, int n_out, int k, int out_f32) { return many_rows(rows, out_f32) ? q4_tc_workspace_bytes(rows, k) : 0; }

cudaError_t launch_q4(const Q4Problem &p) {
    if (many_rows(p.rows, p.out_f32)) return launch_q4_tc(p);
    return p.gated ? by_rows<true>(p) : by_rows<false>(p);
}

}  // namespace gdn
