// gdn_block_norm: the norm after a block, its gate and scale, the residual sum, the norm before the next block.
//
//     y = x rsqrt(mean(x^2) + eps) w_post,   y *= act(gate),   r' = r + s y,   h = r' rsqrt(mean(r'^2) + eps) w_pre
//
// A CTA carries rows one after another, one at a time in registers (pieces of 8 elements, C of them a thread), so x,
// gate and residual are read once and r' and h written once; the two sums of squares are CTA reductions in fp32.  The
// next row's pieces are asked for before this row's sums are formed, and the weights stay in registers: with a row a
// CTA the weights came from L1 for every row, more bytes than the row itself.  Bound by memory: 16383 rows of 2048 with
// gate and fp32 residual, 470 MB, in 77 us = 6.1 TB/s, 0.90 of a copy's rate; one row takes 2.6 us, a launch and its latencies.
#include "kv_cache.cuh"

namespace gdn {
namespace {

// Sum over the CTA; `part` is one float per warp, a different one for each of the two sums.
__device__ __forceinline__ float cta_sum(float v, float *part) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warps = blockDim.x / 32;
    if (warps == 1) return v;
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < warps; ++w) v += part[w];
    return v;
}

// The pieces of one row as they lie in memory.
template <int C, bool RES32>
struct RowPieces {
    uint4 x[C], gate[C], res[C][RES32 ? 2 : 1];
    __device__ __forceinline__ void load(const BlockNormProblem &p, int row, int pieces) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            const size_t at = (size_t)row * p.dim + 8 * (size_t)c;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const bool ok = c < pieces;
            x[i] = ok ? *reinterpret_cast<const uint4 *>(p.x + at) : zero;
            gate[i] = ok && p.gate ? *reinterpret_cast<const uint4 *>(p.gate + at) : zero;
            const uint4 *r = RES32 ? reinterpret_cast<const uint4 *>(static_cast<const float *>(p.residual) + at)
                                   : reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.residual) + at);
            res[i][0] = ok ? r[0] : zero;
            if constexpr (RES32) res[i][1] = ok ? r[1] : zero;
        }
    }
};

// STAY: the next row and the weights are held in registers (4000 x 8192: 70 us against 105 without, fp32 residual; 55 / 98,
// bf16).  A row of more than 8192 needs the registers for itself, and is one of few: its CTA loads it when it comes to it,
// and the weights where they are used.
template <int C, bool RES32, bool STAY>
__global__ void __launch_bounds__(STAY ? 512 : 1024, C == 1 ? 2 : 1) block_norm_kernel(const __grid_constant__ BlockNormProblem p) {
    __shared__ float part[2][2][32];   // by sum, and by turn: a row's last reader may still be at the other turn's
    int turn = 0;
    const int pieces = p.dim / 8, nt = blockDim.x;
    const float inv_dim = 1.f / p.dim;
    RowPieces<C, RES32> next;
    int row = blockIdx.x;
    if (STAY) next.load(p, row, pieces);
    // what y is multiplied by, the norm's weight and the scale, for this thread's piece i; and the weight of h
    auto load_post = [&](int i, float (&w)[8]) {
        const int c = threadIdx.x + i * nt;
        float s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f, s[e] = p.scale;
        if (c < pieces && p.post_w) load8(p.post_w + 8 * c, w);
        if (c < pieces && p.scale_w) load8(p.scale_w + 8 * c, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= s[e];
    };
    auto load_pre = [&](int i, float (&w)[8]) {
        const int c = threadIdx.x + i * nt;
        if (c < pieces) load8(p.pre_w + 8 * c, w);
    };
    float post[C][8], pre[C][8];
    if (STAY) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            load_post(i, post[i]);
            load_pre(i, pre[i]);
        }
    }
    for (; row < p.rows; row += gridDim.x, turn ^= 1) {
        if (!STAY) next.load(p, row, pieces);
        const RowPieces<C, RES32> cur = next;
        if (STAY && row + (int)gridDim.x < p.rows) next.load(p, row + gridDim.x, pieces);
        float y[C][8], r[C][8];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            unpack8(cur.x[i], y[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(y[i][e], y[i][e], ss);
        }
        float f = 1.f;
        if (p.post_w) f = rsqrtf(cta_sum(ss, part[0][turn]) * inv_dim + p.eps);
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if constexpr (RES32) {
                const uint4 a = cur.res[i][0], b = cur.res[i][1];
                const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) r[i][e] = __uint_as_float(w[e]);
            } else {
                unpack8(cur.res[i][0], r[i]);
            }
            float g[8];
            unpack8(cur.gate[i], g);
            if (!STAY) load_post(i, post[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = y[i][e] * f * post[i][e];
                if (p.gate) {
                    const float sig = __fdividef(1.f, 1.f + __expf(-g[e]));
                    v *= p.silu ? g[e] * sig : sig;
                }
                r[i][e] += v;
                ss = fmaf(r[i][e], r[i][e], ss);
            }
            const int c = threadIdx.x + i * nt;
            if (c < pieces) {
                const size_t at = (size_t)row * p.dim + 8 * (size_t)c;
                if (RES32) {
                    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.residual_out) + at);
                    o[0] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
                    o[1] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
                } else {
                    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.residual_out) + at) = pack8(r[i]);
                }
            }
        }
        f = rsqrtf(cta_sum(ss, part[1][turn]) * inv_dim + p.eps);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = threadIdx.x + i * nt;
            if (c >= pieces) continue;
            if (!STAY) load_pre(i, pre[i]);
            float h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = r[i][e] * f * pre[i][e];
            *reinterpret_cast<uint4 *>(p.out + (size_t)row * p.dim + 8 * (size_t)c) = pack8(h);
        }
    }
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormProblem &p) {
    const int pieces = p.dim / 8;
    // One piece a thread up to 512 of them, then two.  Many short rows with an fp32 residual, whose piece is two loads, mostly
    // gain from two as well (us with two / with one): 16383 x 2048 77 / 80, 4096 x 2048 19.9 / 20.4, 60000 x 1536 208 / 220,
    // 32000 x 1024 75 / 79, 16384 x 512 20.3 / 20.5, 16384 x 264 13.4 / 16.0; less so 16384 x 640 26.7 / 24.7 and 4096 x 768
    // 10.1 / 9.0.  Not where one warp holds the row with one (16384 x 256 12.9 / 11.4), at 8000 x 4096 73 / 71, for one row
    // (of 2048 3.1 / 2.9), nor with a bf16 residual (16383 x 2048 52.5 / 52.1).
    const int c = pieces > 512 || (p.residual_f32 && pieces > 32 && pieces <= 256 && p.rows >= 4096) ? 2 : 1;
    const int threads = ((pieces + c - 1) / c + 31) / 32 * 32;
    using Fn = void (*)(const BlockNormProblem);
    const bool f32 = p.residual_f32;
    const Fn fn = c == 1 ? (f32 ? block_norm_kernel<1, true, true> : block_norm_kernel<1, false, true>)
                  : threads <= 512 ? (f32 ? block_norm_kernel<2, true, true> : block_norm_kernel<2, false, true>)
                                   : (f32 ? block_norm_kernel<2, true, false> : block_norm_kernel<2, false, false>);
    // CTAs that stay: what fits on the SMs at once, the same number of rows each as far as that goes
    const int fit = multiprocessor_count() * max(1, min(24, (c == 1 ? 1024 : 512) / threads));
    const int rounds = (p.rows + fit - 1) / fit, ctas = (p.rows + rounds - 1) / rounds;
    fn<<<(unsigned)ctas, (unsigned)threads, 0, p.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gdn
