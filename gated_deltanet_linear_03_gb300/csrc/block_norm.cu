// gdn_block_norm: the norm after a block, its gate and scale, the residual sum, the norm before the next block.
//
//     y = x rsqrt(mean(x^2) + eps) w_post,   y *= act(gate),   r' = r + s y,   h = r' rsqrt(mean(r'^2) + eps) w_pre
//
// One CTA holds one row in registers (pieces of 8 elements, C of them a thread), so x, gate and residual are
// read once and r' and h written once; the two sums of squares are CTA reductions in fp32.  Every load of the
// row and of the weights is issued before the first reduction.  Bound by memory.
#include "kv_cache.cuh"

namespace gdn {
namespace {

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void load8f(const float *p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

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

template <int C, bool RES32>
__global__ void __launch_bounds__(512) block_norm_kernel(const __grid_constant__ BlockNormProblem p) {
    __shared__ float part[2][16];
    const int pieces = p.dim / 8, nt = blockDim.x;
    const size_t base = (size_t)blockIdx.x * p.dim;
    float y[C][8], r[C][8], g[C][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = threadIdx.x + i * nt;
        if (c < pieces) {
            const size_t at = base + 8 * (size_t)c;
            unpack8(*reinterpret_cast<const uint4 *>(p.x + at), y[i]);
            if (p.gate) unpack8(*reinterpret_cast<const uint4 *>(p.gate + at), g[i]);
            if (RES32) load8f(static_cast<const float *>(p.residual) + at, r[i]);
            else unpack8(*reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.residual) + at), r[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[i][e] = r[i][e] = g[i][e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[i][e], y[i][e], ss);
    }
    const float inv_dim = 1.f / p.dim;
    float f = 1.f;
    if (p.post_w) f = rsqrtf(cta_sum(ss, part[0]) * inv_dim + p.eps);
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = threadIdx.x + i * nt;
        if (c >= pieces) continue;
        float w[8], s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f, s[e] = p.scale;
        if (p.post_w) load8f(p.post_w + 8 * c, w);
        if (p.scale_w) load8f(p.scale_w + 8 * c, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = y[i][e] * f * w[e];
            if (p.gate) {
                const float sig = 1.f / (1.f + __expf(-g[i][e]));
                v *= p.silu ? g[i][e] * sig : sig;
            }
            r[i][e] = fmaf(s[e], v, r[i][e]);
            ss = fmaf(r[i][e], r[i][e], ss);
        }
        const size_t at = base + 8 * (size_t)c;
        if (RES32) {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.residual_out) + at);
            o[0] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
            o[1] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.residual_out) + at) = pack8(r[i]);
        }
    }
    f = rsqrtf(cta_sum(ss, part[1]) * inv_dim + p.eps);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = threadIdx.x + i * nt;
        if (c >= pieces) continue;
        float w[8];
        load8f(p.pre_w + 8 * c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= r[i][e] * f;
        *reinterpret_cast<uint4 *>(p.out + base + 8 * (size_t)c) = pack8(w);
    }
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormProblem &p) {
    const int pieces = p.dim / 8;
    // two pieces a thread (enough loads in flight with 8 or more CTAs an SM), four where that would pass 512 threads
    const int c = pieces <= 32 ? 1 : pieces <= 1024 ? 2 : 4;
    const int threads = ((pieces + c - 1) / c + 31) / 32 * 32;
    using Fn = void (*)(const BlockNormProblem);
    const Fn fn = p.residual_f32 ? (c == 1 ? block_norm_kernel<1, true> : c == 2 ? block_norm_kernel<2, true> : block_norm_kernel<4, true>)
                                 : (c == 1 ? block_norm_kernel<1, false> : c == 2 ? block_norm_kernel<2, false> : block_norm_kernel<4, false>);
    fn<<<(unsigned)p.rows, (unsigned)threads, 0, p.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gdn
