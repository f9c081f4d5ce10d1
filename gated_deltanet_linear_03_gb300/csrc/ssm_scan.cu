// gdn_ssm_scan: per channel c, with N numbers of state,
//     h[n] = exp(D a[c, n]) h[n] + D x B[n],   y = (sum_n h[n] C[n] + skip x) z / (1 + e^-z),   D = softplus(dt + bias).
//
// A channel's states lie in the registers of N / S neighbouring lanes, S each, for as long as its sequence lasts.
#include "layer_ops.cuh"

namespace gdn {
namespace {

constexpr int kScanThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float step_width(float v, int softplus) {
    return softplus ? fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))) : v;
}

__device__ __forceinline__ float silu(float z) { return __fdividef(z, 1.f + __expf(-z)); }

template <int S>
__device__ __forceinline__ void load_state(const float *p, float (&h)[S]) {
#pragma unroll
    for (int i = 0; i < S / 4; ++i) {
        const float4 v = *reinterpret_cast<const float4 *>(p + 4 * i);
        h[4 * i] = v.x; h[4 * i + 1] = v.y; h[4 * i + 2] = v.z; h[4 * i + 3] = v.w;
    }
}
template <int S>
__device__ __forceinline__ void store_state(float *p, const float (&h)[S]) {
#pragma unroll
    for (int i = 0; i < S / 4; ++i) *reinterpret_cast<float4 *>(p + 4 * i) = make_float4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
}

// ---------------------------------------------------------------------------------------------- single tokens
// A thread takes 4 states of one channel of one sequence, and reads what it needs of a token itself.  Right for any number of
// tokens, meant for one.
template <int N>
__global__ void __launch_bounds__(kScanThreads) step_kernel(const __grid_constant__ ScanProblem p) {
    constexpr int LANES = N / 4, CH = kScanThreads / LANES;
    const int ctas = (p.channels + CH - 1) / CH;
    const int n = blockIdx.x / ctas, ch = blockIdx.x % ctas * CH + threadIdx.x / LANES, part = threadIdx.x % LANES;
    const int slot = p.seqs.slot(n);
    if (slot < 0) {
        if (threadIdx.x == 0) raise_error(p.seqs.err, kErrInternal);
        return;
    }
    const bool live = ch < p.channels;       // the shuffles want whole warps
    const int c = live ? ch : p.channels - 1;
    const size_t at = ((size_t)slot * p.channels + c) * N + 4 * part;
    float h[4] = {0.f, 0.f, 0.f, 0.f}, a[4];
    if (p.state_in) load_state(p.state_in + at, h);
    load4(p.a + (size_t)c * N + 4 * part, a);
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, skip = p.skip ? p.skip[c] : 0.f;
    const int bc = c / (p.channels / p.groups) * N + 4 * part;
    for (int t = p.seqs.begin(n); t < p.seqs.end(n); ++t) {
        const float x = __bfloat162float(p.x[t * p.x_stride + c]);
        const float d = step_width(__bfloat162float(p.dt[t * p.dt_stride + c]) + bias, p.softplus);
        const float z = p.z ? __bfloat162float(p.z[t * p.z_stride + c]) : 0.f;
        const uint2 bw = *reinterpret_cast<const uint2 *>(p.b + t * p.b_stride + bc);
        const uint2 cw = *reinterpret_cast<const uint2 *>(p.c + t * p.c_stride + bc);
        const float b[4] = {bf16_lo(bw.x), bf16_hi(bw.x), bf16_lo(bw.y), bf16_hi(bw.y)};
        const float cc[4] = {bf16_lo(cw.x), bf16_hi(cw.x), bf16_lo(cw.y), bf16_hi(cw.y)};
        const float u = d * x, dl = d * kLog2e;
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = fmaf(ex2(dl * a[i]), h[i], u * b[i]);
            y = fmaf(h[i], cc[i], y);
        }
#pragma unroll
        for (int o = LANES / 2; o >= 1; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (live && part == 0) {
            y = fmaf(skip, x, y);
            if (p.z) y *= silu(z);
            const size_t to = (size_t)t * p.channels + c;
            if (p.out_f32) static_cast<float *>(p.out)[to] = y;
            else static_cast<__nv_bfloat16 *>(p.out)[to] = __float2bfloat16_rn(y);
        }
    }
    if (live && p.state_out) store_state(p.state_out + at, h);
}

// ---------------------------------------------------------------------------------------------- prompts
template <int N_, int S_>
struct Shape {
    static constexpr int N = N_, S = S_, LANES = N / S, CH = kScanThreads / LANES, CHUNKS = CH / 8;
    static constexpr int TT = kScanThreads / CHUNKS < 32 ? kScanThreads / CHUNKS : 32;   // tokens of a tile
    static constexpr int PARTS = LANES < 4 ? LANES : 4;             // partial sums of y that go through shared memory
    static constexpr int Y_PIECE = 8 * PARTS + 4;                   // floats of 8 channels' partial sums, and 4 against bank conflicts
    struct Tile {
        float2 du[TT][CH];             // step width (times log2 e) and step width times x
        float b[TT][N], c[TT][N];
        float y[TT * CHUNKS][Y_PIECE];
    };
};

// What a thread reads of one tile: one token's 8 channels, and its share of the vectors.
template <class SH>
struct Raw {
    static constexpr int VECTORS = (2 * SH::TT * SH::N / 8 + kScanThreads - 1) / kScanThreads;
    uint4 x, dt, z, bc[VECTORS];
    __device__ __forceinline__ void load(const ScanProblem &p, int t0, int t1, int c0, int c1, int group, bool with_y) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const int t = t0 + threadIdx.x / SH::CHUNKS, c = c0 + 8 * (threadIdx.x % SH::CHUNKS);
        const bool ok = threadIdx.x < SH::TT * SH::CHUNKS && t < t1 && c < c1;
        x = ok ? *reinterpret_cast<const uint4 *>(p.x + t * p.x_stride + c) : zero;
        dt = ok ? *reinterpret_cast<const uint4 *>(p.dt + t * p.dt_stride + c) : zero;
        z = ok && with_y && p.z ? *reinterpret_cast<const uint4 *>(p.z + t * p.z_stride + c) : zero;
#pragma unroll
        for (int i = 0; i < VECTORS; ++i) {
            const int k = threadIdx.x + i * kScanThreads, which = k / (SH::TT * SH::N / 8), at = k % (SH::TT * SH::N / 8);
            const int tb = t0 + at / (SH::N / 8), e = group * SH::N + at % (SH::N / 8) * 8;
            bc[i] = zero;
            if (which < 2 && tb < t1) bc[i] = *reinterpret_cast<const uint4 *>(which ? p.c + tb * p.c_stride + e : p.b + tb * p.b_stride + e);
        }
    }
};

__device__ __forceinline__ float channel_value(const float *p, int c, int channels) { return p && c < channels ? __ldg(p + c) : 0.f; }

// Tokens [t0, t1) of one sequence for the CTA's channels, from c0 and below c1; h is this lane's part of its channel's state.
template <class SH, bool WITH_Y>
__device__ __forceinline__ void scan_tokens(const ScanProblem &p, typename SH::Tile &s, int t0, int t1, int c0, int c1, int group,
                                            const float (&a)[SH::S], float (&h)[SH::S], float *width_sum) {
    constexpr int S = SH::S, TT = SH::TT, N = SH::N;
    const int chan = threadIdx.x / SH::LANES, part = threadIdx.x % SH::LANES;
    const int mt = threadIdx.x / SH::CHUNKS, mc = threadIdx.x % SH::CHUNKS;
    const bool mine = threadIdx.x < TT * SH::CHUNKS;
    Raw<SH> raw;
    raw.load(p, t0, t1, c0, c1, group, WITH_Y);
    float total = 0.f;
    for (int at = t0; at < t1; at += TT) {
        const Raw<SH> cur = raw;
        if (mine) {
            float x[8], d[8];
            unpack8(cur.x, x);
            unpack8(cur.dt, d);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = c0 + 8 * mc + e;
                const float w = at + mt < t1 ? step_width(d[e] + channel_value(p.dt_bias, c, c1), p.softplus) : 0.f;
                s.du[mt][8 * mc + e] = make_float2(w * kLog2e, w * x[e]);      // (a row beyond the end changes nothing)
            }
        }
#pragma unroll
        for (int i = 0; i < Raw<SH>::VECTORS; ++i) {
            const int k = threadIdx.x + i * kScanThreads, which = k / (TT * N / 8), v = k % (TT * N / 8);
            if (which >= 2) continue;
            float f[8];
            unpack8(cur.bc[i], f);
            float4 *to = reinterpret_cast<float4 *>((which ? s.c[0] : s.b[0]) + 8 * v);
            to[0] = make_float4(f[0], f[1], f[2], f[3]);
            to[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
        __syncthreads();
        if (at + TT < t1) raw.load(p, at + TT, t1, c0, c1, group, WITH_Y);
#pragma unroll 8
        for (int t = 0; t < TT; ++t) {
            const float2 du = s.du[t][chan];
            float b[S], c[S];
            load_state(&s.b[t][S * part], b);
            if (WITH_Y) load_state(&s.c[t][S * part], c);
            else total += du.x;
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                h[i] = fmaf(ex2(du.x * a[i]), h[i], du.y * b[i]);
                if (WITH_Y) y = fmaf(h[i], c[i], y);
            }
            if (WITH_Y) {
#pragma unroll
                for (int o = SH::LANES / 2; o >= SH::PARTS; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                if (part < SH::PARTS) s.y[t * SH::CHUNKS + chan / 8][chan % 8 * SH::PARTS + part] = y;
            }
        }
        __syncthreads();
        if (WITH_Y && mine && at + mt < t1 && c0 + 8 * mc < c1) {
            float x[8], z[8], y[8];
            unpack8(cur.x, x);
            unpack8(cur.z, z);
            const float *from = s.y[threadIdx.x];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[e] = 0.f;
#pragma unroll
                for (int q = 0; q < SH::PARTS; ++q) y[e] += from[e * SH::PARTS + q];
                y[e] = fmaf(channel_value(p.skip, c0 + 8 * mc + e, c1), x[e], y[e]);
                if (p.z) y[e] *= silu(z[e]);
            }
            const size_t to = (size_t)(at + mt) * p.channels + c0 + 8 * mc;
            if (p.out_f32) {
                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + to);
                o[0] = make_float4(y[0], y[1], y[2], y[3]);
                o[1] = make_float4(y[4], y[5], y[6], y[7]);
            } else {
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + to) = pack8(y);
            }
        }
    }
    if (!WITH_Y) *width_sum = total;
}

// One CTA carries a whole sequence for its channels.
template <class SH>
__global__ void __launch_bounds__(kScanThreads) scan_kernel(const __grid_constant__ ScanProblem p, int ctas_per_group) {
    extern __shared__ __align__(16) unsigned char smem[];
    typename SH::Tile &s = *reinterpret_cast<typename SH::Tile *>(smem);
    const int per_group = p.channels / p.groups, ctas = ctas_per_group * p.groups;
    const int n = blockIdx.x / ctas, group = blockIdx.x % ctas / ctas_per_group;
    const int c0 = group * per_group + blockIdx.x % ctas_per_group * SH::CH;
    const int slot = p.seqs.slot(n);
    if (slot < 0) {
        if (threadIdx.x == 0) raise_error(p.seqs.err, kErrInternal);
        return;
    }
    const int c1 = (group + 1) * per_group, c = c0 + threadIdx.x / SH::LANES, part = threadIdx.x % SH::LANES;
    const bool live = c < c1;
    const size_t at = ((size_t)slot * p.channels + c) * SH::N + SH::S * part;
    float h[SH::S], a[SH::S];
#pragma unroll
    for (int i = 0; i < SH::S; ++i) h[i] = a[i] = 0.f;
    if (live) {
        if (p.state_in) load_state(p.state_in + at, h);
        load_state(p.a + (size_t)c * SH::N + SH::S * part, a);
    }
    float unused;
    scan_tokens<SH, true>(p, s, p.seqs.begin(n), p.seqs.end(n), c0, c1, group, a, h, &unused);
    if (live && p.state_out) store_state(p.state_out + at, h);
}

template <int N, int S>
cudaError_t launch(const ScanProblem &p) {
    if (!p.seqs.cu || p.max_len == 1) {
        constexpr int CH = kScanThreads / (N / 4);
        const long ctas = (long)((p.channels + CH - 1) / CH) * p.seqs.n;
        step_kernel<N><<<(unsigned)ctas, kScanThreads, 0, p.stream>>>(p);
        return cudaGetLastError();
    }
    using SH = Shape<N, S>;
    const int ctas_per_group = (p.channels / p.groups + SH::CH - 1) / SH::CH;
    const cudaError_t e = cudaFuncSetAttribute(scan_kernel<SH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(typename SH::Tile));
    if (e != cudaSuccess) return e;
    scan_kernel<SH><<<(unsigned)((long)ctas_per_group * p.groups * p.seqs.n), kScanThreads, sizeof(typename SH::Tile), p.stream>>>(p, ctas_per_group);
    return cudaGetLastError();
}

}  // namespace

size_t ssm_scan_workspace_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t launch_ssm_scan(const ScanProblem &p) {
    switch (p.n_state) {
        case 16: return launch<16, 4>(p);
        case 32: return launch<32, 4>(p);
        case 64: return launch<64, 8>(p);
        default: return launch<128, 16>(p);
    }
}

}  // namespace gdn
