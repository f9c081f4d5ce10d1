// gdn_ssm_scan: per channel c, with N numbers of state,
//     h[n] = exp(D a[c, n]) h[n] + D x B[n],   y = (sum_n h[n] C[n] + skip x) z / (1 + e^-z),   D = softplus(dt + bias).
//
// A channel's states lie in the registers of N / S neighbouring lanes, S each, for as long as its sequence lasts.
//
// A prompt is bound by instructions: N exponentials a token and channel (32 a cycle and SM) and four multiplications or sums beside
// each, in packed pairs, which take two of a scheduler's slots.  A warp works on its own, 8 states of 2 channels a lane: B and C of a
// token serve 16 products a lane, and the step widths, gates and stores of 8 tokens are prepared by all lanes at once.  Where there
// are too few sequences and channels for the GPU, the tokens are cut into pieces, and a first pass carries only the states (at 2/3 of
// the cost of a whole one) to the pieces' beginnings.
//
// Measured on a GB300, 4096 channels x 16 states: 64 sequences of 128 tokens 152 us in one pass, 0.38 of the exponentials' rate; 8192 tokens
// of one sequence 259 us (107 for the ends, 152 for the outputs: issue slots 0.63 and 0.61 busy, exponentials 0.58 and 0.46; the bytes are
// 40 us).  7 sequences, 6465 tokens x 1536 channels x 64 states 247 us.  One token: 61 sequences x 4096 x 16 9.5 us, 3.6 TB/s; one sequence 2.1.
#include "layer_ops.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

constexpr int kScanThreads = 128;
// The larger of v and 0; a NaN stays one.
__device__ __forceinline__ float positive(float v) {
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
    return r;
}

// a without infinities: the lowest number forgets as much at every step, and leaves the state as it is at a step of zero, which 0 a of
// an infinite a does not.
__device__ __forceinline__ float finite(float a) { return fabsf(a) == INFINITY ? copysignf(3.402823466e38f, a) : a; }

// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^-|v|, without a branch and to a few units in the last place, down to e = 2^-126;
// a smaller e is zero.  |v| counts as 104 at most, where e is zero: so nothing is infinite in between, and v = -inf, which masks a
// token, or the lowest number gives 0.  The exponential's argument is corrected for its rounding; log(1 + e) = 2 artanh(q) with q = e / (2 + e) <= 1/3, by a
// polynomial for artanh(q) / q in q^2 on [0, 1/9] whose largest relative error is least (Remez's exchange, 4e-9).
__device__ __forceinline__ Pair softplus(Pair v) {
    const auto both = [](float x) { return pair(x, x); };
    float v0, v1, t0, t1;
    halves(v, v0, v1);
    const Pair m = pair(-fminf(fabsf(v0), 104.f), -fminf(fabsf(v1), 104.f)), t = mul2(m, both(kLog2e));
    const Pair r = fma2(m, both(1.925963033500e-8f), fma2(m, both(kLog2e), t ^ 0x8000000080000000ull));       // what t lacks of m log2 e
    halves(t, t0, t1);
    Pair e = pair(ex2(t0), ex2(t1));
    e = fma2(e, mul2(r, both(0.69314718f)), e);
    halves(add2(e, both(2.f)), t0, t1);
    const Pair q = mul2(e, pair(reciprocal(t0), reciprocal(t1))), q2 = mul2(q, q);
    Pair s = fma2(q2, both(0.14089168f), both(0.13980301f));
    s = fma2(q2, s, both(0.20012455f));
    s = fma2(q2, s, both(0.33333157f));
    s = fma2(q2, s, both(1.f));
    return fma2(add2(q, q), s, pair(positive(v0), positive(v1)));
}

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
// A thread takes 4 states each of two channels, and sequences n, n + step, ... one after another, the next one's states on their way
// while one is worked on: the channels' parameters are read once.  It reads what it needs of a token itself.  Right for any number of
// tokens, meant for one.
template <int N>
__global__ void __launch_bounds__(kScanThreads) step_kernel(const __grid_constant__ ScanProblem p, int step) {
    constexpr int LANES = N / 4, CH = kScanThreads / LANES;
    const int ctas = (p.channels + 2 * CH - 1) / (2 * CH);
    const int part = threadIdx.x % LANES, ch0 = blockIdx.x % ctas * 2 * CH + threadIdx.x / LANES;
    const int per_group = p.channels / p.groups;
    const size_t all = (size_t)p.channels * N;
    bool live[2];
    int c[2], bc[2];
    size_t at[2];
    float a[2][4], bias[2], skip[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        live[m] = ch0 + m * CH < p.channels;             // the shuffles want whole warps
        c[m] = live[m] ? ch0 + m * CH : p.channels - 1;
        at[m] = (size_t)c[m] * N + 4 * part;
        bc[m] = c[m] / per_group * N + 4 * part;
        load4(p.a + at[m], a[m]);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[m][i] = finite(a[m][i]);
        bias[m] = p.dt_bias ? __ldg(p.dt_bias + c[m]) : 0.f;
        skip[m] = p.skip ? __ldg(p.skip + c[m]) : 0.f;
    }
    float next[2][4];
    const auto begin = [&](int slot) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int i = 0; i < 4; ++i) next[m][i] = 0.f;
            if (p.state_in && slot >= 0) load_state(p.state_in + slot * all + at[m], next[m]);
        }
    };
    int n = blockIdx.x / ctas, slot = p.seqs.slot(n);
    begin(slot);
    for (; n < p.seqs.n; n += step) {
        float h[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) h[m][i] = next[m][i];
        const int here = slot;
        if (n + step < p.seqs.n) {
            slot = p.seqs.slot(n + step);
            begin(slot);
        }
        if (here < 0) {
            if (threadIdx.x == 0) raise_error(p.seqs.err, kErrInternal);
            continue;
        }
        for (int t = p.seqs.begin(n); t < p.seqs.end(n); ++t) {
            float x[2], z[2] = {0.f, 0.f}, d[2];
            uint2 bw[2], cw[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                x[m] = __bfloat162float(p.x[t * p.x_stride + c[m]]);
                d[m] = __bfloat162float(p.dt[t * p.dt_stride + c[m]]) + bias[m];
                if (p.z) z[m] = __bfloat162float(p.z[t * p.z_stride + c[m]]);
                bw[m] = *reinterpret_cast<const uint2 *>(p.b + t * p.b_stride + bc[m]);
                cw[m] = *reinterpret_cast<const uint2 *>(p.c + t * p.c_stride + bc[m]);
            }
            if (p.softplus) halves(softplus(pair(d[0], d[1])), d[0], d[1]);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float b[4] = {bf16_lo(bw[m].x), bf16_hi(bw[m].x), bf16_lo(bw[m].y), bf16_hi(bw[m].y)};
                const float cc[4] = {bf16_lo(cw[m].x), bf16_hi(cw[m].x), bf16_lo(cw[m].y), bf16_hi(cw[m].y)};
                const float u = d[m] * x[m], dl = d[m] * kLog2e;
                float y = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[m][i] = fmaf(ex2(dl * a[m][i]), h[m][i], u * b[i]);
                    y = fmaf(h[m][i], cc[i], y);
                }
#pragma unroll
                for (int o = LANES / 2; o >= 1; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                if (live[m] && part == 0) {
                    y = fmaf(skip[m], x[m], y);
                    if (p.z) y *= silu(z[m]);
                    const size_t to = (size_t)t * p.channels + c[m];
                    if (p.out_f32) static_cast<float *>(p.out)[to] = y;
                    else static_cast<__nv_bfloat16 *>(p.out)[to] = __float2bfloat16_rn(y);
                }
            }
        }
        if (!p.state_out) continue;
#pragma unroll
        for (int m = 0; m < 2; ++m)
            if (live[m]) store_state(p.state_out + here * all + at[m], h[m]);
    }
}

// ---------------------------------------------------------------------------------------------- prompts
struct alignas(16) Pair2 { Pair x, y; };

constexpr int kPromptWarps = 4, kPromptThreads = 32 * kPromptWarps;      // of a CTA; each goes its own way
constexpr int kPromptCtas = 3;              // CTAs an SM
constexpr int kMaxPiece = 2048;             // tokens of a piece of a scan in pieces
constexpr int kTile = 8;                    // tokens of a turn

template <int N_>
struct Shape {
    static constexpr int N = N_;
    // A lane scans 8 states of 2 neighbouring channels
    static constexpr int LANES = N / 8, V = 64 / LANES;               // lanes of a channel pair; channels of a warp
    // and prepares VH channels of one token (states of 128: half of the lanes do)
    static constexpr int VH = V >= 8 ? V / 4 : 2, CHUNKS = V / VH;
    // A tile's raw rows and vectors are asked for DEEP turns ahead, to cover a read of memory
    static constexpr int DEEP = N == 128 ? 2 : 3, RING = DEEP + 1;
    static constexpr int VECTORS = kTile * N / 8 < 32 ? 1 : kTile * N / 8 / 32;      // pieces of 8 entries of B that a lane copies
    // B and C are widened to 32 bits once, or where they are used: a warp of few channels has too few uses for the former
    static constexpr bool WIDE = N == 16;
    struct Shared {                         // of a warp
        float4 du[kTile][V / 2];            // of two channels: step width D (times log2 e) and D x
        float4 y[kTile][16];                // by lane: its part of y, for two channels
        float b[WIDE ? kTile : 1][N], c[WIDE ? kTile : 1][N];
        uint4 braw[RING][kTile * N / 8], craw[RING][kTile * N / 8];           // as they came, in bf16
        __nv_bfloat16 x[RING][32][VH], dt[RING][32][VH], z[RING][32][VH];      // by preparing lane
    };
    // Of the 16-byte entries of du and y a preparing lane (token t, chunk c) has DU and Y next to one another; they are in the
    // order entry ^ key, key = key of the chunk ^ key of the token, so that what 8 lanes touch at once lies in different banks.
    static constexpr int DU = VH / 2, Y = 16 / CHUNKS;
    __host__ __device__ static constexpr int du_key(int t, int chunk) { return DU == 4 ? 2 * (t & 1) ^ chunk >> 1 : DU == 2 ? t & 1 : 0; }
    __host__ __device__ static constexpr int y_key(int t, int chunk) { return Y == 4 ? 2 * (t & 1) ^ chunk >> 1 : 2 * (t & 3) ^ chunk; }
};

// Copy BYTES (4, 8 or 16) to shared memory behind the thread's back, zeros where there is nothing to read.
template <int BYTES>
__device__ __forceinline__ void copy_async(void *to, const void *from, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(sm100::smem_u32(to)), "l"(from), "n"(BYTES), "r"(there ? BYTES : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// V bf16 values, as they lie in memory.
template <int V> struct Bits { using T = uint4; };
template <> struct Bits<4> { using T = uint2; };
template <> struct Bits<2> { using T = uint32_t; };
template <int V>
__device__ __forceinline__ void unpack(const typename Bits<V>::T &u, Pair (&x)[V / 2]) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&u);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) x[i] = pair(bf16_lo(w[i]), bf16_hi(w[i]));
}

// Tokens [t0, t1) of one sequence for the warp's channels c0 .. and below c1.  h: a lane's part of its channels' states;
// width_sum: the sums of their step widths (times log2 e).
template <class SH, bool WITH_Y>
__device__ __forceinline__ void scan_tokens(const ScanProblem &p, typename SH::Shared &sh, int t0, int t1, int c0, int c1, int group,
                                            const Pair (&a)[2][4], Pair (&h)[2][4], float (&width_sum)[2]) {
    constexpr int N = SH::N, LANES = SH::LANES, VH = SH::VH, CHUNKS = SH::CHUNKS;
    using T = typename Bits<VH>::T;
    const int n = (t1 - t0 + kTile - 1) / kTile, lane = threadIdx.x % 32;
    width_sum[0] = width_sum[1] = 0.f;
    // as a preparing lane: one token's VH channels
    const int my_t = lane / CHUNKS, chunk = lane % CHUNKS, c = c0 + VH * chunk;
    const bool live = my_t < kTile && c < c1;
    Pair bias[VH / 2], skip[VH / 2];
#pragma unroll
    for (int e = 0; e < VH / 2; ++e) {
        const float2 zero = make_float2(0.f, 0.f);
        const float2 b = live && p.dt_bias ? __ldg(reinterpret_cast<const float2 *>(p.dt_bias + c) + e) : zero;
        const float2 k = live && WITH_Y && p.skip ? __ldg(reinterpret_cast<const float2 *>(p.skip + c) + e) : zero;
        bias[e] = pair(b.x, b.y);
        skip[e] = pair(k.x, k.y);
    }
    // what this lane asks for next
    const bool copies = 32 <= kTile * N / 8 || lane < kTile * N / 8;
    const int vec_t = lane / (N / 8);
    long long at_x = (long long)(t0 + my_t) * p.x_stride + c, at_dt = (long long)(t0 + my_t) * p.dt_stride + c;
    long long at_z = (long long)(t0 + my_t) * p.z_stride + c;
    long long at_b = (long long)(t0 + vec_t) * p.b_stride + group * N + lane % (N / 8) * 8;
    long long at_c = (long long)(t0 + vec_t) * p.c_stride + group * N + lane % (N / 8) * 8;
    auto ask = [&](int i) {
        if (i < n) {
            const int left = t1 - (t0 + i * kTile), slot = i % SH::RING;
            const bool there = live && my_t < left;
            copy_async<2 * VH>(sh.x[slot][lane], p.x + (there ? at_x : 0), there);
            copy_async<2 * VH>(sh.dt[slot][lane], p.dt + (there ? at_dt : 0), there);
            if (WITH_Y && p.z) copy_async<2 * VH>(sh.z[slot][lane], p.z + (there ? at_z : 0), there);
            if (copies) {
#pragma unroll
                for (int k = 0; k < SH::VECTORS; ++k) {
                    const int row = k * 32 / (N / 8);
                    const bool held = vec_t + row < left;
                    copy_async<16>(&sh.braw[slot][lane + 32 * k], p.b + (held ? at_b + row * p.b_stride : 0), held);
                    if (WITH_Y) copy_async<16>(&sh.craw[slot][lane + 32 * k], p.c + (held ? at_c + row * p.c_stride : 0), held);
                }
            }
            at_x += kTile * p.x_stride;
            at_dt += kTile * p.dt_stride;
            at_b += kTile * p.b_stride;
            if (WITH_Y) at_z += kTile * p.z_stride, at_c += kTile * p.c_stride;
        }
        copy_commit();                      // (a group for every turn, so that their number says which have arrived)
    };
    // as a scanning lane: where its channels' entry of du is, and its half of an entry of y
    const int entry = lane / LANES, part = lane % LANES, du_chunk = entry / SH::DU, y_chunk = lane / 2 / SH::Y;
    for (int i = 0; i < SH::DEEP; ++i) ask(i);
    for (int i = 0; i < n; ++i) {
        const int slot = i % SH::RING;
        copy_wait<SH::DEEP - 1>();
        __syncwarp();                       // the tile has arrived for all lanes, and all are done with the one before
        ask(i + SH::DEEP);
        const T xr = *reinterpret_cast<const T *>(sh.x[slot][lane]);
        if (SH::WIDE && copies) {
            const auto widen = [&](const uint4 *from, float *to) {
#pragma unroll
                for (int k = 0; k < SH::VECTORS; ++k) {
                    float f[8];
                    unpack8(from[lane + 32 * k], f);
                    float4 *o = reinterpret_cast<float4 *>(to + 8 * (lane + 32 * k));
                    o[0] = make_float4(f[0], f[1], f[2], f[3]);
                    o[1] = make_float4(f[4], f[5], f[6], f[7]);
                }
            };
            widen(sh.braw[slot], sh.b[0]);
            if (WITH_Y) widen(sh.craw[slot], sh.c[0]);
        }
        T zr{};
        if (WITH_Y && p.z) zr = *reinterpret_cast<const T *>(sh.z[slot][lane]);
        {
            Pair x[VH / 2], d[VH / 2];
            unpack<VH>(xr, x);
            unpack<VH>(*reinterpret_cast<const T *>(sh.dt[slot][lane]), d);
#pragma unroll
            for (int e = 0; e < VH / 2; ++e) d[e] = add2(d[e], bias[e]);
            if (p.softplus) {
#pragma unroll
                for (int e = 0; e < VH / 2; ++e) d[e] = softplus(d[e]);
            }
            if (t0 + i * kTile + my_t >= t1) {
#pragma unroll
                for (int e = 0; e < VH / 2; ++e) d[e] = 0;            // (a row beyond the end changes nothing)
            }
            const int key = SH::du_key(my_t, chunk);
            if (32 == kTile * CHUNKS || my_t < kTile) {
                float4 *to = &sh.du[my_t][SH::DU * chunk];
#pragma unroll
                for (int e = 0; e < VH / 2; ++e) {
                    float w0, w1, u0, u1;
                    halves(mul2(d[e], x[e]), u0, u1);
                    halves(mul2(d[e], pair(kLog2e, kLog2e)), w0, w1);
                    to[e ^ key] = make_float4(w0, u0, w1, u1);
                }
            }
        }
        __syncwarp();
        const float *bv = &sh.b[0][8 * part], *cv = &sh.c[0][8 * part];
        const uint4 *bw = &sh.braw[slot][part], *cw = &sh.craw[slot][part];
        float2 *y = reinterpret_cast<float2 *>(&sh.y[0][y_chunk * SH::Y]) + lane % 2;
        // y is stored once for all tokens: the next tokens' reads are not ordered behind it
        float2 outs[kTile];
#pragma unroll
        for (int t = 0; t < kTile; ++t) {
            float2 &out = outs[t];
            const float4 q = sh.du[t][du_chunk * SH::DU + (entry % SH::DU ^ SH::du_key(t, du_chunk))];
            Pair decay[2][4], b[4], cc[4];
            if constexpr (SH::WIDE) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const Pair2 f = *reinterpret_cast<const Pair2 *>(bv + t * N + 4 * k);
                    b[2 * k] = f.x, b[2 * k + 1] = f.y;
                    if (WITH_Y) {
                        const Pair2 f = *reinterpret_cast<const Pair2 *>(cv + t * N + 4 * k);
                        cc[2 * k] = f.x, cc[2 * k + 1] = f.y;
                    }
                }
            } else {
                unpack<8>(bw[t * (N / 8)], b);
                if (WITH_Y) unpack<8>(cw[t * (N / 8)], cc);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float wv = m ? q.z : q.x;
                const Pair w = pair(wv, wv);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float e0, e1;
                    halves(mul2(w, a[m][k]), e0, e1);
                    decay[m][k] = pair(ex2(e0), ex2(e1));
                }
                if (!WITH_Y) width_sum[m] += wv;
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float uv = m ? q.w : q.y;
                const Pair u = pair(uv, uv);
                Pair sum = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    h[m][k] = fma2(decay[m][k], h[m][k], mul2(u, b[k]));
                    if (WITH_Y) sum = k ? fma2(h[m][k], cc[k], sum) : mul2(h[m][k], cc[k]);
                }
                if (WITH_Y) {
                    float lo, hi;
                    halves(sum, lo, hi);
                    (m ? out.y : out.x) = lo + hi;
                }
            }
        }
        if (WITH_Y) {
#pragma unroll
            for (int t = 0; t < kTile; ++t) y[2 * (t * 16 + (lane / 2 % SH::Y ^ SH::y_key(t, y_chunk)))] = outs[t];
        }
        __syncwarp();
        const int t = t0 + i * kTile + my_t;
        if (!WITH_Y || !live || t >= t1) continue;
        Pair x[VH / 2], yv[VH / 2];
        unpack<VH>(xr, x);
        // a channel pair's parts, LANES of them, fill LANES / 2 entries
        const float4 *from = &sh.y[my_t][SH::Y * chunk];
        const int key = SH::y_key(my_t, chunk);
#pragma unroll
        for (int e = 0; e < VH / 2; ++e) {
            Pair q[LANES];
#pragma unroll
            for (int k = 0; k < LANES / 2; ++k) {
                const Pair2 f = *reinterpret_cast<const Pair2 *>(from + ((e * (LANES / 2) + k) ^ key));
                q[2 * k] = f.x;
                q[2 * k + 1] = f.y;
            }
#pragma unroll
            for (int o = LANES / 2; o >= 1; o >>= 1)
#pragma unroll
                for (int k = 0; k < o; ++k) q[k] = add2(q[k], q[k + o]);
            yv[e] = fma2(skip[e], x[e], q[0]);
        }
        if (p.z) {
            Pair z[VH / 2];
            unpack<VH>(zr, z);
#pragma unroll
            for (int e = 0; e < VH / 2; ++e) {                        // z / (1 + e^-z)
                float lo, hi;
                halves(mul2(z[e], pair(-kLog2e, -kLog2e)), lo, hi);
                halves(add2(pair(ex2(lo), ex2(hi)), pair(1.f, 1.f)), lo, hi);
                yv[e] = mul2(yv[e], mul2(z[e], pair(reciprocal(lo), reciprocal(hi))));
            }
        }
        const size_t to = (size_t)t * p.channels + c;
        T o;
        uint32_t *w = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
        for (int k = 0; k < VH / 2; ++k) {
            float lo, hi;
            halves(yv[k], lo, hi);
            if (p.out_f32) reinterpret_cast<float2 *>(static_cast<float *>(p.out) + to)[k] = make_float2(lo, hi);
            else w[k] = pack2(lo, hi);
        }
        if (!p.out_f32) *reinterpret_cast<T *>(static_cast<__nv_bfloat16 *>(p.out) + to) = o;
    }
    __syncwarp();                           // what is in shared memory has been read
}

// How a call's tokens are divided among warps.
struct ScanPlan {
    int piece;                  // tokens of a piece; 0: a warp takes whole sequences
    int pieces, empty;          // pieces, and further warps that look for sequences without tokens
    int units;                  // sequences, or pieces and those further ones
    int warps_per_group;
    float *ends, *widths, *begins;     // [pieces, channels, N], [pieces, channels], [pieces, channels, N]
};
constexpr int kEmptyPerWarp = 64;

enum Pass { kWhole, kEnds, kOutputs };

template <class SH, int PASS>
__global__ void __launch_bounds__(kPromptThreads, kPromptCtas) scan_kernel(const __grid_constant__ ScanProblem p, const __grid_constant__ ScanPlan plan) {
    extern __shared__ __align__(16) unsigned char smem[];
    typename SH::Shared &sh = reinterpret_cast<typename SH::Shared *>(smem)[threadIdx.x / 32];
    constexpr int N = SH::N;
    const int per_group = p.channels / p.groups, warps = plan.warps_per_group * p.groups, lane = threadIdx.x % 32;
    const int w = blockIdx.x * kPromptWarps + threadIdx.x / 32, unit = w / warps, group = w % warps / plan.warps_per_group;
    if (unit >= plan.units) return;
    const int c0 = group * per_group + w % plan.warps_per_group * SH::V, c1 = (group + 1) * per_group;
    // of a scanning lane: its two channels and where their states lie in an array [.., channels, N]
    const int c = c0 + 2 * (lane / SH::LANES), part = lane % SH::LANES;
    const bool live = c < c1;
    const size_t at = (size_t)c * N + 8 * part, all = (size_t)p.channels * N;
    Pair h[2][4], a[2][4];
    auto load = [&](const float *from, Pair (&v)[2][4]) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const Pair2 q = from && live ? *reinterpret_cast<const Pair2 *>(from + at + m * N + 4 * k) : Pair2{0, 0};
                v[m][2 * k] = q.x;
                v[m][2 * k + 1] = q.y;
            }
    };
    auto store = [&](float *to, const Pair (&v)[2][4]) {
        if (!live) return;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int k = 0; k < 2; ++k) *reinterpret_cast<Pair2 *>(to + at + m * N + 4 * k) = Pair2{v[m][2 * k], v[m][2 * k + 1]};
    };
    auto state_in = [&](int slot) { return p.state_in ? p.state_in + slot * all : nullptr; };
    load(p.a, a);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float lo, hi;
        halves(a[k / 4][k % 4], lo, hi);
        a[k / 4][k % 4] = pair(finite(lo), finite(hi));
    }
    float width_sum[2];

    if (PASS == kWhole) {
        const int slot = p.seqs.slot(unit);
        if (slot < 0) {
            if (lane == 0) raise_error(p.seqs.err, kErrInternal);
            return;
        }
        load(state_in(slot), h);
        scan_tokens<SH, true>(p, sh, p.seqs.begin(unit), p.seqs.end(unit), c0, c1, group, a, h, width_sum);
        if (p.state_out) store(p.state_out + slot * all, h);
        return;
    }
    const int t0 = unit * plan.piece, t1 = min(t0 + plan.piece, p.seqs.total);
    if (PASS == kEnds) {
        // the sequence that goes on behind this piece: what its state is at the piece's end, from its state at the piece's
        // beginning if that is known (or else from zero), and the widths' sum, by which the rest decays until then
        const int n = p.seqs.of(t1 - 1), b = p.seqs.begin(n), slot = p.seqs.slot(n);
        if (p.seqs.end(n) <= t1 || b >= t1 || slot < 0) return;
        load(b >= t0 ? state_in(slot) : nullptr, h);
        if (b >= t0 && p.state_in) store(plan.begins + unit * all, h);       // (state_out may be state_in, and is written by others)
        scan_tokens<SH, false>(p, sh, max(b, t0), t1, c0, c1, group, a, h, width_sum);
        store(plan.ends + unit * all, h);
        if (live && part == 0) *reinterpret_cast<float2 *>(plan.widths + (size_t)unit * p.channels + c) = make_float2(width_sum[0], width_sum[1]);
        return;
    }
    if (unit >= plan.pieces) {
        const int first = (unit - plan.pieces) * kEmptyPerWarp;
        for (int n = first; n < min(first + kEmptyPerWarp, p.seqs.n); ++n) {
            if (p.seqs.end(n) > p.seqs.begin(n)) continue;
            const int slot = p.seqs.slot(n);
            if (slot < 0) {
                if (lane == 0) raise_error(p.seqs.err, kErrInternal);
                continue;
            }
            if (!p.state_out || p.state_out == p.state_in) continue;
            load(state_in(slot), h);
            store(p.state_out + slot * all, h);
        }
        return;
    }
    for (int t = t0, n = p.seqs.of(t0); t < t1 && n < p.seqs.n; ++n) {
        const int b = p.seqs.begin(n), e = p.seqs.end(n), slot = p.seqs.slot(n);
        if (e <= b || e <= t || b >= t1) {
            if (b >= t1) break;
            continue;
        }
        if (slot < 0) {
            if (lane == 0) raise_error(p.seqs.err, kErrInternal);
            continue;
        }
        if (b >= t0) {
            load(e > t1 && p.state_in ? plan.begins + unit * all : state_in(slot), h);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) h[k / 4][k % 4] = 0;
#pragma unroll 4
            for (int j = b / plan.piece; j < unit; ++j) {
                Pair end[2][4];
                load(plan.ends + j * all, end);
                const float2 w = live ? *reinterpret_cast<const float2 *>(plan.widths + (size_t)j * p.channels + c) : make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    // e^(a sum of widths) may leave fp32 where what a state becomes does not (and zero stays zero): by three
                    // factors, none of which leaves it, as 2^378 makes infinity, and 2^-378 zero, of any number
                    float e0, e1;
                    const float wv = k < 4 ? w.x : w.y;
                    halves(mul2(pair(wv, wv), a[k / 4][k % 4]), e0, e1);
                    const auto third = [](float e) { return ex2(fminf(fmaxf(e, -378.f), 378.f) * (1.f / 3)); };
                    const Pair f = pair(third(e0), third(e1));
                    Pair &v = h[k / 4][k % 4];
                    v = add2(mul2(mul2(mul2(v, f), f), f), end[k / 4][k % 4]);
                }
            }
        }
        scan_tokens<SH, true>(p, sh, max(b, t0), min(e, t1), c0, c1, group, a, h, width_sum);
        if (e <= t1 && p.state_out) store(p.state_out + slot * all, h);
        t = e;
    }
}

template <int N>
ScanPlan plan_scan(int n_seqs, int total, int channels, int groups, int max_len) {
    using SH = Shape<N>;
    ScanPlan s{};
    s.warps_per_group = (channels / groups + SH::V - 1) / SH::V;
    s.units = n_seqs;
    const long warps = (long)s.warps_per_group * groups, at_once = (long)kPromptCtas * kPromptWarps * multiprocessor_count();
    const long longest = max_len > 0 && max_len < total ? max_len : total;
    // Tokens that one warp walks through, one after another: whole sequences, or pieces twice.  Measured, 4096 channels x 16 states,
    // whole and in pieces: 16 x 512 tokens 180 and 216 us, 32 x 500 293 and 355, 4 x 2000 244 and 253, 1 x 100 14.8 and 17.5; but 1 x 600
    // 74 and 35, 1 x 8192 990 and 259; 7 x 60 .. 4000 of 1536 x 64 456 and 247
    const long whole = max(longest, (long)total * warps / at_once);
    const long halves = 2 * max(64L, (long)total * warps / at_once);
    if (whole <= halves * 5 / 4) return s;
    const long pieces = max(1L, at_once / warps);
    long piece = ((total + pieces - 1) / pieces + kTile - 1) / kTile * kTile;
    piece = min((long)kMaxPiece, max(64L, piece));
    s.piece = (int)piece;
    s.units = s.pieces = (int)((total + piece - 1) / piece);
    return s;
}

template <int N>
cudaError_t launch(const ScanProblem &p) {
    using SH = Shape<N>;
    if (!p.seqs.cu || p.max_len == 1) {
        constexpr int CH = 2 * kScanThreads / (N / 4);
        const long ctas = (p.channels + CH - 1) / CH;
        const int step = (int)min((long)p.seqs.n, max(1L, 7L * multiprocessor_count() / ctas));
        step_kernel<N><<<(unsigned)(ctas * step), kScanThreads, 0, p.stream>>>(p, step);
        return cudaGetLastError();
    }
    constexpr int smem = kPromptWarps * (int)sizeof(typename SH::Shared);
    ScanPlan s = plan_scan<N>(p.seqs.n, p.seqs.total, p.channels, p.groups, p.max_len);
    const long warps = (long)s.warps_per_group * p.groups;
    using Fn = void (*)(const ScanProblem, const ScanPlan);
    auto run = [&](Fn fn, long units) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        s.units = (int)units;
        fn<<<(unsigned)((units * warps + kPromptWarps - 1) / kPromptWarps), kPromptThreads, smem, p.stream>>>(p, s);
        return cudaGetLastError();
    };
    if (s.piece == 0) return run(scan_kernel<SH, kWhole>, p.seqs.n);
    const size_t states = (size_t)s.pieces * p.channels * N;
    s.ends = static_cast<float *>(p.workspace);
    s.begins = s.ends + states;
    s.widths = s.begins + states;
    // sequences without tokens have nobody who keeps their state, unless it stays where it is, or looks at their slot
    if ((p.state_out && p.state_out != p.state_in) || p.seqs.slots) s.empty = (p.seqs.n + kEmptyPerWarp - 1) / kEmptyPerWarp;
    const cudaError_t e = run(scan_kernel<SH, kEnds>, s.pieces);
    return e != cudaSuccess ? e : run(scan_kernel<SH, kOutputs>, s.pieces + s.empty);
}

template <int N>
size_t workspace_bytes(int n_seqs, int total, int channels, int groups, int max_len) {
    const ScanPlan s = plan_scan<N>(n_seqs, total, channels, groups, max_len);
    return (size_t)s.pieces * channels * (2 * N + 1) * 4;
}

}  // namespace

size_t ssm_scan_workspace_bytes(int n_seqs, int total, int channels, int n_state, int groups, int max_len) {
    if (max_len == 1 || total == 0) return 0;
    switch (n_state) {
        case 16: return workspace_bytes<16>(n_seqs, total, channels, groups, max_len);
        case 32: return workspace_bytes<32>(n_seqs, total, channels, groups, max_len);
        case 64: return workspace_bytes<64>(n_seqs, total, channels, groups, max_len);
        default: return workspace_bytes<128>(n_seqs, total, channels, groups, max_len);
    }
}

cudaError_t launch_ssm_scan(const ScanProblem &p) {
    switch (p.n_state) {
        case 16: return launch<16>(p);
        case 32: return launch<32>(p);
        case 64: return launch<64>(p);
        default: return launch<128>(p);
    }
}

}  // namespace gdn
