// gdn_ssm_scan: per channel c, with N numbers of state,
//     h[n] = exp(D a[c, n]) h[n] + D x B[n],   y = (sum_n h[n] C[n] + skip x) z / (1 + e^-z),   D = softplus(dt + bias).
//
// A channel's states lie in the registers of N / S neighbouring lanes, S each, for as long as its sequence lasts.
#include "layer_ops.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

constexpr int kScanThreads = 128;
// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^-|v|, without a branch and to a few units in the last place however small e is.
// The exponential's argument is corrected for its rounding; log(1 + e) = 2 artanh(q) with q = e / (2 + e) <= 1/3, by its series.
__device__ __forceinline__ float softplus(float v) {
    const float m = -fabsf(v), t = m * kLog2e;
    const float r = fmaf(m, 1.925963033500e-8f, fmaf(m, kLog2e, -t));       // what t lacks of m log2 e
    float e = ex2(t);
    e = fmaf(e, r * 0.69314718f, e);
    const float q = e * reciprocal(2.f + e), q2 = q * q;
    float s = fmaf(q2, 1.f / 13, 1.f / 11);
    s = fmaf(q2, s, 1.f / 9);
    s = fmaf(q2, s, 1.f / 7);
    s = fmaf(q2, s, 1.f / 5);
    s = fmaf(q2, s, 1.f / 3);
    s = fmaf(q2, s, 1.f);
    return fmaf(2.f * q, s, fmaxf(v, 0.f));
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
        const float v = __bfloat162float(p.dt[t * p.dt_stride + c]) + bias, d = p.softplus ? softplus(v) : v;
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
struct alignas(16) Pair2 { Pair x, y; };

constexpr int kTile = 32;                   // tokens of one turn
constexpr int kPromptThreads = 256;         // 4 warps that scan, 4 that prepare the next tile and finish the last one
constexpr int kMaxPiece = 2048;             // tokens of a piece of a scan in pieces

template <int N_, int S_>
struct Shape {
    static constexpr int N = N_, S = S_, LANES = N / S, V = 32 / LANES, CH = 4 * V;     // V: channels of a warp
    // A tile's raw rows and vectors are asked for DEEP turns before it is prepared, to cover a read of memory; that of turn
    // i + 1 + DEEP while tile i is scanned, so they need two places more.  (States of 128: two CTAs an SM leave room for less.)
    static constexpr int DEEP = N == 128 ? 2 : 4, RING = DEEP + 2;
    struct Tile {
        float2 du[kTile][CH];               // step width D (times log2 e) and D x
        float y[4 * kTile][36];             // by token and warp: the lanes' parts of y; 4 floats of padding against bank conflicts
    };
    struct Shared {
        Tile tile[2];                       // prepared, and scanned
        uint4 bc[RING][kTile][N / 4];      // by 4 states: B and C as they came, in bf16
        __nv_bfloat16 x[RING][128][V], dt[RING][128][V], z[RING][128][V];      // by preparing thread
    };
    // Row id = 4 token + warp of V channels of du holds its pairs of channels in the order pair ^ key, so that 8 rows written at
    // once meet few banks twice.
    __device__ static __forceinline__ int key(int id) { return V == 8 ? (id >> 1) & 3 : V == 4 ? (id >> 2) & 1 : 0; }
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
__device__ __forceinline__ void unpack(const typename Bits<V>::T &u, float (&x)[V]) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&u);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

// All of the CTA's warps meet here, those that scan and those that prepare, from different places.
__device__ __forceinline__ void turn() { asm volatile("barrier.sync 1, %0;" ::"n"(kPromptThreads) : "memory"); }

// Tokens [t0, t1) of one sequence for the CTA's channels c0 .. and below c1.  h: a scanning lane's part of its channel's
// state; *width_sum: the sum of its step widths (times log2 e).
template <class SH, bool WITH_Y>
__device__ __forceinline__ void scan_tokens(const ScanProblem &p, typename SH::Shared &sh, int t0, int t1, int c0, int c1, int group,
                                            const Pair (&a)[SH::S / 2], Pair (&h)[SH::S / 2], float *width_sum) {
    constexpr int S = SH::S, N = SH::N, V = SH::V, LANES = SH::LANES;
    const int n = (t1 - t0 + kTile - 1) / kTile;
    if (n <= 0) return;
    if (threadIdx.x < 128) {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, part = lane % LANES;
        float total = 0.f;
        turn();
        // Steps go by batches: a batch's exponentials depend on nothing but its inputs, which are asked for a batch ahead
        constexpr int BATCH = S == 4 ? 4 : 2;
        struct Step { float2 w; uint4 bc[S / 4]; };
        const int ch = lane / LANES;
        for (int i = 0; i < n; ++i) {
            typename SH::Tile &s = sh.tile[i & 1];
            const float2 *du = &s.du[0][warp * V];
            const uint4 *bc = &sh.bc[i % SH::RING][0][S / 4 * part];
            float *y = &s.y[warp][lane];
            auto fetch = [&](int t, Step (&q)[BATCH]) {
#pragma unroll
                for (int j = 0; j < BATCH; ++j) {
                    q[j].w = du[(t + j) * SH::CH + (ch ^ 2 * SH::key(4 * (t + j) + warp))];
#pragma unroll
                    for (int k = 0; k < S / 4; ++k) {
                        const uint4 *from = bc + (t + j) * (N / 4) + k;
                        if (WITH_Y) q[j].bc[k] = *from;
                        else {
                            const uint2 only = *reinterpret_cast<const uint2 *>(from);
                            q[j].bc[k].x = only.x, q[j].bc[k].y = only.y;
                        }
                    }
                }
            };
            Step next[BATCH];
            fetch(0, next);
#pragma unroll
            for (int t = 0; t < kTile; t += BATCH) {
                Step q[BATCH];
#pragma unroll
                for (int j = 0; j < BATCH; ++j) q[j] = next[j];
                if (t + BATCH < kTile) fetch(t + BATCH, next);
                Pair decay[BATCH][S / 2];
#pragma unroll
                for (int j = 0; j < BATCH; ++j) {
                    const Pair w = pair(q[j].w.x, q[j].w.x);
#pragma unroll
                    for (int k = 0; k < S / 2; ++k) {
                        float e0, e1;
                        halves(mul2(w, a[k]), e0, e1);
                        decay[j][k] = pair(ex2(e0), ex2(e1));
                    }
                }
#pragma unroll
                for (int j = 0; j < BATCH; ++j) {
                    const Pair u = pair(q[j].w.y, q[j].w.y);
                    Pair sum = 0;
#pragma unroll
                    for (int k = 0; k < S / 2; ++k) {
                        const uint32_t b = k & 1 ? q[j].bc[k / 2].y : q[j].bc[k / 2].x;
                        h[k] = fma2(decay[j][k], h[k], mul2(u, pair(bf16_lo(b), bf16_hi(b))));
                        if (WITH_Y) {
                            const uint32_t c = k & 1 ? q[j].bc[k / 2].w : q[j].bc[k / 2].z;
                            const Pair cv = pair(bf16_lo(c), bf16_hi(c));
                            sum = k ? fma2(h[k], cv, sum) : mul2(h[k], cv);
                        }
                    }
                    if (WITH_Y) {
                        float lo, hi;
                        halves(sum, lo, hi);
                        y[(t + j) * 4 * 36] = lo + hi;
                    } else {
                        total += q[j].w.x;
                    }
                }
            }
            turn();
        }
        if (!WITH_Y) *width_sum = total;
        return;
    }
    const int id = threadIdx.x - 128, c = c0 + V * (id % 4);
    const bool live = c < c1;
    float bias[V], skip[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        bias[e] = live && p.dt_bias ? __ldg(p.dt_bias + c + e) : 0.f;
        skip[e] = live && WITH_Y && p.skip ? __ldg(p.skip + c + e) : 0.f;
    }
    using T = typename Bits<V>::T;
    auto ask = [&](int i) {
        if (i < n) {
            const int t = t0 + i * kTile + id / 4, slot = i % SH::RING;
            const bool there = live && t < t1;
            copy_async<2 * V>(sh.x[slot][id], p.x + (there ? t * p.x_stride + c : 0), there);
            copy_async<2 * V>(sh.dt[slot][id], p.dt + (there ? t * p.dt_stride + c : 0), there);
            if (WITH_Y && p.z) copy_async<2 * V>(sh.z[slot][id], p.z + (there ? t * p.z_stride + c : 0), there);
#pragma unroll
            for (int k = 0; k < N / 16; ++k) {
                const int at = id + k * 128, tv = t0 + i * kTile + at / (N / 4), e = group * N + at % (N / 4) * 4;
                uint2 *to = reinterpret_cast<uint2 *>(&sh.bc[slot][0][at]);
                copy_async<8>(to, p.b + (tv < t1 ? tv * p.b_stride + e : 0), tv < t1);
                if (WITH_Y) copy_async<8>(to + 1, p.c + (tv < t1 ? tv * p.c_stride + e : 0), tv < t1);
            }
        }
        copy_commit();                      // (a group for every turn, so that their number says which have arrived)
    };
    T x1{}, z1{}, x0{}, z0{};               // of the tile that is scanned, and of the one before it
    auto prepare = [&](int i) {
        typename SH::Tile &s = sh.tile[i & 1];
        copy_wait<SH::DEEP - 1>();
        const int slot = i % SH::RING;
        const T xr = *reinterpret_cast<const T *>(sh.x[slot][id]), dr = *reinterpret_cast<const T *>(sh.dt[slot][id]);
        x0 = x1, z0 = z1, x1 = xr;
        if (WITH_Y && p.z) z1 = *reinterpret_cast<const T *>(sh.z[slot][id]);
        float x[V], d[V];
        unpack<V>(xr, x);
        unpack<V>(dr, d);
        const bool inside = t0 + i * kTile + id / 4 < t1;
        float4 *to = reinterpret_cast<float4 *>(&s.du[id / 4][V * (id % 4)]);
        const int key = SH::key(id);
#pragma unroll
        for (int e = 0; e < V; ++e) d[e] += bias[e];
        if (p.softplus) {
#pragma unroll
            for (int e = 0; e < V; ++e) d[e] = softplus(d[e]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            d[e] = inside ? d[e] : 0.f;                               // (a row beyond the end changes nothing)
            x[e] *= d[e];
            d[e] *= kLog2e;
        }
#pragma unroll
        for (int e = 0; e < V / 2; ++e) to[e ^ key] = make_float4(d[2 * e], x[2 * e], d[2 * e + 1], x[2 * e + 1]);
        ask(i + SH::DEEP);
    };
    auto finish = [&](int i, const T &xr, const T &zr) {
        const int t = t0 + i * kTile + id / 4;
        if (!WITH_Y || !live || t >= t1) return;
        float x[V], z[V], y[V];
        unpack<V>(xr, x);
        unpack<V>(zr, z);
        const float *from = sh.tile[i & 1].y[id];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float q[LANES];
#pragma unroll
            for (int k = 0; k < LANES / 4; ++k) {
                const float4 f = *reinterpret_cast<const float4 *>(from + e * LANES + 4 * k);
                q[4 * k] = f.x; q[4 * k + 1] = f.y; q[4 * k + 2] = f.z; q[4 * k + 3] = f.w;
            }
#pragma unroll
            for (int o = LANES / 2; o >= 1; o >>= 1)
#pragma unroll
                for (int k = 0; k < o; ++k) q[k] += q[k + o];
            y[e] = fmaf(skip[e], x[e], q[0]);
        }
        if (p.z) {
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] *= silu(z[e]);
        }
        const size_t to = (size_t)t * p.channels + c;
        if (p.out_f32) {
            float2 *o = reinterpret_cast<float2 *>(static_cast<float *>(p.out) + to);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) o[k] = make_float2(y[2 * k], y[2 * k + 1]);
        } else {
            T o;
            uint32_t *w = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) w[k] = pack2(y[2 * k], y[2 * k + 1]);
            *reinterpret_cast<T *>(static_cast<__nv_bfloat16 *>(p.out) + to) = o;
        }
    };
    for (int i = 0; i < SH::DEEP; ++i) ask(i);
    prepare(0);
    turn();
    for (int i = 0; i < n; ++i) {
        // x1, z1 are tile i's; after prepare(i + 1) they are x0, z0
        const T xp = x0, zp = z0;
        if (i + 1 < n) prepare(i + 1);
        else x0 = x1, z0 = z1;
        if (i > 0) finish(i - 1, xp, zp);
        turn();
    }
    finish(n - 1, x0, z0);
}

// How a call's tokens are divided among CTAs.
struct ScanPlan {
    int piece;                  // tokens of a piece; 0: a CTA takes whole sequences
    int pieces, empty;          // pieces, and further CTAs that look for sequences without tokens
    int ctas_per_group;
    float *ends, *widths, *begins;     // [pieces, channels, N], [pieces, channels], [pieces, channels, N]
};
constexpr int kEmptyPerCta = 64;

enum Pass { kWhole, kEnds, kOutputs };

template <class SH, int PASS>
__global__ void __launch_bounds__(kPromptThreads, 2) scan_kernel(const __grid_constant__ ScanProblem p, const __grid_constant__ ScanPlan plan) {
    extern __shared__ __align__(16) unsigned char smem[];
    typename SH::Shared &sh = *reinterpret_cast<typename SH::Shared *>(smem);
    constexpr int N = SH::N, S = SH::S;
    const int per_group = p.channels / p.groups, ctas = plan.ctas_per_group * p.groups;
    const int unit = blockIdx.x / ctas, group = blockIdx.x % ctas / plan.ctas_per_group;
    const int c0 = group * per_group + blockIdx.x % plan.ctas_per_group * SH::CH, c1 = (group + 1) * per_group;
    // of a scanning lane: its channel and where its states lie in an array [.., channels, N]
    const int c = c0 + threadIdx.x / SH::LANES, part = threadIdx.x % SH::LANES;
    const bool live = threadIdx.x < 128 && c < c1;
    const size_t at = (size_t)c * N + S * part, all = (size_t)p.channels * N;
    Pair h[S / 2], a[S / 2];
    auto load = [&](const float *from, Pair (&v)[S / 2]) {
#pragma unroll
        for (int k = 0; k < S / 4; ++k) {
            const Pair2 q = from && live ? *reinterpret_cast<const Pair2 *>(from + at + 4 * k) : Pair2{0, 0};
            v[2 * k] = q.x;
            v[2 * k + 1] = q.y;
        }
    };
    auto store = [&](float *to, const Pair (&v)[S / 2]) {
        if (!live) return;
#pragma unroll
        for (int k = 0; k < S / 4; ++k) *reinterpret_cast<Pair2 *>(to + at + 4 * k) = Pair2{v[2 * k], v[2 * k + 1]};
    };
    auto state_in = [&](int slot) { return p.state_in ? p.state_in + slot * all : nullptr; };
    load(p.a, a);
    float width_sum;

    if (PASS == kWhole) {
        const int slot = p.seqs.slot(unit);
        if (slot < 0) {
            if (threadIdx.x == 0) raise_error(p.seqs.err, kErrInternal);
            return;
        }
        load(state_in(slot), h);
        scan_tokens<SH, true>(p, sh, p.seqs.begin(unit), p.seqs.end(unit), c0, c1, group, a, h, &width_sum);
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
        scan_tokens<SH, false>(p, sh, max(b, t0), t1, c0, c1, group, a, h, &width_sum);
        store(plan.ends + unit * all, h);
        if (live && part == 0) plan.widths[(size_t)unit * p.channels + c] = width_sum;
        return;
    }
    if (unit >= plan.pieces) {
        const int first = (unit - plan.pieces) * kEmptyPerCta;
        for (int n = first; n < min(first + kEmptyPerCta, p.seqs.n); ++n) {
            if (p.seqs.end(n) > p.seqs.begin(n)) continue;
            const int slot = p.seqs.slot(n);
            if (slot < 0) {
                if (threadIdx.x == 0) raise_error(p.seqs.err, kErrInternal);
                continue;
            }
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
            if (threadIdx.x == 0) raise_error(p.seqs.err, kErrInternal);
            continue;
        }
        if (b >= t0) {
            load(e > t1 && p.state_in ? plan.begins + unit * all : state_in(slot), h);
        } else {
#pragma unroll
            for (int k = 0; k < S / 2; ++k) h[k] = 0;
#pragma unroll 4
            for (int j = b / plan.piece; j < unit; ++j) {
                Pair end[S / 2];
                load(plan.ends + j * all, end);
                const float w = live ? plan.widths[(size_t)j * p.channels + c] : 0.f;
#pragma unroll
                for (int k = 0; k < S / 2; ++k) {
                    float e0, e1;
                    halves(mul2(pair(w, w), a[k]), e0, e1);
                    h[k] = fma2(pair(ex2(e0), ex2(e1)), h[k], end[k]);
                }
            }
        }
        scan_tokens<SH, true>(p, sh, max(b, t0), min(e, t1), c0, c1, group, a, h, &width_sum);
        if (e <= t1 && p.state_out) store(p.state_out + slot * all, h);
        t = e;
    }
}

// S: states of a lane.
template <int N> struct ShapeOf { using T = Shape<N, N == 128 ? 8 : 4>; };

template <int N>
ScanPlan plan_scan(int n_seqs, int total, int channels, int groups, int max_len) {
    using SH = typename ShapeOf<N>::T;
    ScanPlan s{};
    s.ctas_per_group = (channels / groups + SH::CH - 1) / SH::CH;
    const long ctas = (long)s.ctas_per_group * groups, at_once = 2L * multiprocessor_count();
    const long longest = max_len > 0 && max_len < total ? max_len : total;
    // Tokens that one CTA walks through, one after another: whole sequences, or pieces twice
    const long whole = max(longest, (long)total * ctas / at_once);
    const long halves = 2 * max(64L, (long)total * ctas / at_once);
    if (whole <= halves * 5 / 4) return s;
    const long pieces = max(1L, at_once / ctas);
    long piece = ((total + pieces - 1) / pieces + kTile - 1) / kTile * kTile;
    piece = min((long)kMaxPiece, max(64L, piece));
    s.piece = (int)piece;
    s.pieces = (int)((total + piece - 1) / piece);
    return s;
}

template <int N>
cudaError_t launch(const ScanProblem &p) {
    using SH = typename ShapeOf<N>::T;
    if (!p.seqs.cu || p.max_len == 1) {
        constexpr int CH = kScanThreads / (N / 4);
        const long ctas = (long)((p.channels + CH - 1) / CH) * p.seqs.n;
        step_kernel<N><<<(unsigned)ctas, kScanThreads, 0, p.stream>>>(p);
        return cudaGetLastError();
    }
    constexpr int smem = (int)sizeof(typename SH::Shared);
    ScanPlan s = plan_scan<N>(p.seqs.n, p.seqs.total, p.channels, p.groups, p.max_len);
    const long ctas = (long)s.ctas_per_group * p.groups;
    using Fn = void (*)(const ScanProblem, const ScanPlan);
    auto run = [&](Fn fn, long units) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        fn<<<(unsigned)(units * ctas), kPromptThreads, smem, p.stream>>>(p, s);
        return cudaGetLastError();
    };
    if (s.piece == 0) return run(scan_kernel<SH, kWhole>, p.seqs.n);
    const size_t states = (size_t)s.pieces * p.channels * N;
    s.ends = static_cast<float *>(p.workspace);
    s.begins = s.ends + states;
    s.widths = s.begins + states;
    if (p.state_out && p.state_out != p.state_in) s.empty = (p.seqs.n + kEmptyPerCta - 1) / kEmptyPerCta;
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
