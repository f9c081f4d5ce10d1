// What the attention kernels share: the unit line of a call, masks, and small conversions.
#pragma once

#include "kv_cache.cuh"
#include "sm100.cuh"

namespace gdn {
namespace attend {

constexpr int kMaxSplitCtas = 1024;   // CTAs of the split kernel, and
constexpr int kMaxTcCtas = 256;       // of the tensor-core kernel, that workspaces have room for

// One entry a merge CTA reads: the item's first CTA and the slot it used there, and its last CTA (-1: the item
// did not cross CTAs).
struct MergeMeta {
    int first, slot, last, n, h, mt;
};
constexpr size_t kMetaBytes = (kMaxSplitCtas * sizeof(MergeMeta) + 255) / 256 * 256;

struct SplitPlan {
    MergeMeta *meta;      // by item where the items are at most the CTAs, else by first CTA
    float *parts;         // two slots a CTA: its first segment, and one that starts later in its range
    int meta_by_item, mt_max;
};

// A sequence as the kernels see it: first query row, queries, cached tokens (cut to the call's bounds).
struct Sequence {
    int q0, qlen, kvlen;
};

__device__ __forceinline__ Sequence load_sequence(const AttendProblem &p, int n) {
    Sequence s;
    s.q0 = min(max(__ldg(p.cu + n), 0), p.total);
    s.qlen = min(min(max(__ldg(p.cu + n + 1), s.q0), p.total) - s.q0, p.max_q_len);
    s.kvlen = min(max(__ldg(p.kv_lens + n), 0), p.max_kv_len);
    return s;
}

// Lengths beyond the call's bounds are recorded (one thread of every CTA looks at some sequences).
__device__ __forceinline__ void report_lengths(const AttendProblem &p, int cta) {
    for (int n = cta; n < p.n_seqs; n += gridDim.x)
        if (__ldg(p.cu + n + 1) - __ldg(p.cu + n) > p.max_q_len || __ldg(p.kv_lens + n) > p.max_kv_len ||
            __ldg(p.kv_lens + n) < 0 || __ldg(p.cu + n + 1) > p.total || __ldg(p.cu + n) < 0 || __ldg(p.cu + n + 1) < __ldg(p.cu + n))
            raise_error(p.err, kErrInternal);
}

template <int ROWS>
__host__ __device__ __forceinline__ int row_tiles(int qlen, int group) {
    return (qlen * group + ROWS - 1) / ROWS;   // rows of a call stay below 2^31 - 4096
}

// The tokens that ROWS consecutive query rows see together, in tiles: [0, near) of the sinks, then from `far` on.
struct Item {
    int lo_pos, hi_pos;   // positions of its first and last row
    int near_tiles, far_tile, tiles;
    __device__ __forceinline__ int token(int j, int tile) const { return (j < near_tiles ? j : far_tile + j - near_tiles) * tile; }
    // Does every row see all of tokens [a, b)?
    __device__ __forceinline__ bool all_seen(int a, int b, int window, int sinks) const {
        return b - 1 <= lo_pos && (window == 0 || a > hi_pos - window || b <= sinks);
    }
};

__device__ __forceinline__ bool sees(int pos, int token, int window, int sinks) {
    return token <= pos && (window == 0 || token > pos - window || token < sinks);
}

// Does any of the rows at lo_pos .. hi_pos see any of tokens [a, b)?  A block of the cache that none sees is not looked up: the
// pages that a window has left may belong to somebody else.
__device__ __forceinline__ bool in_sight(int lo_pos, int hi_pos, int a, int b, int window, int sinks) {
    return a <= hi_pos && (window == 0 || b - 1 > lo_pos - window || a < sinks);
}

template <int ROWS, int TILE>
__device__ __forceinline__ Item make_item(const AttendProblem &p, const Sequence &s, int group, int mt) {
    Item it;
    const int i0 = mt * ROWS / group, i1 = min(s.qlen - 1, (mt * ROWS + ROWS - 1) / group);
    it.lo_pos = s.kvlen - s.qlen + i0;
    it.hi_pos = s.kvlen - s.qlen + i1;
    const int end = max(0, it.hi_pos + 1), end_tile = (end + TILE - 1) / TILE;
    it.near_tiles = 0;
    it.far_tile = 0;
    if (p.window) {
        const int near = (min(p.sinks, end) + TILE - 1) / TILE, far = max(0, it.lo_pos - p.window + 1) / TILE;
        if (far > near) {
            it.near_tiles = near;
            it.far_tile = far;
        }
    }
    it.tiles = max(1, it.near_tiles + max(0, end_tile - it.far_tile));   // an item that sees nothing still writes its zeros
    return it;
}

// Units of all heads of a sequence.
template <int ROWS, int TILE>
__device__ __forceinline__ int sequence_cost(const AttendProblem &p, const Sequence &s, int group) {
    int c = 0;
    const int mts = row_tiles<ROWS>(s.qlen, group);
    for (int mt = 0; mt < mts; ++mt) c += make_item<ROWS, TILE>(p, s, group, mt).tiles;
    return c * p.pool.hkv;
}

// Powers of two, down * up = 1, that bring a row with this largest magnitude below 2: bf16 components then turn
// to fp16 exactly, except ones below 2^-14 of the largest, which keep an error below 2^-24 of it.  A row of zeros, or
// one with an infinity or NaN, is left as it is.
__device__ __forceinline__ void power_of_two_scale(uint32_t big, float &down, float &up) {
    const int e = (int)(big >> 23) - 127;   // big >= 0
    const int k = big == 0 || e == 128 ? 0 : max(e, -126);
    down = k == 127 ? 5.877471754111438e-39f : __uint_as_float((uint32_t)(127 - k) << 23);   // 2^-127 is subnormal
    up = __uint_as_float((uint32_t)(127 + k) << 23);
}

__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float f) {
    const __half2 h = __floats2half2_rn(bf16_lo(w) * f, bf16_hi(w) * f);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 2^x by the hardware's approximation (relative error 2^-22); results below 2^-126 are 0.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations in one instruction: (a, b) = (a, b) * f + c, and (a, b) += (c, d).
__device__ __forceinline__ void fma2(float &a, float &b, float f, float c) {
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n mov.b64 z, {%3, %3};\n"
        " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
        : "+f"(a), "+f"(b)
        : "f"(f), "f"(c));
}
__device__ __forceinline__ void add2(float &a, float &b, float c, float d) {
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}

__device__ __forceinline__ void lds128(uint32_t a, uint32_t (&w)[4]) {
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a) : "memory");
}

// N consecutive outputs from element `at` of `out`, rounded once to its type.
template <int N>
__device__ __forceinline__ void store_row(const AttendProblem &p, size_t at, const float (&y)[N]) {
    if (p.out_f32) {
        float *o = static_cast<float *>(p.out) + at;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            if constexpr (N == 2) *reinterpret_cast<float2 *>(o) = make_float2(y[0], y[1]);
            else *reinterpret_cast<float4 *>(o + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
        }
        return;
    }
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + at;
    uint32_t w[N / 2];
    static_assert(N == 2 || N % 4 == 0, "pieces of 4, 8 or 16 bytes");
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    if constexpr (N >= 8) {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) reinterpret_cast<uint4 *>(o)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (N == 4) {
        *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
    } else {
        *reinterpret_cast<uint32_t *>(o) = w[0];
    }
}

// Launch as the programmatic dependent of the stream's last kernel: its CTAs may become resident early and wait
// for that kernel's end with grid_dependency_wait.
template <typename... P, typename... A>
cudaError_t launch_after(cudaStream_t stream, dim3 grid, int threads, size_t smem, void (*fn)(P...), const A &...args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

// Joins the parts of the items that cross CTAs, meta by first CTA: a warp per row, lanes over the columns.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ AttendProblem p, const MergeMeta *meta, const float *parts) {
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31, row = blockIdx.y * 8 + (threadIdx.x >> 5), group = p.hq / p.pool.hkv;
    sm100::grid_dependency_wait();
    const MergeMeta mm = meta[blockIdx.x];
    if (mm.last < 0) return;
    const Sequence s = load_sequence(p, mm.n);
    const int grow = mm.mt * ROWS + row;
    if (grow / group >= s.qlen) return;
    const size_t stride = ROWS * D + 2 * ROWS;
    const int count = mm.last - mm.first + 1;
    auto part = [&](int k) { return parts + (size_t)(2 * (mm.first + k) + (k == 0 ? mm.slot : 0)) * stride; };
    float top = -INFINITY;
    for (int k = lane; k < count; k += 32) top = fmaxf(top, part(k)[ROWS * D + row]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == -INFINITY ? 0.f : top;
    float l = 0.f, y[PER] = {};
    for (int k0 = 0; k0 < count; k0 += 32) {
        // a lane to a part for the weights, then the parts one after another, eight asked for at a time
        const bool mine = k0 + lane < count;
        const float w = mine ? exp2f(part(k0 + lane)[ROWS * D + row] - base) : 0.f;
        if (mine) l = fmaf(w, part(k0 + lane)[ROWS * D + ROWS + row], l);
        const int many = min(32, count - k0);
#pragma unroll 8
        for (int k = 0; k < many; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            const float *o = part(k0 + k) + row * D + lane * PER;
#pragma unroll
            for (int e = 0; e < PER; e += 2) {
                const float2 x = *reinterpret_cast<const float2 *>(o + e);
                y[e] = fmaf(wk, x.x, y[e]);
                y[e + 1] = fmaf(wk, x.y, y[e + 1]);
            }
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < PER; ++e) y[e] *= inv;
    store_row<PER>(p, ((size_t)(s.q0 + grow / group) * p.hq + mm.h * group + grow % group) * D + lane * PER, y);
}

}  // namespace attend
}  // namespace gdn
