// What the kernels around the recurrence share: the sequences' conventions (include/gdn.h) and the problems that the
// entry points pass to the launchers.
#pragma once

#include <cuda.h>

#include "kv_cache.cuh"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float silu(float z) { return z * reciprocal(1.f + ex2(-kLog2e * z)); }

// Pairs of fp32 numbers in one 64-bit register: a product or fused product-sum of both is one instruction.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float x, float y) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void halves(Pair p, float &x, float &y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p)); }
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Sequences of one call, and the states that they carry.
struct Sequences {
    int n, total;
    const int32_t *cu;          // null: one token each
    const int32_t *slots;       // null: slot n
    int n_slots;
    unsigned int *err;
    __device__ __forceinline__ int of(int t) const { return cu ? sequence_of(cu, n, t) : t; }
    __device__ __forceinline__ int begin(int i) const { return cu ? min(max(cu[i], 0), total) : i; }
    __device__ __forceinline__ int end(int i) const { return cu ? min(max(cu[i + 1], 0), total) : i + 1; }
    // the slot of sequence i, or -1 where there is none
    __device__ __forceinline__ int slot(int i) const {
        const int s = slots ? slots[i] : i;
        return (unsigned)s < (unsigned)n_slots ? s : -1;
    }
};

struct ConvProblem {
    Sequences seqs;
    int channels, width;
    const __nv_bfloat16 *x;
    long long x_stride;
    const float *weight, *bias;
    int silu;
    const __nv_bfloat16 *state_in;
    __nv_bfloat16 *state_out;
    __nv_bfloat16 *out;
    cudaStream_t stream;
};
cudaError_t launch_short_conv(const ConvProblem &p);

struct ScanProblem {
    Sequences seqs;
    int channels, n_state, groups, max_len;
    const __nv_bfloat16 *x, *dt, *z, *b, *c;
    long long x_stride, dt_stride, z_stride, b_stride, c_stride;
    const float *a, *skip, *dt_bias;
    int softplus;
    const float *state_in;
    float *state_out;
    void *out;
    int out_f32;
    void *workspace;
    cudaStream_t stream;
};
cudaError_t launch_ssm_scan(const ScanProblem &p);
size_t ssm_scan_workspace_bytes(int n_seqs, int total, int channels, int n_state, int groups, int max_len);

// A matrix in 4 bits.
struct Q4Matrix {
    const uint8_t *codes;
    const __nv_bfloat16 *scales, *offsets;
};

struct Q4Problem {
    int rows, n_out, k, group;
    const __nv_bfloat16 *x;
    long long x_stride;
    Q4Matrix w, up;             // up: of the gated form only
    int gated, gelu;
    void *out;
    int out_f32;
    void *workspace;
    cudaStream_t stream;
};
cudaError_t launch_q4(const Q4Problem &p);
size_t q4_workspace_bytes(int rows, int n_out, int k, int group, int out_f32);
// the kernel for one or two rows
bool q4_vec_takes(int rows, int k);
cudaError_t launch_q4_vec(const Q4Problem &p);
// the kernel for many rows
cudaError_t launch_q4_tc(const Q4Problem &p);
size_t q4_tc_workspace_bytes(int rows, int k, int group);
// [rows, bytes of a row, `pitch` bytes apart] read in boxes of box_bytes of box_rows rows, 128-byte swizzled or not; the second
// form: of 128 bytes, swizzled.
bool box_map(CUtensorMap *m, const void *at, uint64_t rows, uint64_t row_bytes, uint64_t pitch, uint32_t box_bytes, uint32_t box_rows,
             bool swizzled);
bool byte_map(CUtensorMap *m, const void *at, uint64_t rows, uint64_t row_bytes, uint64_t pitch, uint32_t box_rows);

// Scales and offsets of a row's groups of 256 inputs (4 of 64 inputs or 2 of 128), as they lie in memory.
struct ChunkScales {
    uint2 s, o;
};

// `wanted`: a bit for each that is needed; the others may be anything.
template <bool OFFSETS>
__device__ __forceinline__ ChunkScales chunk_scales(const Q4Matrix &w, size_t row, int groups, int first, int count, bool vector, int wanted = 15) {
    ChunkScales c{};
    const __nv_bfloat16 *s = w.scales + row * groups + first, *o = OFFSETS ? w.offsets + row * groups + first : nullptr;
    if (vector) {                                        // the row's groups are a multiple of the chunk's
        if (first >= groups) return c;
        if (count == 4) {
            c.s = *reinterpret_cast<const uint2 *>(s);
            if (OFFSETS) c.o = *reinterpret_cast<const uint2 *>(o);
        } else {
            c.s.x = *reinterpret_cast<const uint32_t *>(s);
            if (OFFSETS) c.o.x = *reinterpret_cast<const uint32_t *>(o);
        }
        return c;
    }
    if (groups % 2 == 0 && count == 4) {                 // pairs
        if (wanted & 3 && first < groups) {
            c.s.x = *reinterpret_cast<const uint32_t *>(s);
            if (OFFSETS) c.o.x = *reinterpret_cast<const uint32_t *>(o);
        }
        if (wanted & 12 && first + 2 < groups) {
            c.s.y = *reinterpret_cast<const uint32_t *>(s + 2);
            if (OFFSETS) c.o.y = *reinterpret_cast<const uint32_t *>(o + 2);
        }
        return c;
    }
    uint32_t v[4] = {0, 0, 0, 0}, u[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < count && first + i < groups && wanted >> i & 1) {
            v[i] = __bfloat16_as_ushort(s[i]);
            if (OFFSETS) u[i] = __bfloat16_as_ushort(o[i]);
        }
    c.s = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
    c.o = make_uint2(u[0] | u[1] << 16, u[2] | u[3] << 16);
    return c;
}

__device__ __forceinline__ float nth_bf16(const uint2 &v, int i) {
    const uint32_t w = i & 2 ? v.y : v.x;
    return i & 1 ? bf16_hi(w) : bf16_lo(w);
}

// The activation of a gated feed-forward block: u / (1 + e^-v), with v = u or, for gelu, 2 sqrt(2/pi) (u + 0.044715 u^3), as
// 1 + tanh(w) = 2 / (1 + e^-2w) has no difference of nearly equal numbers.
__device__ __forceinline__ float ffn_argument(float u, int gelu) {
    return gelu ? 1.5957691216057308f * (u + 0.044715f * u * u * u) : u;
}
__device__ __forceinline__ float ffn_act(float u, int gelu) { return u / (1.f + expf(-ffn_argument(u, gelu))); }
// The same to 2^-19 for |v| < 32, where it is rounded to bf16 next.
__device__ __forceinline__ float ffn_act_fast(float u, int gelu) {
    return u * reciprocal(1.f + ex2(-kLog2e * ffn_argument(u, gelu)));
}

}  // namespace gdn
