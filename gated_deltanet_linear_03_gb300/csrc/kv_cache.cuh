// The paged 8-bit cache: formats, conversions and lookups that its kernels share (layout: include/gdn.h).
#pragma once

#include <cuda_fp16.h>

#include "gdn_internal.cuh"

namespace gdn {

constexpr int kKvBlock = GDN_KV_BLOCK;               // tokens that share a scale
constexpr float kAmaxFloor = 8.673617379884035e-19f;  // 2^-60: the scale of an all-zero block, and no reciprocal overflows

template <int FMT>
__host__ __device__ constexpr float kv_code_max() { return FMT == GDN_KV_INT8 ? 127.f : 448.f; }

// The pool and the table of one call.
struct KvPool {
    const int32_t *table;   // [n_seqs, max_pages]
    int max_pages, n_pages, page_size, hkv;
    int page_shift;         // log2 of page_size where that is a power of two, else -1
    __device__ __forceinline__ int page_of(int token) const { return page_shift >= 0 ? token >> page_shift : token / page_size; }
};

// Four codes (one 32-bit word) to two fp16 pairs, exactly: (byte 0, byte 1) and (byte 2, byte 3).
// int8: with its sign bit flipped a byte is x + 128, which under the exponent byte 0x64 is the fp16 number
// 1024 + 128 + x; subtracting 1152 leaves x.
template <int FMT>
__device__ __forceinline__ void codes_to_f16x2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if (FMT == GDN_KV_INT8) {
        w ^= 0x80808080u;
        const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
        const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), off);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
        lo = *reinterpret_cast<const uint32_t *>(&x);
        hi = *reinterpret_cast<const uint32_t *>(&y);
    } else {
        asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    }
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t p) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&p));
}

// Four values, already divided by their block's scale, to four codes (ties to even; out of range saturates).
template <int FMT>
__device__ __forceinline__ uint32_t values_to_codes(float a, float b, float c, float d) {
    if (FMT == GDN_KV_INT8) {
        // |x| <= 127 (1 + 2^-22): adding 1.5 * 2^23 rounds to an integer in the low mantissa bits
        const float m = 12582912.f;
        const uint32_t ab = __byte_perm(__float_as_uint(__fadd_rn(a, m)), __float_as_uint(__fadd_rn(b, m)), 0x0040);
        const uint32_t cd = __byte_perm(__float_as_uint(__fadd_rn(c, m)), __float_as_uint(__fadd_rn(d, m)), 0x0040);
        return __byte_perm(ab, cd, 0x5410);
    }
    uint32_t w;
    asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
        " mov.b32 %0, {l, h};\n}\n"
        : "=r"(w)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return w;
}

// 8 bf16 values (16 bytes) to 32 bits and back, rounded once.
__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// 4 or 8 consecutive entries of a table that the call does not write.
template <int N>
__device__ __forceinline__ void load4(const float *p, float (&x)[N]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
}
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// Largest magnitude of 8 bf16 values as the bits of a float: ordered like the magnitudes, with infinity above
// every finite number and NaN above infinity.
__device__ __forceinline__ uint32_t amax_bits(const uint4 &u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max((w[i] << 16) & 0x7fff0000u, w[i] & 0x7fff0000u));
    return m;
}

// The sequence that holds row t of n packed ones: the last i with cu[i] <= t (t < cu[n]).
__device__ __forceinline__ int sequence_of(const int32_t *__restrict__ cu, int n, int t) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

struct AppendProblem {
    int n_seqs, total, hq, d, rot;
    const __nv_bfloat16 *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    const float *cos, *sin;
    int max_len, interleaved;       // longest sequence that the cos and sin tables and the block table hold
    const int32_t *cu, *past;
    KvPool pool;
    int format;
    uint8_t *k_pages, *v_pages;
    float *k_scales, *v_scales;
    const __nv_bfloat16 *open_in;
    __nv_bfloat16 *open_out;
    const int32_t *slots;
    int n_slots;
    __nv_bfloat16 *q_out;
    unsigned int *err;
    cudaStream_t stream;
};
cudaError_t launch_kv_append(const AppendProblem &p);
bool append_supported(int n_seqs, int total, int hq, int hkv, int d);   // the kernel counts its CTAs and query warps in 32 bits

struct ReadProblem {
    int n_seqs, total, d;
    const int32_t *cu;
    KvPool pool;
    int format;
    const uint8_t *k_pages, *v_pages;
    const float *k_scales, *v_scales;
    void *k_out, *v_out;
    int out_f32;
    unsigned int *err;
    cudaStream_t stream;
};
cudaError_t launch_kv_read(const ReadProblem &p);

struct AttendProblem {
    int n_seqs, total, hq, d;
    const __nv_bfloat16 *q;
    KvPool pool;
    int format;
    const uint8_t *k_pages, *v_pages;
    const float *k_scales, *v_scales;
    const int32_t *cu, *kv_lens;
    int max_q_len, max_kv_len;
    float sm_scale;
    int window, sinks;
    void *out;
    int out_f32;
    void *workspace;
    unsigned int *err;
    cudaStream_t stream;
};
cudaError_t launch_attend(const AttendProblem &p);
size_t attend_workspace_bytes(int n_seqs, int total, int hq, int hkv, int d, int max_q_len, int max_kv_len);
bool attend_supported(int n_seqs, int hq, int hkv, int d, int max_q_len, int max_kv_len);
// the tensor-core kernel, for many query rows
cudaError_t launch_attend_tc(const AttendProblem &p);
size_t attend_tc_workspace_bytes(int n_seqs, int total, int hq, int hkv, int d);

struct BlockNormProblem {
    int rows, dim;
    const __nv_bfloat16 *x, *gate;
    int silu;
    const void *residual;
    int residual_f32;
    const float *post_w, *pre_w, *scale_w;
    float scale, eps;
    void *residual_out;
    __nv_bfloat16 *out;
    cudaStream_t stream;
};
cudaError_t launch_block_norm(const BlockNormProblem &p);

}  // namespace gdn
