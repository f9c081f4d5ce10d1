// gdn_kv_append and gdn_kv_read: the paged 8-bit cache's writer and reader.
//
// Append.  For a 16-token block of one head, with rows x_0 .. x_15 in bf16 (keys after their rotation),
//     A = max(max |x|, 2^-60),   scale = A / Q,   code = round(x * (Q / A)).
// A block is quantised as a whole, so its scale needs all of its rows; a sequence's unfinished block keeps its
// rows in bf16 (open_in / open_out) and is quantised afresh from them whenever it grows.  That costs at most
// 15 rows a head and call, and makes the cache independent of how tokens were divided into calls.
// One CTA takes one (block, head): D threads hold K and V, two 8-element pieces of each per thread, so the
// rows are read once, the maximum is a CTA reduction, and codes leave as 8-byte pieces of full lines.  The
// queries' rotation, most of the bytes with grouped heads, runs in the same launch on further CTAs.
// Bound by memory: T (hq + 2 hkv) d 2-byte reads, T hq d 2-byte and 2 T hkv d 1-byte writes.  16384 tokens of 16 heads over
// 2 of d = 256 56 us, 0.85 of a copy's rate (of 32 heads over 8 of d = 128 72 us, 0.77); one token 3.1 us, a launch and three
// dependent latencies, 61 sequences' tokens 4.6 us, where the search for a token's sequence adds six.
// Read: codes and scales in, values out, one pass.  16384 tokens of 2 heads of d = 256 12.7 us, 0.58 of a copy's rate.
#include "kv_cache.cuh"

namespace gdn {
namespace {

// Interleaved pairs inside one piece of 8 elements, by cos and sin of its four pairs (the first of c and s).
template <int N>
__device__ __forceinline__ void rotate_pairs(float (&x)[8], const float (&c)[N], const float (&s)[N]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * c[i] - b * s[i];
        x[2 * i + 1] = b * c[i] + a * s[i];
    }
}

// Piece c (8 elements) of a key head vector `row`, rotated.
__device__ __forceinline__ uint4 rotated_piece(const __nv_bfloat16 *__restrict__ row, int c, int rot, int interleaved,
                                               const float *__restrict__ cos, const float *__restrict__ sin) {
    const uint4 raw = *reinterpret_cast<const uint4 *>(row + 8 * c);
    if (8 * c >= rot) return raw;
    float x[8];
    unpack8(raw, x);
    if (interleaved) {
        float cc[4], ss[4];
        load4(cos + 4 * c, cc);
        load4(sin + 4 * c, ss);
        rotate_pairs(x, cc, ss);
    } else {
        const bool first = 16 * c < rot;                     // the a-half of the pairs
        const int other = first ? c + rot / 16 : c - rot / 16;
        float y[8], cc[8], ss[8];
        unpack8(*reinterpret_cast<const uint4 *>(row + 8 * other), y);
        const int at = 8 * (first ? c : other);
        load8(cos + at, cc);
        load8(sin + at, ss);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = first ? x[i] * cc[i] - y[i] * ss[i] : x[i] * cc[i] + y[i] * ss[i];
    }
    return pack8(x);
}

template <int FMT>
__device__ __forceinline__ uint2 quantise8(const uint4 &u, float inv) {
    float x[8];
    unpack8(u, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= inv;
    return make_uint2(values_to_codes<FMT>(x[0], x[1], x[2], x[3]), values_to_codes<FMT>(x[4], x[5], x[6], x[7]));
}

// Does the call take a sequence of `len` new tokens?  Its positions have cosines and sines and a place in the table, and its
// slot exists; otherwise all of it is left out.
__device__ __forceinline__ bool taken(const AppendProblem &p, int past, int len, int slot) {
    return past >= 0 && past <= p.max_len - len && (unsigned)slot < (unsigned)p.n_slots;
}

// Query warps.  A warp takes one token and up to kHeadPasses passes over its heads (a pass is 256 / D heads, a piece of 8
// elements a lane): position, cosines and sines are found once, and all of the warp's loads are in flight together.
// The other piece of a pair comes from its lane, so every piece is read before any is written: q_out may be q.
constexpr int kHeadPasses = 4;

template <int D>
__host__ __device__ inline int head_parts(int hq) { return (hq * (D / 8) + 32 * kHeadPasses - 1) / (32 * kHeadPasses); }

template <int D>
__device__ __forceinline__ void rotate_queries(const AppendProblem &p, int warp, int lane) {
    constexpr int LPR = D / 8, HEADS = 32 / LPR;
    const int parts = head_parts<D>(p.hq), t = warp / parts, h0 = (warp % parts) * kHeadPasses * HEADS + lane / LPR;
    if (t >= p.total) return;
    const int c = lane % LPR;
    const bool turned = 8 * c < p.rot, first = 16 * c < p.rot;
    const bool moves = turned || p.q_out != p.q;     // in place, the pieces past rot stay where they are
    const __nv_bfloat16 *src = p.q + t * p.q_stride + (long)h0 * D + 8 * c;
    __nv_bfloat16 *dst = p.q_out + ((long)t * p.hq + h0) * D + 8 * c;
    const int n = sequence_of(p.cu, p.n_seqs, t);
    const int c0 = max(p.cu[n], 0), c1 = min(p.cu[n + 1], p.total), past = p.past[n];
    if (t < c0 || t >= c1) return;                  // no sequence's
    if (!taken(p, past, c1 - c0, p.slots ? p.slots[n] : n)) {
        if (lane == 0) raise_error(p.err, kErrInternal);
        return;
    }
    const int pos = past + t - c0;
    uint4 x[kHeadPasses];
#pragma unroll
    for (int i = 0; i < kHeadPasses; ++i)
        x[i] = moves && h0 + i * HEADS < p.hq ? *reinterpret_cast<const uint4 *>(src + i * HEADS * D) : make_uint4(0, 0, 0, 0);
    float cc[8], ss[8];
    const int other = first ? lane + p.rot / 16 : lane - p.rot / 16;
    if (turned) {
        const float *cos = p.cos + (size_t)pos * (p.rot / 2), *sin = p.sin + (size_t)pos * (p.rot / 2);
        if (p.interleaved) {
            load4(cos + 4 * c, cc);
            load4(sin + 4 * c, ss);
        } else {
            const int at = 8 * (first ? c : c - p.rot / 16);
            load8(cos + at, cc);
            load8(sin + at, ss);
            if (first) {
#pragma unroll
                for (int e = 0; e < 8; ++e) ss[e] = -ss[e];     // a cos - b sin in one half, b cos + a sin in the other
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kHeadPasses; ++i) {
        if (h0 - lane / LPR + i * HEADS >= p.hq) break;          // the same for the whole warp
        if (p.rot > 0 && p.interleaved) {
            if (turned) {
                float y[8];
                unpack8(x[i], y);
                rotate_pairs(y, cc, ss);
                x[i] = pack8(y);
            }
        } else if (p.rot > 0) {
            uint4 z;
            z.x = __shfl_sync(0xffffffffu, x[i].x, other);
            z.y = __shfl_sync(0xffffffffu, x[i].y, other);
            z.z = __shfl_sync(0xffffffffu, x[i].z, other);
            z.w = __shfl_sync(0xffffffffu, x[i].w, other);
            if (turned) {
                float y[8], o[8];
                unpack8(x[i], y);
                unpack8(z, o);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = y[e] * cc[e] + o[e] * ss[e];
                x[i] = pack8(y);
            }
        }
        if (moves && h0 + i * HEADS < p.hq) *reinterpret_cast<uint4 *>(dst + i * HEADS * D) = x[i];
    }
}

// CTAs that hold blocks: sequence n's blocks start at slot cu[n] / 16 + 2 n, which leaves room for
// ceil((past % 16 + new) / 16) <= floor(new / 16) + 2 of them without a scan over the sequences.
__host__ __device__ inline long block_slots(int n_seqs, int total) { return total / kKvBlock + 2L * n_seqs; }

// 1280 threads an SM, 48 registers each.  16384 tokens with the read-back, us for (passes, threads):
//   16 heads over 2 of d = 256   (4, 1280) 68.5, (4, 768) 78, (4, 1536) 71.7, (8, 768) 72.3, (8, 1024) 70.0, (8, 1280) 80, (2, 1280) 75
//   32 heads over 8 of d = 128   (4, 1280) 93.8, (4, 768) 99, (4, 1536) 95.2, (8, 768) 96.4, (8, 1024) 94.9, (8, 1280) 103, (2, 1280) 101
//   16 heads over 4 of d = 64    (4, 1280) 27.2, (4, 768) 29, (4, 1536) 29.6, (8, 768) 29.0, (8, 1024) 28.6, (8, 1280) 34, (2, 1280) 29
// and within 4 % of one another for single tokens of 61 sequences, but (2, 2048) 7 % slower.
template <int D, int FMT>
__global__ void __launch_bounds__(D, 1280 / D) kv_append_kernel(const __grid_constant__ AppendProblem p) {
    constexpr int PIECES = D / 8, ROWS = D / PIECES;   // 8 rows per pass of the CTA, two passes
    __shared__ uint32_t part[2][D / 32];
    const long kv_ctas = block_slots(p.n_seqs, p.total) * p.pool.hkv;
    if (blockIdx.x >= kv_ctas) {
        rotate_queries<D>(p, (int)(blockIdx.x - kv_ctas) * (D / 32) + threadIdx.x / 32, threadIdx.x % 32);
        return;
    }
    const int slot = blockIdx.x / p.pool.hkv, h = blockIdx.x % p.pool.hkv;
    // the sequence whose slots hold this one
    int n = 0;
    for (int hi = p.n_seqs; hi - n > 1;) {
        const int mid = (n + hi) >> 1;
        if (p.cu[mid] / kKvBlock + 2 * mid <= slot) n = mid;
        else hi = mid;
    }
    const int c0 = min(max(p.cu[n], 0), p.total), len = min(max(p.cu[n + 1], c0), p.total) - c0;
    const int past = p.past[n], os = p.slots ? p.slots[n] : n;
    const int local = slot - (p.cu[n] / kKvBlock + 2 * n);
    if (len == 0 && past >= 0 && past % kKvBlock == 0) return;
    if (!taken(p, past, len, os)) {
        if (threadIdx.x == 0) raise_error(p.err, kErrInternal);
        return;
    }
    const int end = past + len, first = past / kKvBlock, last = (end - 1) / kKvBlock;
    if (local > last - first) return;
    // The first block reads open_in, the last writes open_out, which may be the same memory: when they are
    // different blocks, one CTA does both, in that order.
    const bool open = end % kKvBlock != 0;
    if (open && local > 0 && local == last - first) return;
    const int c = threadIdx.x % PIECES, r0 = threadIdx.x / PIECES;

    for (int blk = first + local;; blk = last) {
        uint4 x[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = r0 + i * ROWS, at = blk * kKvBlock + row;
            x[0][i] = x[1][i] = make_uint4(0, 0, 0, 0);
            if (at < past) {
                const __nv_bfloat16 *o = p.open_in + (((size_t)os * 2 * p.pool.hkv + h) * kKvBlock + row) * D + 8 * c;
                x[0][i] = *reinterpret_cast<const uint4 *>(o);
                x[1][i] = *reinterpret_cast<const uint4 *>(o + (size_t)p.pool.hkv * kKvBlock * D);
            } else if (at < end) {
                const long t = c0 + at - past;
                x[1][i] = *reinterpret_cast<const uint4 *>(p.v + t * p.v_stride + (long)h * D + 8 * c);
                x[0][i] = rotated_piece(p.k + t * p.k_stride + (long)h * D, c, p.rot, p.interleaved,
                                        p.cos + (size_t)at * (p.rot / 2), p.sin + (size_t)at * (p.rot / 2));
            }
        }
        uint32_t m[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            m[j] = __reduce_max_sync(0xffffffffu, max(amax_bits(x[j][0]), amax_bits(x[j][1])));
            if (threadIdx.x % 32 == 0) part[j][threadIdx.x / 32] = m[j];
        }
        __syncthreads();
        float amax[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t a = 0;
#pragma unroll
            for (int w = 0; w < D / 32; ++w) a = max(a, part[j][w]);
            amax[j] = __uint_as_float(max(a, __float_as_uint(kAmaxFloor)));
        }
        const int page = p.pool.table[(size_t)n * p.pool.max_pages + blk * kKvBlock / p.pool.page_size];
        const int in_page = blk * kKvBlock % p.pool.page_size;
        if (page < 0 || page >= p.pool.n_pages) {
            if (threadIdx.x == 0) raise_error(p.err, kErrInternal);
        } else {
            const size_t head = (size_t)page * p.pool.hkv + h;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bool finite = amax[j] <= 3.4028234e38f;     // false for infinity and NaN: codes 0, scale as it is
                const float inv = kv_code_max<FMT>() / amax[j];
                uint8_t *dst = (j ? p.v_pages : p.k_pages) + (head * p.pool.page_size + in_page) * D;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<uint2 *>(dst + (size_t)(r0 + i * ROWS) * D + 8 * c) =
                        finite ? quantise8<FMT>(x[j][i], inv) : make_uint2(0, 0);
                if (threadIdx.x == 0)
                    (j ? p.v_scales : p.k_scales)[head * (p.pool.page_size / kKvBlock) + in_page / kKvBlock] =
                        amax[j] / kv_code_max<FMT>();
            }
        }
        if (open && blk == last) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = r0 + i * ROWS;
                if (row >= end % kKvBlock) continue;
                __nv_bfloat16 *o = p.open_out + (((size_t)os * 2 * p.pool.hkv + h) * kKvBlock + row) * D + 8 * c;
                *reinterpret_cast<uint4 *>(o) = x[0][i];
                *reinterpret_cast<uint4 *>(o + (size_t)p.pool.hkv * kKvBlock * D) = x[1][i];
            }
        }
        if (!open || local > 0 || blk == last) return;
        __syncthreads();   // part is free again
    }
}

// One thread reads 16 codes of K and of V (one 16-byte load each) and writes 16 values of each.
template <int FMT, bool F32>
__global__ void __launch_bounds__(256) kv_read_kernel(const __grid_constant__ ReadProblem p) {
    const int units = p.d / 16, shift = 31 - __clz(units);            // d is a power of two
    const long i = (long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long)p.total * p.pool.hkv * units) return;
    const int u = (int)i & (units - 1);
    const long row = i >> shift;                      // (token, head)
    const int t = row >> 32 == 0 ? (int)((unsigned)row / (unsigned)p.pool.hkv) : (int)(row / p.pool.hkv), h = (int)(row - (long)t * p.pool.hkv);
    const int n = sequence_of(p.cu, p.n_seqs, t);
    const int at = t - p.cu[n];
    int page = -1, in_page = 0;
    if (at >= 0 && at < (long)p.pool.max_pages * p.pool.page_size) {
        const int nth = p.pool.page_of(at);
        in_page = at - nth * p.pool.page_size;
        page = p.pool.table[(size_t)n * p.pool.max_pages + nth];
    }
    const bool ok = page >= 0 && page < p.pool.n_pages;
    if (!ok) raise_error(p.err, kErrInternal);
    const size_t head = (size_t)(ok ? page : 0) * p.pool.hkv + h;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint4 codes = make_uint4(0, 0, 0, 0);
        float scale = 0.f;
        if (ok) {
            codes = __ldg(reinterpret_cast<const uint4 *>((j ? p.v_pages : p.k_pages) + (head * p.pool.page_size + in_page) * p.d + 16 * u));
            scale = __ldg((j ? p.v_scales : p.k_scales) + head * (p.pool.page_size / kKvBlock) + in_page / kKvBlock);
        }
        const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
        float x[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t lo, hi;
            codes_to_f16x2<FMT>(w[e], lo, hi);
            const float2 a = f16x2_to_float2(lo), b = f16x2_to_float2(hi);
            x[4 * e] = a.x * scale; x[4 * e + 1] = a.y * scale; x[4 * e + 2] = b.x * scale; x[4 * e + 3] = b.y * scale;
        }
        void *out = j ? p.v_out : p.k_out;
        const size_t o = (size_t)row * p.d + 16 * u;
        if (F32) {
            float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(out) + o);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        } else {
            uint4 *b = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + o);
            b[0] = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
            b[1] = make_uint4(pack2(x[8], x[9]), pack2(x[10], x[11]), pack2(x[12], x[13]), pack2(x[14], x[15]));
        }
    }
}

}  // namespace

namespace {
long append_query_ctas(int total, int hq, int d) {
    const int parts = d == 64 ? head_parts<64>(hq) : d == 128 ? head_parts<128>(hq) : head_parts<256>(hq);
    return ((long)total * parts + d / 32 - 1) / (d / 32);
}
}  // namespace

bool append_supported(int n_seqs, int total, int hq, int hkv, int d) {
    return (double)hq * d < 2147483648.0 && (double)block_slots(n_seqs, total) * hkv + append_query_ctas(total, hq, d) <= 2147483647 / 8;
}

cudaError_t launch_kv_append(const AppendProblem &p) {
    const long kv_ctas = block_slots(p.n_seqs, p.total) * p.pool.hkv, q_ctas = p.q ? append_query_ctas(p.total, p.hq, p.d) : 0;
    using Fn = void (*)(const AppendProblem);
    const bool e4m3 = p.format == GDN_KV_E4M3;
    const Fn fn = p.d == 64 ? (e4m3 ? kv_append_kernel<64, GDN_KV_E4M3> : kv_append_kernel<64, GDN_KV_INT8>)
                  : p.d == 128 ? (e4m3 ? kv_append_kernel<128, GDN_KV_E4M3> : kv_append_kernel<128, GDN_KV_INT8>)
                               : (e4m3 ? kv_append_kernel<256, GDN_KV_E4M3> : kv_append_kernel<256, GDN_KV_INT8>);
    fn<<<(unsigned)(kv_ctas + q_ctas), p.d, 0, p.stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const ReadProblem &p) {
    const long ctas = ((long)p.total * p.pool.hkv * (p.d / 16) + 255) / 256;
    if (ctas == 0) return cudaSuccess;
    if (ctas > 2147483647L) return cudaErrorInvalidValue;
    using Fn = void (*)(const ReadProblem);
    const bool e4m3 = p.format == GDN_KV_E4M3;
    const Fn fn = p.out_f32 ? (e4m3 ? kv_read_kernel<GDN_KV_E4M3, true> : kv_read_kernel<GDN_KV_INT8, true>)
                            : (e4m3 ? kv_read_kernel<GDN_KV_E4M3, false> : kv_read_kernel<GDN_KV_INT8, false>);
    fn<<<(unsigned)ctas, 256, 0, p.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gdn
