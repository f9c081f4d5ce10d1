// extern "C" entry points of the cache, attention and block-norm calls: arguments are checked on the host (the
// CUDA runtime is asked only once they are well formed), then the matching kernel is launched.
#include <limits.h>
#include <math.h>

#include "kv_cache.cuh"

namespace {

bool aligned(const void *p, uintptr_t n = 16) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Range {
    const void *p;
    size_t n;
};

bool overlaps(const Range &a, const Range &b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}

// No output may overlap an input or another output.
template <size_t N, size_t M>
bool disjoint(const Range (&outs)[N], const Range (&ins)[M]) {
    for (size_t i = 0; i < N; ++i) {
        for (const Range &in : ins)
            if (overlaps(outs[i], in)) return false;
        for (size_t j = i + 1; j < N; ++j)
            if (overlaps(outs[i], outs[j])) return false;
    }
    return true;
}

// bytes of `tokens` rows of h * d bf16 elements, `stride` elements apart
size_t rows_bytes(int tokens, long long stride, long long row) {
    return tokens > 0 ? ((size_t)(tokens - 1) * stride + row) * 2 : 0;
}

gdn_status check_pool(int hkv, int d, int max_pages, int n_pages, int page_size, int format) {
    if (hkv <= 0 || d <= 0 || max_pages <= 0 || n_pages <= 0 || page_size <= 0) return GDN_ERR_INVALID_ARG;
    if (d != 64 && d != 128 && d != 256) return GDN_ERR_UNSUPPORTED;
    if (page_size % GDN_KV_BLOCK != 0 || page_size > 4096) return GDN_ERR_UNSUPPORTED;
    if (format != GDN_KV_INT8 && format != GDN_KV_E4M3) return GDN_ERR_UNSUPPORTED;
    if ((double)n_pages * hkv * page_size >= 2147483648.0) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

int page_shift(int page_size) { return (page_size & (page_size - 1)) == 0 ? __builtin_ctz((unsigned)page_size) : -1; }

size_t pool_bytes(int hkv, int d, int n_pages, int page_size) { return (size_t)n_pages * hkv * page_size * d; }

}  // namespace

extern "C" {

gdn_status gdn_kv_append(int n_seqs, int total_tokens, int hq, int hkv, int d, int rot, const void *q,
                         long long q_stride, const void *k, long long k_stride, const void *v, long long v_stride,
                         const float *cos, const float *sin, int n_positions, int interleaved,
                         const int32_t *cu_seqlens, const int32_t *past_lens, const int32_t *block_table,
                         int max_pages, int n_pages, int page_size, int format, void *k_pages, void *v_pages,
                         float *k_scales, float *v_scales, const void *open_in, void *open_out,
                         const int32_t *slots, int n_slots, void *q_out, void *stream) {
    gdn_status st = check_pool(hkv, d, max_pages, n_pages, page_size, format);
    if (st != GDN_OK) return st;
    if (n_seqs < 0 || total_tokens < 0 || hq < 0 || n_slots < 0 || (interleaved != 0 && interleaved != 1)) return GDN_ERR_INVALID_ARG;
    if (rot < 0 || rot > d || n_positions < 0) return GDN_ERR_INVALID_ARG;
    if (rot % 16 != 0) return GDN_ERR_UNSUPPORTED;
    if ((q == nullptr) != (q_out == nullptr) || (q && (hq == 0 || hq % hkv != 0))) return GDN_ERR_INVALID_ARG;
    if (rot > 0 && (!cos || !sin)) return GDN_ERR_INVALID_ARG;
    const long long kv_row = (long long)hkv * d, q_row = (long long)hq * d;
    if (k_stride < kv_row || v_stride < kv_row || (q && q_stride < q_row)) return GDN_ERR_INVALID_ARG;
    if (k_stride % 8 || v_stride % 8 || (q && q_stride % 8)) return GDN_ERR_ALIGNMENT;
    if (n_seqs == 0 && total_tokens > 0) return GDN_ERR_INVALID_ARG;
    if (!gdn::append_supported(n_seqs, total_tokens, hq, hkv, d)) return GDN_ERR_UNSUPPORTED;
    if (n_seqs == 0) return GDN_OK;
    if (!slots && n_slots < n_seqs) return GDN_ERR_INVALID_ARG;
    if (!cu_seqlens || !past_lens || !block_table || !k_pages || !v_pages || !k_scales || !v_scales || !open_in || !open_out)
        return GDN_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!k || !v)) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, cos, sin, cu_seqlens, past_lens, block_table, k_pages, v_pages, k_scales, v_scales,
                          open_in, open_out, slots, q_out};
    for (const void *p : ptrs)
        if (!aligned(p)) return GDN_ERR_ALIGNMENT;

    const size_t pool = pool_bytes(hkv, d, n_pages, page_size), scales = pool / d / GDN_KV_BLOCK * 4;
    const size_t open = (size_t)n_slots * 2 * hkv * GDN_KV_BLOCK * d * 2;
    const Range outs[] = {{k_pages, pool}, {v_pages, pool}, {k_scales, scales}, {v_scales, scales}, {open_out, open},
                          {q_out, rows_bytes(total_tokens, q_row, q_row)}};
    const bool q_in_place = q && q == q_out;
    if (q_in_place && q_stride != q_row) return GDN_ERR_INVALID_ARG;
    const Range ins[] = {{q_in_place ? nullptr : q, rows_bytes(total_tokens, q_stride, q_row)},
                         {k, rows_bytes(total_tokens, k_stride, kv_row)},
                         {v, rows_bytes(total_tokens, v_stride, kv_row)},
                         {cos, (size_t)n_positions * (rot / 2) * 4},
                         {sin, (size_t)n_positions * (rot / 2) * 4},
                         {cu_seqlens, (size_t)(n_seqs + 1) * 4},
                         {past_lens, (size_t)n_seqs * 4},
                         {block_table, (size_t)n_seqs * max_pages * 4},
                         {open_in == open_out ? nullptr : open_in, open},
                         {slots, (size_t)n_seqs * 4}};
    if (!disjoint(outs, ins)) return GDN_ERR_INVALID_ARG;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const void *anchors[] = {k, k_pages, open_out, q_out};
    st = gdn::on_current_device(anchors, sizeof(anchors) / sizeof(anchors[0]), cs);
    if (st != GDN_OK) return st;

    gdn::AppendProblem p{};
    p.n_seqs = n_seqs; p.total = total_tokens; p.hq = hq; p.d = d; p.rot = rot;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.cos = cos; p.sin = sin; p.interleaved = interleaved;
    const long long held = (long long)max_pages * page_size;
    p.max_len = (int)(held < INT_MAX ? held : INT_MAX);
    if (rot > 0 && n_positions < p.max_len) p.max_len = n_positions;
    p.cu = cu_seqlens; p.past = past_lens;
    p.pool = {block_table, max_pages, n_pages, page_size, hkv, page_shift(page_size)};
    p.format = format;
    p.k_pages = static_cast<uint8_t *>(k_pages); p.v_pages = static_cast<uint8_t *>(v_pages);
    p.k_scales = k_scales; p.v_scales = v_scales;
    p.open_in = static_cast<const __nv_bfloat16 *>(open_in);
    p.open_out = static_cast<__nv_bfloat16 *>(open_out);
    p.slots = slots; p.n_slots = n_slots;
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.err = gdn::error_word();
    p.stream = cs;
    if (!p.err) return GDN_ERR_CUDA;
    return gdn::launch_kv_append(p) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_kv_read(int n_seqs, int total_tokens, int hkv, int d, const int32_t *cu_tokens,
                       const int32_t *block_table, int max_pages, int n_pages, int page_size, int format,
                       const void *k_pages, const void *v_pages, const float *k_scales, const float *v_scales,
                       void *k_out, void *v_out, int out_dtype, void *stream) {
    gdn_status st = check_pool(hkv, d, max_pages, n_pages, page_size, format);
    if (st != GDN_OK) return st;
    if (n_seqs < 0 || total_tokens < 0 || (n_seqs == 0 && total_tokens > 0)) return GDN_ERR_INVALID_ARG;
    if (out_dtype != GDN_DTYPE_BF16 && out_dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
    if (total_tokens == 0) return GDN_OK;
    if (!cu_tokens || !block_table || !k_pages || !v_pages || !k_scales || !v_scales || !k_out || !v_out) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {cu_tokens, block_table, k_pages, v_pages, k_scales, v_scales, k_out, v_out};
    for (const void *p : ptrs)
        if (!aligned(p)) return GDN_ERR_ALIGNMENT;
    const size_t pool = pool_bytes(hkv, d, n_pages, page_size), scales = pool / d / GDN_KV_BLOCK * 4;
    const size_t out = (size_t)total_tokens * hkv * d * (out_dtype == GDN_DTYPE_F32 ? 4 : 2);
    const Range outs[] = {{k_out, out}, {v_out, out}};
    const Range ins[] = {{k_pages, pool}, {v_pages, pool}, {k_scales, scales}, {v_scales, scales},
                         {cu_tokens, (size_t)(n_seqs + 1) * 4}, {block_table, (size_t)n_seqs * max_pages * 4}};
    if (!disjoint(outs, ins)) return GDN_ERR_INVALID_ARG;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const void *anchors[] = {k_pages, k_out, v_out};
    st = gdn::on_current_device(anchors, sizeof(anchors) / sizeof(anchors[0]), cs);
    if (st != GDN_OK) return st;

    gdn::ReadProblem p{};
    p.n_seqs = n_seqs; p.total = total_tokens; p.d = d;
    p.cu = cu_tokens;
    p.pool = {block_table, max_pages, n_pages, page_size, hkv, page_shift(page_size)};
    p.format = format;
    p.k_pages = static_cast<const uint8_t *>(k_pages); p.v_pages = static_cast<const uint8_t *>(v_pages);
    p.k_scales = k_scales; p.v_scales = v_scales;
    p.k_out = k_out; p.v_out = v_out; p.out_f32 = out_dtype == GDN_DTYPE_F32;
    p.err = gdn::error_word();
    p.stream = cs;
    if (!p.err) return GDN_ERR_CUDA;
    return gdn::launch_kv_read(p) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"

static gdn_status check_attend_shape(int n_seqs, int total_tokens, int hq, int hkv, int d, int max_q_len, int max_kv_len) {
    if (n_seqs < 0 || total_tokens < 0 || hq <= 0 || hkv <= 0 || d <= 0 || max_q_len < 0 || max_kv_len < 0) return GDN_ERR_INVALID_ARG;
    if (n_seqs == 0 && total_tokens > 0) return GDN_ERR_INVALID_ARG;
    if (total_tokens < max_q_len) max_q_len = total_tokens;
    if (hq % hkv != 0 || (total_tokens > 0 && max_q_len == 0)) return GDN_ERR_INVALID_ARG;
    if (d != 64 && d != 128 && d != 256) return GDN_ERR_UNSUPPORTED;
    if (max_kv_len > INT_MAX - 4096) return GDN_ERR_UNSUPPORTED;                        // a tile's tokens are counted in 32 bits
    if ((double)total_tokens * hq >= 2147483648.0 - 4096) return GDN_ERR_UNSUPPORTED;   // the kernels count query rows in 32 bits
    if (!gdn::attend_supported(n_seqs, hq, hkv, d, max_q_len, max_kv_len)) return GDN_ERR_UNSUPPORTED;         // and units of work
    return GDN_OK;
}

extern "C" {

size_t gdn_attend_workspace_size(int n_seqs, int total_tokens, int hq, int hkv, int d, int max_q_len, int max_kv_len,
                                 gdn_status *status) {
    const gdn_status st = check_attend_shape(n_seqs, total_tokens, hq, hkv, d, max_q_len, max_kv_len);
    if (status) *status = st;
    if (max_q_len > total_tokens) max_q_len = total_tokens;
    return st == GDN_OK ? gdn::attend_workspace_bytes(n_seqs, total_tokens, hq, hkv, d, max_q_len, max_kv_len) : 0;
}

gdn_status gdn_attend(int n_seqs, int total_tokens, int hq, int hkv, int d, const void *q, const void *k_pages,
                      const void *v_pages, const float *k_scales, const float *v_scales, const int32_t *block_table,
                      int max_pages, int n_pages, int page_size, int format, const int32_t *cu_seqlens,
                      const int32_t *kv_lens, int max_q_len, int max_kv_len, float sm_scale, int window, int sinks,
                      void *out, int out_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    gdn_status st = check_attend_shape(n_seqs, total_tokens, hq, hkv, d, max_q_len, max_kv_len);
    if (st == GDN_OK) st = check_pool(hkv, d, max_pages, n_pages, page_size, format);
    if (st != GDN_OK) return st;
    if (!isfinite(sm_scale) || window < 0 || sinks < 0) return GDN_ERR_INVALID_ARG;
    if ((long long)max_kv_len > (long long)max_pages * page_size) return GDN_ERR_INVALID_ARG;
    if (out_dtype != GDN_DTYPE_BF16 && out_dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
    if (total_tokens == 0) return GDN_OK;
    if (!q || !k_pages || !v_pages || !k_scales || !v_scales || !block_table || !cu_seqlens || !kv_lens || !out) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k_pages, v_pages, k_scales, v_scales, block_table, cu_seqlens, kv_lens, out};
    for (const void *p : ptrs)
        if (!aligned(p)) return GDN_ERR_ALIGNMENT;
    max_q_len = max_q_len < total_tokens ? max_q_len : total_tokens;
    const size_t need = gdn::attend_workspace_bytes(n_seqs, total_tokens, hq, hkv, d, max_q_len, max_kv_len);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return GDN_ERR_ALIGNMENT;
    const size_t pool = pool_bytes(hkv, d, n_pages, page_size), scales = pool / d / GDN_KV_BLOCK * 4;
    const size_t elems = (size_t)total_tokens * hq * d;
    const Range outs[] = {{out, elems * (out_dtype == GDN_DTYPE_F32 ? 4 : 2)}, {workspace, need}};
    const Range ins[] = {{q, elems * 2}, {k_pages, pool}, {v_pages, pool}, {k_scales, scales}, {v_scales, scales},
                         {block_table, (size_t)n_seqs * max_pages * 4}, {cu_seqlens, (size_t)(n_seqs + 1) * 4},
                         {kv_lens, (size_t)n_seqs * 4}};
    if (!disjoint(outs, ins)) return GDN_ERR_INVALID_ARG;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const void *anchors[] = {q, k_pages, out, workspace};
    st = gdn::on_current_device(anchors, sizeof(anchors) / sizeof(anchors[0]), cs);
    if (st != GDN_OK) return st;

    gdn::AttendProblem p{};
    p.n_seqs = n_seqs; p.total = total_tokens; p.hq = hq; p.d = d;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.pool = {block_table, max_pages, n_pages, page_size, hkv, page_shift(page_size)};
    p.format = format;
    p.k_pages = static_cast<const uint8_t *>(k_pages); p.v_pages = static_cast<const uint8_t *>(v_pages);
    p.k_scales = k_scales; p.v_scales = v_scales;
    p.cu = cu_seqlens; p.kv_lens = kv_lens;
    p.max_q_len = max_q_len; p.max_kv_len = max_kv_len;
    p.sm_scale = sm_scale;
    // a window that reaches past every cached token is none (and positions minus it stay in range)
    p.window = window >= max_kv_len ? 0 : window; p.sinks = sinks;
    p.out = out; p.out_f32 = out_dtype == GDN_DTYPE_F32;
    p.workspace = workspace;
    p.err = gdn::error_word();
    p.stream = cs;
    if (!p.err) return GDN_ERR_CUDA;
    return gdn::launch_attend(p) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_block_norm(int rows, int dim, const void *x, const void *gate, int gate_act, const void *residual,
                          int residual_dtype, const float *post_weight, const float *pre_weight,
                          const float *scale_weight, float scale, float eps, void *residual_out, void *out, void *stream) {
    if (rows < 0 || dim <= 0) return GDN_ERR_INVALID_ARG;
    if (dim % 8 != 0 || dim > 16384) return GDN_ERR_UNSUPPORTED;
    if (rows > INT_MAX - 65536) return GDN_ERR_UNSUPPORTED;                             // a CTA's next row is counted in 32 bits
    if (residual_dtype != GDN_DTYPE_BF16 && residual_dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
    if (gate_act != GDN_GATE_SIGMOID && gate_act != GDN_GATE_SILU) return GDN_ERR_UNSUPPORTED;
    if (!isfinite(scale) || !isfinite(eps) || eps < 0.f) return GDN_ERR_INVALID_ARG;
    if (rows == 0) return GDN_OK;
    if (!x || !residual || !pre_weight || !residual_out || !out) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {x, gate, residual, post_weight, pre_weight, scale_weight, residual_out, out};
    for (const void *p : ptrs)
        if (!aligned(p)) return GDN_ERR_ALIGNMENT;
    const size_t n = (size_t)rows * dim, res = n * (residual_dtype == GDN_DTYPE_F32 ? 4 : 2), w = (size_t)dim * 4;
    const Range outs[] = {{residual_out, res}, {out, 2 * n}};
    const Range ins[] = {{x == out ? nullptr : x, 2 * n}, {gate == out ? nullptr : gate, 2 * n},
                         {residual == residual_out ? nullptr : residual, res}, {post_weight, w}, {pre_weight, w}, {scale_weight, w}};
    if (!disjoint(outs, ins)) return GDN_ERR_INVALID_ARG;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const void *anchors[] = {x, residual_out, out};
    gdn_status st = gdn::on_current_device(anchors, sizeof(anchors) / sizeof(anchors[0]), cs);
    if (st != GDN_OK) return st;

    gdn::BlockNormProblem p{};
    p.rows = rows; p.dim = dim;
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.gate = static_cast<const __nv_bfloat16 *>(gate);
    p.silu = gate_act == GDN_GATE_SILU;
    p.residual = residual; p.residual_f32 = residual_dtype == GDN_DTYPE_F32;
    p.post_w = post_weight; p.pre_w = pre_weight; p.scale_w = scale_weight;
    p.scale = scale; p.eps = eps;
    p.residual_out = residual_out;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.stream = cs;
    return gdn::launch_block_norm(p) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
