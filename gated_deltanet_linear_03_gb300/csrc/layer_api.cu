// extern "C" entry points of the short convolution, the selective scan and the 4-bit products: arguments are checked on
// the host (the CUDA runtime is asked only once they are well formed), then the matching kernel is launched.
#include <limits.h>
#include <math.h>

#include "api_checks.cuh"
#include "layer_ops.cuh"

using namespace gdn::api;

namespace {

constexpr long long kMaxStride = 1ll << 38;       // bytes between rows are counted in 40 bits, row times stride in 64

// A bf16 row argument: its elements and their distance.
gdn_status check_rows(const void *p, long long stride, long long row) {
    if (stride < row || stride > kMaxStride) return GDN_ERR_INVALID_ARG;
    return stride % 8 || !aligned(p) ? GDN_ERR_ALIGNMENT : GDN_OK;
}

// Sequences and states of one call; `entry` bytes of state a slot.
gdn_status check_sequences(int n_seqs, int total_tokens, const int32_t *cu_seqlens, const void *state_in, const void *state_out,
                           const int32_t *slots, int n_slots) {
    if (n_seqs < 0 || total_tokens < 0 || n_slots < 0) return GDN_ERR_INVALID_ARG;
    if (!cu_seqlens && total_tokens != n_seqs) return GDN_ERR_INVALID_ARG;
    if (n_seqs == 0 && total_tokens > 0) return GDN_ERR_INVALID_ARG;
    if ((state_in || state_out) && !slots && n_slots < n_seqs) return GDN_ERR_INVALID_ARG;
    if (!aligned(cu_seqlens) || !aligned(state_in) || !aligned(state_out) || !aligned(slots)) return GDN_ERR_ALIGNMENT;
    return GDN_OK;
}

gdn::Sequences sequences(int n_seqs, int total_tokens, const int32_t *cu_seqlens, bool states, const int32_t *slots, int n_slots) {
    gdn::Sequences s{};
    s.n = n_seqs; s.total = total_tokens; s.cu = cu_seqlens;
    s.slots = states ? slots : nullptr;             // without states, slots say nothing
    s.n_slots = states ? n_slots : INT_MAX;
    s.err = gdn::error_word();
    return s;
}

gdn_status check_scan_shape(int n_seqs, int total_tokens, int channels, int n_state, int groups, int max_len) {
    if (n_seqs < 0 || total_tokens < 0 || channels <= 0 || n_state <= 0 || groups <= 0 || max_len < 0) return GDN_ERR_INVALID_ARG;
    if (n_seqs == 0 && total_tokens > 0) return GDN_ERR_INVALID_ARG;
    if (n_state != 16 && n_state != 32 && n_state != 64 && n_state != 128) return GDN_ERR_UNSUPPORTED;
    if (channels % 8 != 0 || channels % groups != 0 || channels / groups % 8 != 0) return GDN_ERR_UNSUPPORTED;
    // warps, of 4 channels each at the least, are counted in 32 bits
    if (((double)n_seqs + total_tokens + 64) * (channels / 4 + groups) >= 2147000000.0) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status check_q4_shape(int rows, int n_out, int k, int group) {
    if (rows < 0 || n_out <= 0 || k <= 0) return GDN_ERR_INVALID_ARG;
    if (group != 64 && group != 128) return GDN_ERR_UNSUPPORTED;
    if (k % group != 0 || k > 65536) return GDN_ERR_UNSUPPORTED;
    if (rows > INT_MAX - 65536 || n_out > INT_MAX - 65536) return GDN_ERR_UNSUPPORTED;
    // CTAs and tiles are counted in 32 bits: 8 rows of x and 8 of weights each at the least
    if (((double)rows / 8 + 1) * ((double)n_out / 8 + 1) >= 2147000000.0) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status q4(int rows, int n_out, int k, int group, const void *x, long long x_stride, const gdn::Q4Matrix &w,
              const gdn::Q4Matrix *up, int gelu, void *out, int out_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    gdn_status st = check_q4_shape(rows, n_out, k, group);
    if (st != GDN_OK) return st;
    if (out_dtype != GDN_DTYPE_BF16 && out_dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
    if (rows == 0) return GDN_OK;
    if (!x || !w.codes || !w.scales || !out || (up && (!up->codes || !up->scales))) return GDN_ERR_INVALID_ARG;
    if (up && (w.offsets == nullptr) != (up->offsets == nullptr)) return GDN_ERR_INVALID_ARG;
    st = check_rows(x, x_stride, k);
    if (st != GDN_OK) return st;
    const gdn::Q4Matrix none{}, &v = up ? *up : none;
    const void *ptrs[] = {w.codes, w.scales, w.offsets, v.codes, v.scales, v.offsets, out};
    for (const void *p : ptrs)
        if (!aligned(p)) return GDN_ERR_ALIGNMENT;
    const size_t codes = (size_t)n_out * (k / 2), scales = (size_t)n_out * (k / group) * 2;
    const size_t need = gdn::q4_workspace_bytes(rows, n_out, k, group, out_dtype == GDN_DTYPE_F32);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return GDN_ERR_ALIGNMENT;
    const Range outs[] = {{out, (size_t)rows * n_out * (out_dtype == GDN_DTYPE_F32 ? 4 : 2)}, {workspace, need}};
    const Range ins[] = {{x, rows_bytes(rows, x_stride, k)}, {w.codes, codes}, {w.scales, scales}, {w.offsets, scales},
                         {v.codes, codes}, {v.scales, scales}, {v.offsets, scales}};
    if (!disjoint(outs, ins)) return GDN_ERR_INVALID_ARG;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const void *anchors[] = {x, w.codes, out, workspace};
    st = gdn::on_current_device(anchors, sizeof(anchors) / sizeof(anchors[0]), cs);
    if (st != GDN_OK) return st;
    gdn::Q4Problem p{};
    p.rows = rows; p.n_out = n_out; p.k = k; p.group = group;
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.x_stride = x_stride;
    p.w = w; p.up = v; p.gated = up != nullptr; p.gelu = gelu;
    p.out = out; p.out_f32 = out_dtype == GDN_DTYPE_F32;
    p.workspace = workspace;
    p.stream = cs;
    return gdn::launch_q4(p) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn::Q4Matrix matrix(const void *codes, const void *scales, const void *offsets) {
    return {static_cast<const uint8_t *>(codes), static_cast<const __nv_bfloat16 *>(scales), static_cast<const __nv_bfloat16 *>(offsets)};
}

}  // namespace

extern "C" {

gdn_status gdn_short_conv(int n_seqs, int total_tokens, int channels, int width, const void *x, long long x_stride,
                          const float *weight, const float *bias, int act, const int32_t *cu_seqlens, const void *state_in,
                          void *state_out, const int32_t *slots, int n_slots, void *out, void *stream) {
    if (channels <= 0 || width <= 0) return GDN_ERR_INVALID_ARG;
    if (channels % 8 != 0 || width < 2 || width > 4) return GDN_ERR_UNSUPPORTED;
    if (act != GDN_CONV_NONE && act != GDN_CONV_SILU) return GDN_ERR_UNSUPPORTED;
    gdn_status st = check_sequences(n_seqs, total_tokens, cu_seqlens, state_in, state_out, slots, n_slots);
    if (st != GDN_OK) return st;
    // CTAs are counted in 32 bits: a token and 512 channels each at the least
    if (((double)n_seqs + total_tokens + 64) * (channels / 512 + 1) >= 2147483648.0) return GDN_ERR_UNSUPPORTED;
    if (n_seqs == 0) return GDN_OK;
    if (!weight || (total_tokens > 0 && (!x || !out))) return GDN_ERR_INVALID_ARG;
    st = check_rows(x, x_stride, channels);
    if (st != GDN_OK) return st;
    if (!aligned(weight) || !aligned(bias) || !aligned(out)) return GDN_ERR_ALIGNMENT;
    const size_t state = (size_t)n_slots * (width - 1) * channels * 2;
    const Range outs[] = {{out, rows_bytes(total_tokens, channels, channels)}, {state_out, state}};
    const Range ins[] = {{x, rows_bytes(total_tokens, x_stride, channels)}, {weight, (size_t)channels * width * 4},
                         {bias, (size_t)channels * 4}, {cu_seqlens, (size_t)(n_seqs + 1) * 4},
                         {state_in == state_out ? nullptr : state_in, state}, {slots, (size_t)n_seqs * 4}};
    if (!disjoint(outs, ins)) return GDN_ERR_INVALID_ARG;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const void *anchors[] = {x, weight, state_out, out};
    st = gdn::on_current_device(anchors, sizeof(anchors) / sizeof(anchors[0]), cs);
    if (st != GDN_OK) return st;

    gdn::ConvProblem p{};
    p.seqs = sequences(n_seqs, total_tokens, cu_seqlens, state_in || state_out, slots, n_slots);
    if (!p.seqs.err) return GDN_ERR_CUDA;
    p.channels = channels; p.width = width;
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.x_stride = x_stride;
    p.weight = weight; p.bias = bias; p.silu = act == GDN_CONV_SILU;
    p.state_in = static_cast<const __nv_bfloat16 *>(state_in);
    p.state_out = static_cast<__nv_bfloat16 *>(state_out);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.stream = cs;
    return gdn::launch_short_conv(p) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_ssm_scan_workspace_size(int n_seqs, int total_tokens, int channels, int n_state, int groups, int max_len,
                                   gdn_status *status) {
    const gdn_status st = check_scan_shape(n_seqs, total_tokens, channels, n_state, groups, max_len);
    if (status) *status = st;
    return st == GDN_OK ? gdn::ssm_scan_workspace_bytes(n_seqs, total_tokens, channels, n_state, groups, max_len) : 0;
}

gdn_status gdn_ssm_scan(int n_seqs, int total_tokens, int channels, int n_state, int groups, const void *x,
                        long long x_stride, const void *dt, long long dt_stride, const float *a, const void *b,
                        long long b_stride, const void *c, long long c_stride, const float *skip, const void *z,
                        long long z_stride, const float *dt_bias, int dt_softplus, const int32_t *cu_seqlens, int max_len,
                        const float *state_in, float *state_out, const int32_t *slots, int n_slots, void *out,
                        int out_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    gdn_status st = check_scan_shape(n_seqs, total_tokens, channels, n_state, groups, max_len);
    if (st != GDN_OK) return st;
    if (out_dtype != GDN_DTYPE_BF16 && out_dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
    if (dt_softplus != 0 && dt_softplus != 1) return GDN_ERR_INVALID_ARG;
    st = check_sequences(n_seqs, total_tokens, cu_seqlens, state_in, state_out, slots, n_slots);
    if (st != GDN_OK) return st;
    if (n_seqs == 0) return GDN_OK;
    if (!a || (total_tokens > 0 && (!x || !dt || !b || !c || !out))) return GDN_ERR_INVALID_ARG;
    const long long row = (long long)groups * n_state;
    const struct { const void *p; long long stride, row; } rows[] = {
        {x, x_stride, channels}, {dt, dt_stride, channels}, {b, b_stride, row}, {c, c_stride, row}, {z, z ? z_stride : channels, channels}};
    for (const auto &r : rows)
        if ((st = check_rows(r.p, r.stride, r.row)) != GDN_OK) return st;
    const void *ptrs[] = {a, skip, dt_bias, out};
    for (const void *p : ptrs)
        if (!aligned(p)) return GDN_ERR_ALIGNMENT;
    const size_t need = gdn::ssm_scan_workspace_bytes(n_seqs, total_tokens, channels, n_state, groups, cu_seqlens ? max_len : 1);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return GDN_ERR_ALIGNMENT;
    const size_t state = (size_t)n_slots * channels * n_state * 4, per_channel = (size_t)channels * 4;
    const Range outs[] = {{out, (size_t)total_tokens * channels * (out_dtype == GDN_DTYPE_F32 ? 4 : 2)}, {state_out, state}, {workspace, need}};
    const Range ins[] = {{x, rows_bytes(total_tokens, x_stride, channels)}, {dt, rows_bytes(total_tokens, dt_stride, channels)},
                         {z, rows_bytes(total_tokens, z_stride, channels)}, {b, rows_bytes(total_tokens, b_stride, row)},
                         {c, rows_bytes(total_tokens, c_stride, row)}, {a, per_channel * n_state}, {skip, per_channel},
                         {dt_bias, per_channel}, {cu_seqlens, (size_t)(n_seqs + 1) * 4},
                         {state_in == state_out ? nullptr : state_in, state}, {slots, (size_t)n_seqs * 4}};
    if (!disjoint(outs, ins)) return GDN_ERR_INVALID_ARG;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const void *anchors[] = {x, a, state_out, out, workspace};
    st = gdn::on_current_device(anchors, sizeof(anchors) / sizeof(anchors[0]), cs);
    if (st != GDN_OK) return st;

    gdn::ScanProblem p{};
    p.seqs = sequences(n_seqs, total_tokens, cu_seqlens, state_in || state_out, slots, n_slots);
    if (!p.seqs.err) return GDN_ERR_CUDA;
    p.channels = channels; p.n_state = n_state; p.groups = groups; p.max_len = cu_seqlens ? max_len : 1;
    p.x = static_cast<const __nv_bfloat16 *>(x); p.x_stride = x_stride;
    p.dt = static_cast<const __nv_bfloat16 *>(dt); p.dt_stride = dt_stride;
    p.z = static_cast<const __nv_bfloat16 *>(z); p.z_stride = z_stride;
    p.b = static_cast<const __nv_bfloat16 *>(b); p.b_stride = b_stride;
    p.c = static_cast<const __nv_bfloat16 *>(c); p.c_stride = c_stride;
    p.a = a; p.skip = skip; p.dt_bias = dt_bias; p.softplus = dt_softplus;
    p.state_in = state_in; p.state_out = state_out;
    p.out = out; p.out_f32 = out_dtype == GDN_DTYPE_F32;
    p.workspace = workspace;
    p.stream = cs;
    return gdn::launch_ssm_scan(p) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_q4_workspace_size(int rows, int n_out, int k, int group, int out_dtype, gdn_status *status) {
    gdn_status st = check_q4_shape(rows, n_out, k, group);
    if (st == GDN_OK && out_dtype != GDN_DTYPE_BF16 && out_dtype != GDN_DTYPE_F32) st = GDN_ERR_UNSUPPORTED;
    if (status) *status = st;
    return st == GDN_OK ? gdn::q4_workspace_bytes(rows, n_out, k, group, out_dtype == GDN_DTYPE_F32) : 0;
}

gdn_status gdn_q4_linear(int rows, int n_out, int k, int group, const void *x, long long x_stride, const void *codes,
                         const void *scales, const void *offsets, void *out, int out_dtype, void *workspace,
                         size_t workspace_bytes, void *stream) {
    return q4(rows, n_out, k, group, x, x_stride, matrix(codes, scales, offsets), nullptr, 0, out, out_dtype, workspace,
              workspace_bytes, stream);
}

gdn_status gdn_q4_gated(int rows, int n_out, int k, int group, const void *x, long long x_stride, const void *gate_codes,
                        const void *gate_scales, const void *gate_offsets, const void *up_codes, const void *up_scales,
                        const void *up_offsets, int act, void *out, int out_dtype, void *workspace, size_t workspace_bytes,
                        void *stream) {
    if (act != GDN_FFN_SILU && act != GDN_FFN_GELU) return GDN_ERR_UNSUPPORTED;
    const gdn::Q4Matrix up = matrix(up_codes, up_scales, up_offsets);
    return q4(rows, n_out, k, group, x, x_stride, matrix(gate_codes, gate_scales, gate_offsets), &up, act == GDN_FFN_GELU, out,
              out_dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
