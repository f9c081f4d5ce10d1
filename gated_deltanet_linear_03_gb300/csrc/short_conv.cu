// gdn_short_conv: y[t, c] = act(bias[c] + sum_j w[c, j] x[t - (W - 1) + j, c]), rows before a sequence from its state.
//
// A thread carries a piece of 8 channels (16 bytes) down a tile of L tokens with the last W - 1 inputs in registers, so
// every input is read once, but for the W - 1 rows in front of a tile.  Tiles are cut from the packed tokens, whatever
// sequences they hold; a thread that comes to a sequence's first token takes the inputs before it from the state, and
// writes the sequence's new state as well: its old state is read by this thread alone and before that, so that
// state_out may be state_in.
#include "layer_ops.cuh"

namespace gdn {
namespace {

constexpr int kConvThreads = 128;
constexpr int kEmptyPerCta = 64;      // sequences without tokens are looked for by further CTAs, this many each

template <int W>
__device__ __forceinline__ uint4 state_row(const ConvProblem &p, int slot, int i, int c) {
    if (!p.state_in) return make_uint4(0, 0, 0, 0);
    return *reinterpret_cast<const uint4 *>(p.state_in + ((size_t)slot * (W - 1) + i) * p.channels + c);
}

// A sequence's state after its tokens [c0, c1), for this thread's channels.
template <int W>
__device__ __forceinline__ void keep_state(const ConvProblem &p, int slot, int c0, int c1, int c) {
    uint4 row[W - 1];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        const int t = c1 - (W - 1) + i;
        row[i] = t >= c0 ? *reinterpret_cast<const uint4 *>(p.x + t * p.x_stride + c) : state_row<W>(p, slot, t - c0 + W - 1, c);
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
        *reinterpret_cast<uint4 *>(p.state_out + ((size_t)slot * (W - 1) + i) * p.channels + c) = row[i];
}

template <int W, int L>
__global__ void __launch_bounds__(kConvThreads) short_conv_kernel(const __grid_constant__ ConvProblem p, int piece_ctas, int tiles) {
    const int c = 8 * (blockIdx.x % piece_ctas * kConvThreads + threadIdx.x), tile = blockIdx.x / piece_ctas;
    if (c >= p.channels) return;
    if (tile >= tiles) {
        const int first = (tile - tiles) * kEmptyPerCta;
        for (int n = first; n < min(first + kEmptyPerCta, p.seqs.n); ++n) {
            const int c0 = p.seqs.begin(n), slot = p.seqs.slot(n);
            if (p.seqs.end(n) > c0) continue;
            if (slot >= 0) keep_state<W>(p, slot, c0, c0, c);
            else raise_error(p.seqs.err, kErrInternal);
        }
        return;
    }
    float w[8][W], bias[8];
    {
        float flat[8 * W];
#pragma unroll
        for (int i = 0; i < 2 * W; ++i) {
            float q[4];
            load4(p.weight + (size_t)c * W + 4 * i, q);
#pragma unroll
            for (int e = 0; e < 4; ++e) flat[4 * i + e] = q[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int j = 0; j < W; ++j) w[e][j] = flat[e * W + j];
#pragma unroll
        for (int e = 0; e < 8; ++e) bias[e] = 0.f;
        if (p.bias) load8(p.bias + c, bias);
    }
    const int t0 = tile * L, t1 = min(t0 + L, p.seqs.total);
    uint4 x[L];
#pragma unroll
    for (int i = 0; i < L; ++i)
        x[i] = t0 + i < t1 ? *reinterpret_cast<const uint4 *>(p.x + (t0 + i) * p.x_stride + c) : make_uint4(0, 0, 0, 0);
    int n = p.seqs.of(t0), c0 = p.seqs.begin(n), c1 = p.seqs.end(n), slot = p.seqs.slot(n);
    float before[W - 1][8];            // the inputs before this token, oldest first
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        const int t = t0 - (W - 1) + i;
        uint4 row = make_uint4(0, 0, 0, 0);
        if (t >= c0 && t0 < c1) row = *reinterpret_cast<const uint4 *>(p.x + t * p.x_stride + c);
        else if (t0 > c0 && t0 < c1 && slot >= 0) row = state_row<W>(p, slot, t - c0 + W - 1, c);
        unpack8(row, before[i]);
    }
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const int t = t0 + i;
        if (t >= t1) break;
        if (t >= c1 && n + 1 < p.seqs.n) {       // the next sequence that has tokens
            n = p.seqs.of(t);
            c0 = p.seqs.begin(n);
            c1 = p.seqs.end(n);
            slot = p.seqs.slot(n);
        }
        const bool held = t >= c0 && t < c1;
        if (t == c0 && held) {
            if (slot < 0) raise_error(p.seqs.err, kErrInternal);
            else {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) unpack8(state_row<W>(p, slot, j, c), before[j]);
                if (p.state_out) keep_state<W>(p, slot, c0, c1, c);
            }
        }
        float now[8], y[8];
        unpack8(x[i], now);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[e] = bias[e];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) y[e] = fmaf(w[e][j], before[j][e], y[e]);
            y[e] = fmaf(w[e][W - 1], now[e], y[e]);
            if (p.silu) y[e] = __fdividef(y[e], 1.f + __expf(-y[e]));
        }
        if (held && slot >= 0) *reinterpret_cast<uint4 *>(p.out + (size_t)t * p.channels + c) = pack8(y);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) before[j][e] = j + 1 < W - 1 ? before[j + 1][e] : now[e];
    }
}

template <int W>
cudaError_t launch(const ConvProblem &p) {
    const int piece_ctas = (p.channels / 8 + kConvThreads - 1) / kConvThreads;
    const long pieces = (long)p.channels / 8 * p.seqs.total;
    const int l = pieces >= 8L * 1024 * multiprocessor_count() ? 16 : 1;
    const int tiles = (p.seqs.total + l - 1) / l;
    // sequences without tokens have nobody who keeps their state, unless it stays where it is
    const int empty = p.seqs.cu && p.state_out && p.state_out != p.state_in ? (p.seqs.n + kEmptyPerCta - 1) / kEmptyPerCta : 0;
    const long ctas = (long)(tiles + empty) * piece_ctas;
    if (ctas == 0) return cudaSuccess;
    (l == 1 ? short_conv_kernel<W, 1> : short_conv_kernel<W, 16>)<<<(unsigned)ctas, kConvThreads, 0, p.stream>>>(p, piece_ctas, tiles);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_short_conv(const ConvProblem &p) {
    return p.width == 2 ? launch<2>(p) : p.width == 3 ? launch<3>(p) : launch<4>(p);
}

}  // namespace gdn
