// gdn_short_conv: y[t, c] = act(bias[c] + sum_j w[c, j] x[t - (W - 1) + j, c]), rows before a sequence from its state.
//
// A thread carries 4 channels (8 bytes) down a run of tokens with the last W - 1 inputs in registers, so that
// every input is read once, but for the W - 1 rows in front of a run.  Runs are cut from the packed tokens, whatever
// sequences they hold; a thread that comes to a sequence's first token takes the inputs before it from the state, and
// writes the sequence's new state as well.  Nobody else reads that state (the tokens that need it all belong to this
// run), so that state_out may be state_in.
//
// Bound by memory: 4 bytes a token and channel.  Six tokens' inputs are on their way while one is worked on, eight CTAs an SM, 6 KB an
// SM and CTA.  Measured on a GB300: packed prompts of 12545 tokens x 8192 channels, width 4, with bias and SiLU, 71.2 us: 5.8 TB/s, 0.85
// of the copy rate (issue slots 0.48 busy, exponentials 0.33).  One token x 8192 channels 2.4 us, which is a launch.
#include "layer_ops.cuh"

namespace gdn {
namespace {

constexpr int kConvThreads = 128, kConvCtas = 8;       // CTAs an SM
constexpr int kRing = 6;
constexpr int kEmptyPerCta = 64;      // sequences without tokens are looked for by further CTAs, this many each

__device__ __forceinline__ void unpack_pairs(const uint2 &u, Pair (&x)[2]) {
    x[0] = pair(bf16_lo(u.x), bf16_hi(u.x));
    x[1] = pair(bf16_lo(u.y), bf16_hi(u.y));
}

template <int W>
__device__ __forceinline__ uint2 state_row(const ConvProblem &p, int slot, int i, int c) {
    if (!p.state_in) return make_uint2(0, 0);
    return *reinterpret_cast<const uint2 *>(p.state_in + ((size_t)slot * (W - 1) + i) * p.channels + c);
}

// A sequence's state after its tokens [c0, c1), for this thread's channels.
template <int W>
__device__ __forceinline__ void keep_state(const ConvProblem &p, int slot, int c0, int c1, int c) {
    uint2 row[W - 1];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        const int t = c1 - (W - 1) + i;
        row[i] = t >= c0 ? *reinterpret_cast<const uint2 *>(p.x + t * p.x_stride + c) : state_row<W>(p, slot, t - c0 + W - 1, c);
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
        *reinterpret_cast<uint2 *>(p.state_out + ((size_t)slot * (W - 1) + i) * p.channels + c) = row[i];
}

// RING: inputs of that many tokens are on their way while one is worked on.
template <int W, int RING>
__global__ void __launch_bounds__(kConvThreads, kConvCtas) short_conv_kernel(const __grid_constant__ ConvProblem p, int piece_ctas, int tiles, int length) {
    const int c = 4 * (blockIdx.x % piece_ctas * kConvThreads + threadIdx.x), tile = blockIdx.x / piece_ctas;
    if (c >= p.channels) return;
    if (tile >= tiles) {
        const int first = (tile - tiles) * kEmptyPerCta;
        for (int n = first; n < min(first + kEmptyPerCta, p.seqs.n); ++n) {
            const int c0 = p.seqs.begin(n), slot = p.seqs.slot(n);
            if (p.seqs.end(n) > c0) continue;
            if (slot < 0) raise_error(p.seqs.err, kErrInternal);
            else if (p.state_out && p.state_out != p.state_in) keep_state<W>(p, slot, c0, c0, c);
        }
        return;
    }
    Pair w[2][W], bias[2] = {0, 0};         // of channels 2 i and 2 i + 1
    {
        float flat[4 * W], one[4];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            load4(p.weight + (size_t)c * W + 4 * i, one);
#pragma unroll
            for (int e = 0; e < 4; ++e) flat[4 * i + e] = one[e];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int j = 0; j < W; ++j) w[e][j] = pair(flat[2 * e * W + j], flat[(2 * e + 1) * W + j]);
        if (p.bias) {
            load4(p.bias + c, one);
            bias[0] = pair(one[0], one[1]);
            bias[1] = pair(one[2], one[3]);
        }
    }
    const int t0 = tile * length;
    int t1 = t0 + min(length, p.seqs.total - t0), begin = t0;      // (t0 + length may pass 2^31)
    int n = p.seqs.of(t0), c0 = p.seqs.begin(n), c1 = p.seqs.end(n), slot = p.seqs.slot(n);
    if (p.seqs.cu) {
        // A sequence's first W - 1 tokens belong to the run that its first one lies in, which alone reads its state: this run leaves
        // those of a sequence that began before it to the one before, and goes on over its own end for its last sequence's
        if (c0 < t0 && t0 < c1) begin = min(max(t0, c0 + W - 1), c1);
        int e0 = c0, e1 = c1;
        if (length > 1) {
            const int m = p.seqs.of(t1 - 1);
            e0 = p.seqs.begin(m);
            e1 = p.seqs.end(m);
        }
        if (e0 >= t0 && e0 < t1 && e1 > t1) t1 = max(t1, min(e1, e0 + W - 1));
        if (begin >= t1) return;
    }
    const __nv_bfloat16 *from = p.x + begin * p.x_stride + c;
    uint2 x[RING];
#pragma unroll
    for (int i = 0; i < RING; ++i) {
        if (begin + i < t1) x[i] = *reinterpret_cast<const uint2 *>(from);
        from += p.x_stride;
    }
    Pair before[W - 1][2];             // the inputs before this token, oldest first
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        const int t = begin - (W - 1) + i;
        unpack_pairs(t >= c0 && begin < c1 ? *reinterpret_cast<const uint2 *>(p.x + t * p.x_stride + c) : make_uint2(0, 0), before[i]);
    }
    __nv_bfloat16 *to = p.out + (size_t)begin * p.channels + c;
    const auto token = [&](const uint2 &raw, bool written) {
        Pair now[2];
        unpack_pairs(raw, now);
        uint32_t out[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            Pair y = bias[e];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) y = fma2(w[e][j], before[j][e], y);
            y = fma2(w[e][W - 1], now[e], y);
            float lo, hi;
            if (p.silu) {                      // y / (1 + e^-y)
                halves(mul2(y, pair(-kLog2e, -kLog2e)), lo, hi);
                halves(add2(pair(ex2(lo), ex2(hi)), pair(1.f, 1.f)), lo, hi);
                y = mul2(y, pair(reciprocal(lo), reciprocal(hi)));
            }
            halves(y, lo, hi);
            out[e] = pack2(lo, hi);
        }
        if (written) *reinterpret_cast<uint2 *>(to) = make_uint2(out[0], out[1]);
        to += p.channels;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) before[j][e] = j + 1 < W - 1 ? before[j + 1][e] : now[e];
    };
    for (int base = begin; base < t1; base += RING) {
        if (RING > 1 && base > c0 && base + RING <= c1 && base + 2 * RING <= t1 && slot >= 0) {     // inside one sequence
#pragma unroll
            for (int i = 0; i < RING; ++i) {
                const uint2 now = x[i];
                x[i] = *reinterpret_cast<const uint2 *>(from);
                from += p.x_stride;
                token(now, true);
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < RING; ++i) {
            const int t = base + i;
            if (t >= t1) break;
            const uint2 now = x[i];
            if (t + RING < t1) x[i] = *reinterpret_cast<const uint2 *>(from);
            from += p.x_stride;
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
                    for (int j = 0; j < W - 1; ++j) unpack_pairs(state_row<W>(p, slot, j, c), before[j]);
                    if (p.state_out) keep_state<W>(p, slot, c0, c1, c);
                }
            }
            token(now, held && slot >= 0);
        }
    }
}

template <int W>
cudaError_t launch(const ConvProblem &p) {
    const int piece_ctas = (p.channels / 4 + kConvThreads - 1) / kConvThreads;
    // Few tokens: one a thread.  Many: as many CTAs as are on the SMs at once, each down an equal run of tokens.  61 tokens x 8192
    // channels take 3.7 us as few, 6.4 as many; 500 take 21.5 and 16.6; 3000 in prompts 86.6 and 24.0
    const long pieces = (long)p.channels / 4 * p.seqs.total;
    const bool many = pieces >= (long)kConvCtas * kConvThreads * kRing * multiprocessor_count();
    const int runs = max(1, kConvCtas * multiprocessor_count() / piece_ctas);
    const int length = many ? max(kRing, (p.seqs.total + runs - 1) / runs) : 1;
    const int tiles = (p.seqs.total + length - 1) / length;
    // sequences without tokens have nobody who keeps their state, unless it stays where it is, or looks at their slot
    const bool looked_at = (p.state_out && p.state_out != p.state_in) || p.seqs.slots;
    const int empty = p.seqs.cu && looked_at ? (p.seqs.n + kEmptyPerCta - 1) / kEmptyPerCta : 0;
    const long ctas = (long)(tiles + empty) * piece_ctas;
    if (ctas == 0) return cudaSuccess;
    (many ? short_conv_kernel<W, kRing> : short_conv_kernel<W, 1>)<<<(unsigned)ctas, kConvThreads, 0, p.stream>>>(p, piece_ctas, tiles, length);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_short_conv(const ConvProblem &p) {
    return p.width == 2 ? launch<2>(p) : p.width == 3 ? launch<3>(p) : launch<4>(p);
}

}  // namespace gdn
