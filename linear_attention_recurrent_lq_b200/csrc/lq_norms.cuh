// lq_norms.cuh -- the norms and gates around the recurrence (sm_100a).
// Before it: q and k rows to unit length (q also scaled), and the decay and
// write strength from their logits,
//     q' = s q / sqrt(sum q^2 + eps),  k' = k / sqrt(sum k^2 + eps),
//     decay = exp(-exp(A_h) softplus(a + dt)),  beta = 1 / (1 + exp(-b)).
// After it: the head's root-mean-square norm, its weight and output gate,
//     y = o / sqrt(mean o^2 + eps) * w * act(g).
// Both are bound by HBM: each value is read once with 16-byte loads, several
// rows in flight per thread, sums and gates in FP32, one rounding at the end.
// Measured, bf16, d = 128: qk_norm of 16384 tokens of 12 heads with a gate per key
// channel 73.0 us (54.0 at the copy's rate; bound by instruction issue), out_norm of
// 16384 tokens of 32 heads 90.6 us, 5930 GB/s (82.0).
#pragma once

#include "lq_linear.cuh"

namespace lq {

struct QkNormArgs {
    const void *q, *k;  // [rows, Hk, D]
    const void *a;      // [rows, H] or [rows, H, D]
    const void *b;      // [rows, H]
    const float *a_log;   // [H]
    const float *dt_bias; // [H] or [H, D]
    void *q_out, *k_out;
    float *decay, *beta;
    float q_scale, eps;
    long long qk_rows;  // rows * Hk
    unsigned heads_n;   // rows * H
    int H, kda;
    unsigned norm_blocks, gate_blocks;  // blocks for q and k rows, and for the gates
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool BF16>
__device__ __forceinline__ void store_piece(void *p, const float (&x)[BF16 ? 8 : 4]) {
    uint4 w;
    if constexpr (BF16)
        w = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    else
        w = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    *reinterpret_cast<uint4 *>(p) = w;
}

// exp(-rate softplus(x)) of two, softplus(x) = max(x, 0) + log(1 + e), e =
// exp(-|x|).  Small ones have to keep their digits, so log(1 + e) is not taken of
// a rounded 1 + e but from its series 2 artanh(r), r = e / (2 + e) <= 1/3; the
// first term left out is r^14 / 15 <= 1.4e-8 of the sum.  With log1pf and expf
// the gates of a key-channel layer took as long as its memory traffic twice.
__device__ __forceinline__ float2 gate_decay2(float2 x, float rate) {
    const float2 e = make_float2(__expf(-fabsf(x.x)), __expf(-fabsf(x.y)));
    const float2 r = make_float2(__fdividef(e.x, 2.f + e.x), __fdividef(e.y, 2.f + e.y)), r2 = __fmul2_rn(r, r);
    auto both = [](float c) { return make_float2(c, c); };
    float2 p = __ffma2_rn(r2, both(1.f / 13.f), both(1.f / 11.f));
    p = __ffma2_rn(r2, p, both(1.f / 9.f));
    p = __ffma2_rn(r2, p, both(1.f / 7.f));
    p = __ffma2_rn(r2, p, both(1.f / 5.f));
    p = __ffma2_rn(r2, p, both(1.f / 3.f));
    p = __ffma2_rn(r2, p, both(1.f));
    const float2 soft = __ffma2_rn(__fmul2_rn(both(2.f), r), p, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
    const float2 t = __fmul2_rn(both(-rate), soft);
    return make_float2(__expf(t.x), __expf(t.y));
}

// 1 / (1 + exp(-x)) from e = exp(-|x|), which never overflows: e / (1 + e) below
// zero, so that a gate far below keeps its digits down to FP32's smallest values.
__device__ __forceinline__ float sigmoidf(float x) {
    const float e = expf(-fabsf(x));
    return __fdiv_rn(x < 0.f ? e : 1.f, 1.f + e);
}
// The same for a result that is rounded to bf16 (2^-8) next, from 2^24 e: the
// exponent -|x| log2(e) + 24 is rounded by at most 2^-18, so the result is within
// 1e-5, and nothing is flushed to zero before x = -104, where a silu is below
// bf16's smallest value.
__device__ __forceinline__ float sigmoid_fast(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(-fabsf(x), 1.44269504f, 24.f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 0x1p24f));
    return (x < 0.f ? e : 0x1p24f) * r;
}

template <bool BF16>
__device__ __forceinline__ void unpack_piece(const uint4 &w, float (&x)[BF16 ? 8 : 4]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        } else {
            x[i] = __uint_as_float(u[i]);
        }
    }
}

// Pieces of 16 bytes a thread loads before it uses the first: 8 for q and k
// rows, 4 for the gates of key channels (4 and 1: 95 us for 16384 tokens of 12
// heads, d = 128, 54 us of memory traffic).
constexpr int kNormUnroll = 8, kGateUnroll = 4;

template <int D, bool BF16>
__global__ void __launch_bounds__(256) qk_norm_kernel(QkNormArgs A) {
    constexpr int V = BF16 ? 8 : 4, E = BF16 ? 2 : 4, LR = D / V;  // values and lanes per row piece
    constexpr int G = 256 / LR;                                    // rows per pass of the block
    const int tid = threadIdx.x, c = (tid % LR) * V;
    // the two kinds of block alternate over the grid, so that an SM has the one
    // bound by memory and the one bound by its exponentials at the same time
    const unsigned blocks = A.norm_blocks + A.gate_blocks;
    const unsigned gates = (unsigned)((unsigned long long)blockIdx.x * A.gate_blocks / blocks);  // before this block
    const bool is_gate = (unsigned)((unsigned long long)(blockIdx.x + 1u) * A.gate_blocks / blocks) > gates;
    pdl_wait();
    pdl_trigger();
    if (!is_gate) {
        const long long r0 = (long long)(blockIdx.x - gates) * (G * kNormUnroll) + tid / LR;
        uint4 w[kNormUnroll];
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            const long long r = r0 + u * G;
            const bool isk = r >= A.qk_rows;
            const size_t o = ((size_t)(isk ? r - A.qk_rows : r) * D + c) * E;
            w[u] = r < 2 * A.qk_rows ? __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(isk ? A.k : A.q) + o))
                                     : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            float x[V], ss = 0.f;
            unpack_piece<BF16>(w[u], x);
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int off = LR / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
            const long long r = r0 + u * G;
            const bool isk = r >= A.qk_rows;
            const float f = (isk ? 1.f : A.q_scale) * rsqrtf(ss + A.eps);
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] *= f;
            if (r < 2 * A.qk_rows) {
                const size_t o = ((size_t)(isk ? r - A.qk_rows : r) * D + c) * E;
                store_piece<BF16>(static_cast<uint8_t *>(isk ? A.k_out : A.q_out) + o, x);
            }
        }
        return;
    }
    if (A.kda) {  // V channels of one head
        const unsigned r0 = gates * (G * kGateUnroll) + tid / LR;  // rows * H < 2^31
        // heads of the rows u G apart: one division, then steps
        unsigned h = r0 % (unsigned)A.H;
        const unsigned step = G % (unsigned)A.H;
        uint4 w[kGateUnroll];
#pragma unroll
        for (int u = 0; u < kGateUnroll; ++u) {
            const unsigned r = r0 + u * G;
            w[u] = r < A.heads_n ? __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(A.a) + ((size_t)r * D + c) * E))
                                 : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < kGateUnroll; ++u) {
            const unsigned r = r0 + u * G;
            if (r >= A.heads_n) return;
            const float rate = __expf(A.a_log[h]);
            float x[V];
            unpack_piece<BF16>(w[u], x);
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 d = __ldg(reinterpret_cast<const float4 *>(A.dt_bias + (size_t)h * D + c + i));
                const float2 g0 = gate_decay2(__fadd2_rn(make_float2(x[i], x[i + 1]), make_float2(d.x, d.y)), rate);
                const float2 g1 = gate_decay2(__fadd2_rn(make_float2(x[i + 2], x[i + 3]), make_float2(d.z, d.w)), rate);
                *reinterpret_cast<float4 *>(A.decay + (size_t)r * D + c + i) = make_float4(g0.x, g0.y, g1.x, g1.y);
            }
            if (c == 0) A.beta[r] = sigmoidf(load_in(A.b, (size_t)r, BF16));
            h += step;
            if (h >= (unsigned)A.H) h -= (unsigned)A.H;
        }
        return;
    }
    const unsigned x = gates * 256u + tid;
    if (x >= A.heads_n) return;
    const unsigned h = x % (unsigned)A.H;
    const float z = load_in(A.a, (size_t)x, BF16) + A.dt_bias[h];
    A.decay[x] = gate_decay2(make_float2(z, z), expf(A.a_log[h])).x;
    A.beta[x] = sigmoidf(load_in(A.b, (size_t)x, BF16));
}

struct OutNormArgs {
    const float *o;       // [n, D]
    const float *weight;  // [D] or null
    const void *gate;     // [n, D] or null
    void *y;              // [n, D]
    float eps;
    long long n;  // rows * H
};

constexpr int kGateNone = 0, kGateSilu = 1, kGateSigmoid = 2;
constexpr int kOutNormUnroll = 2;

template <int D, bool BF16, int GATE>
__global__ void __launch_bounds__(256) out_norm_kernel(OutNormArgs A) {
    constexpr int LR = D / 8, G = 256 / LR, E = BF16 ? 2 : 4;
    const int tid = threadIdx.x, c = 8 * (tid % LR);
    const long long r0 = (long long)blockIdx.x * (G * kOutNormUnroll) + tid / LR;
    pdl_wait();
    pdl_trigger();
    float x[kOutNormUnroll][8], g[kOutNormUnroll][8], w[8];
#pragma unroll
    for (int u = 0; u < kOutNormUnroll; ++u) {
        const long long r = r0 + u * G;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[u][i] = g[u][i] = 0.f;
        if (r < A.n) {
            const size_t o = (size_t)r * D + c;
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 f = __ldcs(reinterpret_cast<const float4 *>(A.o + o + i));
                x[u][i] = f.x; x[u][i + 1] = f.y; x[u][i + 2] = f.z; x[u][i + 3] = f.w;
            }
            if constexpr (GATE != kGateNone) {
                const uint8_t *gp = static_cast<const uint8_t *>(A.gate) + o * E;
                if constexpr (BF16) {
                    unpack_piece<true>(__ldcs(reinterpret_cast<const uint4 *>(gp)), g[u]);
                } else {
                    float h[4];
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        unpack_piece<false>(__ldcs(reinterpret_cast<const uint4 *>(gp + 4 * i)), h);
                        g[u][i] = h[0]; g[u][i + 1] = h[1]; g[u][i + 2] = h[2]; g[u][i + 3] = h[3];
                    }
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    if (A.weight) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(A.weight + c + i));
            w[i] = f.x; w[i + 1] = f.y; w[i + 2] = f.z; w[i + 3] = f.w;
        }
    }
#pragma unroll
    for (int u = 0; u < kOutNormUnroll; ++u) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[u][i], x[u][i], ss);
#pragma unroll
        for (int off = LR / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
        const float f = rsqrtf(fmaf(ss, 1.f / D, A.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float y = x[u][i] * f * w[i];
            if constexpr (GATE != kGateNone) {
                const float sg = BF16 ? sigmoid_fast(g[u][i]) : sigmoidf(g[u][i]);
                y *= GATE == kGateSilu ? g[u][i] * sg : sg;
            }
            x[u][i] = y;
        }
        const long long r = r0 + u * G;
        if (r < A.n) {
            uint8_t *yp = static_cast<uint8_t *>(A.y) + ((size_t)r * D + c) * E;
            if constexpr (BF16) {
                store_piece<true>(yp, x[u]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float h[4] = {x[u][i], x[u][i + 1], x[u][i + 2], x[u][i + 3]};
                    store_piece<false>(yp + 4 * i, h);
                }
            }
        }
    }
}

}  // namespace lq
