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
// channel 74 us (54.0 at the copy's rate; the latency of the gates' exponentials, with
// a third of the warps that an SM holds), out_norm of 16384 tokens of 32 heads 92 us,
// 5840 GB/s (82.0).
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

// 2^x and 1 / x within 2 and 1 units of 2^-23; results below FP32's normal numbers
// are zeros.
__device__ __forceinline__ float ex2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596303e-8f;  // log2(e), and what its rounding left
constexpr float kLn2 = 0.693147181f;

// -rate log2(e) in two floats, rate = exp(a_log).
struct GateRate {
    float hi, lo;
    __device__ __forceinline__ explicit GateRate(float a_log) {
        const float y = a_log * kLog2e, z = ex2_ftz(y);
        const float rate = fmaf(z, kLn2 * fmaf(a_log, kLog2eRest, fmaf(a_log, kLog2e, -y)), z);
        hi = -rate * kLog2e;
        lo = fmaf(-rate, kLog2eRest, fmaf(-rate, kLog2e, -hi));
    }
    // times a softplus up to 2^63 it stays inside FP32, and the decay is 0 there
    __device__ __forceinline__ bool usual() const { return hi <= -0x1p-55f && hi >= -0x1p63f; }
};

// exp(-exp(a_log) softplus(x)) for rates outside GateRate's usual range.
__device__ __noinline__ float gate_decay_far(float x, float a_log) {
    return expf(-expf(a_log) * (fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)))));
}

// exp(-rate softplus(x)) of two for a usual rate, softplus(x) = max(x, 0) +
// log(1 + e), e = exp(-|x|).  Small ones have to keep their digits, so log(1 + e) is
// not taken of a rounded 1 + e but as 2 artanh(r), r = e / (2 + e) <= 1/3, r times a
// polynomial in r^2 (least maximum of the relative error, 5e-9).  e is within
// (4 + 2.4 |x|) units of 2^-24, of the order of what the rounded sum a + dt_bias
// does to it (|x| units).  The exponent of the result may be large, so the rounding
// error of the product rate times softplus, a unit for each unit of the exponent,
// is kept and put back: the result is as exact as its two factors are.
__device__ __forceinline__ float2 gate_decay2(float2 x, const GateRate &rate) {
    auto both = [](float c) { return make_float2(c, c); };
    const float2 e = make_float2(ex2_ftz(-kLog2e * fabsf(x.x)), ex2_ftz(-kLog2e * fabsf(x.y)));
    const float2 e2 = __fadd2_rn(e, both(2.f));
    const float2 r = __fmul2_rn(e, make_float2(rcp_ftz(e2.x), rcp_ftz(e2.y))), r2 = __fmul2_rn(r, r);
    float2 p = __ffma2_rn(r2, both(0.280244589f), both(0.279991418f));
    p = __ffma2_rn(r2, p, both(0.400216997f));
    p = __ffma2_rn(r2, p, both(0.666664124f));
    p = __ffma2_rn(r2, p, both(2.f));
    // beyond 2^63 the decay is 0, as it is at 2^63
    const float2 soft = __ffma2_rn(r, p, make_float2(fminf(fmaxf(x.x, 0.f), 0x1p63f), fminf(fmaxf(x.y, 0.f), 0x1p63f)));
    const float2 y = __fmul2_rn(both(rate.hi), soft);
    float2 left = __ffma2_rn(both(rate.hi), soft, make_float2(-y.x, -y.y));
    left = __fmul2_rn(both(kLn2), __ffma2_rn(both(rate.lo), soft, left));
    float2 z;
    asm("ex2.approx.f32 %0, %1;" : "=f"(z.x) : "f"(y.x));
    asm("ex2.approx.f32 %0, %1;" : "=f"(z.y) : "f"(y.y));
    return __ffma2_rn(z, left, z);
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
    const float e = ex2_ftz(fmaf(-fabsf(x), kLog2e, 24.f));
    return (x < 0.f ? e : 0x1p24f) * rcp_ftz(e + 0x1p24f);
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
// rows, 32 values for the gates of key channels (16384 tokens of 12 heads, d = 128,
// bf16: 2, 4 and 8 pieces 76.7, 71.6 and 91.4 us; f32: 130, 118 and 111 us).
constexpr int kNormUnroll = 8;
template <bool BF16>
constexpr int kGateUnroll = BF16 ? 4 : 8;

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
        const unsigned r0 = gates * (G * kGateUnroll<BF16>) + tid / LR;  // rows * H < 2^31
        // heads of the rows u G apart: one division, then steps
        unsigned h = r0 % (unsigned)A.H;
        const unsigned step = G % (unsigned)A.H;
        uint4 w[kGateUnroll<BF16>];
        float a_log[kGateUnroll<BF16>];
#pragma unroll
        for (int u = 0; u < kGateUnroll<BF16>; ++u) {
            const unsigned r = r0 + u * G;
            a_log[u] = __ldg(A.a_log + h);
            h += step;
            if (h >= (unsigned)A.H) h -= (unsigned)A.H;
            w[u] = r < A.heads_n ? __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(A.a) + ((size_t)r * D + c) * E))
                                 : make_uint4(0u, 0u, 0u, 0u);
        }
        h = r0 % (unsigned)A.H;
#pragma unroll
        for (int u = 0; u < kGateUnroll<BF16>; ++u) {
            const unsigned r = r0 + u * G;
            if (r >= A.heads_n) return;
            const GateRate rate(a_log[u]);
            float x[V];
            unpack_piece<BF16>(w[u], x);
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 d = __ldg(reinterpret_cast<const float4 *>(A.dt_bias + (size_t)h * D + c + i));
                if (!rate.usual()) {
                    *reinterpret_cast<float4 *>(A.decay + (size_t)r * D + c + i) =
                        make_float4(gate_decay_far(x[i] + d.x, a_log[u]), gate_decay_far(x[i + 1] + d.y, a_log[u]),
                                    gate_decay_far(x[i + 2] + d.z, a_log[u]), gate_decay_far(x[i + 3] + d.w, a_log[u]));
                    continue;
                }
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
    const float a_log = A.a_log[h];
    const GateRate rate(a_log);
    A.decay[x] = rate.usual() ? gate_decay2(make_float2(z, z), rate).x : gate_decay_far(z, a_log);
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
