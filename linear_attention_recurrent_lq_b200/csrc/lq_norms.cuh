// lq_norms.cuh -- the norms and gates around the recurrence (sm_100a).
// Before it: q and k rows to unit length (q also scaled), and the decay and
// write strength from their logits,
//     q' = s q / sqrt(sum q^2 + eps),  k' = k / sqrt(sum k^2 + eps),
//     decay = exp(-exp(A_h) softplus(a + dt)),  beta = 1 / (1 + exp(-b)).
// After it: the head's root-mean-square norm, its weight and output gate,
//     y = o / sqrt(mean o^2 + eps) * w * act(g).
// Both are bound by HBM: each value is read once with 16-byte loads, several
// rows in flight per thread, sums and gates in FP32, one rounding at the end.
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
    long long heads_n;  // rows * H
    int H, kda;
    unsigned norm_blocks;  // the first blocks take q and k rows, the others the gates
};

template <bool BF16>
__device__ __forceinline__ void load_piece(const void *p, float (&x)[BF16 ? 8 : 4]) {
    const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p));
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

// exp(-rate softplus(x)); softplus by log1p, so that small ones keep their digits
__device__ __forceinline__ float gate_decay(float x, float rate) {
    const float soft = fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
    return expf(-rate * soft);
}

__device__ __forceinline__ float sigmoidf(float x) { return __fdiv_rn(1.f, 1.f + expf(-x)); }

constexpr int kNormUnroll = 4;

template <int D, bool BF16>
__global__ void __launch_bounds__(256) qk_norm_kernel(QkNormArgs A) {
    constexpr int V = BF16 ? 8 : 4, E = BF16 ? 2 : 4, LR = D / V;  // values and lanes per row piece
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x < A.norm_blocks) {
        constexpr int G = 256 / LR;  // rows per pass of the block
        const long long r0 = (long long)blockIdx.x * (G * kNormUnroll) + tid / LR;
        const int c = tid % LR;
        float x[kNormUnroll][V];
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            const long long r = r0 + u * G;
            if (r < 2 * A.qk_rows) {
                const bool isk = r >= A.qk_rows;
                const size_t o = ((size_t)(isk ? r - A.qk_rows : r) * D + c * V) * E;
                load_piece<BF16>(static_cast<const uint8_t *>(isk ? A.k : A.q) + o, x[u]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) x[u][i] = 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(x[u][i], x[u][i], ss);
#pragma unroll
            for (int off = LR / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
            const long long r = r0 + u * G;
            const bool isk = r >= A.qk_rows;
            const float f = __fdiv_rn(isk ? 1.f : A.q_scale, __fsqrt_rn(ss + A.eps));
#pragma unroll
            for (int i = 0; i < V; ++i) x[u][i] *= f;
            if (r < 2 * A.qk_rows) {
                const size_t o = ((size_t)(isk ? r - A.qk_rows : r) * D + c * V) * E;
                store_piece<BF16>(static_cast<uint8_t *>(isk ? A.k_out : A.q_out) + o, x[u]);
            }
        }
        return;
    }
    const long long x = (long long)(blockIdx.x - A.norm_blocks) * 256 + tid;
    if (A.kda) {  // V channels of one head
        const long long hr = x / LR;
        if (hr >= A.heads_n) return;
        const int h = (int)(hr % A.H), c = (int)(x % LR) * V;
        float av[V];
        load_piece<BF16>(static_cast<const uint8_t *>(A.a) + ((size_t)hr * D + c) * E, av);
        const float rate = expf(A.a_log[h]);
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 d = *reinterpret_cast<const float4 *>(A.dt_bias + (size_t)h * D + c + i);
            const float4 g = make_float4(gate_decay(av[i] + d.x, rate), gate_decay(av[i + 1] + d.y, rate),
                                         gate_decay(av[i + 2] + d.z, rate), gate_decay(av[i + 3] + d.w, rate));
            *reinterpret_cast<float4 *>(A.decay + (size_t)hr * D + c + i) = g;
        }
        if (c == 0) A.beta[hr] = sigmoidf(load_in(A.b, (size_t)hr, BF16));
        return;
    }
    if (x >= A.heads_n) return;
    const int h = (int)(x % A.H);
    A.decay[x] = gate_decay(load_in(A.a, (size_t)x, BF16) + A.dt_bias[h], expf(A.a_log[h]));
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
                    load_piece<true>(gp, g[u]);
                } else {
                    float h[4];
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        load_piece<false>(gp + 4 * i, h);
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
        const float f = __fdiv_rn(1.f, __fsqrt_rn(fmaf(ss, 1.f / D, A.eps)));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float y = x[u][i] * f * w[i];
            if constexpr (GATE == kGateSilu) y *= g[u][i] * sigmoidf(g[u][i]);
            if constexpr (GATE == kGateSigmoid) y *= sigmoidf(g[u][i]);
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
