// lq_linear_chunked.cuh -- a prompt of linear attention in the chunkwise form
// on the tensor cores (bf16 q, k, v; sm_100a, tcgen05).
//
// Over a chunk of 64 tokens, with a_t the gates, S the state before it, and
//     R_ts = prod_{s < u <= t} a_u,   G_t = prod_{u <= t} a_u,
//     W_s = prod_{u > s} a_u          (products, so a gate of 0 is exact),
// the outputs and the state after it are
//     o_t = G_t S^T q_t + sum_{s <= t} R_ts (q_t . k_s) v_s,
//     S'  = G_last S + sum_s W_s k_s v_s^T.
//
// Precision: the state and the weights are FP32, the tensor cores take bf16
// with FP32 accumulation.  q, k and v are bf16 as they come; every FP32
// operand (S, the weighted scores P, the weighted keys K') is cut into three
// bf16 pieces of 8 mantissa bits each, which hold its 24 bits exactly, and
// multiplied piece by piece, smallest first.  Against that, a cut into two
// pieces would leave 2^-17 of each operand, and TF32 (11 bits) two pieces at
// twice the cost of bf16 each.
//
// One CTA of 256 threads takes one head (or one segment of a prompt cut along
// time), two CTAs share an SM: while one waits for its products the other
// computes.  The state stays in registers (lane = value channel, the two
// groups of four warps take half of the key channels each).  Per chunk:
//  * q, k, v arrive by cp.async into 128-byte-swizzled tiles; rows behind the
//    prompt arrive as zeros, whatever lies there;
//  * Q K^T (64 x 64) in tensor memory, read back, weighted with R and written
//    as the three pieces of P;
//  * S^T in three pieces to tensor memory, where it is the A operand of
//    Y^T = S^T Q^T; Y^T is scaled by G in place;
//  * O^T = Y^T + V^T P^T, and V^T K' beside it; the outputs go straight from
//    tensor memory to global memory, a warp 128 bytes of a row at a time.
// Products with V^T and K' read the tiles along their rows (MN-major).
#pragma once

#include "lq_linear.cuh"
#include "lq_umma.cuh"

namespace lq {

constexpr int kLcTokens = 64;
constexpr int kLcThreads = 256;
constexpr uint32_t kLcCols = 256;              // tensor-memory columns of a CTA
constexpr uint32_t kLcO = 0, kLcR = 64;        // O^T (and Q K^T) | S pieces, then V^T K'

// Shared memory from a 1024-aligned base: [D / 64] blocks of 128 rows x 128
// bytes (64 rows of Q, 64 of K, later K' high) | V, [D / 64] blocks of 64 rows
// | P, three pieces of 64 rows | K' middle and low, [D / 64] blocks each |
// control.
template <int D>
struct LcShape {
    static constexpr int KB = D / 64;
    static constexpr uint32_t QK = 0, V = KB * 16384u, P = V + KB * 8192u, KM = P + 3u * 8192u;
    static constexpr uint32_t CTL = KM + 2u * KB * 8192u;
    // barriers [2], tensor-memory base | gates | G | products from token 32 on | W
    static constexpr uint32_t SMEM_USED = CTL + 64u + 4u * 64u * 4u + 1024u;
    // D = 64 too: at most two CTAs per SM, which is all tensor memory has columns for
    static constexpr uint32_t SMEM = SMEM_USED > 90u * 1024u ? SMEM_USED : 90u * 1024u;
};

// Shared-memory matrix descriptors (128-byte swizzle, 1024 bytes between
// groups of eight rows) differ in their low word only: the address and, for an
// operand read along its rows, the distance of its 64-element blocks.  The
// issuing thread adds to that word; the high word is a constant.
constexpr uint32_t kLcDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t lc_desc(uint32_t saddr, uint32_t lbo) {
    return ((saddr >> 4) & 0x3FFFu) | (((lbo >> 4) & 0x3FFFu) << 16);
}

// D in FP32, A and B in bf16; a bit per operand read along its rows (MN-major).
__host__ __device__ constexpr uint32_t lc_idesc(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void lc_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kLcDescHi)
        : "memory");
}

__device__ __forceinline__ void lc_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kLcDescHi)
        : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool lc_elect() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
          "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two FP32 values in three pairs of bf16 pieces: the 8 leading bits, the next
// 8, the rest (cut off, not rounded), so that x = hi - mid + lo exactly.  The
// middle piece comes out negated, because the subtraction that takes a bf16
// half of a register as it is (no masks: 6.6 clocks of a scheduler a pair,
// 9.6 with them) has it first; the products with it negate it back.
__device__ __forceinline__ void lc_split2(float x, float y, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    float x1, y1, x2, y2;
    hi = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tsub.rn.f32.bf16 %0, a, %3;\n\tsub.rn.f32.bf16 %1, b, %4;\n\t}"
        : "=f"(x1), "=f"(y1) : "r"(hi), "f"(x), "f"(y));
    mid = __byte_perm(__float_as_uint(x1), __float_as_uint(y1), 0x7632);
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tsub.rn.f32.bf16 %0, a, %3;\n\tsub.rn.f32.bf16 %1, b, %4;\n\t}"
        : "=f"(x2), "=f"(y2) : "r"(mid), "f"(x1), "f"(y1));
    lo = __byte_perm(__float_as_uint(x2), __float_as_uint(y2), 0x7632);
}
constexpr uint32_t kLcNegA = 1u << 13, kLcNegB = 1u << 14;  // of the instruction descriptor

template <int D, bool PARTIAL>
__global__ void __launch_bounds__(kLcThreads, 2) lin_chunk_kernel(LinArgs A) {
    using SH = LcShape<D>;
    constexpr int KB = SH::KB, C = kLcTokens, HD = D / 2;  // HD: key channels a thread holds
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int w = blockIdx.x, seg = blockIdx.y;
    const int row = w / A.map.heads, hh = w - row * A.map.heads;
    const int j = 32 * (warp & 3) + lane, half = warp >> 2;  // tensor-memory lane, column half
    const bool holds = j < D;                                // this lane is a value channel

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + SH::CTL);
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + SH::CTL + 16);
    float *s_a = reinterpret_cast<float *>(smem + SH::CTL + 64), *s_G = s_a + C, *s_G2 = s_G + C, *s_W = s_G2 + C;
    const uint32_t base = smem_u32(smem);

    if (tid == 0) {
        mbar_init(&bar[0], 1);
        mbar_init(&bar[1], 1);
        fence_mbar_init();
    }
    pdl_wait();
    // after the wait: a kernel still running may need all of tensor memory
    if (warp == 0) tmem_alloc(s_tmem, kLcCols);
    pdl_trigger();
    const int len = lin_length(A, row), last = lin_last_segment(A, len);
    const int bi = A.map.blob(w);
    uint8_t *blob = A.state + (size_t)(bi < 0 ? 0 : bi) * A.L.blob;
    bool run = bi >= 0 && !(PARTIAL && seg >= last);
    if (!PARTIAL && A.cont && run) run = A.nseg > 1 ? A.ws_run[w] != 0 : lin_may_run(blob, tid == 0);
    const int t_begin = seg * A.seg_len, t_end = min(A.tokens, t_begin + A.seg_len);
    if (!PARTIAL && run && seg <= last)
        for (int s = 0; s < seg; ++s)
            if (A.ws_bad[(size_t)w * A.nseg + s] != kNoBad) run = false;
    const int t_stop = run ? min(len, t_end) : t_begin;

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    const uint32_t tlane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);

    // ---- loads of one chunk: rows of 16-byte pieces, swizzled
    const uint8_t *qg = static_cast<const uint8_t *>(A.q), *kg = static_cast<const uint8_t *>(A.k);
    const uint8_t *vg = static_cast<const uint8_t *>(A.v);
    constexpr int NP = 8 * KB;  // pieces per row
    const int pr = tid / NP, pc = tid % NP;
    auto tile_off = [&](int r, int c, uint32_t block) -> uint32_t {
        return (uint32_t)(c >> 3) * block + (uint32_t)r * 128u + (uint32_t)(((c & 7) ^ (r & 7)) << 4);
    };
    auto load_rows = [&](const uint8_t *g, bool is_v, uint32_t at, uint32_t block, int t0) {
#pragma unroll
        for (int x = 0; x < C * NP / kLcThreads; ++x) {
            const int r = pr + x * (kLcThreads / NP);
            const bool in = t0 + r < t_stop;
            const int t = in ? t0 + r : t_begin;
            const size_t o = is_v ? lin_v_row(A, row, hh, t) : lin_qk_row(A, row, hh, t);
            cp_async16(smem + at + tile_off(r, pc, block), g + o * (size_t)(2 * D) + 16 * pc, in);
        }
    };
    auto load_q = [&](int t0) { load_rows(qg, false, SH::QK, 16384u, t0); };
    auto load_kv = [&](int t0) {
        load_rows(kg, false, SH::QK + 8192u, 16384u, t0);
        load_rows(vg, true, SH::V, 8192u, t0);
        if (tid < C) {
            const bool in = t0 + tid < t_stop;
            cp_async4(s_a + tid, A.decay + lin_v_row(A, row, hh, in ? t0 + tid : t_begin), in);
        }
    };
    if (t_begin < t_stop) {
        if (!PARTIAL) load_q(t_begin);
        load_kv(t_begin);
    }
    cp_async_commit();

    // ---- the state this segment starts from: S[i][j], i = HD half + x
    float S[HD];
    {
        const float *src = nullptr;
        if (!PARTIAL && run && seg <= last) {
            if (A.nseg > 1) src = A.ws_S + ((size_t)w * A.nseg + seg) * (D * D);
            else if (A.cont) src = reinterpret_cast<const float *>(blob + kHdrBytes);
            else if (A.S0) src = A.S0 + (size_t)w * (D * D);
        }
#pragma unroll
        for (int x = 0; x < HD; ++x) S[x] = src && holds ? src[(size_t)(HD * half + x) * D + j] : 0.f;
    }

    uint32_t ph0 = 0, ph1 = 0;
    bool failed = false;
    auto wait_mma = [&](uint64_t *b, uint32_t &ph) {
        if (!mbar_wait_bounded(b, ph & 1u)) failed = true;
        ++ph;
        tc_fence_after();
    };
    float gprod = 1.f;
    int bad = kNoBad, t_done = t_stop;

#pragma unroll 1
    for (int t0 = t_begin; t0 < t_stop && bad == kNoBad; t0 += C) {
        int n = min(C, t_stop - t0);
        cp_async_wait<0>();
        fence_async_smem();
        tc_fence_before();
        if (__syncthreads_or(failed)) {
            failed = true;
            break;
        }
        // ---- gates: a prompt ends before its first bad one (uniform over the CTA)
        float a0 = 2 * lane < n ? s_a[2 * lane] : 1.f, a1 = 2 * lane + 1 < n ? s_a[2 * lane + 1] : 1.f;
        {
            const unsigned w0 = __ballot_sync(0xFFFFFFFFu, !lin_gate_ok(a0));
            const unsigned w1 = __ballot_sync(0xFFFFFFFFu, !lin_gate_ok(a1));
            if (w0 | w1) {
                n = min(w0 ? 2 * (__ffs(w0) - 1) : C, w1 ? 2 * (__ffs(w1) - 1) + 1 : C);
                bad = t_done = t0 + n;
                if (2 * lane >= n) a0 = 1.f;
                if (2 * lane + 1 >= n) a1 = 1.f;
                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                for (int x = tid; x < (C - n) * NP; x += kLcThreads) {
                    const int r = n + x / NP, c = x % NP;
                    *reinterpret_cast<uint4 *>(smem + SH::QK + 8192u + tile_off(r, c, 16384u)) = zero;
                    *reinterpret_cast<uint4 *>(smem + SH::V + tile_off(r, c, 8192u)) = zero;
                }
                fence_async_smem();
                __syncthreads();
            }
        }
        if (!PARTIAL && tid == 0) {  // Q K^T; rows 64 .. 127 (K K^T) are not used
            tc_fence_after();
            constexpr uint32_t id = lc_idesc(128, 64, 0, 0);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t o = base + SH::QK + (uint32_t)(ks >> 2) * 16384u + (uint32_t)(ks & 3) * 32u;
                lc_mma_ss(tmem + kLcO, lc_desc(o, 16u), lc_desc(o + 8192u, 16u), id, ks > 0);
            }
            umma_commit(&bar[0]);
        }
        // ---- products of gates; a lane holds tokens 2 lane and 2 lane + 1,
        // scans run over 16 lanes (32 tokens) and then over the two halves
        if (warp == 1) {
            float pre = a0 * a1, suf = pre;
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) {
                const float x = __shfl_up_sync(0xFFFFFFFFu, pre, d, 16), y = __shfl_down_sync(0xFFFFFFFFu, suf, d, 16);
                if ((lane & 15) >= d) pre *= x;
                if ((lane & 15) + d < 16) suf *= y;
            }
            // pre: tokens of the half up to 2 lane + 1; suf: from 2 lane on
            const float before = __shfl_up_sync(0xFFFFFFFFu, pre, 1, 16), after = __shfl_down_sync(0xFFFFFFFFu, suf, 1, 16);
            const float first = __shfl_sync(0xFFFFFFFFu, pre, 15), second = __shfl_sync(0xFFFFFFFFu, pre, 31);
            const float p0 = (lane & 15) ? before * a0 : a0;           // up to 2 lane
            const float s1 = (lane & 15) < 15 ? after : 1.f;           // behind 2 lane + 1
            const float f = lane < 16 ? 1.f : first, g = lane < 16 ? second : 1.f;
            *reinterpret_cast<float2 *>(s_a + 2 * lane) = make_float2(a0, a1);
            *reinterpret_cast<float2 *>(s_G2 + 2 * lane) = make_float2(p0, pre);
            *reinterpret_cast<float2 *>(s_G + 2 * lane) = make_float2(f * p0, f * pre);
            *reinterpret_cast<float2 *>(s_W + 2 * lane) = make_float2(s1 * a1 * g, s1 * g);
        }
        if (!PARTIAL) {
            // ---- S^T in three pieces to tensor memory (pairs of key channels)
            if (holds) {
#pragma unroll
                for (int x = 0; x < HD; x += 32) {
                    uint32_t hi[16], mid[16], lo[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y) lc_split2(S[x + 2 * y], S[x + 2 * y + 1], hi[y], mid[y], lo[y]);
                    const uint32_t at = tlane + kLcR + (uint32_t)(half * (HD / 2) + x / 2);
                    tmem_st16u(at, hi);
                    tmem_st16u(at + HD, mid);
                    tmem_st16u(at + 2 * HD, lo);
                }
                tmem_st_wait();
            }
        }
        __syncthreads();  // the products of gates
        if (!PARTIAL) {
            wait_mma(&bar[0], ph0);
            // ---- P_ts = R_ts (q_t . k_s), s <= t, in three pieces; a thread
            // takes 32 columns of one row, from the diagonal down
            if ((warp & 3) < 2) {
                const int t = j, c0 = 32 * half;
                float r = (t >= 32 && half == 0) ? s_G2[t] : 1.f;
                const uint32_t prow = SH::P + (uint32_t)t * 128u;
#pragma unroll
                for (int x = 16; x >= 0; x -= 16) {
                    float v[16];
                    tmem_ld16(tlane + kLcO + (uint32_t)(c0 + x), v);
#pragma unroll
                    for (int y = 15; y >= 0; --y) {
                        const int s = c0 + x + y;
                        const bool in = s <= t;
                        v[y] = in ? v[y] * r : 0.f;
                        if (in) r *= s_a[s];
                    }
#pragma unroll
                    for (int y = 0; y < 16; y += 8) {
                        uint32_t hi[4], mid[4], lo[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) lc_split2(v[y + 2 * z], v[y + 2 * z + 1], hi[z], mid[z], lo[z]);
                        const uint32_t o = prow + (uint32_t)((((c0 + x + y) >> 3) ^ (t & 7)) << 4);
                        *reinterpret_cast<uint4 *>(smem + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4 *>(smem + o + 8192u) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
                        *reinterpret_cast<uint4 *>(smem + o + 16384u) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
            }
            fence_async_smem();
            tc_fence_before();
            __syncthreads();
            if (tid == 0) {  // Y^T = S^T Q^T, low pieces first
                tc_fence_after();
                constexpr uint32_t id = lc_idesc(128, 64, 0, 0);
#pragma unroll
                for (int x = 2; x >= 0; --x)
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        lc_mma_ts(tmem + kLcO, tmem + kLcR + (uint32_t)(x * HD + 8 * ks),
                                  lc_desc(base + SH::QK + (uint32_t)(ks >> 2) * 16384u + (uint32_t)(ks & 3) * 32u, 16u),
                                  id | (x == 1 ? kLcNegA : 0u), x < 2 || ks > 0);
                umma_commit(&bar[0]);
            }
        }
        // ---- K'_s = W_s k_s in three pieces, the high one in place of k
#pragma unroll
        for (int x = 0; x < C * NP / kLcThreads; ++x) {
            const int r = pr + x * (kLcThreads / NP);
            uint8_t *kp = smem + SH::QK + 8192u + tile_off(r, pc, 16384u);
            uint8_t *mp = smem + SH::KM + tile_off(r, pc, 8192u);
            const uint4 kk = *reinterpret_cast<const uint4 *>(kp);
            const uint32_t u[4] = {kk.x, kk.y, kk.z, kk.w};
            const float f = s_W[r];
            uint32_t hi[4], mid[4], lo[4];
#pragma unroll
            for (int z = 0; z < 4; ++z)
                lc_split2(f * __uint_as_float(u[z] << 16), f * __uint_as_float(u[z] & 0xFFFF0000u), hi[z], mid[z], lo[z]);
            *reinterpret_cast<uint4 *>(kp) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(mp) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
            *reinterpret_cast<uint4 *>(mp + KB * 8192) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        const float g_last = s_G[C - 1];  // tokens behind the prompt have gate 1
        if (PARTIAL) gprod *= g_last;
        if (!PARTIAL) {
            wait_mma(&bar[0], ph0);
            // ---- Y_t scaled by G_t in place
            if (holds) {
#pragma unroll
                for (int x = 0; x < 32; x += 16) {
                    float v[16];
                    const int c0 = 32 * half + x;
                    tmem_ld16(tlane + kLcO + (uint32_t)c0, v);
#pragma unroll
                    for (int y = 0; y < 16; ++y) v[y] *= s_G[c0 + y];
                    tmem_st16(tlane + kLcO + (uint32_t)c0, v);
                }
            }
        }
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
            constexpr uint32_t vlbo = KB > 1 ? 8192u : 0u;  // D = 64: lanes 64 .. repeat the others
            if (!PARTIAL) {  // O^T = Y^T + V^T P^T
                constexpr uint32_t id = lc_idesc(128, 64, 1, 0);
#pragma unroll
                for (int x = 2; x >= 0; --x)
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks)
                        lc_mma_ss(tmem + kLcO, lc_desc(base + SH::V + (uint32_t)ks * 2048u, vlbo),
                                  lc_desc(base + SH::P + (uint32_t)x * 8192u + (uint32_t)ks * 32u, 16u),
                                  id | (x == 1 ? kLcNegB : 0u), 1u);
                umma_commit(&bar[0]);
            }
            constexpr uint32_t id = lc_idesc(128, D, 1, 1);  // V^T K'
#pragma unroll
            for (int x = 2; x >= 0; --x)
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks) {
                    const uint32_t kb = x == 0 ? SH::QK + 8192u : SH::KM + (uint32_t)(x - 1) * (KB * 8192u);
                    lc_mma_ss(tmem + kLcR, lc_desc(base + SH::V + (uint32_t)ks * 2048u, vlbo),
                              lc_desc(base + kb + (uint32_t)ks * 2048u, x == 0 ? 16384u : 8192u),
                              id | (x == 1 ? kLcNegB : 0u), x < 2 || ks > 0);
                }
            umma_commit(&bar[1]);
        }
        if (!PARTIAL) {
            if (t0 + C < t_stop && bad == kNoBad) load_q(t0 + C);  // Q has been used
            wait_mma(&bar[0], ph0);
            if (A.out && holds) {
#pragma unroll
                for (int x = 0; x < 32; x += 16) {
                    float v[16];
                    const int c0 = 32 * half + x;
                    tmem_ld16(tlane + kLcO + (uint32_t)c0, v);
                    float *o = A.out + lin_v_row(A, row, hh, t0 + c0) * D + j;
                    const size_t step = (size_t)A.map.heads * D;
#pragma unroll
                    for (int y = 0; y < 16; ++y)
                        if (c0 + y < n) o[y * step] = v[y];
                }
            }
        }
        wait_mma(&bar[1], ph1);
        if (t0 + C < t_stop && bad == kNoBad) load_kv(t0 + C);  // K' and V have been used
        cp_async_commit();
        if (holds) {
#pragma unroll
            for (int x = 0; x < HD; x += 16) {
                float v[16];
                tmem_ld16(tlane + kLcR + (uint32_t)(HD * half + x), v);
#pragma unroll
                for (int y = 0; y < 16; ++y) S[x + y] = fmaf(g_last, S[x + y], v[y]);
            }
        }
    }
    cp_async_wait<0>();
    tc_fence_before();
    failed = __syncthreads_or(failed);
    if (failed && tid == 0) {  // let what is still in flight end
        mbar_wait_bounded(&bar[0], ph0 & 1u);
        mbar_wait_bounded(&bar[1], ph1 & 1u);
    }
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, kLcCols);
    if (failed) {
        if (tid == 0 && bi >= 0) set_status(blob, LQ_DEV_TIMEOUT);
        return;
    }
    if (PARTIAL) {
        if (!run) return;
        float *dst = A.ws_S + ((size_t)w * A.nseg + seg) * (D * D);
        if (holds)
#pragma unroll
            for (int x = 0; x < HD; ++x) dst[(size_t)(HD * half + x) * D + j] = S[x];
        if (tid == 0) {
            A.ws_g[(size_t)w * A.nseg + seg] = gprod;
            A.ws_bad[(size_t)w * A.nseg + seg] = bad;
        }
        return;
    }
    if (A.out)  // no outputs past the prompt's end
        for (int x = tid; x < (t_end - t_done) * (D / 4); x += kLcThreads)
            *reinterpret_cast<float4 *>(A.out + lin_v_row(A, row, hh, t_done + x / (D / 4)) * D + 4 * (x % (D / 4))) =
                make_float4(0.f, 0.f, 0.f, 0.f);
    if (run && (bad != kNoBad || seg == last)) {  // this segment holds the prompt's end
        float *dst = reinterpret_cast<float *>(blob + kHdrBytes);
        if (holds)
#pragma unroll
            for (int x = 0; x < HD; ++x) dst[(size_t)(HD * half + x) * D + j] = S[x];
        if (tid == 0) lin_write_header(blob, A.cont, bad != kNoBad);
    }
}

}  // namespace lq
