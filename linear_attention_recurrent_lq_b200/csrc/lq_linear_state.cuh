// lq_linear_state.cuh -- what a segment of a prompt leaves behind, on the tensor
// cores: the first pass over a prompt that is cut along time (bf16 k, v;
// sm_100a: TMA, tcgen05, tensor memory).
//
// From a zero state, a segment of tokens t0 .. t1 ends with
//     S = sum_s W_s k_s v_s^T,   W_s = prod_{s < u <= t1} a_u,
// one long product: the weights refer to the segment's end, so the accumulator
// in tensor memory is never scaled.  The chunks of 64 tokens are taken from the
// last to the first, with the product of the gates behind them carried along
// (a gate of 0 is exact).  W k is cut into three bf16 pieces.
//
// One CTA takes one (head, segment): two groups of eight warps weight the keys
// of even and of odd chunks (one after the other, all sixteen: 2400 clocks per
// chunk, the latency of that work), one thread issues the products, one warp
// loads (TMA), one makes the weights from the gates.  Its floor is HBM: 516
// bytes per token and head (d = 128), 1390 clocks per chunk and SM; 768 are
// tensor time.  32 heads of 16384 tokens in 9 segments: 66 us, of which 37 are
// traffic; their 256 CTAs of 29 chunks are two rounds on 148 SMs, of 2100 clocks
// a chunk (the keys' weights: 16 warps, the latency of a shared-memory round
// trip and a split per chunk).
//
// A wait that gives up marks the segment as lost in the workspace: the blob's
// header is written later, by the pass that joins the segments.
#pragma once

#include "lq_linear_mma.cuh"

namespace lq {

constexpr int kLsKeys = 16;  // warps that weight the keys
constexpr int kLsThreads = (kLsKeys + 3) * 32;
constexpr int kLsStages = 3;
constexpr int kLsGates = 8;  // chunks of gates on their way (a gate is a memory latency of its own)

template <int D>
struct LsShape {
    static constexpr int KB = D / 64;
    // a stage: K and V, KB blocks of 64 rows x 128 bytes each
    static constexpr uint32_t V = KB * 8192u, STAGE = 2u * V, K = kLsStages * STAGE, KBUF = 3u * KB * 8192u;
    static constexpr uint32_t W = K + 2u * KBUF, G = W + kLsStages * 256u, BAR = G + kLsGates * 256u, SMEM = BAR + 128u + 1024u;
};

struct LsBars {
    uint64_t full[kLsStages], empty[kLsStages], k_ready[2], d_done[2], all_done;
    uint32_t tmem;
};
static_assert(sizeof(LsBars) <= 128, "barrier space");

template <int D>
__global__ void __launch_bounds__(kLsThreads, 1)
    lin_state_kernel(const LinArgs A, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using SH = LsShape<D>;
    constexpr int KB = SH::KB, C = 64;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int w = blockIdx.x, seg = blockIdx.y;
    const int row = w / A.map.heads, hh = w - row * A.map.heads;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    LsBars *bars = reinterpret_cast<LsBars *>(smem + SH::BAR);
    const uint32_t base = smem_u32(smem);
    if (tid == 0) {
        for (int i = 0; i < kLsStages; ++i) {
            mbar_init(&bars->full[i], 2);  // the loads, and the weights
            mbar_init(&bars->empty[i], 1);
        }
        mbar_init(&bars->all_done, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->k_ready[i], kLsKeys / 2);
            mbar_init(&bars->d_done[i], 1);
        }
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    // a segment before the one that holds the prompt's end is whole
    if (A.map.blob(w) < 0 || seg >= lin_last_segment(A, lin_length(A, row))) return;  // uniform: not needed
    if (warp == kLsKeys) tmem_alloc(&bars->tmem, 128u);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    const int t_begin = seg * A.seg_len, chunks = A.seg_len / C;
    bool ok = true;
    auto wait = [&](uint64_t *b, uint32_t phase) {  // the outcome is the warp's
        const bool got = mbar_try_wait(b, phase & 1u) || mbar_wait_bounded(b, phase & 1u);
        ok = __all_sync(0xFFFFFFFFu, got) && ok;
    };

    if (warp == kLsKeys + 2) {  // the loads
        const int x = (hh / A.group) * D, xv = hh * D, y0 = row * A.tokens + t_begin;
        int i = 0;  // loads asked for
#pragma unroll 1
        for (; i < chunks; ++i) {
            const uint32_t st = (uint32_t)i % kLsStages;
            if (i >= kLsStages) wait(&bars->empty[st], (uint32_t)i / kLsStages - 1u);
            if (!ok) break;
            if (lc_elect()) {
                uint8_t *sp = smem + st * SH::STAGE;
                const int y = y0 + (chunks - 1 - i) * C;
                mbar_arrive_expect_tx(&bars->full[st], SH::STAGE);
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    tma_load_2d(sp + kb * 8192, &mk, x + 64 * kb, y, &bars->full[st]);
                    tma_load_2d(sp + SH::V + kb * 8192, &mv, xv + 64 * kb, y, &bars->full[st]);
                }
            }
            __syncwarp();
        }
        // they land before the CTA leaves, also where nobody waits for them any more
        for (int j = i > kLsStages ? i - kLsStages : 0; j < i; ++j) wait(&bars->full[j % kLsStages], (uint32_t)(j / kLsStages));
    } else if (warp == kLsKeys + 1) {  // the weights
        const float *gates = A.decay + lin_v_row(A, row, hh, t_begin);
        const size_t gs = (size_t)A.map.heads;
        float carry = 1.f;  // product of the gates behind the chunk
        int bad = kNoBad;
        auto ask = [&](int i) {  // gates of the i-th chunk from the end
            if (i < chunks) {
                const float *g = gates + (size_t)((chunks - 1 - i) * C + 2 * lane) * gs;
                uint8_t *to = smem + SH::G + (i % kLsGates) * 256 + 8 * lane;
                cp_async4(to, g, true);
                cp_async4(to + 4, g + gs, true);
            }
            cp_async_commit();
        };
        for (int i = 0; i < kLsGates - 1; ++i) ask(i);
#pragma unroll 1
        for (int i = 0; i < chunks; ++i) {
            const int at = (chunks - 1 - i) * C;
            const uint32_t st = (uint32_t)i % kLsStages;
            if (i >= kLsStages) wait(&bars->empty[st], (uint32_t)i / kLsStages - 1u);
            if (!ok) break;
            ask(i + kLsGates - 1);
            cp_async_wait<kLsGates - 1>();  // a lane reads what it asked for
            const float2 a = *reinterpret_cast<const float2 *>(smem + SH::G + (i % kLsGates) * 256 + 8 * lane);
            const float a0 = a.x, a1 = a.y;
            const unsigned w0 = __ballot_sync(0xFFFFFFFFu, !lin_gate_ok(a0));
            const unsigned w1 = __ballot_sync(0xFFFFFFFFu, !lin_gate_ok(a1));
            if (w0 | w1) bad = t_begin + at + min(w0 ? 2 * (__ffs(w0) - 1) : C, w1 ? 2 * (__ffs(w1) - 1) + 1 : C);
            float suf = a0 * a1;  // products of the gates from token 2 lane on
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const float y = __shfl_down_sync(0xFFFFFFFFu, suf, d);
                if (lane + d < 32) suf *= y;
            }
            const float after = __shfl_down_sync(0xFFFFFFFFu, suf, 1);
            const float b1 = (lane < 31 ? after : 1.f) * carry;
            *reinterpret_cast<float2 *>(smem + SH::W + st * 256u + 8u * lane) = make_float2(a1 * b1, b1);
            carry *= __shfl_sync(0xFFFFFFFFu, suf, 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->full[st]);
        }
        cp_async_wait<0>();
        if (lane == 0) {
            A.ws_g[(size_t)w * A.nseg + seg] = carry;
            A.ws_bad[(size_t)w * A.nseg + seg] = bad;
        }
    } else if (warp == kLsKeys) {  // the issuer: S^T += V^T K'
        auto uni = [](uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
        constexpr uint32_t id = lc_idesc(128, D, 1, 1), vlbo = KB > 1 ? 8192u : 0u;
        const uint32_t v0 = uni(lc_desc(base + SH::V, vlbo)), k0 = uni(lc_desc(base + SH::K, 8192u)), td = uni(tmem);
        int i = 0;  // chunks whose products were issued
#pragma unroll 1
        for (; i < chunks; ++i) {
            wait(&bars->k_ready[i & 1], (uint32_t)i / 2u);  // the chunk's loads have landed, too
            if (!ok) break;
            const uint32_t vd = uni(v0 + (uint32_t)(i % kLsStages) * (SH::STAGE / 16u)), kd = uni(k0 + (uint32_t)(i & 1) * (SH::KBUF / 16u));
            const uint32_t acc = uni(i > 0 ? 1u : 0u);
            if (lc_elect()) {
                tc_fence_after();
#pragma unroll
                for (int x = 2; x >= 0; --x)
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks)
                        lc_mma_ss(td, vd + ks * 128u, kd + x * (KB * 512) + ks * 128u, id | (x == 1 ? kLcNegB : 0u),
                                  x < 2 || ks > 0 ? 1u : acc);
                umma_commit(&bars->d_done[i & 1]);
                umma_commit(&bars->empty[i % kLsStages]);
                if (i == chunks - 1) umma_commit(&bars->all_done);
            }
            __syncwarp();
        }
        // every commit has arrived before shared memory and tensor memory are given back
        for (int j = i > 2 ? i - 2 : 0; j < i; ++j) wait(&bars->d_done[j & 1], (uint32_t)j / 2u);
        for (int j = i > kLsStages ? i - kLsStages : 0; j < i; ++j) wait(&bars->empty[j % kLsStages], (uint32_t)(j / kLsStages));
        if (i == chunks) wait(&bars->all_done, 0u);
    } else {  // the keys, then the state to the workspace
        constexpr int NP = 8 * KB;
#pragma unroll 1
        for (int i = warp / (kLsKeys / 2); i < chunks; i += 2) {
            const uint32_t st = (uint32_t)i % kLsStages;
            // in this order: the products of chunk i - 2 stand behind those of
            // chunk i - 3, so the stage's phase before this one has ended for the
            // group that did not wait for it, too
            if (i >= 2) wait(&bars->d_done[i & 1], (uint32_t)i / 2u - 1u);
            wait(&bars->full[st], (uint32_t)i / kLsStages);
            if (!ok) break;
            const float *W = reinterpret_cast<const float *>(smem + SH::W + st * 256u);
#pragma unroll 2
            for (int x = tid % (kLsKeys * 16); x < C * NP; x += kLsKeys * 16) {
                const int t = x / NP, pc = x % NP;
                const uint32_t o = lc_tile_off(t, pc, 8192u);
                lc_weighted_piece(*reinterpret_cast<const uint4 *>(smem + st * SH::STAGE + o), W[t],
                                  smem + SH::K + (i & 1) * SH::KBUF + o, KB * 8192u);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->k_ready[i & 1]);
        }
        if (ok) wait(&bars->all_done, 0u);
        tc_fence_after();
        constexpr int Q = D / (kLsKeys / 4);  // key channels of a warp
        const int j = 32 * (warp & 3) + lane, i0 = Q * (warp >> 2);
        if (ok && (warp & 3) < D / 32) {
            float *dst = A.ws_S + ((size_t)w * A.nseg + seg) * (D * D) + (size_t)i0 * D + j;
#pragma unroll
            for (int x = 0; x < Q; x += 16) {
                uint32_t v[16];
                tmem_ld16_async(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(i0 + x), v);
                tmem_ld_wait(v);
#pragma unroll
                for (int y = 0; y < 16; ++y) dst[(size_t)(x + y) * D] = __uint_as_float(v[y]);
            }
        }
    }
    tc_fence_before();
    if (__syncthreads_or(!ok) && tid == 0) A.ws_bad[(size_t)w * A.nseg + seg] = kLost;
    if (warp == kLsKeys) tmem_dealloc(tmem, 128u);
}

}  // namespace lq
