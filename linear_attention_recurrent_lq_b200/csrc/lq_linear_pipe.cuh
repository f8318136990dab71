// lq_linear_pipe.cuh -- a prompt of linear attention in the chunkwise form on
// the tensor cores, the chunks of all heads in one pipeline per SM (bf16 q,
// k, v; sm_100a: TMA, tcgen05, tensor memory).
//
// A chunk is up to 64 tokens.  The first token's gate is applied to the
// incoming state (S = a_0 S_before); with G_t the product of the gates behind
// it up to t (G_0 = 1),
//     o_t = G_t ( S^T q_t + sum_{s <= t} (q_t . k_s / G_s) v_s ),
//     S'  = G_last ( S + sum_s (k_s / G_s) v_s^T ),
// so nothing has to be scaled between the two products of o_t.  A chunk ends
// before a token that would take G below 2^-64: 1 / G stays far inside FP32,
// and a gate of 0 starts a chunk, where it clears the state exactly.
//
// There is a CTA for each work item (a head, or a segment of a prompt cut along
// time), but one that runs takes over the items of CTAs that have not started
// (cluster launch control), so one CTA per SM sees a stream of chunks across
// items, and prompts of unequal length keep all SMs busy.  The state is an FP32
// accumulator in tensor memory (lane = value channel) onto which V^T K' is
// summed.  The CTA's warps, one of each kind on every scheduler:
//   0 .. 7   the state: scaled, and cut into the pieces of an A operand in
//            tensor memory; read from and written to global memory
//   8 .. 15  four for the outputs, from tensor memory to global memory, and
//            four, with 20, 22, 23 and 25 .. 27, for K' = k / G, in three pieces to
//            shared memory
//   16, 17, 21  the scores Q K^T, a block of 32 x 32 each: from tensor memory,
//            times 1 / G, masked, in three pieces to shared memory
//   18       one thread issues V^T K', S^T Q^T and V^T P^T
//   24       one thread issues Q K^T, ahead of them
//   19       the feeder: gates and their products, the chunk's bounds, and the
//            TMA loads
// What bounds it (d = 128): a chunk takes an SM about 4600 clocks (2048 heads
// of 256 tokens: 160 us; its traffic alone 123 us at the copy's rate).  Its q, k, v and outputs are 3440 clocks of HBM, its products 2300 of the
// tensor core, its splits and copies 2400 shared-memory wavefronts beside 2000
// of operand reads; what is not hidden is the chain from one chunk's state to
// the next and the issuing warp, whose every satisfied wait is 200 .. 300
// clocks, as its scheduler has six other warps.
//
// They meet in mbarriers only.  A barrier's waiters look at the parity of a
// phase, so none may end twice before all have seen it once: where one side can
// be a chunk ahead, there is a barrier for even and one for odd chunks.
//
// A role whose wait gives up leaves without an arrival, so its chunk's
// description stays in the ring and the roles behind it give up, too.  What the
// ring and the feeder then hold is what may be unfinished; those blobs get
// LQ_DEV_TIMEOUT after the last role has left, when no header store can follow.
#pragma once

#include "lq_linear_mma.cuh"

namespace lq {

constexpr int kLpThreads = 28 * 32;
constexpr int kLpRing = 4;     // chunk descriptions
constexpr float kLpMinGate = 0x1p-64f;
// tensor memory: Q K^T | O^T, two | S pieces | S
constexpr uint32_t kLpQK = 0, kLpO = 64, kLpSp = 192, kLpS = 384;

enum : int { kLpFirst = 1, kLpLast = 2, kLpFinal = 4, kLpBad = 8, kLpNone = 16, kLpEnd = 32 };

struct __align__(16) LpSlot {
    float G[64], inv[64];  // products of gates, and one over them (0 behind the chunk)
    int w, t0, n, flags;
    int zero_end, seg;     // outputs from t0 + n up to here are zeros (last chunk of an item)
    float a_first, g_next; // gate of the item's first token; G_last times the next chunk's first gate
};

template <int D>
struct LpShape {
    static constexpr int KB = D / 64;
    static constexpr int ST = D == 128 ? 3 : 4;  // chunks of q, k, v in shared memory
    static constexpr int NK = D == 128 ? 1 : 2;  // chunks of K'
    // a stage: KB blocks of 128 rows (64 of Q, 64 of K) x 128 bytes, KB blocks of 64 rows of V
    static constexpr uint32_t V = KB * 16384u, STAGE = KB * 24576u;
    static constexpr uint32_t P = ST * STAGE, K = P + 3u * 8192u, KBUF = 3u * KB * 8192u, RING = K + NK * KBUF;
    static constexpr uint32_t BAR = RING + kLpRing * (uint32_t)sizeof(LpSlot);
    static constexpr uint32_t CLAIM = BAR + 320u, SMEM = CLAIM + 16u + 1024u;
    // state warps at work: all, or those whose lanes are < 64
    static constexpr int SW = D / 16;
};

struct LpBars {
    uint64_t full[4], empty[4], ring_full[kLpRing], ring_free[kLpRing];
    uint64_t qk_done, qk_free, p_ready, s_ready, y_done, k_ready[2], d_done[2], o_done[2], o_free[2];
    uint32_t tmem, chunks;  // chunks: how many there are, once the feeder knows
    uint64_t claim_done;
    uint32_t from_zero[4];  // per stage: the chunk starts from a zero state
    int left[2];  // a feeder that gave up: the item it was at, and the one it had claimed
};
static_assert(sizeof(LpBars) <= 320, "barrier space");

// Ask for a CTA of this grid that has not started; the answer (16 bytes)
// arrives on `bar`.  Not to be asked again after a refusal.
__device__ __forceinline__ void claim_cta(uint32_t answer, uint64_t *bar) {
    mbar_arrive_expect_tx(bar, 16u);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 ::"r"(answer), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ int claimed_cta(uint32_t answer) {  // -1: none is left
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\tld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(got), "=r"(x) : "r"(answer) : "memory");
    return got ? (int)x : -1;
}

// Work item w may be unfinished; its header may not have been written yet.
__device__ __forceinline__ void lin_give_up(const LinArgs &A, int w) {
    const int bi = w >= 0 && w < A.work ? A.map.blob(w) : -1;
    if (bi < 0) return;
    uint8_t *blob = A.state + (size_t)bi * A.L.blob;
    if (A.cont || A.nseg > 1) set_status(blob, LQ_DEV_TIMEOUT);
    else lin_new_header(blob, LQ_DEV_TIMEOUT);
}

template <int D>
__global__ void __launch_bounds__(kLpThreads, 1)
    lin_pipe_kernel(const LinArgs A, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv) {
    using SH = LpShape<D>;
    constexpr int KB = SH::KB, HD = D / 2, C = 64, ST = SH::ST, NK = SH::NK;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    LpSlot *ring = reinterpret_cast<LpSlot *>(smem + SH::RING);
    LpBars *bars = reinterpret_cast<LpBars *>(smem + SH::BAR);
    const uint32_t base = smem_u32(smem);

    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&bars->full[i], 1);
            mbar_init(&bars->empty[i], 1);
        }
        for (int i = 0; i < kLpRing; ++i) {
            ring[i].w = -1;
            mbar_init(&bars->ring_full[i], 1);
            mbar_init(&bars->ring_free[i], SH::SW + 17);  // output, key and score warps too
        }
        mbar_init(&bars->qk_done, 1);
        mbar_init(&bars->qk_free, 3);
        mbar_init(&bars->p_ready, 3);
        mbar_init(&bars->s_ready, SH::SW);
        mbar_init(&bars->y_done, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->k_ready[i], 10);
            mbar_init(&bars->d_done[i], 1);
            mbar_init(&bars->o_done[i], 1);
            mbar_init(&bars->o_free[i], 4);
        }
        bars->chunks = 0xFFFFFFFFu;
        bars->left[0] = bars->left[1] = -1;
        mbar_init(&bars->claim_done, 1);
        fence_mbar_init();
    }
    pdl_wait();
    if (warp == 18) tmem_alloc(&bars->tmem, 512u);  // after the wait: a kernel still running may need it
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    const uint32_t tlane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);

    bool ok = true;  // false: a wait gave up; the role then leaves
    auto wait = [&](uint64_t *b, uint32_t phase) {
        // the first try in line: most waits end there.  The outcome is the warp's: a
        // phase may end between two lanes' last looks at it, and tensor memory is read
        // and written by whole warps only
        const bool got = mbar_try_wait(b, phase & 1u) || mbar_wait_bounded(b, phase & 1u);
        ok = __all_sync(0xFFFFFFFFu, got) && ok;
    };
    auto arrive = [&](uint64_t *b) {  // one arrival per warp, after all its lanes
        __syncwarp();
        if (lane == 0) mbar_arrive(b);
    };

    if (warp == 19) {
        // ------------------------------------------------------- the feeder
        uint32_t r = 0, c = 0, claims = 0;
        auto slot_wait = [&]() -> LpSlot * {
            if (r >= kLpRing) wait(&bars->ring_free[r % kLpRing], r / kLpRing - 1u);
            return ring + r % kLpRing;
        };
        // Up to 32 rows of given lengths are taken longest first, so that the last
        // items to start are short: lane r finds the row of rank r.
        const int rows = A.work / A.map.heads;
        const bool ranked = A.lengths != nullptr && rows <= 32;
        int row_of_rank = lane;
        if (ranked) {
            const int mine = lane < rows ? lin_length(A, lane) : -1;
            int rank = 0;
            for (int i = 0; i < 32; ++i) {
                const int other = __shfl_sync(0xFFFFFFFFu, mine, i);
                rank += other > mine || (other == mine && i < lane);
            }
            for (int i = 0; i < 32; ++i)
                if (__shfl_sync(0xFFFFFFFFu, rank, i) == lane) row_of_rank = i;
        }
#pragma unroll 1
        for (int it = blockIdx.x, next = it; it >= 0 && ok; it = next) {
            // the next item, while this one is fed
            if (lane == 0) claim_cta(base + SH::CLAIM, &bars->claim_done);
            auto claimed = [&]() {
                wait(&bars->claim_done, claims++);
                next = claimed_cta(base + SH::CLAIM);
                fence_async_smem();  // the answer has been read before the next one is written
                __syncwarp();
            };
            int w = it / A.nseg;
            const int seg = it - w * A.nseg, hh = w % A.map.heads;
            int row = w / A.map.heads;
            if (ranked) row = __shfl_sync(0xFFFFFFFFu, row_of_rank, row);
            w = row * A.map.heads + hh;
            const int len = lin_length(A, row), last = lin_last_segment(A, len);
            const int bi = A.map.blob(w);
            uint8_t *blob = A.state + (size_t)(bi < 0 ? 0 : bi) * A.L.blob;
            bool run = bi >= 0;
            if (A.nseg == 1) {
                if (A.cont && run) run = lin_may_run(blob, lane == 0);
            } else if (run && seg <= last) {
                bool stop = A.ws_run[w] == 0;
                for (int s = lane; s < seg; s += 32) stop |= A.ws_bad[(size_t)w * A.nseg + s] != kNoBad;
                run = !__any_sync(0xFFFFFFFFu, stop);
            }
            const int t_begin = seg * A.seg_len, t_end = min(A.tokens, t_begin + A.seg_len);
            const int t_stop = lin_stop(run, len, t_begin, t_end);
            const bool holds_end = run && seg == last;
            const float *gates = A.decay + lin_v_row(A, row, hh, 0);
            const size_t gs = (size_t)A.map.heads;
            auto gate = [&](int t) -> float { return t < t_stop ? __ldcg(gates + (size_t)t * gs) : 1.f; };
            float a0 = gate(t_begin + 2 * lane), a1 = gate(t_begin + 2 * lane + 1), a64 = gate(t_begin + C);
            const float first = __shfl_sync(0xFFFFFFFFu, a0, 0);
            const bool first_bad = t_begin < t_stop && !lin_gate_ok(first);
            if (t_begin >= t_stop || first_bad) {  // no chunk
                LpSlot *sl = slot_wait();
                if (ok && lane == 0) {
                    sl->w = w; sl->seg = seg; sl->t0 = t_begin; sl->n = 0; sl->zero_end = t_end;
                    sl->flags = kLpNone | kLpFirst | kLpLast | (holds_end || first_bad ? kLpFinal : 0) |
                                (first_bad ? kLpBad : 0);
                }
                if (ok) arrive(&bars->ring_full[r % kLpRing]);
                ++r;
            }
            const float *src = lin_state_source(A, w, seg, blob);
            const bool from_zero = src == nullptr, some = t_begin < t_stop && !first_bad;
            // the state warps read it some chunks from now
            if (some && src && lane == 0) bulk_prefetch_l2(src, D * D * 4);
            const int xq = (hh / A.group) * D, xv = hh * D, y0 = row * A.tokens;
#pragma unroll 1
            for (int t0 = t_begin; some;) {
                // the gates of the next chunk, if this one has all 64 tokens
                const float n0 = gate(t0 + C + 2 * lane), n1 = gate(t0 + C + 2 * lane + 1), n64 = gate(t0 + 2 * C);
                const unsigned w0 = __ballot_sync(0xFFFFFFFFu, !lin_gate_ok(a0));
                const unsigned w1 = __ballot_sync(0xFFFFFFFFu, !lin_gate_ok(a1));
                const int nb = min(w0 ? 2 * (__ffs(w0) - 1) : C, w1 ? 2 * (__ffs(w1) - 1) + 1 : C);
                float p = (lane ? a0 : 1.f) * a1, pre = p;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const float x = __shfl_up_sync(0xFFFFFFFFu, pre, d);
                    if (lane >= d) pre *= x;
                }
                const float before = __shfl_up_sync(0xFFFFFFFFu, pre, 1);
                const float g0 = lane ? before * a0 : 1.f, g1 = pre;  // up to tokens 2 lane, 2 lane + 1
                const unsigned l0 = __ballot_sync(0xFFFFFFFFu, !(g0 >= kLpMinGate));
                const unsigned l1 = __ballot_sync(0xFFFFFFFFu, !(g1 >= kLpMinGate));
                const int nl = min(l0 ? 2 * (__ffs(l0) - 1) : C, l1 ? 2 * (__ffs(l1) - 1) + 1 : C);
                const int rem = t_stop - t0, n = min(min(C, rem), min(nb, nl));
                const float ev = __shfl_sync(0xFFFFFFFFu, a0, (n >> 1) & 31), od = __shfl_sync(0xFFFFFFFFu, a1, (n >> 1) & 31);
                const float next = n == C ? a64 : (n & 1) ? od : ev;
                const bool bad = n < rem && !lin_gate_ok(next), end = n == rem || bad;
                const float ge = __shfl_sync(0xFFFFFFFFu, g0, ((n - 1) >> 1) & 31), go = __shfl_sync(0xFFFFFFFFu, g1, ((n - 1) >> 1) & 31);
                const float g_last = ((n - 1) & 1) ? go : ge;

                const uint32_t st = c % ST;
                if (c >= ST) wait(&bars->empty[st], c / ST - 1u);
                if (!ok) break;  // c counts what has been asked for
                if (lc_elect()) {
                    uint8_t *sp = smem + st * SH::STAGE;
                    bars->from_zero[st] = from_zero && t0 == t_begin;
                    mbar_arrive_expect_tx(&bars->full[st], SH::STAGE);
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        tma_load_2d(sp + kb * 16384, &mq, xq + 64 * kb, y0 + t0, &bars->full[st]);
                        tma_load_2d(sp + kb * 16384 + 8192, &mk, xq + 64 * kb, y0 + t0, &bars->full[st]);
                        tma_load_2d(sp + SH::V + kb * 8192, &mv, xv + 64 * kb, y0 + t0, &bars->full[st]);
                    }
                }
                ++c;
                LpSlot *sl = slot_wait();
                if (!ok) break;  // the slot is still in use
                *reinterpret_cast<float2 *>(sl->G + 2 * lane) = make_float2(g0, g1);
                *reinterpret_cast<float2 *>(sl->inv + 2 * lane) =
                    make_float2(2 * lane < n ? __fdiv_rn(1.f, g0) : 0.f, 2 * lane + 1 < n ? __fdiv_rn(1.f, g1) : 0.f);
                if (lane == 0) {
                    sl->w = w; sl->seg = seg; sl->t0 = t0; sl->n = n; sl->zero_end = t_end;
                    sl->a_first = first;
                    sl->g_next = end ? g_last : g_last * next;
                    sl->flags = (t0 == t_begin ? kLpFirst : 0) | (end ? kLpLast : 0) |
                                (end && (holds_end || bad) ? kLpFinal : 0) | (bad ? kLpBad : 0);
                }
                arrive(&bars->ring_full[r % kLpRing]);
                ++r;
                t0 += n;
                if (end) break;
                if (n == C) {
                    a0 = n0; a1 = n1; a64 = n64;
                } else {
                    a0 = gate(t0 + 2 * lane); a1 = gate(t0 + 2 * lane + 1); a64 = gate(t0 + C);
                }
            }
            claimed();
            if (!ok) {
                int nw = next >= 0 && next < A.work * A.nseg ? next / A.nseg : w;
                if (ranked) nw = __shfl_sync(0xFFFFFFFFu, row_of_rank, nw / A.map.heads) * A.map.heads + nw % A.map.heads;
                if (lane == 0) {
                    bars->left[0] = w;
                    bars->left[1] = nw;
                }
            }
        }
        if (ok) {
            LpSlot *sl = slot_wait();
            if (ok && lane == 0) {
                sl->w = -1;
                sl->flags = kLpEnd;
                bars->chunks = c;
            }
            if (ok) arrive(&bars->ring_full[r % kLpRing]);
        }
        // what has been asked for lands before the CTA leaves
        for (uint32_t i = c >= ST ? c - ST : 0u; i < c; ++i) wait(&bars->full[i % ST], i / ST);
        if (ok && c >= ST) wait(&bars->empty[c % ST], c / ST - 1u);
        if (ok) arrive(&bars->full[c % ST]);  // warp 24 learns the end here
    } else if (warp == 18 || warp == 24) {
        // ------------------------------------------------------ the issuers
        constexpr uint32_t id64 = lc_idesc(128, 64, 0, 0), idpv = lc_idesc(128, 64, 1, 0),
                           idpv2 = lc_idesc(128, 32, 1, 0), idd = lc_idesc(128, D, 1, 1);
        constexpr uint32_t vlbo = KB > 1 ? 8192u : 0u;  // D = 64: lanes 64 .. repeat the others
        // A tcgen05.mma takes its operands' descriptions from uniform registers:
        // the bases pass through a shuffle, so that the compiler sees them as
        // such and adds to them there.  An issuer gets a sixth of its scheduler's
        // slots, and its products run hardly behind it: what it executes per
        // product and per wait counts (descriptions built one by one: 140 clocks
        // a product, 40 now).
        auto uni = [](uint32_t x) { return __shfl_sync(0xFFFFFFFFu, x, 0); };
        const uint32_t td = uni(tmem), q0 = uni(lc_desc(base, 16u));
        const volatile uint32_t *chunks = &bars->chunks;
        uint32_t c = 0, st = 0, full_ph = 0;
        // Whatever a commit arrives on has to be waited for before the CTA gives its
        // shared memory and tensor memory back, by the warp that made the commit: the
        // last ones have no other waiter, and after a wait that gave up none may have.
        auto landed = [](uint64_t *b, uint32_t phase) { mbar_wait_bounded(b, phase & 1u); };
        if (warp == 24) {
#pragma unroll 1
            for (; ok; ++c) {
                const uint32_t at = uni(st * (SH::STAGE / 16u));
                wait(&bars->full[st], full_ph);
                if (c > 0) wait(&bars->qk_free, c - 1u);
                if (!ok || c >= *chunks) break;
                if (lc_elect()) {  // Q K^T; rows 64 .. 127 (K K^T) are not used
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t qd = q0 + at + (uint32_t)(ks >> 2) * 1024u + (uint32_t)(ks & 3) * 2u;
                        lc_mma_ss(td + kLpQK, qd, qd + 512u, id64, ks > 0);
                    }
                    umma_commit(&bars->qk_done);
                }
                __syncwarp();
                if (++st == (uint32_t)ST) {
                    st = 0;
                    full_ph ^= 1u;
                }
            }
            if (c > 0) landed(&bars->qk_done, c - 1u);
        } else {
            const uint32_t pd = uni(lc_desc(base + SH::P, 16u)), v0 = uni(lc_desc(base + SH::V, vlbo)),
                           k0 = uni(lc_desc(base + SH::K, 8192u));
            uint32_t begun = 0;  // chunks whose first products were issued; c: whose last were
#pragma unroll 1
            for (; ok; ++c) {
                const uint32_t at = uni(st * (SH::STAGE / 16u)), o = uni(td + kLpO + 64u * (c & 1u));
                const uint32_t kd = uni(k0 + (c % NK) * (SH::KBUF / 16u));
                wait(&bars->k_ready[c % NK], c / NK);  // the chunk's loads have landed, too
                if (!ok || c >= *chunks) break;
                const uint32_t acc = uni(*reinterpret_cast<volatile uint32_t *>(&bars->from_zero[st])) ? 0u : 1u;
                wait(&bars->s_ready, c);
                if (!ok) break;
                if (lc_elect()) {
                    tc_fence_after();
#pragma unroll
                    for (int x = 2; x >= 0; --x)  // S += V^T K'
#pragma unroll
                        for (int ks = 0; ks < C / 16; ++ks)
                            lc_mma_ss(td + kLpS, v0 + at + ks * 128u, kd + x * (KB * 512) + ks * 128u, idd | (x == 1 ? kLcNegB : 0u),
                                      x < 2 || ks > 0 ? 1u : acc);
                    umma_commit(&bars->d_done[c % NK]);
                    if (acc) {  // S^T Q^T
#pragma unroll
                        for (int x = 2; x >= 0; --x)
#pragma unroll
                            for (int ks = 0; ks < D / 16; ++ks)
                                lc_mma_ts(o, td + kLpSp + (uint32_t)(x * HD + 8 * ks),
                                          q0 + at + (uint32_t)(ks >> 2) * 1024u + (uint32_t)(ks & 3) * 2u,
                                          id64 | (x == 1 ? kLcNegA : 0u), x < 2 || ks > 0);
                    }
                    umma_commit(&bars->y_done);
                }
                begun = c + 1u;
                __syncwarp();
                wait(&bars->p_ready, c);
                if (!ok) break;
                if (lc_elect()) {  // O^T += V^T P^T
                    tc_fence_after();
#pragma unroll
                    for (int x = 2; x >= 0; --x)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)  // tokens 32 .. reach rows 32 .. only
                            lc_mma_ss(ks < 2 ? o : o + 32u, v0 + at + ks * 128u, pd + x * 512u + (ks < 2 ? 0u : 256u) + ks * 2u,
                                      (ks < 2 ? idpv : idpv2) | (x == 1 ? kLcNegB : 0u), x < 2 || ks > 0 ? 1u : acc);
                    umma_commit(&bars->o_done[c & 1u]);
                    umma_commit(&bars->empty[st]);
                }
                __syncwarp();
                if (++st == (uint32_t)ST) st = 0;
            }
            // a barrier's earlier phase had ended when its last commit was made (the
            // operands of that chunk waited for it), so the parity is not ambiguous
            for (uint32_t i = begun > NK ? begun - NK : 0u; i < begun; ++i) landed(&bars->d_done[i % NK], i / NK);
            if (begun > 0) landed(&bars->y_done, begun - 1u);
            for (uint32_t i = c > 2u ? c - 2u : 0u; i < c; ++i) landed(&bars->o_done[i & 1u], i / 2u);
            for (uint32_t i = c > ST ? c - ST : 0u; i < c; ++i) landed(&bars->empty[i % ST], i / ST);
        }
    } else if (warp == 20 || warp == 22 || warp == 23 || warp >= 25 || (warp >= 8 && warp < 16 && (D == 128 ? warp >= 12 : (warp & 3) >= 2))) {
        // ------------------------------------------------- k / G, in pieces
        constexpr int NP = 8 * KB, NT = 10 * 32;
        const int kw = warp >= 25 ? warp - 18 : warp >= 22 ? warp - 17 : warp == 20 ? 4 : D == 128 ? warp - 12 : (warp & 1) + (warp >= 12 ? 2 : 0);
        const int kt = 32 * kw + lane;
        uint32_t c = 0;
#pragma unroll 1
        for (uint32_t r = 0;; ++r) {
            wait(&bars->ring_full[r % kLpRing], r / kLpRing);
            if (!ok) break;
            const LpSlot *sl = ring + r % kLpRing;
            const int flags = sl->flags;
            if (flags & (kLpEnd | kLpNone)) {
                arrive(&bars->ring_free[r % kLpRing]);
                if (flags & kLpEnd) {  // warp 18 learns it here
                    if (c >= NK) wait(&bars->d_done[c % NK], c / NK - 1u);
                    if (ok) arrive(&bars->k_ready[c % NK]);
                    break;
                }
                continue;
            }
            const int n = sl->n;
            uint8_t *sp = smem + (c % ST) * SH::STAGE;
            wait(&bars->full[c % ST], c / ST);
            if (c >= NK) wait(&bars->d_done[c % NK], c / NK - 1u);
            if (!ok) break;
            {
                // NT is a multiple of NP: a thread keeps its piece of the row
                constexpr int RS = NT / NP, R = (C + RS - 1) / RS;
                const int pc = kt % NP, t0 = kt / NP;
                const uint8_t *kp = sp + 8192 + (pc >> 3) * 16384;
                uint8_t *dp = smem + SH::K + (c % NK) * SH::KBUF + (pc >> 3) * 8192;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int t = t0 + i * RS;
                    if (i == R - 1 && t >= C) break;
                    const uint32_t o = (uint32_t)(t * 128 + (((pc & 7) ^ (t & 7)) << 4));
                    uint4 kk = make_uint4(0u, 0u, 0u, 0u);  // rows behind the chunk
                    if (t < n) kk = *reinterpret_cast<const uint4 *>(kp + o);
                    lc_weighted_piece(kk, sl->inv[t], dp + o, KB * 8192u);
                }
                // rows of V behind the chunk meet zeros of P and K', so they must be finite
                for (int x = kt; x < (C - n) * NP; x += NT)
                    *reinterpret_cast<uint4 *>(sp + SH::V + lc_tile_off(n + x / NP, x % NP, 8192u)) = make_uint4(0u, 0u, 0u, 0u);
                fence_async_smem();
            }
            arrive(&bars->k_ready[c % NK]);
            arrive(&bars->ring_free[r % kLpRing]);
            ++c;
        }
    } else if (warp == 16 || warp == 17 || warp == 21) {
        // ------------------------------------------------------- the scores
        const int t = 32 * (warp & 3) + lane, c0 = warp == 21 ? 32 : 0;  // row, first column
        const int diag = warp == 17 ? 32 : lane;  // last column of the block that the row sees
        uint32_t c = 0;
#pragma unroll 1
        for (uint32_t r = 0;; ++r) {
            wait(&bars->ring_full[r % kLpRing], r / kLpRing);
            if (!ok) break;
            const LpSlot *sl = ring + r % kLpRing;
            const int flags = sl->flags;
            if (flags & (kLpEnd | kLpNone)) {
                arrive(&bars->ring_free[r % kLpRing]);
                if (flags & kLpEnd) break;
                continue;
            }
            wait(&bars->qk_done, c);
            if (!ok) break;
            tc_fence_after();
            uint32_t v[2][16];
            tmem_ld16_async(tlane + kLpQK + (uint32_t)c0, v[0]);
            tmem_ld16_async(tlane + kLpQK + (uint32_t)c0 + 16u, v[1]);
            tmem_ld_wait(v[0]);
            tmem_ld_wait(v[1]);
            tc_fence_before();
            arrive(&bars->qk_free);
            if (c > 0) wait(&bars->o_done[(c - 1u) & 1u], (c - 1u) / 2u);  // P is free
            if (!ok) break;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int y = 0; y < 16; y += 8) {
                    const int s0 = 16 * b + y;  // inside the block
                    const float4 f0 = *reinterpret_cast<const float4 *>(sl->inv + c0 + s0);
                    const float4 f1 = *reinterpret_cast<const float4 *>(sl->inv + c0 + s0 + 4);
                    const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
                    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const float2 x2 = __fmul2_rn(make_float2(__uint_as_float(v[b][y + 2 * z]), __uint_as_float(v[b][y + 2 * z + 1])),
                                                     make_float2(f[2 * z], f[2 * z + 1]));
                        lc_split2(s0 + 2 * z <= diag ? x2.x : 0.f, s0 + 2 * z + 1 <= diag ? x2.y : 0.f, hi[z], mid[z], lo[z]);
                    }
                    uint8_t *o = smem + SH::P + lc_tile_off(t, (c0 + s0) >> 3, 0u);
                    *reinterpret_cast<uint4 *>(o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(o + 8192) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
                    *reinterpret_cast<uint4 *>(o + 16384) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            fence_async_smem();
            arrive(&bars->p_ready);
            arrive(&bars->ring_free[r % kLpRing]);
            ++c;
        }
    } else if (warp >= 8 && warp < 16) {
        // ------------------------------------------------------ the outputs
        // D = 128: 64 tokens of 32 value channels each; D = 64: 32 tokens
        const int j = 32 * (warp & 3) + lane;
        constexpr int TN = D / 2, NT = 128;
        const int x0 = D == 64 && warp >= 12 ? 32 : 0;
        const int ot = 32 * (D == 128 ? warp - 8 : (warp & 1) + (warp >= 12 ? 2 : 0)) + lane;
        const uint32_t step = (uint32_t)A.map.heads * D;  // < 2^31
        uint32_t c = 0;
#pragma unroll 1
        for (uint32_t r = 0;; ++r) {
            wait(&bars->ring_full[r % kLpRing], r / kLpRing);
            if (!ok) break;
            const LpSlot *sl = ring + r % kLpRing;
            const int flags = sl->flags;
            if (flags & kLpEnd) break;
            const int row = sl->w / A.map.heads, hh = sl->w - row * A.map.heads, n = sl->n;
            if (!(flags & kLpNone)) {
                float *o = A.out + lin_v_row(A, row, hh, sl->t0 + x0) * D + j;
                wait(&bars->o_done[c & 1u], c / 2u);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int x = x0; x < x0 + TN; x += 32) {
                    uint32_t v[2][16];
                    tmem_ld16_async(tlane + kLpO + 64u * (c & 1u) + (uint32_t)x, v[0]);
                    tmem_ld16_async(tlane + kLpO + 64u * (c & 1u) + (uint32_t)x + 16u, v[1]);
                    tmem_ld_wait(v[0]);
                    tmem_ld_wait(v[1]);
                    if (x + 32 >= x0 + TN) {
                        tc_fence_before();
                        arrive(&bars->o_free[c & 1u]);
                    }
                    auto put = [&](int left) {
#pragma unroll
                        for (int y = 0; y < 32; y += 4) {
                            const float4 g = *reinterpret_cast<const float4 *>(sl->G + x + y);
                            const float gg[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                if (y + z < left)
                                    o[(uint64_t)(uint32_t)(y + z) * step] = __uint_as_float(v[(y + z) >> 4][(y + z) & 15]) * gg[z];
                        }
                    };
                    if (A.out) {
                        if (n == C) put(32);
                        else put(n - x);
                    }
                    o += (size_t)32 * step;
                }
                ++c;
            }
            if ((flags & kLpLast) && A.out)  // no outputs past the prompt's end (tokens x columns may pass 2^31)
                for (int t = sl->t0 + n + ot / (D / 4), end = sl->zero_end; t < end; t += NT / (D / 4))
                    *reinterpret_cast<float4 *>(A.out + lin_v_row(A, row, hh, t) * D + 4 * (ot % (D / 4))) =
                        make_float4(0.f, 0.f, 0.f, 0.f);
            arrive(&bars->ring_free[r % kLpRing]);
        }
    } else if (warp < 8 && (warp & 3) < D / 32) {
        // -------------------------------------------------------- the state
        const int j = 32 * (warp & 3) + lane, half = warp >> 2;
        const uint32_t ts = tlane + kLpS + (uint32_t)(HD * half), tp = tlane + kLpSp + (uint32_t)(HD / 2 * half);
        uint32_t c = 0;
        float g = 1.f;  // scale of the accumulator
        bool from_zero = false;
#pragma unroll 1
        for (uint32_t r = 0;; ++r) {
            wait(&bars->ring_full[r % kLpRing], r / kLpRing);
            if (!ok) break;
            const LpSlot *sl = ring + r % kLpRing;
            const int flags = sl->flags, w = sl->w;
            if (flags & kLpEnd) {
                arrive(&bars->ring_free[r % kLpRing]);
                break;
            }
            // S^T Q^T of the chunk before, and with it V^T K', which was issued before it
            if (c > 0) wait(&bars->y_done, c - 1u);
            if (c > 1) wait(&bars->o_free[c & 1u], c / 2u - 1u);  // for S^T Q^T of this chunk
            if (!ok) break;
            tc_fence_after();
            if (flags & kLpFirst) {
                const int bi = A.map.blob(w);
                const float *src = nullptr;
                if (!(flags & kLpNone) || (flags & kLpFinal)) src = lin_state_source(A, w, sl->seg, A.state + (size_t)bi * A.L.blob);
                from_zero = src == nullptr && !(flags & kLpNone);
                if (src) src += (size_t)(HD * half) * D + j;
#pragma unroll 1
                for (int x = 0; x < HD && !from_zero; x += 32) {
                    uint32_t v[32];
#pragma unroll
                    for (int y = 0; y < 32; ++y) v[y] = src ? __float_as_uint(src[(size_t)(x + y) * D]) : 0u;
                    uint32_t lo[16], up[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        lo[y] = v[y];
                        up[y] = v[16 + y];
                    }
                    tmem_st16u(ts + (uint32_t)x, lo);
                    tmem_st16u(ts + (uint32_t)x + 16u, up);
                }
                tmem_st_wait();
                g = (flags & kLpNone) ? 1.f : sl->a_first;
            }
            if (!(flags & kLpNone)) {
                // ---- S scaled, and S^T in three pieces (pairs of key channels); from a
                // zero state nothing is to be done: the products overwrite
#pragma unroll 1
                for (int x = 0; x < HD && !from_zero; x += 32) {
                    uint32_t v[2][16];
                    tmem_ld16_async(ts + (uint32_t)x, v[0]);
                    tmem_ld16_async(ts + (uint32_t)x + 16u, v[1]);
                    tmem_ld_wait(v[0]);
                    tmem_ld_wait(v[1]);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        uint32_t hi[8], mid[8], lo[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const float2 s2 = __fmul2_rn(make_float2(g, g), make_float2(__uint_as_float(v[b][2 * y]), __uint_as_float(v[b][2 * y + 1])));
                            v[b][2 * y] = __float_as_uint(s2.x);
                            v[b][2 * y + 1] = __float_as_uint(s2.y);
                            lc_split2(s2.x, s2.y, hi[y], mid[y], lo[y]);
                        }
                        tmem_st16u(ts + (uint32_t)(x + 16 * b), v[b]);
                        tmem_st8u(tp + (uint32_t)(x / 2 + 8 * b), hi);
                        tmem_st8u(tp + HD + (uint32_t)(x / 2 + 8 * b), mid);
                        tmem_st8u(tp + 2 * HD + (uint32_t)(x / 2 + 8 * b), lo);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                arrive(&bars->s_ready);
                from_zero = false;
                g = sl->g_next;
                ++c;
            }
            if (flags & kLpFinal) {  // the prompt's end
                if (!(flags & kLpNone)) wait(&bars->y_done, c - 1u);
                if (!ok) break;
                tc_fence_after();
                uint8_t *blob = A.state + (size_t)A.map.blob(w) * A.L.blob;
                float *dst = reinterpret_cast<float *>(blob + kHdrBytes) + (size_t)(HD * half) * D + j;
#pragma unroll 1
                for (int x = 0; x < HD; x += 16) {
                    uint32_t v[16];
                    tmem_ld16_async(ts + (uint32_t)x, v);
                    tmem_ld_wait(v);
#pragma unroll
                    for (int y = 0; y < 16; ++y) dst[(size_t)(x + y) * D] = g * __uint_as_float(v[y]);
                }
                tc_fence_before();
                if (tid == 0) lin_write_header(A, blob, (flags & kLpBad) != 0);
            }
            arrive(&bars->ring_free[r % kLpRing]);
        }
    }
    tc_fence_before();
    if (__syncthreads_or(!ok) && tid < kLpRing + 2) lin_give_up(A, tid < kLpRing ? ring[tid].w : bars->left[tid - kLpRing]);
    if (warp == 18) tmem_dealloc(tmem, 512u);
}

}  // namespace lq
