// linear.cu -- host side of the linear-attention entry points of
// include/leapquant.h: argument checks and launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include "leapquant.h"
#include "lq_common.cuh"
#include "lq_host.cuh"
#include "lq_linear.cuh"
#include "lq_linear_pipe.cuh"
#include "lq_linear_state.cuh"
#include "lq_norms.cuh"

using namespace lq;

namespace {

// The choices below were measured on a B200 and count its SMs; on a part with
// another number they would cost time, not results.
constexpr int kSms = 148;

// Token after token, a CTA takes 16, 64 or (d = 128) 128 columns of a head.
// Of 16: the latency of a token is lowest, but a cluster of 4 or 8 CTAs reads
// each q and k anew.  f32, 200 tokens, 16 and 64 columns: d = 128, 12 heads 25.1
// and 43.8 us, 24 heads 39.4 and 43.9, 36 heads 67.9 and 44.2; d = 64, 24 heads
// 17.3 and 24.5, 36 heads 24.9 and 24.6, 74 heads 39.6 and 24.6.
bool narrow(const lq_config &c, int64_t work) { return work * (c.dk / 16) <= kSms * 4 / 3; }

// Of 128 columns, eight per lane: shared memory is read half as often.  What
// decides is how many CTAs an SM gets.  f32, 200 tokens, 64 and 128 columns: 74
// heads 44.5 and 60.6 us, 100 heads 64.6 and 60.8, 140 heads 86.4 and 61.1, 200
// heads 88.3 and 101.5, 296 heads 121 and 102, 600 heads 251 and 242.
bool wide(const lq_config &c, int64_t work) {
    return c.dv == 128 && work > kSms / 2 && (work <= kSms || work > 3 * kSms / 2);
}

// Whether a bf16 prompt takes the chunkwise form on the tensor cores.  It costs
// a chunk of 64 tokens whatever the prompt's length; token after token the time
// grows with the tokens.  Chunkwise and token after token, d = 128: 12 heads, 64
// tokens 11.0 and 7.8 us, 100 tokens 13.2 and 11.5, 128 tokens (nothing in L2)
// 14.3 and 18.4; 24 heads, 64 tokens 11.1 and 10.7, 100 tokens 13.3 and 16.4; 60
// heads, 17 tokens 8.2 and 6.8, 32 tokens 8.3 and 8.6; 140 heads, 8 tokens 9.0
// and 6.7, 17 tokens 9.1 and 10.4; 600 heads, 4 tokens 20.1 and 16.8, 8 tokens
// 19.8 and 20.8.  d = 64: 24 heads, 100 tokens 10.7 and 8.8, 200 tokens 16.3 and
// 15.0; 100 heads, 48 tokens 9.7 and 8.2, 64 tokens 9.7 and 10.0; 2048 heads, 48
// tokens 80 and 63, 64 tokens 78.7 and 80.3.
bool chunked(const lq_config &c, int64_t work, int tokens) {
    if (c.in_dtype != 1) return false;
    // all clusters of 16-column CTAs at once, an SM each (a few SMs stay outside)
    if (work * (c.dk / 16) <= 128) return tokens > (c.dk == 128 ? 96 : 128);
    if (c.dk == 64) return tokens >= 64;
    if (narrow(c, work)) return tokens > 64;
    return tokens >= 32 || (tokens >= 8 && work * tokens >= 2000);
}

// Where the heads alone leave SMs idle, a prompt is cut along time into `nseg`
// segments of `seg_len` tokens.  That costs a pass over k and v for what the
// segments leave behind, and a scan over those states.
constexpr int kMaxSegments = 64;

// Token after token: segments of 32 tokens or more.
int64_t most_segments(int tokens) { return tokens / 32 < kMaxSegments ? tokens / 32 : kMaxSegments; }

// The CTAs of a prompt cut along time, token after token, d = 128: 128 columns
// where there are enough for two per SM.  64 and 128 columns: 8 heads of 777
// tokens 46 and 52 us, 24 heads of 400 tokens 49 and 55; 8 heads of 2000 tokens
// 76 and 68, 36 heads 220 and 202.
bool wide_cut(const lq_config &c, int64_t work, int tokens) { return c.dv == 128 && work * most_segments(tokens) > 300; }

struct Cut {
    int seg_len, nseg;
};

Cut cut_of(const lq_config &c, int64_t work, int tokens) {
    Cut best{tokens > 0 ? tokens : 1, 1};
    if (work <= 0 || tokens < 256) return best;
    if (chunked(c, work, tokens)) {
        // One CTA per SM and kind of pass.  In units of 0.1 us, as measured at
        // d = 128: 27 for a chunk of 64 tokens in the main pass and 12 in the
        // first, 15 and 30 for each segment's start, 0.3 a segment in the scan,
        // 60 for the launches.  32 heads of 16384 tokens: 230 us in 9 segments
        // (this choice), 275 us in 32.
        auto cost = [&](int64_t n, int64_t chunks) {
            const int64_t t = (work * n + kSms - 1) / kSms * (chunks * 27 + 15);
            return n == 1 ? t : t + (work * (n - 1) + kSms - 1) / kSms * (chunks * 12 + 30) + work * n * 3 / 10 + 60;
        };
        const int64_t all = (tokens + 63) / 64;
        int64_t least = cost(1, all);
        for (int64_t n = 2; n <= kMaxSegments && n * 2 <= all; ++n) {
            const int64_t chunks = (all + n - 1) / n, got = (all + chunks - 1) / chunks;
            if (cost(got, chunks) < least) {
                least = cost(got, chunks);
                best = Cut{(int)(chunks * 64), (int)got};
            }
        }
        return best;
    }
    // Token after token (f32).  Both passes together take about 0.85 ns (d = 128:
    // 2.5 ns) per head and token and 15 us (28), the uncut prompt 113 ns (210) per
    // token.  Cut and uncut, d = 64: 74 heads of 256 tokens 31 and 32 us, 100 heads
    // 39 and 32, 100 heads of 2000 tokens 171 and 225, 148 heads 224 and 226;
    // d = 128: 36 heads of 256 tokens 53 and 57 us, 50 heads of 777 tokens 124 and
    // 164, 60 heads of 400 tokens 103 and 87, 74 heads of 2000 tokens 385 and 422,
    // 148 heads 638 and 569.
    const int64_t most = most_segments(tokens);
    int64_t n;
    if (c.dv == 64) {
        if (work * tokens >= 133 * (int64_t)tokens - 14000) return best;
        // CTAs per SM: 36 heads of 777 tokens 36 us, with three 47 us.  Not the best
        // everywhere: 36 heads of 400 tokens 33 us (segments of 48), 27 in segments of 32
        n = 6 * kSms / work;
    } else {
        if (work * tokens >= 84 * (int64_t)tokens - 11500) return best;
        // CTAs of 128 columns two per SM, or twice as many: 36 heads of 2000 tokens
        // 202 us in 8 segments and 213 in 16, 64 heads 379 in 4 and 353 in 12
        n = most;
        if (wide_cut(c, work, tokens)) n = (2 * kSms / work >= 6 ? 2 : 4) * kSms / work;
    }
    if (n > most) n = most;
    if (n < 2) return best;
    best.seg_len = (int)align_up((uint32_t)((tokens + n - 1) / n), 16u);
    best.nseg = (tokens + best.seg_len - 1) / best.seg_len;
    return best;
}

// [work, nseg, dk, dv] f32 states | [work, nseg] gate products | [work, nseg]
// first bad tokens | [work] run flags
size_t workspace_bytes(const lq_config &c, int64_t work, const Cut &cut) {
    if (cut.nseg < 2) return 0;
    const size_t n = (size_t)work * cut.nseg;
    return (n * ((size_t)c.dk * c.dv + 2) + (size_t)work) * 4u;
}

lq_status check_linear(const lq_config *cfg, int qk_heads) {
    const lq_status st = check_config(cfg);
    if (st != LQ_OK) return st;
    if (qk_heads <= 0 || cfg->num_heads % qk_heads != 0) return LQ_ERR_INVALID_ARG;
    if (cfg->bits != 32 || cfg->decay_kind != 0) return LQ_ERR_UNSUPPORTED;
    return LQ_OK;
}

template <int D, bool BF16>
lq_status launch_step(const LinArgs &a, cudaStream_t s) {
    // d = 128, few heads: four CTAs per head, so that every SM has loads in flight.
    // Four and one: 12 heads 1.8 and 2.6 us, 148 heads 4.9 and 4.9, 280 heads 7.4
    // and 8.1, 400 heads 9.8 and 10.0; d = 64, 32 heads 1.7 and 1.8, 200 heads 3.8
    // and 3.0
    if constexpr (D == 128)
        if (a.work < 2 * kSms) return launched(launch_pdl(lin_step_kernel<D, BF16, D / 4>, a.work * 4, 256, 0u, s, a));
    return launched(launch_pdl(lin_step_kernel<D, BF16, D>, a.work, 256, 0u, s, a));
}

lq_status step_rows(const lq_config &c, void *state, const int32_t *slots, int rows, int qk_heads, const void *q,
                    const void *k, const void *v, const float *decay, float *out, lq_stream_t stream) {
    if (rows > 0 && (!q || !k || !v || !decay || !out)) return LQ_ERR_INVALID_ARG;
    if ((int64_t)rows * c.num_heads > 0x7FFFFFFF / 8) return LQ_ERR_UNSUPPORTED;
    if (!aligned(state, 256) || !aligned(slots, 4) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(decay, 4) || !aligned(out, 16))
        return LQ_ERR_MISALIGNED;
    if (rows == 0) return LQ_OK;
    LinArgs a{};
    a.state = static_cast<uint8_t *>(state);
    a.L = make_layout(c);
    a.map = SlotMap{slots, c.num_heads, c.num_slots};
    a.q = q; a.k = k; a.v = v; a.decay = decay; a.out = out;
    a.tokens = 1;
    a.work = rows * c.num_heads;
    a.qk_heads = qk_heads;
    a.group = c.num_heads / qk_heads;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (c.dk == 128) return c.in_dtype ? launch_step<128, true>(a, s) : launch_step<128, false>(a, s);
    return c.in_dtype ? launch_step<64, true>(a, s) : launch_step<64, false>(a, s);
}

template <int D, bool BF16, int C>
lq_status launch_recurrent(const LinArgs &a, cudaStream_t s) {
    using SH = LinShape<D, BF16, C>;
    if constexpr (!BF16 && C > 1) if (a.nseg > 1) {  // others are not cut (cut_of)
        auto k = lin_recurrent_kernel<D, BF16, C, true>;
        if (allow_smem(k, SH::SMEM) != cudaSuccess) return LQ_ERR_CUDA;
        if (launch_pdl(k, dim3((unsigned)(a.work * SH::NB), (unsigned)(a.nseg - 1)), kLinThreads, 1, SH::SMEM, s,
                       a) != cudaSuccess)
            return LQ_ERR_CUDA;
        if (launch_pdl(lin_scan_kernel<D>, a.work * (D * D / 1024), 256, 0u, s, a) != cudaSuccess) return LQ_ERR_CUDA;
    }
    auto k = lin_recurrent_kernel<D, BF16, C, false>;
    if (allow_smem(k, SH::SMEM) != cudaSuccess) return LQ_ERR_CUDA;
    return launched(launch_pdl(k, dim3((unsigned)(a.work * SH::NB), (unsigned)a.nseg), kLinThreads, SH::NB,
                               SH::SMEM, s, a));
}

// A [rows, cols] bf16 tensor as boxes of 64 rows x 64 columns, 128-byte swizzle.
bool make_map(CUtensorMap *m, const void *p, uint64_t cols, uint64_t rows) {
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return false;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols * 2};
    const cuuint32_t box[2] = {64, 64}, step[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
lq_status launch_chunked(const LinArgs &a, cudaStream_t s) {
    CUtensorMap mq, mk, mv;
    const uint64_t rows = (uint64_t)(a.work / a.map.heads) * a.tokens;
    if (!make_map(&mq, a.q, (uint64_t)a.qk_heads * D, rows) || !make_map(&mk, a.k, (uint64_t)a.qk_heads * D, rows) ||
        !make_map(&mv, a.v, (uint64_t)a.map.heads * D, rows))
        return LQ_ERR_CUDA;
    if (a.nseg > 1) {
        const uint32_t smem = LsShape<D>::SMEM;
        auto k = lin_state_kernel<D>;
        if (allow_smem(k, smem) != cudaSuccess) return LQ_ERR_CUDA;
        if (launch_pdl(k, dim3((unsigned)a.work, (unsigned)(a.nseg - 1)), kLsThreads, 1, smem, s, a, mk, mv) != cudaSuccess)
            return LQ_ERR_CUDA;
        if (launch_pdl(lin_scan_kernel<D>, a.work * (D * D / 1024), 256, 0u, s, a) != cudaSuccess) return LQ_ERR_CUDA;
    }
    const uint32_t smem = LpShape<D>::SMEM;
    auto k = lin_pipe_kernel<D>;
    if (allow_smem(k, smem) != cudaSuccess) return LQ_ERR_CUDA;
    return launched(launch_pdl(k, a.work * a.nseg, kLpThreads, smem, s, a, mq, mk, mv));
}

template <int D, bool BF16>
lq_status launch_prefill(const lq_config &c, const LinArgs &a, cudaStream_t s) {
    if constexpr (BF16)
        if (chunked(c, a.work, a.tokens)) return launch_chunked<D>(a, s);
    if (a.nseg == 1 && narrow(c, a.work)) return launch_recurrent<D, BF16, 1>(a, s);
    if constexpr (D == 128)
        if (a.nseg == 1 ? wide(c, a.work) : wide_cut(c, a.work, a.tokens)) return launch_recurrent<D, BF16, 8>(a, s);
    return launch_recurrent<D, BF16, 4>(a, s);
}

lq_status prefill_rows(const lq_config &c, void *state, const int32_t *slots, int rows, int tokens,
                       const int32_t *lengths, const float *S0, int qk_heads, const void *q, const void *k,
                       const void *v, const float *decay, float *out, uint32_t flags, void *workspace,
                       size_t workspace_size, lq_stream_t stream) {
    if (tokens < 0 || (flags & ~LQ_PREFILL_CONTINUE)) return LQ_ERR_INVALID_ARG;
    if ((flags & LQ_PREFILL_CONTINUE) && S0) return LQ_ERR_INVALID_ARG;
    if ((int64_t)rows * (tokens > 0 ? tokens : 1) * c.num_heads > 0x7FFFFFFF) return LQ_ERR_UNSUPPORTED;
    if ((int64_t)rows * c.num_heads > 0x7FFFFFFF / 16 || c.num_heads > 0x7FFFFFFF / 128) return LQ_ERR_UNSUPPORTED;
    if (rows > 0 && tokens > 0 && (!q || !k || !v || !decay)) return LQ_ERR_INVALID_ARG;
    if (!aligned(state, 256) || !aligned(slots, 4) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(decay, 4) || !aligned(out, 16) || !aligned(S0, 16) || !aligned(lengths, 4) || !aligned(workspace, 16))
        return LQ_ERR_MISALIGNED;
    if (rows == 0) return LQ_OK;
    LinArgs a{};
    a.state = static_cast<uint8_t *>(state);
    a.L = make_layout(c);
    a.map = SlotMap{slots, c.num_heads, c.num_slots};
    a.S0 = S0;
    a.q = q; a.k = k; a.v = v; a.decay = decay; a.lengths = lengths;
    a.out = tokens > 0 ? out : nullptr;
    a.tokens = tokens;
    a.work = rows * c.num_heads;
    a.qk_heads = qk_heads;
    a.group = c.num_heads / qk_heads;
    a.cont = (flags & LQ_PREFILL_CONTINUE) != 0u;
    Cut cut = cut_of(c, a.work, tokens);
    if (workspace) {
        if (workspace_size < workspace_bytes(c, a.work, cut)) return LQ_ERR_INVALID_ARG;
    } else {
        cut = Cut{tokens > 0 ? tokens : 1, 1};
    }
    a.seg_len = cut.seg_len;
    a.nseg = cut.nseg;
    if (a.nseg > 1) {
        const size_t n = (size_t)a.work * a.nseg;
        a.ws_S = static_cast<float *>(workspace);
        a.ws_g = a.ws_S + n * (size_t)(c.dk * c.dv);
        a.ws_bad = reinterpret_cast<int *>(a.ws_g + n);
        a.ws_run = a.ws_bad + n;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (c.dk == 128) return c.in_dtype ? launch_prefill<128, true>(c, a, s) : launch_prefill<128, false>(c, a, s);
    return c.in_dtype ? launch_prefill<64, true>(c, a, s) : launch_prefill<64, false>(c, a, s);
}

lq_status check_linear_slots(const lq_config *cfg, const void *state, const int32_t *slots, int n_active,
                             int qk_heads) {
    const lq_status st = check_linear(cfg, qk_heads);
    if (st != LQ_OK) return st;
    if (!state || n_active < 0 || (n_active > 0 && !slots)) return LQ_ERR_INVALID_ARG;
    return LQ_OK;
}

template <int D, bool BF16>
cudaError_t launch_qk_norm(QkNormArgs a, cudaStream_t s) {
    constexpr int G = 256 / (D / (BF16 ? 8 : 4));  // rows a block takes at once
    const long long nb = (2 * a.qk_rows + G * kNormUnroll - 1) / (G * kNormUnroll);
    const long long per = a.kda ? G * kGateUnroll<BF16> : 256, ng = (a.heads_n + per - 1) / per;
    if (nb + ng > 0x7FFFFFFF) return cudaErrorInvalidValue;
    a.norm_blocks = (unsigned)nb;
    a.gate_blocks = (unsigned)ng;
    return launch_pdl(qk_norm_kernel<D, BF16>, (int)(nb + ng), 256, 0u, s, a);
}

template <int D, bool BF16>
cudaError_t launch_out_norm(const OutNormArgs &a, int gate, cudaStream_t s) {
    constexpr int per = 256 / (D / 8) * kOutNormUnroll;
    const int grid = (int)((a.n + per - 1) / per);
    switch (gate) {
        case kGateNone: return launch_pdl(out_norm_kernel<D, BF16, kGateNone>, grid, 256, 0u, s, a);
        case kGateSilu: return launch_pdl(out_norm_kernel<D, BF16, kGateSilu>, grid, 256, 0u, s, a);
        default: return launch_pdl(out_norm_kernel<D, BF16, kGateSigmoid>, grid, 256, 0u, s, a);
    }
}

}  // namespace

extern "C" {

lq_status lq_linear_step(const lq_config *cfg, void *state, int qk_heads, const void *q, const void *k, const void *v,
                         const float *decay, float *out, lq_stream_t stream) {
    const lq_status st = check_linear(cfg, qk_heads);
    if (st != LQ_OK) return st;
    if (!state) return LQ_ERR_INVALID_ARG;
    return step_rows(*cfg, state, nullptr, cfg->num_slots, qk_heads, q, k, v, decay, out, stream);
}

lq_status lq_linear_step_slots(const lq_config *cfg, void *state, const int32_t *slots, int n_active, int qk_heads,
                               const void *q, const void *k, const void *v, const float *decay, float *out,
                               lq_stream_t stream) {
    const lq_status st = check_linear_slots(cfg, state, slots, n_active, qk_heads);
    if (st != LQ_OK) return st;
    return step_rows(*cfg, state, slots, n_active, qk_heads, q, k, v, decay, out, stream);
}

size_t lq_linear_prefill_workspace(const lq_config *cfg, int rows, int tokens) {
    if (check_linear(cfg, 1) != LQ_OK || rows <= 0 || tokens <= 0) return 0;
    const int64_t work = (int64_t)rows * cfg->num_heads;
    return workspace_bytes(*cfg, work, cut_of(*cfg, work, tokens));
}

lq_status lq_linear_prefill(const lq_config *cfg, void *state, int tokens, const int32_t *lengths, const float *S0,
                            int qk_heads, const void *q, const void *k, const void *v, const float *decay, float *out,
                            uint32_t flags, void *workspace, size_t workspace_bytes, lq_stream_t stream) {
    const lq_status st = check_linear(cfg, qk_heads);
    if (st != LQ_OK) return st;
    if (!state) return LQ_ERR_INVALID_ARG;
    return prefill_rows(*cfg, state, nullptr, cfg->num_slots, tokens, lengths, S0, qk_heads, q, k, v, decay, out, flags,
                        workspace, workspace_bytes, stream);
}

lq_status lq_linear_prefill_slots(const lq_config *cfg, void *state, const int32_t *slots, int n_active, int tokens,
                                  const int32_t *lengths, const float *S0, int qk_heads, const void *q, const void *k,
                                  const void *v, const float *decay, float *out, uint32_t flags, void *workspace,
                                  size_t workspace_bytes, lq_stream_t stream) {
    const lq_status st = check_linear_slots(cfg, state, slots, n_active, qk_heads);
    if (st != LQ_OK) return st;
    return prefill_rows(*cfg, state, slots, n_active, tokens, lengths, S0, qk_heads, q, k, v, decay, out, flags,
                        workspace, workspace_bytes, stream);
}

lq_status lq_qk_norm(const lq_config *cfg, int rows, int qk_heads, const void *q, const void *k, const void *a,
                     const void *b, const float *a_log, const float *dt_bias, float q_scale, float eps, void *q_out,
                     void *k_out, float *decay, float *beta, lq_stream_t stream) {
    const lq_status st = check_config(cfg);
    if (st != LQ_OK) return st;
    if (rows < 0 || qk_heads <= 0 || cfg->num_heads % qk_heads != 0 || !(eps >= 0.f)) return LQ_ERR_INVALID_ARG;
    if (rows > 0 && (!q || !k || !a || !b || !a_log || !dt_bias || !q_out || !k_out || !decay || !beta))
        return LQ_ERR_INVALID_ARG;
    const lq_config &c = *cfg;
    if ((int64_t)rows * c.num_heads > 0x7FFFFFFF) return LQ_ERR_UNSUPPORTED;
    const uintptr_t e = c.in_dtype ? 2 : 4;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
        !aligned(a, c.decay_kind ? 16 : e) || !aligned(b, e) || !aligned(a_log, 4) ||
        !aligned(dt_bias, c.decay_kind ? 16 : 4) || !aligned(decay, c.decay_kind ? 16 : 4) || !aligned(beta, 4))
        return LQ_ERR_MISALIGNED;
    if (rows == 0) return LQ_OK;
    QkNormArgs n{q, k, a, b, a_log, dt_bias, q_out, k_out, decay, beta, q_scale, eps, (long long)rows * qk_heads,
                 (unsigned)(rows * c.num_heads), c.num_heads, c.decay_kind, 0u, 0u};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (c.dk == 128)
        return launched(c.in_dtype ? launch_qk_norm<128, true>(n, s) : launch_qk_norm<128, false>(n, s));
    return launched(c.in_dtype ? launch_qk_norm<64, true>(n, s) : launch_qk_norm<64, false>(n, s));
}

lq_status lq_out_norm(const lq_config *cfg, int rows, const float *o, const float *weight, const void *gate,
                      int gate_kind, float eps, void *y, lq_stream_t stream) {
    const lq_status st = check_config(cfg);
    if (st != LQ_OK) return st;
    if (rows < 0 || gate_kind < LQ_GATE_NONE || gate_kind > LQ_GATE_SIGMOID || !(eps >= 0.f)) return LQ_ERR_INVALID_ARG;
    if ((gate_kind == LQ_GATE_NONE) != (gate == nullptr) && rows > 0) return LQ_ERR_INVALID_ARG;
    if (rows > 0 && (!o || !y)) return LQ_ERR_INVALID_ARG;
    const lq_config &c = *cfg;
    if ((int64_t)rows * c.num_heads > 0x7FFFFFFF) return LQ_ERR_UNSUPPORTED;
    if (!aligned(o, 16) || !aligned(weight, 16) || !aligned(gate, 16) || !aligned(y, 16)) return LQ_ERR_MISALIGNED;
    if (rows == 0) return LQ_OK;
    OutNormArgs n{o, weight, gate, y, eps, (long long)rows * c.num_heads};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (c.dv == 128)
        return launched(c.in_dtype ? launch_out_norm<128, true>(n, gate_kind, s)
                                   : launch_out_norm<128, false>(n, gate_kind, s));
    return launched(c.in_dtype ? launch_out_norm<64, true>(n, gate_kind, s)
                               : launch_out_norm<64, false>(n, gate_kind, s));
}

}  // extern "C"
