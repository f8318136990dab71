// lq_linear.cuh -- linear attention with one decay per head over the FP32
// state blobs (bits = 32), sm_100a:
//     S_t = a_t S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,
// S dk x dv, row i = key channel.  Unlike the delta rule the update does not
// read the state, so columns of S are independent and a prompt may be cut
// along time: over tokens t0 .. t1 the state is G S + P with G the product of
// their gates and P the state the same tokens leave from zero.
//
// Kernels here: one token (lin_step_kernel), a prompt token after token
// (lin_recurrent_kernel, also the first pass of a prompt cut along time), and
// the pass that joins the cuts (lin_scan_kernel).  The chunkwise form on the
// tensor cores is in lq_linear_pipe.cuh and lq_linear_state.cuh.  Grouped queries
// and keys: value head h reads query / key head h / (H / Hk).
#pragma once

#include "lq_common.cuh"

namespace lq {

struct LinArgs {
    uint8_t *state;
    Layout L;
    SlotMap map;
    const float *S0;         // [rows, H, dk, dv] or null (zero state)
    const void *q, *k;       // [rows, T, Hk, dk]
    const void *v;           // [rows, T, H, dv]
    const float *decay;      // [rows, T, H]
    const int32_t *lengths;  // [rows] or null (all T)
    float *out;              // [rows, T, H, dv] or null
    int tokens;              // T
    int work;                // rows * H
    int group;               // value heads per query / key head
    int qk_heads;            // Hk
    int cont;                // 1: go on from the blob's state
    // a prompt cut along time (nseg > 1): segment s holds tokens
    // [s seg_len, (s + 1) seg_len)
    int seg_len, nseg;
    float *ws_S;   // [work, nseg, dk, dv]: a segment's own state, then the state before it
    float *ws_g;   // [work, nseg]: product of a segment's gates
    int *ws_bad;   // [work, nseg]: its first token with a bad gate, or kNoBad or kLost
    int *ws_run;   // [work]: 0 if the blob's header refuses the call or a segment was lost
};

constexpr int kNoBad = 0x7FFFFFFF;  // no gate is bad
constexpr int kLost = -1;           // a wait of the first pass gave up: the segment's state is not there

// The forms of a prompt divide by products of gates, which must not grow past
// FP32's range: a gate above 1 is as wrong as a negative one.
__device__ __forceinline__ bool lin_gate_ok(float a) { return a >= 0.f && a <= 1.f; }

// Row indices of token t of work item (row, hh).
__device__ __forceinline__ size_t lin_v_row(const LinArgs &A, int row, int hh, int t) {
    return ((size_t)row * A.tokens + t) * A.map.heads + hh;
}
__device__ __forceinline__ size_t lin_qk_row(const LinArgs &A, int row, int hh, int t) {
    return ((size_t)row * A.tokens + t) * A.qk_heads + hh / A.group;
}

__device__ __forceinline__ int lin_length(const LinArgs &A, int row) {
    return A.lengths ? min(max(__ldcg(A.lengths + row), 0), A.tokens) : A.tokens;
}

// The segment that holds a prompt's last token (0 for an empty prompt).
__device__ __forceinline__ int lin_last_segment(const LinArgs &A, int len) {
    return len > 0 ? (len - 1) / A.seg_len : 0;
}

// Where the tokens that a segment [t_begin, t_end) takes in end: at its start
// if it does not run or lies behind the prompt.  From there to t_end its outputs
// are zeros, so the segments of a row write each output once.
__host__ __device__ __forceinline__ int lin_stop(bool run, int len, int t_begin, int t_end) {
    const int t = len < t_end ? len : t_end;
    return run && t > t_begin ? t : t_begin;
}

// Where work item w's segment starts from; null: a zero state.
__device__ __forceinline__ const float *lin_state_source(const LinArgs &A, int w, int seg, const uint8_t *blob) {
    const size_t n = A.L.pairs_off - A.L.qs_off;  // bytes of a state
    if (A.nseg > 1) return A.ws_S + ((size_t)w * A.nseg + seg) * (n / 4);
    if (A.cont) return reinterpret_cast<const float *>(blob + kHdrBytes);
    return A.S0 ? A.S0 + (size_t)w * (n / 4) : nullptr;
}

// A new header with the given status.
__device__ __forceinline__ void lin_new_header(uint8_t *blob, uint32_t status) {
    *reinterpret_cast<uint4 *>(blob) = make_uint4(0u, status, 0u, kMagic);
    *reinterpret_cast<float *>(blob + kHdrG) = 1.f;
}

// Header of a blob whose prompt has been taken in.  That of a prompt cut along
// time was written by the pass that joins the cuts: several CTAs add to its
// status, so none of them may store it.
__device__ __forceinline__ void lin_write_header(const LinArgs &A, uint8_t *blob, bool bad) {
    if (A.cont || A.nseg > 1) {
        if (bad) set_status(blob, LQ_DEV_RANGE);
    } else {
        lin_new_header(blob, bad ? LQ_DEV_RANGE : 0u);
    }
}

// Whether a call that goes on from the blob may run; sets LQ_DEV_CORRUPT in a
// header without the magic (`report`: one caller per blob).
__device__ __forceinline__ bool lin_may_run(uint8_t *blob, bool report) {
    const uint4 hdr = __ldcg(reinterpret_cast<const uint4 *>(blob));
    if (report && hdr.y == 0u && hdr.w != kMagic) set_status(blob, LQ_DEV_CORRUPT);
    return hdr.y == 0u && hdr.w == kMagic;
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(void *dst, const void *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four consecutive inputs as floats.
template <bool BF16>
__device__ __forceinline__ float4 lin_load4(const uint8_t *p) {
    if constexpr (BF16) {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                           __uint_as_float(w.y & 0xFFFF0000u));
    } else {
        return *reinterpret_cast<const float4 *>(p);
    }
}

// ------------------------------------------------------------- one token
// Bound by HBM: the state is read and written once.  A CTA takes CB columns
// of one head, all its loads in flight before the first use, a thread four
// columns of R rows.  d = 128: 64 x 32 heads 43.1 us, 6290 GB/s (41.4 us at the
// copy's rate), 512 x 36 heads through a slot list 290.6 us (279.4).
template <int D, bool BF16, int CB>
__global__ void __launch_bounds__(256, 3) lin_step_kernel(LinArgs A) {
    constexpr int E = BF16 ? 2 : 4, NB = D / CB, CQ = CB / 4, RG = 256 / CQ, R = D / RG;
    __shared__ float s_q[D], s_k[D];
    __shared__ float4 s_part[RG][CQ];
    const int tid = threadIdx.x, cq = tid % CQ, rg = tid / CQ;
    const int w = blockIdx.x / NB, j0 = (blockIdx.x % NB) * CB + 4 * cq;
    const int row = w / A.map.heads, hh = w - row * A.map.heads;

    pdl_wait();
    pdl_trigger();
    const int bi = A.map.blob(w);
    float *out = A.out + (size_t)w * D;
    if (bi < 0) {  // no such slot (uniform over the CTA)
        if (rg == 0) *reinterpret_cast<float4 *>(out + j0) = make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    uint8_t *blob = A.state + (size_t)bi * A.L.blob;
    float *S = reinterpret_cast<float *>(blob + kHdrBytes) + j0;
    float4 s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = __ldcs(reinterpret_cast<const float4 *>(S + (size_t)(rg + RG * r) * D));
    const uint4 hdr = __ldcg(reinterpret_cast<const uint4 *>(blob));
    const float a = A.decay[w];
    const float4 v = lin_load4<BF16>(static_cast<const uint8_t *>(A.v) + ((size_t)w * D + j0) * E);
    const size_t qk = ((size_t)row * A.qk_heads + hh / A.group) * D;
    if (tid < D) s_q[tid] = load_in(A.q, qk + tid, BF16);
    if (tid >= 256 - D) s_k[tid - (256 - D)] = load_in(A.k, qk + tid - (256 - D), BF16);
    const bool ok = hdr.y == 0u && hdr.w == kMagic && lin_gate_ok(a);
    __syncthreads();
    if (!ok) {  // uniform: every CTA of this head decides the same
        if (tid == 0 && hdr.y == 0u) set_status(blob, hdr.w == kMagic ? LQ_DEV_RANGE : LQ_DEV_CORRUPT);
        if (rg == 0) *reinterpret_cast<float4 *>(out + j0) = make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float ki = s_k[rg + RG * r], qi = s_q[rg + RG * r];
        s[r].x = fmaf(a, s[r].x, ki * v.x);
        s[r].y = fmaf(a, s[r].y, ki * v.y);
        s[r].z = fmaf(a, s[r].z, ki * v.z);
        s[r].w = fmaf(a, s[r].w, ki * v.w);
        __stcs(reinterpret_cast<float4 *>(S + (size_t)(rg + RG * r) * D), s[r]);
        o.x = fmaf(s[r].x, qi, o.x);
        o.y = fmaf(s[r].y, qi, o.y);
        o.z = fmaf(s[r].z, qi, o.z);
        o.w = fmaf(s[r].w, qi, o.w);
    }
    s_part[rg][cq] = o;
    __syncthreads();
    if (tid < CB) {
        const float *p = reinterpret_cast<const float *>(s_part) + tid;
        float sum = 0.f;
#pragma unroll
        for (int g = 0; g < RG; ++g) sum += p[g * CB];
        out[j0 - 4 * cq + tid] = sum;
    }
}

// ------------------------------------------- a prompt, token after token
// 128 threads hold 64 columns of one head's state in registers (16 where heads
// are few): lane % 8 takes the rows 4 (lane % 8) + 32 m .. + 3, lane / 8 and the
// warp take four columns (one).  q, k, v and the gates arrive 16 tokens at a
// time through a ring of three shared-memory stages; rows past the prompt arrive
// as zeros.  The outputs of four (eight) tokens are summed over the eight row
// lanes at once.
//
// Bound by FP32 multiply-adds.  The registers hold S / G with G the product of
// the gates so far, so a token costs two per entry instead of three,
//     S / G_t += k_t (v_t / G_t),   o_t = G_t (S / G_t)^T q_t,
// and S is brought back to G = 1 before 16 tokens that start from G < 2^-16.
// 16 tokens whose gates multiply to less than 2^-48 (gates of 0 among them)
// are taken one by one from G = 1: S = a_t S + k_t v_t^T.  f32, 2048 heads of 256
// tokens: d = 128 833 us, 462 of them multiply-adds at their peak rate; d = 64
// 266 us (115); the rest are reads of q, k and v from shared memory.  Of 64 columns,
// f32 and d = 128, the kernel fills its 128 registers and spills 84 bytes.
constexpr int kLinTokens = 16;  // tokens per stage
constexpr int kLinStages = 3;
constexpr int kLinThreads = 128;

template <int D, bool BF16, int C>
struct LinShape {
    static constexpr int E = BF16 ? 2 : 4;
    static constexpr int U = C == 1 ? 8 : C == 4 ? 4 : 2;          // tokens summed at once
    static constexpr int COLS = 16 * C;               // columns of one CTA
    static constexpr int NB = D / COLS;               // CTAs of one head (one cluster)
    static constexpr int QB = D * E, VB = COLS * E;   // bytes of a q / k row, of a v row's columns
    static constexpr int K_OFF = kLinTokens * QB, V_OFF = 2 * K_OFF, A_OFF = V_OFF + kLinTokens * VB;
    static constexpr int STAGE = A_OFF + 4 * kLinTokens;
    static constexpr uint32_t SMEM = (uint32_t)(kLinStages * STAGE);
};

// C columns of one state row (null: zeros).
template <int C>
__device__ __forceinline__ void lin_get_row(const float *p, float (&x)[C]) {
    if constexpr (C % 4 == 0) {
#pragma unroll
        for (int c = 0; c < C; c += 4) {
            const float4 v = p ? *reinterpret_cast<const float4 *>(p + c) : make_float4(0.f, 0.f, 0.f, 0.f);
            x[c] = v.x; x[c + 1] = v.y; x[c + 2] = v.z; x[c + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = p ? p[c] : 0.f;
    }
}
template <int C>
__device__ __forceinline__ void lin_put_row(float *p, const float (&x)[C]) {
    if constexpr (C % 4 == 0) {
#pragma unroll
        for (int c = 0; c < C; c += 4) *reinterpret_cast<float4 *>(p + c) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) p[c] = x[c];
    }
}

template <int D, bool BF16, int C, bool PARTIAL>
__global__ void __launch_bounds__(kLinThreads, C == 8 ? 2 : 4) lin_recurrent_kernel(LinArgs A) {
    using SH = LinShape<D, BF16, C>;
    constexpr int E = SH::E, RL = 8, U = SH::U, M = D / 32, TB = kLinTokens;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rl = lane % RL, jt = (32 / RL * warp + lane / RL) * C;  // first column inside the CTA
    const int w = blockIdx.x / SH::NB, jc = (blockIdx.x % SH::NB) * SH::COLS;
    const int seg = blockIdx.y;
    const int row = w / A.map.heads, hh = w - row * A.map.heads;
    extern __shared__ __align__(16) uint8_t smem[];

    pdl_wait();
    pdl_trigger();
    const int len = lin_length(A, row), last = lin_last_segment(A, len);
    if (PARTIAL && seg >= last) return;  // not needed
    const int bi = A.map.blob(w);
    if (PARTIAL && bi < 0) return;
    uint8_t *blob = A.state + (size_t)(bi < 0 ? 0 : bi) * A.L.blob;
    bool run = bi >= 0;
    if (!PARTIAL && A.nseg > 1) {
        if (run && seg <= last) {
            run = A.ws_run[w] != 0;
            for (int s = 0; s < seg; ++s)
                if (A.ws_bad[(size_t)w * A.nseg + s] != kNoBad) run = false;
        }
    } else if (!PARTIAL && A.cont) {
        if (run) run = lin_may_run(blob, tid == 0 && jc == 0);
        // every CTA of the head reads the status before one may change it
        if constexpr (SH::NB > 1)
            asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    }
    const int t_begin = seg * A.seg_len, t_end = min(A.tokens, t_begin + A.seg_len);
    const int t_stop = lin_stop(run, len, t_begin, t_end);

    // ---- the state this segment starts from
    float2 S[2 * M][C];
    {
        const float *src = nullptr;
        if (!PARTIAL && run && seg <= last) src = lin_state_source(A, w, seg, blob);
#pragma unroll
        for (int p = 0; p < 2 * M; ++p) {
            float a[C], b[C];
            const int i = 4 * rl + 4 * RL * (p >> 1) + 2 * (p & 1);
            lin_get_row<C>(src ? src + (size_t)i * D + jc + jt : nullptr, a);
            lin_get_row<C>(src ? src + (size_t)(i + 1) * D + jc + jt : nullptr, b);
#pragma unroll
            for (int c = 0; c < C; ++c) S[p][c] = make_float2(a[c], b[c]);
        }
    }

    const uint8_t *qg = static_cast<const uint8_t *>(A.q), *kg = static_cast<const uint8_t *>(A.k);
    const uint8_t *vg = static_cast<const uint8_t *>(A.v);
    auto issue = [&](int st, int t0) {
        uint8_t *b = smem + st * SH::STAGE;
        constexpr int QP = SH::QB / 16, VP = SH::VB / 16;
#pragma unroll
        for (int x = tid; x < TB * QP; x += kLinThreads) {
            const int r = x / QP, c = 16 * (x % QP);
            const bool in = t0 + r < t_stop;
            const size_t o = lin_qk_row(A, row, hh, in ? t0 + r : t_begin) * SH::QB + c;
            if (!PARTIAL) cp_async16(b + r * SH::QB + c, qg + o, in);
            cp_async16(b + SH::K_OFF + r * SH::QB + c, kg + o, in);
        }
#pragma unroll
        for (int x = tid; x < TB * VP; x += kLinThreads) {
            const int r = x / VP, c = 16 * (x % VP);
            const bool in = t0 + r < t_stop;
            cp_async16(b + SH::V_OFF + r * SH::VB + c,
                       vg + lin_v_row(A, row, hh, in ? t0 + r : t_begin) * (size_t)(D * E) + (size_t)jc * E + c, in);
        }
        if (tid < TB) {
            const bool in = t0 + tid < t_stop;
            cp_async4(b + SH::A_OFF + 4 * tid, A.decay + lin_v_row(A, row, hh, in ? t0 + tid : t_begin), in);
        }
    };
    const int n_stage = t_stop > t_begin ? (t_stop - t_begin + TB - 1) / TB : 0;
#pragma unroll
    for (int i = 0; i < kLinStages - 1; ++i) {
        if (i < n_stage) issue(i, t_begin + i * TB);
        cp_async_commit();
    }

    float G = 1.f, gprod = 1.f;
    int bad = kNoBad, t_done = t_stop;
#pragma unroll 1
    for (int i = 0; i < n_stage && bad == kNoBad; ++i) {
        const int t0 = t_begin + i * TB;
        cp_async_wait<kLinStages - 2>();
        __syncthreads();
        if (i + kLinStages - 1 < n_stage) issue((i + kLinStages - 1) % kLinStages, t0 + (kLinStages - 1) * TB);
        cp_async_commit();
        uint8_t *b = smem + (i % kLinStages) * SH::STAGE;
        int n = min(TB, t_stop - t0);
        float al = lane < n ? reinterpret_cast<const float *>(b + SH::A_OFF)[lane] : 1.f;
        const unsigned wrong = __ballot_sync(0xFFFFFFFFu, !lin_gate_ok(al));
        if (wrong) {  // the prompt ends before its first bad gate (uniform over the CTA)
            n = __ffs(wrong) - 1;
            bad = t0 + n;
            t_done = bad;
            if (lane >= n) al = 1.f;
            for (int x = tid; x < (TB - n) * SH::QB / 16; x += kLinThreads)
                *reinterpret_cast<uint4 *>(b + SH::K_OFF + n * SH::QB + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
            for (int x = tid; x < (TB - n) * SH::VB / 16; x += kLinThreads)
                *reinterpret_cast<uint4 *>(b + SH::V_OFF + n * SH::VB + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
            __syncthreads();
        }
        // products of the gates: pre up to token lane, all 16 in `total`
        float pre = al;
#pragma unroll
        for (int d = 1; d < TB; d <<= 1) {
            const float x = __shfl_up_sync(0xFFFFFFFFu, pre, d, TB);
            if ((lane & (TB - 1)) >= d) pre *= x;
        }
        const float total = __shfl_sync(0xFFFFFFFFu, pre, TB - 1);
        const bool apart = !(total >= 0x1p-48f);
        if (apart || G < 0x1p-16f) {
            const float2 g2 = make_float2(G, G);
#pragma unroll
            for (int p = 0; p < 2 * M; ++p)
#pragma unroll
                for (int c = 0; c < C; ++c) S[p][c] = __fmul2_rn(g2, S[p][c]);
            G = 1.f;
        }
        const float Gl = G * pre, inv = __fdiv_rn(1.f, Gl);  // of token `lane`
        if (PARTIAL) gprod *= total;
        if (!apart) G *= total;
        // S += k v^T of token t, v times f; returns S^T q of this lane's rows
        auto token = [&](int t, float f, float (&o)[C]) {
            const uint8_t *qs = b + t * SH::QB + 4 * rl * E, *ks = qs + SH::K_OFF;
            float v[C];
#pragma unroll
            for (int c = 0; c < C; ++c) v[c] = f * load_in(b + SH::V_OFF + t * SH::VB, jt + c, BF16);
            float2 acc[C];
#pragma unroll
            for (int c = 0; c < C; ++c) acc[c] = make_float2(0.f, 0.f);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const float4 k4 = lin_load4<BF16>(ks + 4 * RL * m * E);
                float4 q4 = make_float4(0.f, 0.f, 0.f, 0.f);
                if (!PARTIAL) q4 = lin_load4<BF16>(qs + 4 * RL * m * E);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float2 v2 = make_float2(v[c], v[c]);
                    S[2 * m][c] = __ffma2_rn(make_float2(k4.x, k4.y), v2, S[2 * m][c]);
                    S[2 * m + 1][c] = __ffma2_rn(make_float2(k4.z, k4.w), v2, S[2 * m + 1][c]);
                    if (!PARTIAL) {
                        acc[c] = __ffma2_rn(S[2 * m][c], make_float2(q4.x, q4.y), acc[c]);
                        acc[c] = __ffma2_rn(S[2 * m + 1][c], make_float2(q4.z, q4.w), acc[c]);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c) o[c] = acc[c].x + acc[c].y;
        };
        if (apart) {
#pragma unroll 1
            for (int t = 0; t < n; ++t) {
                const float a = __shfl_sync(0xFFFFFFFFu, al, t);
                float o[C];
#pragma unroll
                for (int r = 0; r < 2 * M; ++r)
#pragma unroll
                    for (int c = 0; c < C; ++c) S[r][c] = __fmul2_rn(make_float2(a, a), S[r][c]);
                token(t, 1.f, o);
#pragma unroll
                for (int c = 0; c < C; ++c) {
#pragma unroll
                    for (int d = RL / 2; d >= 1; d >>= 1) o[c] += __shfl_xor_sync(0xFFFFFFFFu, o[c], d);
                    if (!PARTIAL && A.out && rl == 0) A.out[lin_v_row(A, row, hh, t0 + t) * D + jc + jt + c] = o[c];
                }
            }
            continue;
        }
#pragma unroll 1
        for (int g = 0; g < TB && g < n; g += U) {
            float p[U][C];
#pragma unroll
            for (int u = 0; u < U; ++u) token(g + u, __shfl_sync(0xFFFFFFFFu, inv, g + u), p[u]);
            if (!PARTIAL && A.out) {
                // sums over the row lanes; a lane keeps NV columns of one token
                constexpr int N = U * C, NV = N / RL;
                float x[N];
#pragma unroll
                for (int e = 0; e < N; ++e) x[e] = p[e / C][e % C];
#pragma unroll
                for (int d = RL / 2; d >= 1; d >>= 1)
#pragma unroll
                    for (int e = 0; e < d * NV; ++e) {
                        const bool up = (rl & d) != 0;
                        x[e] = (up ? x[e + d * NV] : x[e]) + __shfl_xor_sync(0xFFFFFFFFu, up ? x[e] : x[e + d * NV], d);
                    }
                const int t = g + rl * NV / C;
                const float go = __shfl_sync(0xFFFFFFFFu, Gl, t);
                if (t < n) {
                    float *o = A.out + lin_v_row(A, row, hh, t0 + t) * D + jc + jt + rl * NV % C;
                    if constexpr (NV == 2) *reinterpret_cast<float2 *>(o) = make_float2(go * x[0], go * x[1]);
                    else *o = go * x[0];
                }
            }
        }
    }
    cp_async_wait<0>();
#pragma unroll
    for (int p = 0; p < 2 * M; ++p)
#pragma unroll
        for (int c = 0; c < C; ++c) S[p][c] = __fmul2_rn(make_float2(G, G), S[p][c]);

    if (PARTIAL) {
        float *dst = A.ws_S + ((size_t)w * A.nseg + seg) * (D * D) + jc + jt;
#pragma unroll
        for (int p = 0; p < 2 * M; ++p) {
            float a[C], b[C];
            const int i = 4 * rl + 4 * RL * (p >> 1) + 2 * (p & 1);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                a[c] = S[p][c].x;
                b[c] = S[p][c].y;
            }
            lin_put_row<C>(dst + (size_t)i * D, a);
            lin_put_row<C>(dst + (size_t)(i + 1) * D, b);
        }
        if (tid == 0 && jc == 0) {
            A.ws_g[(size_t)w * A.nseg + seg] = gprod;
            A.ws_bad[(size_t)w * A.nseg + seg] = bad;
        }
        return;
    }
    if (A.out)  // no outputs past the prompt's end (tokens x columns may pass 2^31)
        for (int t = t_done + tid / SH::COLS; t < t_end; t += kLinThreads / SH::COLS)
            A.out[lin_v_row(A, row, hh, t) * D + jc + tid % SH::COLS] = 0.f;
    if (run && (bad != kNoBad || seg == last)) {  // this segment holds the prompt's end
        float *dst = reinterpret_cast<float *>(blob + kHdrBytes) + jc + jt;
#pragma unroll
        for (int p = 0; p < 2 * M; ++p) {
            float a[C], b[C];
            const int i = 4 * rl + 4 * RL * (p >> 1) + 2 * (p & 1);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                a[c] = S[p][c].x;
                b[c] = S[p][c].y;
            }
            lin_put_row<C>(dst + (size_t)i * D, a);
            lin_put_row<C>(dst + (size_t)(i + 1) * D, b);
        }
        if (tid == 0 && jc == 0) lin_write_header(A, blob, bad != kNoBad);
    }
}

// ------------------------------------- joining a prompt cut along time
// In place: each segment's own state becomes the state before that segment.
// One thread takes four entries of one head through all segments.  The first
// CTA of a head also writes its header, before the main pass, whose CTAs only
// add to the status; a head with a lost segment gets LQ_DEV_TIMEOUT and does
// not run, so its outputs are zeros and its state stays as it was.
template <int D>
__global__ void __launch_bounds__(256) lin_scan_kernel(LinArgs A) {
    constexpr int NB = D * D / 1024;
    const int w = blockIdx.x / NB, e = (blockIdx.x % NB) * 1024 + 4 * threadIdx.x;
    const int row = w / A.map.heads;
    pdl_wait();
    pdl_trigger();
    const int bi = A.map.blob(w);
    if (bi < 0) return;
    uint8_t *blob = A.state + (size_t)bi * A.L.blob;
    float4 carry = make_float4(0.f, 0.f, 0.f, 0.f);
    const int last = lin_last_segment(A, lin_length(A, row));
    const bool run = !A.cont || lin_may_run(blob, e == 0);
    if (blockIdx.x % NB == 0 && threadIdx.x < 32) {
        bool lost = false;
        for (int s = threadIdx.x; s < last; s += 32) lost |= A.ws_bad[(size_t)w * A.nseg + s] == kLost;
        lost = __any_sync(0xFFFFFFFFu, lost);
        if (threadIdx.x == 0) {
            A.ws_run[w] = run && !lost;
            if (!A.cont) lin_new_header(blob, lost ? LQ_DEV_TIMEOUT : 0u);
            else if (run && lost) set_status(blob, LQ_DEV_TIMEOUT);
        }
    }
    if (A.cont) {
        if (!run) return;
        carry = *reinterpret_cast<const float4 *>(blob + kHdrBytes + 4 * (size_t)e);
    } else if (A.S0) {
        carry = *reinterpret_cast<const float4 *>(A.S0 + (size_t)w * (D * D) + e);
    }
    float *S = A.ws_S + (size_t)w * A.nseg * (D * D) + e;
    const float *g = A.ws_g + (size_t)w * A.nseg;
    // sixteen segments' loads in flight (one at a time: 30 us for 32 heads of 9
    // segments, d = 128)
    constexpr int U = 16;
#pragma unroll 1
    for (int s0 = 0; s0 < last; s0 += U) {
        float4 own[U];
        float gs[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + u < last) {
                own[u] = __ldcg(reinterpret_cast<const float4 *>(S + (size_t)(s0 + u) * (D * D)));
                gs[u] = __ldcg(g + s0 + u);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + u < last) {
                *reinterpret_cast<float4 *>(S + (size_t)(s0 + u) * (D * D)) = carry;
                carry.x = fmaf(gs[u], carry.x, own[u].x);
                carry.y = fmaf(gs[u], carry.y, own[u].y);
                carry.z = fmaf(gs[u], carry.z, own[u].z);
                carry.w = fmaf(gs[u], carry.w, own[u].w);
            }
    }
    *reinterpret_cast<float4 *>(S + (size_t)last * (D * D)) = carry;
}

}  // namespace lq
