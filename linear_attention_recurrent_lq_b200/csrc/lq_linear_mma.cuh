// lq_linear_mma.cuh -- tensor-core helpers of the linear-attention prompts:
// bf16 products with FP32 accumulation (tcgen05.mma kind::f16), TMA tile
// loads, and FP32 operands cut into three bf16 pieces (sm_100a).
//
// Precision: q, k and v are bf16 as they come; the state, the scores and the
// weighted keys are FP32, and the tensor cores take bf16.  Three bf16 pieces
// of 8 mantissa bits hold an FP32 value's 24 bits exactly; they are multiplied
// piece by piece, smallest first, and summed in FP32.  Two pieces would leave
// 2^-17 of each operand, and TF32 (11 bits) two pieces at twice the cost of
// bf16 each.
#pragma once

#include <cuda.h>

#include "lq_linear.cuh"
#include "lq_umma.cuh"

namespace lq {

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

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// 16 columns, without the wait (tmem_ld_wait before the first use)
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// Wait for the loads above; the registers pass through, so that no use is
// scheduled before it.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 ::"memory");
}

__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Offset of 16-byte piece c of row r in tiles of 64 elements a row (`block`
// bytes from one tile to the next), 128-byte swizzle.
__device__ __forceinline__ uint32_t lc_tile_off(int r, int c, uint32_t block) {
    return (uint32_t)(c >> 3) * block + (uint32_t)r * 128u + (uint32_t)(((c & 7) ^ (r & 7)) << 4);
}

// One piece (8 bf16 keys) times f, in three pieces, to dst and `step` bytes
// behind it each.
__device__ __forceinline__ void lc_weighted_piece(const uint4 &kk, float f, uint8_t *dst, uint32_t step) {
    const uint32_t u[4] = {kk.x, kk.y, kk.z, kk.w};
    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
    for (int z = 0; z < 4; ++z) {
        const float2 kf = __fmul2_rn(make_float2(f, f), make_float2(__uint_as_float(u[z] << 16), __uint_as_float(u[z] & 0xFFFF0000u)));
        lc_split2(kf.x, kf.y, hi[z], mid[z], lo[z]);
    }
    *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4 *>(dst + step) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
    *reinterpret_cast<uint4 *>(dst + 2 * step) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

}  // namespace lq
