// Attention over the 8-bit cache on the 5th-generation tensor cores: the block's shape and the tensor-core and TMEM operations that the
// kernels of kv8_prompt.cu and kv8_shared.cu share.
#pragma once

#include "kv8_attn.cuh"

namespace cac {

constexpr int PT_ROWS = 128, PT_KEYS = 128, PT_HALF = 64;

// TILES: row tiles of a block, two at most: what shared memory and TMEM hold
template <class T, int HDP, int TILES = sizeof(T) == 4 && HDP == 128 ? 1 : 2> struct PShape {
    static constexpr bool WIDE = sizeof(T) == 4;             // queries and weights as hi + lo
    static constexpr int NM = TILES;
    static constexpr int PARTS = WIDE ? 2 : 1;
    static constexpr int PANEL = 128 * 128;                  // 128 rows of 64 fp16
    static constexpr int TILE = HDP / 64 * PANEL;
    static constexpr int OFF_K = NM * PARTS * TILE, OFF_V = OFF_K + 2 * TILE, OFF_SC = OFF_V + 2 * TILE;
    static constexpr int OFF_BAR = OFF_SC + 4 * 24 * 4;      // [4 tiles][K scale, log2 and reciprocal of V scale][8]
    static constexpr int BYTES = OFF_BAR + 21 * 8 + 16 + 1024;
    static constexpr int SMEM = BYTES > 120 * 1024 ? BYTES : 120 * 1024;  // one block an SM
    static constexpr int SOFT = NM * 4, CONV = 6, WARPS = SOFT + CONV + 2, THREADS = WARPS * 32;
    // TMEM columns: scores (two times 64 a row tile, the weights of 64 tokens in their first 32 and, for fp32, the low halves in the
    // other 32), sums (HDP a row tile)
    // The tensor core cuts sums off where fp32 would round.  For fp32 results its sums are of FLUSH pieces of 64 tokens, which are
    // added up in columns of their own (measured over windows of 2,047 tokens: off by 4.3e-6 of the result without that).
    static constexpr int FLUSH = WIDE ? 4 : 1 << 30;
    static constexpr int COL_S = 0, COL_O = NM * 128, COL_SUM = COL_O + NM * HDP;
    static_assert(COL_SUM + (WIDE ? NM * HDP : 0) <= 512, "TMEM");
    static constexpr float SLACK = WIDE ? 2.f : 8.f, LIFT = 15.f - SLACK, NORM = norm_factor(WIDE ? 13 : 7);
};

// D[tmem] (+)= A[smem] B[smem], fp16 operands
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    tc_mma_bf16(d, a, b, idesc, add);  // kind::f16; the descriptor names the operands' type
}
// D[tmem] (+)= A[tmem] B[smem], fp16 operands
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// fp16 A (K-major) and B, fp32 D; mn: B's rows are the contracted index
constexpr uint32_t idesc_f16(int M, int N, bool mn) {
    return (1u << 4) | ((uint32_t)mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// V tile: rows (tokens) of 64 elements (128 bytes, swizzled), 8-row groups 1024 bytes apart, panels of 64 elements PANEL apart
__device__ __forceinline__ uint64_t sdesc_mn_sw128(const void* tile, uint32_t panel) {
    return (sdesc_k_sw128(tile) & ~((uint64_t)0x3FFFu << 16)) | ((uint64_t)(panel >> 4) << 16);
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 64 or 16 columns of the thread's lane.  The wait stands in the same statement: between the two the compiler could move a value
// that has not arrived.
__device__ __forceinline__ void tmem_ld64(uint32_t addr, float (&v)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
          "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
          "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
          "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]),
          "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(addr)
        : "memory");
}
// two at once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 columns of the thread's lane times r
__device__ __forceinline__ void scale16(uint32_t col, float r) {
    float o[16];
    uint32_t u[16];
    tmem_ld16(col, o);
#pragma unroll
    for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(o[k] * r);
    tmem_st16(col, u);
}

// mbar_wait and mbar_arrive for a whole warp, with one answer for all of it.  All lanes poll (one polling for the others measured 3 %
// slower); one arrives.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

}  // namespace cac
