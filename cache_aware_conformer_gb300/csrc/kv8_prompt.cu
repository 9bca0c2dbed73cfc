// Attention over the paged 8-bit K/V cache for calls with many query rows to a K/V head
// (prompts and pieces of them), on the 5th-generation tensor cores.  The mathematics is that of
// kv8_attn.cu: codes enter as exact fp16, the block scales sit in the exponent.
//
// Arithmetic bounds it: 4 * head_dim operations a pair of query and token.  A block takes
// NM tiles of 128 query rows (row = query * group + head of the group, so the heads that share K and V
// share the tile too) of one sequence and K/V head, and walks over its 128-token tiles:
//   converters  6 warps, 16 tokens of K or of V at a time in turn: 16-byte loads of codes, the next piece
//               under way, turned into fp16 in the 128-byte-swizzled layout that the tensor core reads
//               (K as [token][element]: its rows are the columns of the scores; V the same
//               way, read with the token as the contracted index), a ring of two tiles each
//   MMA         a thread for each row tile: S = Q K^T into TMEM, O += P V with P from TMEM, 64 tokens at a time
//   softmax     4 warps for each row tile, a thread per row: 64 scores from TMEM into registers, maximum, weights
//               back into TMEM in place of the scores, row sums
// A call goes to this kernel or to kv_attend_kernel as a whole, by its mean row count, and a block walks all tokens of its rows: a
// single token over a long cache in one call with prompts occupies a block of 256 rows (64 tokens over up to 32,000 and
// a prompt of 4,096: 1,401 us in one call, 332 and 152 in two), and few blocks over a long cache leave SMs idle (512 queries of 32
// heads on 30,000 tokens: 500 us, as much as 1,024).
// A row tile has two places for scores, so that those of the next 64 tokens are there when the softmax of these is done;
// with two row tiles the tensor core always has one to work on.  A row's sums are only rescaled when its
// maximum has grown by more than 2^SLACK since the last time, which after the first tiles is hardly ever;
// until then weights may pass 1, and their lift leaves room for it.
//
// Every wait is bounded; one that gives up latches CAC_E_TIMEOUT, and the block unwinds.
// Measured: two prompts of 5,001 and 8,000 tokens, 8 K/V heads, group 4, 128 wide, int8, bf16: 688 us, 1.0 PFLOP/s of the
// arithmetic under the mask, tensor core active 43 % of the time.  A 128-token tile takes 4,280 clocks where its products alone take 2,048:
// the scores' operands pass through shared memory at 128 KB a tile beside the converters' 64 KB, and a softmax warp waits for TMEM, the
// maximum and the exponentials in turn.  Some 16,000 clocks of a block are its beginning and end.
// Shared and tensor memory allow one block an SM.  The TMEM is taken after the wait on the
// kernel before and before the next kernel may start, so that no block can hold it
// while it waits for one that needs it.
#include <algorithm>
#include <atomic>

#include "kv8_attn.cuh"

namespace cac {
namespace {

constexpr int PT_ROWS = 128, PT_KEYS = 128, PT_HALF = 64;

template <class T, int HDP> struct PShape {
    static constexpr bool WIDE = sizeof(T) == 4;             // queries and weights as hi + lo
    static constexpr int NM = WIDE && HDP == 128 ? 1 : 2;    // row tiles of a block: what shared memory and TMEM hold
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

// The block's rows and the tokens that any of them sees, in tiles of 128.
struct PWork {
    SeqWork s;
    int head, r0, rows;        // rows r0 .. r0 + rows - 1 of the sequence's m * group
    int lot, skt, tiles;       // the window's first tile, sink tiles before it, tiles in all (0: nothing is seen)
    int halves;                // pieces of 64 tokens in them: the last tile may need one only
    __device__ __forceinline__ int token(int j) const { return (j < skt ? j : lot + j - skt) * PT_KEYS; }
};

template <class T, int CODE, int HDP>
__global__ void __launch_bounds__(PShape<T, HDP>::THREADS, 1)
    kv_prompt_kernel(const __grid_constant__ KvAttend a) {
    using S = PShape<T, HDP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* s_scale = reinterpret_cast<float*>(smem + S::OFF_SC);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);
    uint64_t *q_full = bar, *k_full = bar + 1, *k_empty = bar + 3, *v_full = bar + 5, *v_empty = bar + 7;
    uint64_t *s_full = bar + 9, *p_full = bar + 13, *o_done = bar + 17;  // s_full, p_full, o_done: [row tile][place]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 21);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, D = a.c.head_dim, kvh = a.c.kv_heads;
    pdl_wait();

    // a sequence's last row tiles see the most tokens and go first
    PWork w;
    const int number = (int)(blockIdx.x / kvh), all = (int)(gridDim.x / kvh);
    int2 tile;
    if (a.rows.starts) {
        tile = a.tile_at(all - 1 - number, S::NM * PT_ROWS);
    } else {
        tile = make_int2(number % a.rows.n, all / a.rows.n - 1 - number / a.rows.n);
    }
    if (tile.x < 0) {
        pdl_trigger();
        return;
    }
    w.head = (int)(blockIdx.x % kvh);
    w.s = seq_work(a, tile.x);
    const int R = w.s.m * a.group;
    w.r0 = tile.y * S::NM * PT_ROWS;
    w.rows = min(S::NM * PT_ROWS, R - w.r0);
    w.lot = w.skt = w.tiles = w.halves = 0;
    if (w.rows > 0 && w.s.len > 0) {
        const int p0 = w.s.len - w.s.m + w.r0 / a.group, p1 = w.s.len - w.s.m + (w.r0 + w.rows - 1) / a.group;
        if (p1 >= 0) {
            const int low = a.win.low(max(p0, 0)), high = a.win.high(p1, w.s.len);
            w.lot = low / PT_KEYS;
            w.skt = min((min(a.win.sinks, high) + PT_KEYS - 1) / PT_KEYS, w.lot);
            w.tiles = w.skt + (high + PT_KEYS - 1) / PT_KEYS - w.lot;
            w.halves = 2 * w.tiles - (w.token(w.tiles - 1) + PT_HALF >= high);
        }
    }
    const long long out0 = w.s.row0;
    if (w.tiles == 0) {  // nothing is seen: an empty sequence, one that the call may not name, positions before 0
        pdl_trigger();
        for (int e = threadIdx.x; e < max(w.rows, 0) * D; e += S::THREADS) {
            const int row = w.r0 + e / D, query = a.query_of(row), qh = w.head * a.group + row - query * a.group;
            static_cast<T*>(a.out)[(out0 + query) * a.out_stride + (long long)qh * D + e % D] = from_f<T>(0.f);
            if (a.lse && e % D == 0) a.lse[(out0 + query) * a.heads + qh] = -INFINITY;
        }
        return;
    }
    const int nm = w.rows > PT_ROWS ? 2 : 1;

    if (threadIdx.x == 0) {
        mbar_init(q_full, nm * 4);
        for (int k = 0; k < 2; ++k) {
            mbar_init(k_full + k, 8);
            mbar_init(v_full + k, 8);
            mbar_init(k_empty + k, nm);
            mbar_init(v_empty + k, nm);
            mbar_init(s_full + k, 1);
            mbar_init(s_full + 2 + k, 1);
            mbar_init(p_full + k, 4);
            mbar_init(p_full + 2 + k, 4);
            mbar_init(o_done + k, 1);
            mbar_init(o_done + 2 + k, 1);
        }
        fence_mbar_init();
    }
    if (warp == S::WARPS - 1) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;

    if (warp < S::SOFT) {
        // -------------------------------------------------------------- softmax: a thread per row
        const int x = warp >> 2, r = (warp & 3) * 32 + lane, row = w.r0 + x * PT_ROWS + r;
        if (x < nm) {
            const bool on = row < R;
            const int query = on ? a.query_of(row) : 0, qh = w.head * a.group + (on ? row - query * a.group : 0);
            const int p = w.s.len - w.s.m + query;
            const int low = on && p >= 0 ? a.win.low(p) : 0, high = on && p >= 0 ? a.win.high(p, w.s.len) : 0;
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t col_s = tmem + lanes + S::COL_S + x * 128, col_o = tmem + lanes + S::COL_O + x * HDP;
            const uint32_t col_sum = tmem + lanes + S::COL_SUM + x * HDP;
            // The warp's 32 rows of queries: largest value of a row under 2^15, then fp16 (hi, lo).  CPR lanes load a row, 16 bytes
            // each (a thread per row would touch 32 lines of memory with every load).
            float amax = 0.f;
            {
                constexpr int VEC = 16 / sizeof(T), CPR = HDP / VEC, RPI = 32 / CPR;
                const int c = lane & (CPR - 1), first = x * PT_ROWS + (warp & 3) * 32;
                uint8_t* dst0 = smem + x * S::PARTS * S::TILE + (c * VEC >> 6) * S::PANEL;
                constexpr int GROUP = 8;  // loads on their way at once
#pragma unroll 1
                for (int it0 = 0; it0 < CPR; it0 += GROUP) {
                    uint4 raw[GROUP];
#pragma unroll
                    for (int k = 0; k < GROUP; ++k) {
                        const int row = w.r0 + first + (it0 + k) * RPI + lane / CPR, q = a.query_of(row);
                        const T* src = static_cast<const T*>(a.q) + (out0 + q) * a.q_stride +
                                       (long long)(w.head * a.group + row - q * a.group) * D + c * VEC;
                        raw[k] = row < R && c * VEC < D ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int k = 0; k < GROUP; ++k) {
                        const uint32_t u[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
                        float y[VEC], mx = 0.f;
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            if constexpr (S::WIDE) {
                                y[b] = __uint_as_float(u[b]);
                            } else {
                                y[2 * b] = __uint_as_float(u[b] << 16);
                                y[2 * b + 1] = __uint_as_float(u[b] & 0xffff0000u);
                            }
                        }
#pragma unroll
                        for (int b = 0; b < VEC; ++b) mx = fmaxf(mx, fabsf(y[b]));
#pragma unroll
                        for (int d = CPR / 2; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                        const float of_mine = __shfl_sync(0xffffffffu, mx, (lane & (RPI - 1)) * CPR);
                        if (lane / RPI == it0 + k) amax = of_mine;
                        const float up = lift_to_half(mx) * (a.scale < 0.f ? -1.f : 1.f);
                        const int rr = (warp & 3) * 32 + (it0 + k) * RPI + lane / CPR;
                        uint8_t* dst = dst0 + rr * 128 + (((c * VEC >> 3 & 7) ^ (rr & 7)) << 4);
                        uint32_t hi[VEC / 2], lo[VEC / 2];
#pragma unroll
                        for (int b = 0; b < VEC / 2; ++b) {
                            hi[b] = pack_half(y[2 * b] * up, y[2 * b + 1] * up);
                            if constexpr (S::WIDE) lo[b] = pack_rest(y[2 * b] * up, y[2 * b + 1] * up, hi[b]);
                        }
                        if constexpr (S::WIDE) {
                            *reinterpret_cast<uint2*>(dst + (c & 1) * 8) = make_uint2(hi[0], hi[1]);
                            *reinterpret_cast<uint2*>(dst + S::TILE + (c & 1) * 8) = make_uint2(lo[0], lo[1]);
                        } else {
                            *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        }
                    }
                }
            }
            const float f = fabsf(a.scale) * LOG2E / lift_to_half(amax);  // a power of two: exact
            fence_proxy_async_smem();
            warp_arrive(q_full);

            float m = -INFINITY, l = 0.f;
            for (int h = 0; h < w.halves; ++h) {
                const int j = h >> 1, tok = w.token(j) + (h & 1) * PT_HALF;
                const uint32_t col = col_s + (h & 1) * PT_HALF;
                const float4* sc = reinterpret_cast<const float4*>(s_scale + (j & 3) * 24 + (h & 1) * 4);
                if (!warp_wait(s_full + 2 * x + (h & 1), j & 1)) { ok = false; break; }
                tc_fence_after();
                const float4 ks4 = sc[0], lv4 = sc[2], iv4 = sc[4];
                // Above 0 even where the product underflows (a query of zeros over a block of zeros) or the call's scale is 0: unseen
                // tokens score -inf before they are multiplied.  A score is under 2^31 there, so FLT_MIN times it is nothing.
                const float ks[4] = {fmaxf(ks4.x * f, FLT_MIN), fmaxf(ks4.y * f, FLT_MIN), fmaxf(ks4.z * f, FLT_MIN),
                                     fmaxf(ks4.w * f, FLT_MIN)},
                            lv[4] = {lv4.x, lv4.y, lv4.z, lv4.w}, iv[4] = {iv4.x, iv4.y, iv4.z, iv4.w};
                float v[PT_HALF];
                tmem_ld64(col, v);
                // a token that the row does not see scores -inf
                if (!__all_sync(0xffffffffu, tok + PT_HALF <= high && (tok >= low || tok + PT_HALF <= a.win.sinks))) {
#pragma unroll
                    for (int k = 0; k < PT_HALF; ++k) {
                        const int t = tok + k;
                        if (!(t < high && (t >= low || t < a.win.sinks))) v[k] = -INFINITY;
                    }
                }
                float top = -INFINITY, mb[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) mb[b] = fmaxf(v[16 * b], v[16 * b + 1]);
#pragma unroll
                for (int k = 2; k < 16; k += 2)
#pragma unroll
                    for (int b = 0; b < 4; ++b) mb[b] = max3(mb[b], v[16 * b + k], v[16 * b + k + 1]);
#pragma unroll
                for (int b = 0; b < 4; ++b) top = fmaxf(top, fmaf(mb[b], ks[b], lv[b]));
                const bool grown = top > m + S::SLACK || (m == -INFINITY && top > m);
                if (__any_sync(0xffffffffu, grown)) {
                    const float d = grown ? m - top : 0.f, r = ex2(d);
                    l = move_norm(l, d, r);
                    m = grown ? top : m;
                    __syncwarp();  // the tensor-memory instructions are for a converged warp
                    if (h > 0) {
                        if (!warp_wait(o_done + 2 * x + ((h - 1) & 1), (h - 1) >> 1 & 1)) { ok = false; break; }  // the sums so far are in
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < HDP; c += 16) {
                            scale16(col_o + c, r);
                            if (S::WIDE && h > S::FLUSH) scale16(col_sum + c, r);
                        }
                        if (S::WIDE) tmem_st_wait();  // the flush below loads these columns, and loads do not wait for stores
                    }
                }
                if (S::WIDE && h > 0 && h % S::FLUSH == 0) {
                    if (!warp_wait(o_done + 2 * x + ((h - 1) & 1), (h - 1) >> 1 & 1)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < HDP; c += 16) {
                        float o[16], sum[16] = {};
                        uint32_t u[16];
                        if (h > S::FLUSH) tmem_ld16(col_sum + c, sum);
                        tmem_ld16(col_o + c, o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(o[k] + sum[k]);
                        tmem_st16(col_sum + c, u);
                    }
                }
                const float base = m == -INFINITY ? -S::LIFT : m - S::LIFT;
                // one kind of instruction at a time, none of which waits for another of its kind: a warp has little else to hide
                // their latencies behind
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float off = lv[b] - base;
#pragma unroll
                    for (int k = 16 * b; k < 16 * b + 16; k += 2) {
                        const float2 y = fma2(make_float2(v[k], v[k + 1]), make_float2(ks[b], ks[b]), make_float2(off, off));
                        v[k] = y.x, v[k + 1] = y.y;
                    }
                }
                if (fminf(fminf(lv[0], lv[1]), fminf(lv[2], lv[3])) < FAR) {
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        if (lv[b] < FAR && lv[b] != -INFINITY) {
                            float x = 0.f;
#pragma unroll
                            for (int k = 16 * b; k < 16 * b + 16; ++k) x += ex2(v[k] - lv[b]);
                            l = fmaf(x, S::NORM, l);
                        }
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int k = 32 * c; k < 32 * c + 32; ++k) v[k] = ex2(v[k]);
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        hi[k] = pack_half(v[32 * c + 2 * k], v[32 * c + 2 * k + 1]);
                        if constexpr (S::WIDE) lo[k] = pack_rest(v[32 * c + 2 * k], v[32 * c + 2 * k + 1], hi[k]);
                    }
                    tmem_st16(col + c * 16, hi);
                    if constexpr (S::WIDE) tmem_st16(col + 32 + c * 16, lo);
#pragma unroll
                    for (int b = 2 * c; b < 2 * c + 2; ++b) {
                        float2 sum[4];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float2 y = make_float2(v[16 * b + 2 * k], v[16 * b + 2 * k + 1]);
                            sum[k & 3] = k < 4 ? y : add2(sum[k & 3], y);
                        }
                        const float2 all = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                        l = fmaf((all.x + all.y) * S::NORM, iv[b], l);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(p_full + 2 * x + (h & 1));
            }
            for (int h = max(w.halves - 2, 0); h < w.halves; ++h)
                if (ok && !warp_wait(o_done + 2 * x + (h & 1), h >> 1 & 1)) ok = false;
            tc_fence_after();
            if (ok) {
                const bool seen = l > 0.f || l != l;
                const float inv = seen ? 1.f / l : 0.f;
                T* dst = static_cast<T*>(a.out) + (out0 + query) * a.out_stride + (long long)qh * D;
#pragma unroll
                for (int c = 0; c < HDP / 32; ++c) {
                    float v[32];
                    __syncwarp();  // rows past the last one stored nothing; the loads are for a converged warp
                    tmem_ld32(col_o + c * 32, v);
                    if (S::WIDE && w.halves > S::FLUSH) {
                        float sum[32];
                        tmem_ld32(col_sum + c * 32, sum);
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] += sum[k];
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] *= S::NORM;
                    if (!on) continue;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (c * 32 + h * 16 >= D) continue;
                        T* q = dst + c * 32 + h * 16;
                        if constexpr (S::WIDE) {
#pragma unroll
                            for (int k = 0; k < 16; k += 4)
                                *reinterpret_cast<float4*>(q + k) = make_float4(v[16 * h + k] * inv, v[16 * h + k + 1] * inv,
                                                                                v[16 * h + k + 2] * inv, v[16 * h + k + 3] * inv);
                        } else {
#pragma unroll
                            for (int k = 0; k < 16; k += 8) {
                                uint32_t u[4];
#pragma unroll
                                for (int b = 0; b < 4; ++b) {
                                    const __nv_bfloat162 y =
                                        __floats2bfloat162_rn(v[16 * h + k + 2 * b] * inv, v[16 * h + k + 2 * b + 1] * inv);
                                    u[b] = *reinterpret_cast<const uint32_t*>(&y);
                                }
                                *reinterpret_cast<uint4*>(q + k) = make_uint4(u[0], u[1], u[2], u[3]);
                            }
                        }
                    }
                }
                if (on && a.lse) a.lse[(out0 + query) * a.heads + qh] = seen ? (m + NORM_LOG2 + log2f(l)) * LN2 : -INFINITY;
            }
        }
    } else if (warp < S::SOFT + S::CONV) {
        // -------------------------------------------------------------- converters
        // piece n: 16 tokens (block n % 8) of tile n / 16, K where n / 8 is even, else V; warp cw takes every CONV-th
        const int cw = warp - S::SOFT, pieces = w.tiles * 16;
        const int sub = lane >> 2, c4 = lane & 3;   // token % 8 and chunk % 4 of a lane's loads
        constexpr int NL = HDP / 32;
        // Lane l knows where the warp's l-th piece of the next 32 lies, and its scales (with K: the scores need both).
        struct Spot {
            long long at;      // -1: past the end, or no page
            float ks, lv, iv;
        };
        auto look = [&](int n) {
            Spot t{-1, 1.f, -INFINITY, 0.f};  // a block without a page: any K scale will do, its weights are 2^-inf
            const int tok = n < pieces ? w.token(n >> 4) + (n & 7) * KV_BLOCK : w.s.len;
            if (tok < w.s.len) {
                const int page = a.c.table[(long long)w.s.id * a.c.max_pages + tok / a.c.page_tokens];
                if (page >= 0) {
                    const int in_page = tok % a.c.page_tokens;
                    t.at = kv_head_at(a.c, a.layer, page, w.head) + (long long)in_page * D;
                    if (!(n & 8)) {
                        const long long sc = kv_scale_at(a.c, a.layer, page, w.head) + in_page / KV_BLOCK;
                        t.ks = a.c.k_scale[sc];
                        t.lv = log2f(a.c.v_scale[sc]);
                        t.iv = t.lv < FAR ? 0.f : ex2(-t.lv);
                    }
                }
            }
            return t;
        };
        Spot here = look(cw + S::CONV * lane);
        const int lane_at = sub * D + c4 * 16;
        const uint8_t *k_lane = static_cast<const uint8_t*>(a.c.k) + lane_at, *v_lane = static_cast<const uint8_t*>(a.c.v) + lane_at;
        auto load = [&](int n, long long at, uint4 (&raw)[NL]) {
            const uint8_t* from = (n & 8 ? v_lane : k_lane) + at;
            // rows sub and sub + 8, elements of each 64; past the end of the sequence the codes may be anything, NaN among them
            const int left = at >= 0 ? w.s.len - w.token(n >> 4) - (n & 7) * KV_BLOCK - sub : 0;
#pragma unroll
            for (int y = 0; y < NL; ++y)
                raw[y] = left > (y & 1) * 8 && ((y >> 1) * 4 + c4) * 16 < D
                             ? *reinterpret_cast<const uint4*>(from + (y & 1) * 8 * D + (y >> 1) * 64)
                             : make_uint4(0, 0, 0, 0);
        };
        uint4 raw[2][NL];
        load(cw, __shfl_sync(0xffffffffu, here.at, 0), raw[0]);
        Spot then = here;
        int q = 0;  // the piece's place among the 32
        auto piece = [&](int n, uint4 (&cur)[NL], uint4 (&nxt)[NL]) {
            const float ks = __shfl_sync(0xffffffffu, here.ks, q), lv = __shfl_sync(0xffffffffu, here.lv, q),
                        iv = __shfl_sync(0xffffffffu, here.iv, q);
            if (++q == 32) {
                q = 0;
                here = then;
            }
            if (q == 8) then = look(n + S::CONV * (25 + lane));  // the 32 after these: not before the first are on their way
            load(n + S::CONV, __shfl_sync(0xffffffffu, here.at, q), nxt);
            const int j = n >> 4, st = j & 1, block = n & 7;
            const bool v = n & 8;
            if (j >= 2 && !warp_wait((v ? v_empty : k_empty) + st, (j / 2 - 1) & 1)) return false;
            uint8_t* to = smem + (v ? S::OFF_V : S::OFF_K) + st * S::TILE + (block * 16 + sub) * 128;
#pragma unroll
            for (int y = 0; y < NL; ++y) {
                const uint32_t u[4] = {cur[y].x, cur[y].y, cur[y].z, cur[y].w};
                uint32_t h[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) half4<CODE>(u[k], h[2 * k], h[2 * k + 1]);
                uint8_t* dst = to + (y >> 1) * S::PANEL + (y & 1) * 1024;
                *reinterpret_cast<uint4*>(dst + (((2 * c4) ^ sub) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(dst + (((2 * c4 + 1) ^ sub) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (!v) {
                    float* sc = s_scale + (j & 3) * 24 + block;
                    sc[0] = ks, sc[8] = lv, sc[16] = iv;
                }
                mbar_arrive((v ? v_full : k_full) + st);
            }
            return true;
        };
#pragma unroll 1
        for (int n = cw; n < pieces; n += 2 * S::CONV) {
            if (!piece(n, raw[0], raw[1])) { ok = false; break; }
            if (n + S::CONV < pieces && !piece(n + S::CONV, raw[1], raw[0])) { ok = false; break; }
        }
    } else {
        // -------------------------------------------------------------- MMA: a thread per row tile
        const int x = warp - S::SOFT - S::CONV;
        if (lane == 0 && x < nm) {
            constexpr uint32_t qk = idesc_f16(128, PT_HALF, false), pv = idesc_f16(128, HDP, true);
            auto scores = [&](int h) {
                const uint64_t kd = sdesc_k_sw128(smem + S::OFF_K + (h >> 1 & 1) * S::TILE + (h & 1) * (PT_HALF * 128));
#pragma unroll
                for (int part = 0; part < S::PARTS; ++part) {
                    const uint64_t qd = sdesc_k_sw128(smem + (x * S::PARTS + part) * S::TILE);
#pragma unroll
                    for (int k = 0; k < HDP / 16; ++k) {
                        const uint32_t step = (k >> 2) * (S::PANEL >> 4) + 2 * (k & 3);
                        mma_ss(tmem + S::COL_S + x * 128 + (h & 1) * PT_HALF, qd + step, kd + step, qk, part > 0 || k > 0);
                    }
                }
                tc_commit(s_full + 2 * x + (h & 1));
                if (h & 1) tc_commit(k_empty + (h >> 1 & 1));
            };
            ok = mbar_wait(q_full, 0) && mbar_wait(k_full, 0);
            if (ok) {
                tc_fence_after();
                scores(0);
            }
            for (int h = 0; ok && h < w.halves; ++h) {
                const int st = h >> 1 & 1, next = h + 1;
                if (next < w.halves) {
                    // the next scores take the place of the weights before these: products into other accumulators need
                    // not run in order
                    if ((!(next & 1) && !mbar_wait(k_full + (next >> 1 & 1), next >> 2 & 1)) ||
                        (h > 0 && !mbar_wait(o_done + 2 * x + ((h - 1) & 1), (h - 1) >> 1 & 1))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    scores(next);
                }
                if ((!(h & 1) && !mbar_wait(v_full + st, h >> 2 & 1)) || !mbar_wait(p_full + 2 * x + (h & 1), h >> 1 & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t vd = sdesc_mn_sw128(smem + S::OFF_V + st * S::TILE + (h & 1) * (PT_HALF * 128), S::PANEL);
#pragma unroll
                for (int part = 0; part < S::PARTS; ++part)
#pragma unroll
                    for (int k = 0; k < PT_HALF / 16; ++k)
                        mma_ts(tmem + S::COL_O + x * HDP, tmem + S::COL_S + x * 128 + (h & 1) * PT_HALF + part * 32 + 8 * k,
                               vd + k * (2048 >> 4), pv, h % S::FLUSH > 0 || part > 0 || k > 0);
                tc_commit(o_done + 2 * x + (h & 1));
                if (h & 1) tc_commit(v_empty + st);
            }
        }
    }
    if (!ok) latch_error(a.c.status, CAC_E_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == S::WARPS - 1) tmem_dealloc(tmem, 512);
}

template <class T, int CODE, int HDP> cudaError_t launch_prompt(const KvAttend& a, cudaStream_t s) {
    using S = PShape<T, HDP>;
    const auto kernel = kv_prompt_kernel<T, CODE, HDP>;
    static std::atomic<uint64_t> ready{0};
    const uint64_t bit = 1ull << (a.c.device & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    const unsigned blocks = (unsigned)a.tiles_of_all(S::NM * PT_ROWS) * a.c.kv_heads;
    return launch_k(kernel, dim3(blocks), dim3(S::THREADS), S::SMEM, s, 1, a);
}
template <class T, int CODE> cudaError_t launch_prompt(const KvAttend& a, cudaStream_t s) {
    return a.c.head_dim <= 64 ? launch_prompt<T, CODE, 64>(a, s) : launch_prompt<T, CODE, 128>(a, s);
}

}  // namespace

// Against kv_attend_kernel, which deals 16-row tiles out over the whole card (and re-reads K and V for each): a 128-token tile of a
// block here takes as long as it takes an SM for two to three of its 16-row tiles, but the card fills in steps of a block an SM.  Measured
// (bf16, group 4, head_dim 128; us for 16 / 32 / 64 / 128 / 256 rows): 32 sequences of 4,000 tokens, 8 K/V heads,
// 87 / 130 / 223 / 404 / 764 there, 155 / 156 / 155 / 155 / 172 here; 4 of 8,000, 41 / 55 / 81 / 128 / 217 and 128 / 127 /
// 127 / 122 / 140; one of 30,000, 2 heads, 31 / 33 / 38 / 49 / 70 and 454 / 454 / 455 / 424 / 489; 64 of 1,000, 8 heads of 64, group 1,
// 39 / 53 / 84 for 16 / 32 / 64 rows and 75 here.  The ratio at the crossings is 1.6 to 2.8.
bool kv_prompt_takes(const KvAttend& a, int dtype, int sms, long long rows) {
    if (a.c.head_dim > 128) return false;
    const int block = dtype == CAC_DTYPE_F32 && a.c.head_dim > 64 ? PT_ROWS : 2 * PT_ROWS;
    const long long units = (long long)a.rows.n * a.c.kv_heads;
    const long long waves = (units * ((rows + block - 1) / block) + sms - 1) / sms;
    return units * ((rows + 15) / 16) > 2 * waves * sms;
}

cudaError_t kv_launch_prompt(const KvAttend& a, int dtype, cudaStream_t s) {
    if (a.c.code == CAC_KV8_INT8)
        return dtype == CAC_DTYPE_BF16 ? launch_prompt<bf16, CAC_KV8_INT8>(a, s) : launch_prompt<float, CAC_KV8_INT8>(a, s);
    return dtype == CAC_DTYPE_BF16 ? launch_prompt<bf16, CAC_KV8_E4M3>(a, s) : launch_prompt<float, CAC_KV8_E4M3>(a, s);
}

}  // namespace cac
