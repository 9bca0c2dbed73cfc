// Attention over the paged 8-bit K/V cache for calls with many query rows to a K/V head
// (prompts and pieces of them), on the 5th-generation tensor cores.  The mathematics is that of
// kv8_attn.cu: codes enter as exact fp16, the block scales sit in the exponent.
//
// Arithmetic bounds it: 4 * head_dim operations a pair of query and token.  A block takes
// NM tiles of 128 query rows (row = query * group + head of the group, so the heads that share K and V
// share the tile too) of one sequence and K/V head, and walks over its 128-token tiles:
//   converters  7 warps, 16 tokens of K or of V at a time in turn: 16-byte loads of codes, the next piece
//               under way, turned into fp16 in the 128-byte-swizzled layout that the tensor core reads
//               (K as [token][element]: its rows are the columns of the scores; V the same
//               way, read with the token as the contracted index), a ring of two tiles each
//   MMA         1 thread: S = Q K^T into TMEM, O += P V with P from TMEM
//   softmax     4 warps for each row tile, a thread per row: the 128 scores from TMEM into registers, maximum, weights
//               back into TMEM in place of the scores, row sums.  These threads take over registers
//               of the others (setmaxnreg), so that the scores are read once.
// With two row tiles the tensor core works on one while the softmax of the other runs.  A
// row's sums are only rescaled when its maximum has grown by more than 2^SLACK since the last
// time, which after the first tiles is hardly ever; until then weights may pass 1, and
// their lift leaves room for it.
//
// Every wait is bounded; one that gives up latches CAC_E_TIMEOUT, and the block unwinds.
// Shared and tensor memory allow one block an SM.  The TMEM is taken after the wait on the
// kernel before and before the next kernel may start, so that no block can hold it
// while it waits for one that needs it.
#include <algorithm>
#include <atomic>

#include "kv8_attn.cuh"

namespace cac {
namespace {

constexpr int PT_ROWS = 128, PT_KEYS = 128;

template <class T, int HDP> struct PShape {
    static constexpr bool WIDE = sizeof(T) == 4;             // queries and weights as hi + lo
    static constexpr int NM = WIDE && HDP == 128 ? 1 : 2;    // row tiles of a block: what shared memory and TMEM hold
    static constexpr int PARTS = WIDE ? 2 : 1;
    static constexpr int PANEL = 128 * 128;                  // 128 rows of 64 fp16
    static constexpr int TILE = HDP / 64 * PANEL;
    static constexpr int OFF_K = NM * PARTS * TILE, OFF_V = OFF_K + 2 * TILE, OFF_SC = OFF_V + 2 * TILE;
    static constexpr int OFF_BAR = OFF_SC + 4 * 24 * 4;      // [4 tiles][K scale, log2 and reciprocal of V scale][8]
    static constexpr int BYTES = OFF_BAR + 16 * 8 + 16 + 1024;
    static constexpr int SMEM = BYTES > 120 * 1024 ? BYTES : 120 * 1024;  // one block an SM
    static constexpr int SOFT = NM * 4, CONV = 7, WARPS = SOFT + CONV + 1, THREADS = WARPS * 32;
    // registers: a launch gets 65,536 / THREADS each, in steps of 8 (128 of 512 threads, 168 of 384); the split may not pass that sum
    static constexpr int LAUNCH = NM == 2 ? 128 : 168, R_SOFT = NM == 2 ? 200 : 232, R_REST = NM == 2 ? 56 : 136;
    static_assert(SOFT * R_SOFT + (WARPS - SOFT) * R_REST <= WARPS * LAUNCH, "registers");
    static_assert(WARPS * 32 * LAUNCH <= 65536 && WARPS % 4 == 0, "registers");
    // TMEM columns: scores (128 each), sums (HDP each), fp32's low halves of the weights (64 each)
    static constexpr int COL_S = 0, COL_O = NM * 128, COL_L = COL_O + NM * HDP;
    static_assert(COL_L + (WIDE ? NM * 64 : 0) <= 512, "TMEM");
    static constexpr float SLACK = WIDE ? 2.f : 8.f, LIFT = 15.f - SLACK;
};

template <int N> __device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

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
// 32 columns of the thread's lane, not yet there: tmem_arrived() makes them so
__device__ __forceinline__ void tmem_ld32_start(uint32_t addr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(addr)
        : "memory");
}
template <int N> __device__ __forceinline__ void tmem_arrived(float (&v)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int k = 0; k < N; k += 16)  // no use of them may move above the wait
        asm volatile("" : "+f"(v[k]), "+f"(v[k + 1]), "+f"(v[k + 2]), "+f"(v[k + 3]), "+f"(v[k + 4]), "+f"(v[k + 5]),
                          "+f"(v[k + 6]), "+f"(v[k + 7]), "+f"(v[k + 8]), "+f"(v[k + 9]), "+f"(v[k + 10]), "+f"(v[k + 11]),
                          "+f"(v[k + 12]), "+f"(v[k + 13]), "+f"(v[k + 14]), "+f"(v[k + 15]));
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
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// mbar_wait by a whole warp, with one answer for all of it
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// The block's rows and the tokens that any of them sees, in tiles of 128.
struct PWork {
    SeqWork s;
    int head, r0, rows;        // rows r0 .. r0 + rows - 1 of the sequence's m * group
    int lot, skt, tiles;       // the window's first tile, sink tiles before it, tiles in all (0: nothing is seen)
    __device__ __forceinline__ int token(int j) const { return (j < skt ? j : lot + j - skt) * PT_KEYS; }
};

template <class T, int CODE, int HDP>
__global__ void __launch_bounds__(PShape<T, HDP>::THREADS, 1)
    kv_prompt_kernel(const __grid_constant__ KvAttend a, int row_tiles) {
    using S = PShape<T, HDP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* s_scale = reinterpret_cast<float*>(smem + S::OFF_SC);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);
    uint64_t *q_full = bar, *k_full = bar + 1, *k_empty = bar + 3, *v_full = bar + 5, *v_empty = bar + 7;
    uint64_t *s_full = bar + 9, *p_full = bar + 11, *o_full = bar + 13;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 16);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, D = a.c.head_dim, kvh = a.c.kv_heads;
    pdl_wait();

    // the last row tiles see the most tokens and go first
    PWork w;
    const int per = a.rows.n * kvh;
    int tile = row_tiles - 1 - (int)(blockIdx.x / per);
    w.head = (int)(blockIdx.x % per) % kvh;
    w.s = seq_work(a, (int)(blockIdx.x % per) / kvh);
    const int R = w.s.m * a.group;
    w.r0 = tile * S::NM * PT_ROWS;
    w.rows = min(S::NM * PT_ROWS, R - w.r0);
    w.lot = w.skt = w.tiles = 0;
    if (w.rows > 0 && w.s.len > 0) {
        const int p0 = w.s.len - w.s.m + w.r0 / a.group, p1 = w.s.len - w.s.m + (w.r0 + w.rows - 1) / a.group;
        if (p1 >= 0) {
            const int low = a.win.low(max(p0, 0)), high = a.win.high(p1, w.s.len);
            w.lot = low / PT_KEYS;
            w.skt = min((min(a.win.sinks, high) + PT_KEYS - 1) / PT_KEYS, w.lot);
            w.tiles = w.skt + (high + PT_KEYS - 1) / PT_KEYS - w.lot;
        }
    }
    const long long out0 = w.s.row0;
    if (w.tiles == 0) {  // nothing is seen: an empty sequence, one that the call may not name, positions before 0
        pdl_trigger();
        const int step = w.s.len > 0 ? 1 << 30 : row_tiles * S::NM * PT_ROWS;  // a count above max_new has rows past the last tile
        for (long long r0 = w.r0; r0 < R; r0 += step)
            for (int e = threadIdx.x; e < min(S::NM * PT_ROWS, (int)(R - r0)) * D; e += S::THREADS) {
                const int row = (int)r0 + e / D, query = row / a.group, qh = w.head * a.group + row - query * a.group;
                static_cast<T*>(a.out)[(out0 + query) * a.out_stride + (long long)qh * D + e % D] = from_f<T>(0.f);
                if (a.lse && e % D == 0) a.lse[(out0 + query) * a.heads + qh] = -INFINITY;
            }
        return;
    }
    const int nm = w.rows > PT_ROWS ? 2 : 1;

    if (threadIdx.x == 0) {
        mbar_init(q_full, nm * 128);
        for (int k = 0; k < 2; ++k) {
            mbar_init(k_full + k, 8);
            mbar_init(v_full + k, 8);
            mbar_init(k_empty + k, 1);
            mbar_init(v_empty + k, 1);
            mbar_init(s_full + k, 1);
            mbar_init(p_full + k, 128);
        }
        mbar_init(o_full, 1);
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
        take_registers<S::R_SOFT>();
        // -------------------------------------------------------------- softmax: a thread per row
        const int x = warp >> 2, r = (warp & 3) * 32 + lane, row = w.r0 + x * PT_ROWS + r;
        if (x < nm) {
            const bool on = row < R;
            const int query = on ? row / a.group : 0, qh = w.head * a.group + (on ? row - query * a.group : 0);
            const int p = w.s.len - w.s.m + query;
            const int low = on && p >= 0 ? a.win.low(p) : 0, high = on && p >= 0 ? a.win.high(p, w.s.len) : 0;
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t col_s = tmem + lanes + S::COL_S + x * 128, col_o = tmem + lanes + S::COL_O + x * HDP;
            // the row's queries: largest value under 2^15, then fp16 (hi, lo)
            float f;
            {
                const T* src = static_cast<const T*>(a.q) + (out0 + query) * a.q_stride + (long long)qh * D;
                constexpr int VEC = 16 / sizeof(T);  // values of a 16-byte load
                uint4 raw[HDP / VEC];
#pragma unroll
                for (int c = 0; c < HDP / VEC; ++c)
                    raw[c] = on && c * VEC < D ? *reinterpret_cast<const uint4*>(src + c * VEC) : make_uint4(0, 0, 0, 0);
                auto value = [&](int e) {
                    const uint4& q = raw[e / VEC];
                    const int k = e % VEC, wd = S::WIDE ? k : k >> 1;
                    const uint32_t u = wd == 0 ? q.x : wd == 1 ? q.y : wd == 2 ? q.z : q.w;
                    return __uint_as_float(S::WIDE ? u : k & 1 ? u & 0xffff0000u : u << 16);
                };
                float amax = 0.f;
#pragma unroll
                for (int e = 0; e < HDP; ++e) amax = fmaxf(amax, fabsf(value(e)));
                const int e = min(268 - (int)(__float_as_uint(amax) >> 23), 254);
                const float up = __uint_as_float((uint32_t)e << 23) * (a.scale < 0.f ? -1.f : 1.f);
                f = fabsf(a.scale) * LOG2E * __uint_as_float((uint32_t)max(254 - e, 1) << 23) * (e == 254 ? 0.5f : 1.f);
#pragma unroll
                for (int c = 0; c < HDP / 8; ++c) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float y0 = value(8 * c + 2 * k) * up, y1 = value(8 * c + 2 * k + 1) * up;
                        hi[k] = pack_half(y0, y1);
                        if constexpr (S::WIDE) lo[k] = pack_rest(y0, y1, hi[k]);
                    }
                    uint8_t* dst = smem + x * S::PARTS * S::TILE + (c >> 3) * S::PANEL + r * 128 + (((c & 7) ^ (r & 7)) << 4);
                    *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if constexpr (S::WIDE) *reinterpret_cast<uint4*>(dst + S::TILE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(q_full);

            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < w.tiles; ++j) {
                const int tok = w.token(j);
                const float* sc = s_scale + (j & 3) * 24;
                if (!warp_wait(s_full + x, j & 1)) { ok = false; break; }
                tc_fence_after();
                float v[PT_KEYS];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32_start(col_s + c * 32, v + c * 32);
                tmem_arrived(v);
                // a token that the row does not see scores -inf
                if (!__all_sync(0xffffffffu, tok + PT_KEYS <= high && (tok >= low || tok + PT_KEYS <= a.win.sinks))) {
#pragma unroll
                    for (int k = 0; k < PT_KEYS; ++k) {
                        const int t = tok + k;
                        if (!(t < high && (t >= low || t < a.win.sinks))) v[k] = -INFINITY;
                    }
                }
                float top = -INFINITY;
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    float m0 = fmaxf(v[16 * b], v[16 * b + 1]), m1 = fmaxf(v[16 * b + 2], v[16 * b + 3]);
#pragma unroll
                    for (int k = 4; k < 16; k += 4) {
                        m0 = fmaxf(fmaxf(m0, v[16 * b + k]), v[16 * b + k + 1]);
                        m1 = fmaxf(fmaxf(m1, v[16 * b + k + 2]), v[16 * b + k + 3]);
                    }
                    top = fmaxf(top, fmaf(fmaxf(m0, m1), f * sc[b], sc[8 + b]));
                }
                const bool grown = top > m + S::SLACK || (m == -INFINITY && top > m);
                if (__any_sync(0xffffffffu, grown)) {
                    const float r = grown ? ex2(m - top) : 1.f;
                    if (grown) m = top, l *= r;
                    if (j > 0) {
#pragma unroll
                        for (int c = 0; c < HDP / 32; ++c) {
                            float v[32];
                            tmem_ld32(col_o + c * 32, v);
                            uint32_t u[16];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
#pragma unroll
                                for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(v[16 * h + k] * r);
                                tmem_st16(col_o + c * 32 + 16 * h, u);
                            }
                        }
                    }
                }
                const float base = m == -INFINITY ? -S::LIFT : m - S::LIFT;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int b = 2 * c; b < 2 * c + 2; ++b) {
                        const float ck = f * sc[b], off = sc[8 + b] - base;
                        const float2 ck2 = make_float2(ck, ck), off2 = make_float2(off, off);
                        float2 sum[2];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            float2 y = fma2(make_float2(v[16 * b + 2 * k], v[16 * b + 2 * k + 1]), ck2, off2);
                            y.x = ex2(y.x), y.y = ex2(y.y);
                            sum[k & 1] = k < 2 ? y : add2(sum[k & 1], y);
                            hi[8 * (b & 1) + k] = pack_half(y.x, y.y);
                            if constexpr (S::WIDE) lo[8 * (b & 1) + k] = pack_rest(y.x, y.y, hi[8 * (b & 1) + k]);
                        }
                        const float2 all = add2(sum[0], sum[1]);
                        l = fmaf(all.x + all.y, sc[16 + b], l);
                    }
                    tmem_st16(col_s + c * 16, hi);
                    if constexpr (S::WIDE) tmem_st16(tmem + lanes + S::COL_L + x * 64 + c * 16, lo);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(p_full + x);
            }
            if (ok && !warp_wait(o_full, 0)) ok = false;
            tc_fence_after();
            if (ok) {
                const bool seen = l > 0.f || l != l;
                const float inv = seen ? 1.f / l : 0.f;
                T* dst = static_cast<T*>(a.out) + (out0 + query) * a.out_stride + (long long)qh * D;
#pragma unroll
                for (int c = 0; c < HDP / 32; ++c) {
                    float v[32];
                    tmem_ld32(col_o + c * 32, v);
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
                if (on && a.lse) a.lse[(out0 + query) * a.heads + qh] = seen ? (m - S::LIFT + log2f(l)) * LN2 : -INFINITY;
            }
        }
    } else if (warp < S::SOFT + S::CONV) {
        give_registers<S::R_REST>();
        // -------------------------------------------------------------- converters
        // piece n: 16 tokens (block n % 8) of tile n / 16, K where n / 8 is even, else V; warp cw takes every seventh
        const int cw = warp - S::SOFT, pieces = w.tiles * 16;
        const int sub = lane >> 2, c4 = lane & 3;   // token % 8 and chunk % 4 of a lane's loads
        constexpr int NL = HDP / 32;
        auto page_of = [&](int n) {  // -1: past the end, or released
            const int tok = n < pieces ? w.token(n >> 4) + (n & 7) * KV_BLOCK : w.s.len;
            return tok < w.s.len ? a.c.table[(long long)w.s.id * a.c.max_pages + tok / a.c.page_tokens] : -1;
        };
        auto load = [&](int n, int page, uint4 (&raw)[NL], float2& scale) {
            const int in_page = (w.token(n >> 4) + (n & 7) * KV_BLOCK) % a.c.page_tokens;
            const uint8_t* from = static_cast<const uint8_t*>(n & 8 ? a.c.v : a.c.k);
            if (page >= 0) {
                from += kv_head_at(a.c, a.layer, page, w.head) + (long long)(in_page + sub) * D + c4 * 16;
                const long long sc = kv_scale_at(a.c, a.layer, page, w.head) + in_page / KV_BLOCK;
                if (!(n & 8)) scale = make_float2(a.c.k_scale[sc], a.c.v_scale[sc]);
            }
#pragma unroll
            for (int y = 0; y < NL; ++y)  // rows sub and sub + 8, elements of each 64
                raw[y] = page >= 0 && ((y >> 1) * 4 + c4) * 16 < D
                             ? *reinterpret_cast<const uint4*>(from + (y & 1) * 8 * D + (y >> 1) * 64)
                             : make_uint4(0, 0, 0, 0);
        };
        int page = page_of(cw), page1 = page_of(cw + S::CONV);
        uint4 raw[NL], next[NL];
        float2 scale = make_float2(0.f, 0.f), scale1 = scale;
        load(cw, page, raw, scale);
#pragma unroll 1
        for (int n = cw; n < pieces; n += S::CONV) {
            const int page2 = page_of(n + 2 * S::CONV);
            load(min(n + S::CONV, pieces - 1), n + S::CONV < pieces ? page1 : -1, next, scale1);
            const int j = n >> 4, st = j & 1, block = n & 7;
            const bool v = n & 8;
            if (j >= 2 && !warp_wait((v ? v_empty : k_empty) + st, (j / 2 - 1) & 1)) { ok = false; break; }
            uint8_t* to = smem + (v ? S::OFF_V : S::OFF_K) + st * S::TILE + (block * 16 + sub) * 128;
#pragma unroll
            for (int y = 0; y < NL; ++y) {
                const uint32_t u[4] = {raw[y].x, raw[y].y, raw[y].z, raw[y].w};
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
                if (!v) {  // both scales with K: the scores need them.  A block without a page: weights of 2^-inf
                    float* sc = s_scale + (j & 3) * 24 + block;
                    const float lv = log2f(scale.y) + (CODE == CAC_KV8_INT8 ? 0.f : 8.f);
                    sc[0] = page >= 0 ? scale.x * code_unit<CODE>() : 1.f;
                    sc[8] = page >= 0 ? lv : -INFINITY;
                    sc[16] = page >= 0 ? ex2(-lv) : 0.f;
                }
                mbar_arrive((v ? v_full : k_full) + st);
            }
            page = page1, page1 = page2, scale = scale1;
#pragma unroll
            for (int y = 0; y < NL; ++y) raw[y] = next[y];
        }
    } else {
        give_registers<S::R_REST>();
        if (lane == 0) {
        // -------------------------------------------------------------- MMA
        constexpr uint32_t qk = idesc_f16(128, 128, false), pv = idesc_f16(128, HDP, true);
        auto scores = [&](int x, int st) {
            const uint64_t kd = sdesc_k_sw128(smem + S::OFF_K + st * S::TILE);
#pragma unroll
            for (int part = 0; part < S::PARTS; ++part) {
                const uint64_t qd = sdesc_k_sw128(smem + (x * S::PARTS + part) * S::TILE);
#pragma unroll
                for (int k = 0; k < HDP / 16; ++k) {
                    const uint32_t step = (k >> 2) * (S::PANEL >> 4) + 2 * (k & 3);
                    mma_ss(tmem + S::COL_S + x * 128, qd + step, kd + step, qk, part > 0 || k > 0);
                }
            }
            tc_commit(s_full + x);
        };
        if (!mbar_wait(q_full, 0) || !mbar_wait(k_full, 0)) ok = false;
        if (ok) {
            tc_fence_after();
            for (int x = 0; x < nm; ++x) scores(x, 0);
            tc_commit(k_empty);
        }
        for (int j = 0; ok && j < w.tiles; ++j) {
            const int st = j & 1, sn = st ^ 1;
            for (int x = 0; ok && x < nm; ++x) {
                if ((x == 0 && !mbar_wait(v_full + st, (j / 2) & 1)) || !mbar_wait(p_full + x, j & 1)) { ok = false; break; }
                tc_fence_after();
                const uint64_t vd = sdesc_mn_sw128(smem + S::OFF_V + st * S::TILE, S::PANEL);
#pragma unroll
                for (int part = 0; part < S::PARTS; ++part)
#pragma unroll
                    for (int k = 0; k < PT_KEYS / 16; ++k)
                        mma_ts(tmem + S::COL_O + x * HDP, tmem + (part ? S::COL_L + x * 64 : S::COL_S + x * 128) + 8 * k,
                               vd + k * (2048 >> 4), pv, j > 0 || part > 0 || k > 0);
                if (x == nm - 1) tc_commit(v_empty + st);
                if (j + 1 < w.tiles) {
                    if (x == 0 && !mbar_wait(k_full + sn, ((j + 1) / 2) & 1)) { ok = false; break; }
                    tc_fence_after();
                    scores(x, sn);
                    if (x == nm - 1) tc_commit(k_empty + sn);
                }
            }
        }
        tc_commit(o_full);
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
    const int row_tiles = (int)(((long long)a.max_new * a.group + S::NM * PT_ROWS - 1) / (S::NM * PT_ROWS));
    const long long blocks = (long long)a.rows.n * a.c.kv_heads * row_tiles;
    return launch_k(kernel, dim3((unsigned)blocks), dim3(S::THREADS), S::SMEM, s, 1, a, row_tiles);
}
template <class T, int CODE> cudaError_t launch_prompt(const KvAttend& a, cudaStream_t s) {
    return a.c.head_dim <= 64 ? launch_prompt<T, CODE, 64>(a, s) : launch_prompt<T, CODE, 128>(a, s);
}

}  // namespace

bool kv_prompt_takes(const KvAttend& a, int dtype) {
    (void)dtype;
    return a.c.head_dim <= 128 && (long long)a.max_new * a.group > 32;
}

cudaError_t kv_launch_prompt(const KvAttend& a, int dtype, cudaStream_t s) {
    if (a.c.code == CAC_KV8_INT8)
        return dtype == CAC_DTYPE_BF16 ? launch_prompt<bf16, CAC_KV8_INT8>(a, s) : launch_prompt<float, CAC_KV8_INT8>(a, s);
    return dtype == CAC_DTYPE_BF16 ? launch_prompt<bf16, CAC_KV8_E4M3>(a, s) : launch_prompt<float, CAC_KV8_E4M3>(a, s);
}

}  // namespace cac
