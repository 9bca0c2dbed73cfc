// Attention over the paged 8-bit K/V cache (include/cac_kv8.h) for calls with few
// query rows to a K/V head: single tokens and short pushes.
//
//   t_j = scale log2(e) ks_b (q . kc_j)      kc, vc: codes of token j; ks_b, vs_b: scales of its block of 16
//   w_j = 2^(t_j + log2(vs_b) - m),  m the running maximum of t_j + log2(vs_b)
//   out = sum_j w_j vc_j / (sum_j w_j / vs_b)
//
// With the value scale inside the exponent, the codes enter both products as they
// are (whole numbers or e4m3 values, exact in fp16), no product of a weight and a
// scale can leave the range of fp16, and the scales cost one multiply and one add per
// block.  Queries enter as fp16 after a power of two that brings the row's largest
// value under 2^15: a bf16 query is exact but for elements 2^29 smaller than the
// row's largest; an fp32 query enters as hi + lo.  Weights are rounded to fp16 (11 bits, against
// the 8 of a bf16 result) or, for fp32 results, enter as hi + lo.  Maxima, sums and
// accumulators are fp32.
//
// The work is one pass over the cache's bytes, so memory bounds it.  A unit is (sequence, K/V head, 16 query rows); its tiles are the
// 16-token blocks that any of its rows sees.  All tiles of the call, in order, are
// dealt out evenly to the warps of one block per SM, wherever that cuts a
// sequence; a warp that holds all of a unit writes its rows, the others leave partial
// sums that kv_join_kernel adds up in order.  So one sequence of 120,000 tokens and
// 64 of unlike lengths both keep every SM busy to the end, and the result does not
// depend on timing.
//
// Measured (bf16, head_dim 128, 8 K/V heads): 64 sequences of up to 32,000 tokens, group 4, int8: 345 us for 2.14 GB, 92 % of the rate of a
// plain copy; 128 windows of 4,096 tokens, group 8, e4m3: 201 us for 0.98 GB, 72 %; one sequence of 120,000: 62 us for
// 0.25 GB, 59 %.  What is above the bytes' time is 9 us until the first copies are queued (the call's lengths, a tile's place and scales, the
// queries: dependent reads), then a spread of about 10 % in what the SMs get of the memory's rate, and 10 us of joins.
//
// Each warp streams its tiles through a ring of its own in shared memory with
// 16-byte asynchronous copies, several tiles ahead of the mathematics, across
// the borders of units: there is no barrier between warps and nothing to wait for
// but its own copies.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kv8_attn.cuh"

#ifndef KV8_ATTN_CODE
#define KV8_ATTN_CODE 0  // CAC_KV8_INT8
#endif

namespace cac {
namespace {

// Weights are held times 2^LIFT: fp16 keeps 11 bits of every weight down to 2^-27 of the largest (a small weight may meet a large
// value).  SLACK is what a maximum may lag behind (RowsLow): at LIFT + SLACK = 15 a weight is 32,768 at most.
constexpr float LIFT = 13.f, SLACK = 2.f, NORM = norm_factor(13);

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// an 8 x 8 matrix of fp16 spread over a warp, two neighbours of a row to a thread, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// Where chunk c (16 bytes) of token row r of a tile lies: every quarter-warp of the
// fragment reads below touches all 32 banks once.
template <int HDP> __device__ __forceinline__ int tile_at(int r, int c) {
    if constexpr (HDP == 64) return ((r & ~1) | ((r ^ (r >> 2)) & 1)) * 64 + ((c ^ (r & 2)) << 4);
    return r * HDP + ((c ^ (r & 7)) << 4);
}

struct Tile {
    long long at;              // its codes (K and V alike), -1: nothing there
    float ks, lv, iv;          // K scale; log2 and reciprocal of the V scale (0 where that is FAR)
    int j0;                    // its first token
};
template <int CODE, class W>
__device__ __forceinline__ Tile tile_of(const KvAttend& a, const W& s, int kt, int head) {
    Tile t{-1, 0.f, 0.f, 0.f, 0};
    t.j0 = s.block(kt) * KV_BLOCK;
    if (t.j0 < s.len) {
        const int page = a.c.table[(long long)s.id * a.c.max_pages + t.j0 / a.c.page_tokens];
        if (page >= 0) {
            const int in_page = t.j0 % a.c.page_tokens;
            const long long sc = kv_scale_at(a.c, a.layer, page, head) + in_page / KV_BLOCK;
            t.at = kv_head_at(a.c, a.layer, page, head) + (long long)in_page * a.c.head_dim;
            t.ks = a.c.k_scale[sc];
            t.lv = log2f(a.c.v_scale[sc]);
            t.iv = t.lv < FAR ? 0.f : ex2(-t.lv);  // of the rounded logarithm, so that weight and norm have the same factor
        }
    }
    return t;
}
__device__ __forceinline__ Tile tile_from(const Tile& t, int lane) {
    Tile r;
    r.at = __shfl_sync(0xffffffffu, t.at, lane);
    r.ks = __shfl_sync(0xffffffffu, t.ks, lane);
    r.lv = __shfl_sync(0xffffffffu, t.lv, lane);
    r.iv = __shfl_sync(0xffffffffu, t.iv, lane);
    r.j0 = __shfl_sync(0xffffffffu, t.j0, lane);
    return r;
}

// A row's queries in the order of the fragments: contraction step s = 4 j + x, thread t of a row's four has elements 64 j + 16 t + 4 x +
// {0, 1} in a[s] and + {2, 3} in b[s], times the power of two that is returned; al, bl: what fp16 left over.
template <class T, int HDP, int LO>
__device__ __forceinline__ float load_query(const T* src, bool on, int t, int D, uint32_t (&a)[HDP / 16], uint32_t (&b)[HDP / 16],
                                            uint32_t (&al)[LO], uint32_t (&bl)[LO]) {
    constexpr int STEPS = HDP / 16;
    float x[STEPS][4];
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < HDP / 64; ++j) {
        const int e = 64 * j + 16 * t;
        if (on && e < D) {
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 v = *reinterpret_cast<const float4*>(src + e + 4 * k);
                    x[4 * j + k][0] = v.x, x[4 * j + k][1] = v.y, x[4 * j + k][2] = v.z, x[4 * j + k][3] = v.w;
                }
            } else {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint4 v = *reinterpret_cast<const uint4*>(src + e + 8 * k);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        x[4 * j + 2 * k + (c >> 1)][2 * (c & 1)] = __uint_as_float(w[c] << 16);
                        x[4 * j + 2 * k + (c >> 1)][2 * (c & 1) + 1] = __uint_as_float(w[c] & 0xffff0000u);
                    }
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[4 * j + k][0] = x[4 * j + k][1] = x[4 * j + k][2] = x[4 * j + k][3] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(x[4 * j + (k >> 2)][k & 3]));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const float up = lift_to_half(amax);
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        a[k] = pack_half(x[k][0] * up, x[k][1] * up);
        b[k] = pack_half(x[k][2] * up, x[k][3] * up);
        if constexpr (LO > 1) {
            al[k] = pack_rest(x[k][0] * up, x[k][1] * up, a[k]);
            bl[k] = pack_rest(x[k][2] * up, x[k][3] * up, b[k]);
        }
    }
    return up;
}

// The tokens that rows r0 .. r0 + size - 1 (of those there are) see: a tile is looked at from hi_max and lo_min, and whole
// for all of them between lo_max and hi_min.
struct Seen {
    int lo_max, hi_min, lo_min, hi_max;
    __device__ __forceinline__ void set(const KvAttend& a, const PieceWork& s, int r0, int size) {
        if (s.whole) hi_min = hi_max = s.len, lo_max = lo_min = s.lot * KV_BLOCK;
        else set(a, static_cast<const SeqWork&>(s), r0, size);
    }
    __device__ __forceinline__ void set(const KvAttend& a, const SeqWork& s, int r0, int size) {
        // rows in order of their positions: the first and last bound the windows
        const int p0 = s.len - s.m + a.query_of(r0), p1 = s.len - s.m + a.query_of(min(r0 + size, s.m * a.group) - 1);
        const bool any = s.len > 0 && p1 >= 0;
        hi_min = any && p0 >= 0 ? a.win.high(p0, s.len) : 0;
        hi_max = any ? a.win.high(p1, s.len) : 0;
        lo_max = any ? a.win.low(p1) : 0;
        lo_min = any ? a.win.low(max(p0, 0)) : 0;
    }
    // whether a tile holds a token that one of the rows sees (nothing where its V scale is 0: no write has filled it), and whether all see all of it
    __device__ __forceinline__ bool sees(const Tile& d, int sinks) const {
        return d.at >= 0 && d.lv != -INFINITY && d.j0 < hi_max && (d.j0 + KV_BLOCK > lo_min || d.j0 < sinks);
    }
    __device__ __forceinline__ bool whole(const Tile& d, int sinks) const {
        return d.j0 + KV_BLOCK <= hi_min && (d.j0 >= lo_max || d.j0 + KV_BLOCK <= sinks);
    }
};

// RUN consecutive results of a row
template <class T, int RUN> __device__ __forceinline__ void store_run(T* dst, const float (&x)[RUN]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < RUN; k += 4) *reinterpret_cast<float4*>(dst + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
    } else {
#pragma unroll
        for (int k = 0; k < RUN; k += 8) {
            uint32_t w[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[k + 2 * b], x[k + 2 * b + 1]);
                w[b] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(dst + k) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

constexpr int MOST_WARPS = 12;   // of a block (16 at most: join_warp has a lane for each)

// Partial sums of units that were cut.  Slot 2 w: the unit that warp w's share begins in; slot 2 w + 1: the one that it ends in,
// when that is another.  After the warps' slots the same for the blocks.
struct Partials {
    float *o, *ml;               // [slot][16][HDP], [slot][16][2]
    long long* first;            // [TA_SEQS + 1] tiles before each sequence
    int warps;
};
// RUN elements from e on of row `row` of a unit whose rows begin at r0: the result itself, or, with cut, its part in slot `slot`
template <class T, int HDP, int RUN>
__device__ __forceinline__ void put_run(const KvAttend& a, const SeqWork& s, int head, int row, int r0, int e, float (&y)[RUN], float l,
                                        const Partials* cut, int slot) {
    if (cut) {
        store_run<float, RUN>(cut->o + ((size_t)slot * 16 + row - r0) * HDP + e, y);
    } else if (e < a.c.head_dim) {
        const int query = a.query_of(row), qh = head * a.group + row - query * a.group;
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
        for (int k = 0; k < RUN; ++k) y[k] = y[k] * NORM * inv;  // NORM * inv may be too small a number
        store_run<T, RUN>(static_cast<T*>(a.out) + (s.row0 + (long long)query) * a.out_stride + (long long)qh * a.c.head_dim + e, y);
    }
}
template <class T, int HDP>
__device__ __forceinline__ void put_sums(const KvAttend& a, const SeqWork& s, int head, int row, int r0, float m, float l,
                                         const Partials* cut, int slot) {
    if (cut) {
        cut->ml[((size_t)slot * 16 + row - r0) * 2] = m;
        cut->ml[((size_t)slot * 16 + row - r0) * 2 + 1] = l;
    } else if (a.lse) {
        const int query = a.query_of(row), qh = head * a.group + row - query * a.group;
        a.lse[(s.row0 + (long long)query) * a.heads + qh] =
            l > 0.f || l != l ? (m + NORM_LOG2 + log2f(l)) * LN2 : -INFINITY;
    }
}

// Sixteen query rows and their running sums, spread over a warp as the tensor core's
// fragments: a thread has rows g and g + 8 (g = lane / 4, t = lane % 4).
template <class T, int CODE, int HDP> struct Rows : Seen {
    static constexpr bool WIDE = sizeof(T) == 4;          // hi + lo
    static constexpr int STEPS = HDP / 16, NT = HDP / 8, LO = WIDE ? STEPS : 1;
    uint32_t q[STEPS][4], ql[LO][4];
    float o[NT][4];
    float m[2], l[2], f[2];                               // maximum, sum, score factor of rows g, g + 8
    int low[2], high[2];

    // Queries of K/V head `head`, rows r0 .. r0 + 15 of the sequence's m * group
    template <class W> __device__ __forceinline__ void load(const KvAttend& a, const W& s, int head, int r0) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, D = a.c.head_dim;
        set(a, s, r0, 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = r0 + g + 8 * h, query = a.query_of(r);
            const bool on = r < s.m * a.group;
            const RowSeen see = row_seen(a, s, r);
            m[h] = -INFINITY, l[h] = 0.f;
            low[h] = see.low, high[h] = see.high;
            uint32_t x[STEPS], y[STEPS], xl[LO], yl[LO];
            f[h] = a.scale * LOG2E / load_query<T, HDP>(static_cast<const T*>(a.q) + (s.row0 + (long long)query) * a.q_stride +
                                                            (long long)(head * a.group + r - query * a.group) * D,
                                                        on, t, D, x, y, xl, yl);  // by a power of two: exact
#pragma unroll
            for (int k = 0; k < STEPS; ++k) q[k][h] = x[k], q[k][2 + h] = y[k];
            if constexpr (WIDE)
#pragma unroll
                for (int k = 0; k < STEPS; ++k) ql[k][h] = xl[k], ql[k][2 + h] = yl[k];
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    }

    // Two tiles of 16 tokens, their codes at shared addresses k[u] (V after K); on[u]: take part (one that does not may be another
    // sequence's, and its scales anything).  Column n of score tile i is
    // token (n / 2) + 4 (2 i + n % 2), so that a thread's four weights of a row are tokens t, t + 4, t + 8, t + 12.
    __device__ __forceinline__ void tiles(const Tile (&d)[2], const uint8_t* const (&k)[2], const bool (&on)[2], int sinks) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        float s[2][2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int i = 0; i < 2; ++i) s[u][i][0] = s[u][i][1] = s[u][i][2] = s[u][i][3] = on[u] ? 0.f : -INFINITY;
            if (!on[u]) continue;
#pragma unroll
            for (int j = 0; j < HDP / 64; ++j) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = (g >> 1) + 4 * (2 * i + (g & 1));
                    const uint4 w = *reinterpret_cast<const uint4*>(k[u] + tile_at<HDP>(r, 4 * j + t));
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint32_t b0, b1;
                        half4<CODE>(ww[x], b0, b1);
                        mma_f16(s[u][i], q[4 * j + x], b0, b1);
                        if constexpr (WIDE) mma_f16(s[u][i], ql[4 * j + x], b0, b1);
                    }
                }
            }
            const bool full = whole(d[u], sinks);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float c = f[h] * d[u].ks;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int b = 0; b < 2; ++b) s[u][i][2 * h + b] = fmaf(s[u][i][2 * h + b], c, d[u].lv);
            }
            if (!full) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const int j = d[u].j0 + t + 4 * (2 * i + b);
                            if (!(j < high[h] && (j >= low[h] || j < sinks))) s[u][i][2 * h + b] = -INFINITY;
                        }
            }
        }
        float top[2];
        bool moved = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float mx = fmaxf(fmaxf(s[0][0][2 * h], s[0][0][2 * h + 1]), fmaxf(s[0][1][2 * h], s[0][1][2 * h + 1]));
            mx = fmaxf(mx, fmaxf(fmaxf(s[1][0][2 * h], s[1][0][2 * h + 1]), fmaxf(s[1][1][2 * h], s[1][1][2 * h + 1])));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            top[h] = fmaxf(m[h], mx);
            moved |= top[h] > m[h];
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float d = top[h] == -INFINITY ? 0.f : m[h] - top[h], r = ex2(d);
                m[h] = top[h];
                l[h] = move_norm(l[h], d, r);
#pragma unroll
                for (int n = 0; n < NT; ++n) o[n][2 * h] *= r, o[n][2 * h + 1] *= r;
            }
        }
        uint32_t p[2][4], pl[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float base = m[h] == -INFINITY ? 0.f : m[h] - LIFT;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float w[2][2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int b = 0; b < 2; ++b) w[i][b] = ex2(s[u][i][2 * h + b] - base);
                l[h] = fmaf(((w[0][0] + w[0][1]) + (w[1][0] + w[1][1])) * NORM, on[u] ? d[u].iv : 0.f, l[h]);
                if (on[u] && d[u].lv < FAR) {
                    float x = 0.f;
#pragma unroll
                    for (int i = 0; i < 2; ++i) x += ex2(s[u][i][2 * h] - d[u].lv - base) + ex2(s[u][i][2 * h + 1] - d[u].lv - base);
                    l[h] = fmaf(x, NORM, l[h]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    p[u][2 * i + h] = pack_half(w[i][0], w[i][1]);
                    if constexpr (WIDE) pl[u][2 * i + h] = pack_rest(w[i][0], w[i][1], p[u][2 * i + h]);
                }
            }
        }
        // value columns: column n of output tile y is element first(n) + y (see `element`)
        constexpr int PER = HDP == 64 ? 8 : 16;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (!on[u]) continue;
            const uint8_t* v = k[u] + KV_BLOCK * HDP;
#pragma unroll
            for (int z = 0; z < HDP / (8 * PER); ++z) {
                const int c = HDP == 64 ? g >> 1 : (((g & 1) << 2) | (g >> 1)) + 8 * z;
                uint32_t w[4][PER / 4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint8_t* at = v + tile_at<HDP>(t + 4 * y, c);
                    if constexpr (HDP == 64) {
                        const uint2 e = *reinterpret_cast<const uint2*>(at + (g & 1) * 8);
                        w[y][0] = e.x, w[y][1] = e.y;
                    } else {
                        const uint4 e = *reinterpret_cast<const uint4*>(at);
                        w[y][0] = e.x, w[y][1] = e.y, w[y][2] = e.z, w[y][3] = e.w;
                    }
                    if (CODE == CAC_KV8_E4M3 && d[u].j0 + KV_BLOCK > hi_max && d[u].j0 + t + 4 * y >= hi_max) {
                        // a token past the end: its codes may be anything, and a weight of 0 times NaN is NaN
#pragma unroll
                        for (int x = 0; x < PER / 4; ++x) w[y][x] = 0;
                    }
                }
#pragma unroll
                for (int x = 0; x < PER / 4; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {  // elements 4 x + 2 y and 4 x + 2 y + 1 of four tokens
                        const uint32_t sel = y ? 0x7362 : 0x5140;
                        uint32_t a0, a1, b0, b1;
                        half4<CODE>(__byte_perm(w[0][x], w[1][x], sel), a0, b0);
                        half4<CODE>(__byte_perm(w[2][x], w[3][x], sel), a1, b1);
                        const int n = z * PER + 4 * x + 2 * y;
                        if constexpr (WIDE) {
                            // The tensor core cuts sums off where fp32 would round: over a long cache that adds up to more than
                            // an fp32 result may lose, so its sums are of one tile and are added here.
                            float a[4] = {}, b[4] = {};
                            mma_f16(a, pl[u], a0, a1);
                            mma_f16(b, pl[u], b0, b1);
                            mma_f16(a, p[u], a0, a1);
                            mma_f16(b, p[u], b0, b1);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[n][e] += a[e], o[n + 1][e] += b[e];
                        } else {
                            mma_f16(o[n], p[u], a0, a1);
                            mma_f16(o[n + 1], p[u], b0, b1);
                        }
                    }
            }
        }
    }
    // first element of column n's run in piece z
    static __device__ __forceinline__ int element(int n, int z) {
        if constexpr (HDP == 64) return n * 8;
        return (((n & 1) << 2) | (n >> 1)) * 16 + 128 * z;
    }
    static constexpr int RUN = HDP == 64 ? 8 : 16;

    // The rows' results, or, cut, their parts in slot `slot`
    __device__ __forceinline__ void emit(const KvAttend& a, const SeqWork& s, int head, int r0, const Partials* cut, int slot) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            const int row = r0 + g + 8 * h;
            if (row >= s.m * a.group) continue;
#pragma unroll
            for (int z = 0; z < HDP / (8 * RUN); ++z)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float y[RUN];
#pragma unroll
                    for (int k = 0; k < RUN; ++k) y[k] = o[z * RUN + k][2 * h + b];
                    put_run<T, HDP, RUN>(a, s, head, row, r0, element(2 * t + b, z), y, l[h], cut, slot);
                }
            if (t == 0) put_sums<T, HDP>(a, s, head, row, r0, m[h], l[h], cut, slot);
        }
    }
};

// At most eight query rows: the other way round, tokens and elements are the rows of the tensor core's operand A and the queries the
// eight columns of B, which halves its instructions and the registers of the sums (64 sequences of up to 32,000 tokens: 409 -> 358 us).  A thread (g, t) has tokens g / 2 + 4 (g % 2) and 8 more of
// the scores of query rows 2 t and 2 t + 1.  The maximum is only moved (and the sums rescaled, and the warp's lanes asked) when
// it has grown by 2^SLACK; until then weights may pass 1, and LIFT leaves room for it.
template <class T, int CODE, int HDP> struct RowsLow : Seen {
    static constexpr bool WIDE = sizeof(T) == 4;          // hi + lo
    static constexpr int STEPS = HDP / 16, LO = WIDE ? STEPS : 1, MT = HDP / 16;
    static constexpr int PER = HDP == 64 ? 8 : 16;        // elements that a thread has of a piece of the values
    uint32_t q0[STEPS], q1[STEPS], l0[LO], l1[LO];
    float o[MT][4];                                       // pairs of elements (0, 1 and 2, 3) of rows 2 t (0, 2) and 2 t + 1 (1, 3)
    float m[2], l[2], f[2];                               // of rows 2 t, 2 t + 1
    int low[2], high[2];

    template <class W> __device__ __forceinline__ void load(const KvAttend& a, const W& s, int head, int r0) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, D = a.c.head_dim;
        set(a, s, r0, 8);
        const int r = r0 + g, query = a.query_of(r);
        const float up = load_query<T, HDP>(static_cast<const T*>(a.q) + (s.row0 + (long long)query) * a.q_stride +
                                                (long long)(head * a.group + r - query * a.group) * D,
                                            r < s.m * a.group, t, D, q0, q1, l0, l1);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const RowSeen see = row_seen(a, s, r0 + 2 * t + b);
            f[b] = a.scale * LOG2E / __shfl_sync(0xffffffffu, up, 4 * (2 * t + b));  // by a power of two: exact
            m[b] = -INFINITY, l[b] = 0.f;
            low[b] = see.low, high[b] = see.high;
        }
#pragma unroll
        for (int n = 0; n < MT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    }

    __device__ __forceinline__ void tiles(const Tile (&d)[2], const uint8_t* const (&k)[2], const bool (&on)[2], int sinks) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, tok = (g >> 1) + 4 * (g & 1);
        float s[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            s[u][0] = s[u][1] = s[u][2] = s[u][3] = on[u] ? 0.f : -INFINITY;
            if (!on[u]) continue;
#pragma unroll
            for (int j = 0; j < HDP / 64; ++j) {
                const uint4 wa = *reinterpret_cast<const uint4*>(k[u] + tile_at<HDP>(tok, 4 * j + t));
                const uint4 wb = *reinterpret_cast<const uint4*>(k[u] + tile_at<HDP>(tok + 8, 4 * j + t));
                const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w}, b[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t kk[4];
                    half4<CODE>(a[x], kk[0], kk[2]);
                    half4<CODE>(b[x], kk[1], kk[3]);
                    if constexpr (WIDE) mma_f16(s[u], kk, l0[4 * j + x], l1[4 * j + x]);
                    mma_f16(s[u], kk, q0[4 * j + x], q1[4 * j + x]);
                }
            }
            const bool full = whole(d[u], sinks);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const float c = f[b] * d[u].ks;
#pragma unroll
                for (int i = 0; i < 2; ++i) s[u][2 * i + b] = fmaf(s[u][2 * i + b], c, d[u].lv);
            }
            if (!full) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int j = d[u].j0 + tok + 8 * i;
                        if (!(j < high[b] && (j >= low[b] || j < sinks))) s[u][2 * i + b] = -INFINITY;
                    }
            }
        }
        float top[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) top[b] = fmaxf(fmaxf(s[0][b], s[0][2 + b]), fmaxf(s[1][b], s[1][2 + b]));
        if (__any_sync(0xffffffffu, top[0] > m[0] + SLACK || top[1] > m[1] + SLACK)) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) top[b] = fmaxf(top[b], __shfl_xor_sync(0xffffffffu, top[b], x));
                if (top[b] > m[b] + SLACK) {
                    const float d = m[b] - top[b], r = ex2(d);
                    m[b] = top[b];
                    l[b] = move_norm(l[b], d, r);
#pragma unroll
                    for (int n = 0; n < MT; ++n) o[n][b] *= r, o[n][2 + b] *= r;
                }
            }
        }
        uint32_t p[2][2], pl[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = ex2(s[u][e] - (m[e & 1] == -INFINITY ? 0.f : m[e & 1] - LIFT));
            const float iv = on[u] ? d[u].iv : 0.f;
            l[0] = fmaf((w[0] + w[2]) * NORM, iv, l[0]);
            l[1] = fmaf((w[1] + w[3]) * NORM, iv, l[1]);
            if (on[u] && d[u].lv < FAR) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    l[e & 1] = fmaf(ex2(s[u][e] - d[u].lv - (m[e & 1] == -INFINITY ? 0.f : m[e & 1] - LIFT)), NORM, l[e & 1]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // tokens by rows -> rows by tokens: what operand B takes
                const uint32_t hi = pack_half(w[2 * i], w[2 * i + 1]);
                p[u][i] = transpose8(hi);
                if constexpr (WIDE) pl[u][i] = transpose8(pack_rest(w[2 * i], w[2 * i + 1], hi));
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (!on[u]) continue;
            const uint8_t* v = k[u] + KV_BLOCK * HDP;
#pragma unroll
            for (int z = 0; z < HDP / (8 * PER); ++z) {
                const int c = HDP == 64 ? g >> 1 : (((g & 1) << 2) | (g >> 1)) + 8 * z;
                uint32_t w[4][PER / 4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint8_t* at = v + tile_at<HDP>(t + 4 * y, c);
                    if constexpr (HDP == 64) {
                        const uint2 e = *reinterpret_cast<const uint2*>(at + (g & 1) * 8);
                        w[y][0] = e.x, w[y][1] = e.y;
                    } else {
                        const uint4 e = *reinterpret_cast<const uint4*>(at);
                        w[y][0] = e.x, w[y][1] = e.y, w[y][2] = e.z, w[y][3] = e.w;
                    }
                    if (CODE == CAC_KV8_E4M3 && d[u].j0 + KV_BLOCK > hi_max && d[u].j0 + t + 4 * y >= hi_max) {
                        // a token past the end: its codes may be anything, and a weight of 0 times NaN is NaN
#pragma unroll
                        for (int x = 0; x < PER / 4; ++x) w[y][x] = 0;
                    }
                }
#pragma unroll
                for (int x = 0; x < PER / 4; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {  // elements 4 x + 2 y and 4 x + 2 y + 1 of four tokens
                        const uint32_t sel = y ? 0x7362 : 0x5140;
                        uint32_t vv[4];
                        half4<CODE>(__byte_perm(w[0][x], w[1][x], sel), vv[0], vv[1]);
                        half4<CODE>(__byte_perm(w[2][x], w[3][x], sel), vv[2], vv[3]);
                        float(&sum)[4] = o[(z * PER + 4 * x + 2 * y) / 2];
                        if constexpr (WIDE) {
                            // sums of one tile, added here: the tensor core cuts sums off where fp32 would round
                            float part[4] = {};
                            mma_f16(part, vv, pl[u][0], pl[u][1]);
                            mma_f16(part, vv, p[u][0], p[u][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) sum[e] += part[e];
                        } else {
                            mma_f16(sum, vv, p[u][0], p[u][1]);
                        }
                    }
            }
        }
    }

    __device__ __forceinline__ void emit(const KvAttend& a, const SeqWork& s, int head, int r0, const Partials* cut, int slot) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[b] += __shfl_xor_sync(0xffffffffu, l[b], x);
            const int row = r0 + 2 * t + b;
            if (row >= s.m * a.group) continue;
#pragma unroll
            for (int z = 0; z < HDP / (8 * PER); ++z) {
                float y[PER];
#pragma unroll
                for (int k = 0; k < PER; ++k) y[k] = o[(z * PER + k) / 2][2 * (k & 1) + b];
                put_run<T, HDP, PER>(a, s, head, row, r0, HDP == 64 ? g * 8 : (((g & 1) << 2) | (g >> 1)) * 16 + 128 * z, y, l[b],
                                     cut, slot);
            }
            if (g == 0) put_sums<T, HDP>(a, s, head, row, r0, m[b], l[b], cut, slot);
        }
        // only a sequence with more rows than max_new has rows 8 .. 15: they see nothing
        const int row = r0 + 8 + g;
        if (row < s.m * a.group && !cut) {
            const int D = a.c.head_dim, query = a.query_of(row), qh = head * a.group + row - query * a.group;
            T* dst = static_cast<T*>(a.out) + (s.row0 + (long long)query) * a.out_stride + (long long)qh * D;
            for (int e = t; e < D; e += 4) dst[e] = from_f<T>(0.f);
            if (t == 0 && a.lse) a.lse[(s.row0 + (long long)query) * a.heads + qh] = -INFINITY;
        }
    }
};

// The call's split over warps: tile x of `total` belongs to the warp w with
// begin(w) <= x < begin(w + 1).
// A share has LEAST tiles at least: fewer cost more to join than they save.
constexpr int LEAST = 4;
struct Deal {
    long long total;
    int warps;
    long long share;    // tiles of a share; the first `over` have one more
    int over;
    __device__ __forceinline__ Deal(long long tiles, int most)
        : total(tiles), warps(tiles >= (long long)most * LEAST ? most : max((int)(tiles / LEAST), 1)) {
        share = total / warps;
        over = (int)(total - share * warps);
    }
    __device__ __forceinline__ long long begin(int w) const { return w < warps ? share * w + min(w, over) : total; }
    __device__ __forceinline__ int owner(long long x) const {
        const long long head = (share + 1) * over;
        return (int)(x < head ? x / (share + 1) : over + (x - head) / share);
    }
};

template <int HDP> inline size_t partial_bytes(int sms) {
    return (size_t)sms * (MOST_WARPS + 1) * 2 * 16 * (HDP + 2) * 4 + (TA_SEQS + 2) * 8;
}
template <int HDP> __device__ __forceinline__ Partials partials_at(void* space, int blocks, int warps) {
    Partials p;
    p.first = static_cast<long long*>(space);
    p.o = reinterpret_cast<float*>(p.first + TA_SEQS + 2);
    p.ml = p.o + (size_t)(blocks + warps) * 2 * 16 * HDP;
    p.warps = warps;
    return p;
}

// The parts of a unit in slots `first`, then next, next + 2, ... (`more` of those) are added up: this warp does rows mine, mine +
// more, ... and writes them out, or, with to >= 0, into that slot.  ROWS rows and PARTS parts are on their way at once.
template <class T, int HDP, int ROWS, int PARTS>
__device__ __forceinline__ void join_rows(const KvAttend& a, const Partials& p, const SeqWork& s, int unit, int first, int next, int more,
                                          int mine, int to) {
    constexpr int PER = HDP / 32;
    const int lane = threadIdx.x & 31, kvh = a.c.kv_heads, head = unit % kvh, r0 = unit / kvh * 16, step = more;
    const int rows = min(16, s.m * a.group - r0);
    auto slot = [&](int k) { return (size_t)(k == 0 ? first : next + 2 * (k - 1)) * 16; };
#pragma unroll 1
    for (int r = mine; r < rows; r += ROWS * step) {
        float2 ml[ROWS];
#pragma unroll
        for (int b = 0; b < ROWS; ++b) {
            ml[b] = make_float2(-INFINITY, 0.f);
            if (lane <= more && r + b * step < rows) ml[b] = __ldcg(reinterpret_cast<const float2*>(p.ml) + slot(lane) + r + b * step);
        }
        float o[ROWS][PER] = {}, f[ROWS], top[ROWS], l[ROWS];
#pragma unroll 1
        for (int k0 = 0; k0 <= more; k0 += PARTS) {
            float v[PARTS][ROWS][PER];
#pragma unroll
            for (int k = 0; k < PARTS; ++k)
#pragma unroll
                for (int b = 0; b < ROWS; ++b)
#pragma unroll
                    for (int c = 0; c < PER; c += 2) {
                        float2 y = make_float2(0.f, 0.f);
                        if (k0 + k <= more && r + b * step < rows)
                            y = __ldcg(reinterpret_cast<const float2*>(p.o + (slot(k0 + k) + r + b * step) * HDP + lane * PER + c));
                        v[k][b][c] = y.x, v[k][b][c + 1] = y.y;
                    }
            if (k0 == 0) {
#pragma unroll
                for (int b = 0; b < ROWS; ++b) top[b] = ml[b].x;
#pragma unroll
                for (int d = 8; d; d >>= 1)  // lanes 0 .. 15 hold the parts
#pragma unroll
                    for (int b = 0; b < ROWS; ++b) top[b] = fmaxf(top[b], __shfl_xor_sync(0xffffffffu, top[b], d, 16));
#pragma unroll
                for (int b = 0; b < ROWS; ++b) {
                    const float d = ml[b].x - (top[b] == -INFINITY ? 0.f : top[b]);
                    f[b] = ex2(d), l[b] = move_norm(ml[b].y, d, f[b]);
                }
#pragma unroll
                for (int d = 8; d; d >>= 1)
#pragma unroll
                    for (int b = 0; b < ROWS; ++b) l[b] += __shfl_xor_sync(0xffffffffu, l[b], d, 16);
#pragma unroll
                for (int b = 0; b < ROWS; ++b) top[b] = __shfl_sync(0xffffffffu, top[b], 0), l[b] = __shfl_sync(0xffffffffu, l[b], 0);
            }
#pragma unroll
            for (int k = 0; k < PARTS; ++k)
#pragma unroll
                for (int b = 0; b < ROWS; ++b) {
                    const float w = __shfl_sync(0xffffffffu, f[b], k0 + k);
                    if (k0 + k <= more)
#pragma unroll
                        for (int c = 0; c < PER; ++c) o[b][c] = fmaf(v[k][b][c], w, o[b][c]);
                }
        }
#pragma unroll
        for (int b = 0; b < ROWS; ++b) {
            const int at = r + b * step;
            if (at >= rows) break;
            if (to >= 0) {
#pragma unroll
                for (int c = 0; c < PER; ++c) p.o[((size_t)to * 16 + at) * HDP + lane * PER + c] = o[b][c];
                if (lane == 0) p.ml[((size_t)to * 16 + at) * 2] = top[b], p.ml[((size_t)to * 16 + at) * 2 + 1] = l[b];
            } else {
                const int row = r0 + at, query = a.query_of(row), qh = head * a.group + row - query * a.group, D = a.c.head_dim;
                const bool seen = l[b] > 0.f || l[b] != l[b];
                T* dst = static_cast<T*>(a.out) + (s.row0 + (long long)query) * a.out_stride + (long long)qh * D + lane * PER;
#pragma unroll
                for (int c = 0; c < PER; ++c)
                    if (lane * PER + c < D) dst[c] = from_f<T>(seen ? o[b][c] * NORM / l[b] : 0.f);
                if (lane == 0 && a.lse)
                    a.lse[(s.row0 + (long long)query) * a.heads + qh] = seen ? (top[b] + NORM_LOG2 + log2f(l[b])) * LN2 : -INFINITY;
            }
        }
    }
}

// While other blocks still stream, each wait for memory takes 4 us: many warps have few rows each and few have many, and either
// way all of a warp's loads should be on their way at once.
template <class T, int HDP>
__device__ __forceinline__ void join_warp(const KvAttend& a, const Partials& p, const SeqWork& s, int unit, int first, int next, int more,
                                          int mine, int to) {
    constexpr int WIDTH = HDP > 128 ? 2 : 1;
    if (more == 1) join_rows<T, HDP, 8 / WIDTH, 2>(a, p, s, unit, first, next, more, mine, to);
    else if (more < 4) join_rows<T, HDP, 4 / WIDTH, 4>(a, p, s, unit, first, next, more, mine, to);
    else join_rows<T, HDP, 1, MOST_WARPS>(a, p, s, unit, first, next, more, mine, to);
}

// Warps of a block, and the tiles that each has in flight or at hand (two matrices of 16 rows of HDP bytes).  The sums of 16 rows
// take HDP / 2 registers (of 8 rows, HDP / 4) and an fp32 query's two halves HDP / 2 more, which leaves room for 12 warps, or 8.  Measured with
// 8 / 10 / 12 warps of 8 rows of 128 bf16: 357 / 357 / 343 us (64 sequences of up to 32,000), 213 / 210 / 209 (128 windows of 4,096);
// with half of the shared memory 360 and 199, with three quarters 349 and 196.
template <class T, int HDP, bool LOW, bool SPLIT> struct Shape {
    static constexpr int WARPS = !SPLIT ? 4 : HDP == 64 || (HDP == 128 && LOW && sizeof(T) == 2) ? 12 : 8;
    static constexpr int STAGE = 2 * KV_BLOCK * HDP;
    static constexpr int STAGES = !SPLIT ? (HDP == 256 ? 3 : 4) : 196608 / (WARPS * STAGE);
    static constexpr int BYTES = WARPS * STAGES * STAGE;
    static constexpr int BLOCKS = !SPLIT && HDP == 64 ? 4 : 1;  // of an SM
    static_assert(WARPS <= MOST_WARPS && MOST_WARPS <= 16, "the workspace has room for the parts of so many");
    static_assert(BYTES + (SPLIT ? 25 * 1024 : 0) <= 227 * 1024, "shared memory");
};

// SPLIT: tiles are dealt out over a grid of one block per SM.  Otherwise each warp takes one
// whole unit (short windows, where a unit has a handful of tiles): nothing has to be joined.
template <class T, int CODE, int HDP, bool LOW, bool SPLIT>
__global__ void __launch_bounds__(Shape<T, HDP, LOW, SPLIT>::WARPS * 32, (Shape<T, HDP, LOW, SPLIT>::BLOCKS))
    kv_attend_kernel(const __grid_constant__ KvAttend a, void* space) {
    using R = std::conditional_t<LOW, RowsLow<T, CODE, HDP>, Rows<T, CODE, HDP>>;
    using S = Shape<T, HDP, LOW, SPLIT>;
    constexpr int STAGES = S::STAGES, STAGE = S::STAGE, WARPS = S::WARPS, CH = HDP / 16;
    extern __shared__ __align__(128) uint8_t ring_all[];
    __shared__ long long s_first[SPLIT ? TA_SEQS + 1 : 1];
    __shared__ long long s_part[WARPS];
    __shared__ SeqWork s_seq[SPLIT ? TA_SEQS : 1];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = a.rows.n, kvh = a.c.kv_heads;
    uint8_t* ring = ring_all + warp * STAGES * STAGE;
    const int D = a.c.head_dim;

    const Partials part = partials_at<HDP>(space, gridDim.x, gridDim.x * WARPS);

    long long x0 = 0, x1 = 0;   // this warp's share of the tiles
    int i = 0, unit = 0;        // SPLIT = false: its unit
    SeqWork s{};
    if constexpr (SPLIT) {
        // tiles before each sequence
        long long before = 0;
        for (int base = 0; base < n; base += WARPS * 32) {
            const int k = base + threadIdx.x;
            long long mine = 0;
            if (k < n) {
                const SeqWork w = seq_work(a, k);
                s_seq[k] = w;
                mine = (long long)w.tiles * kvh * ((w.m * a.group + 15) / 16);
            }
            long long sum = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += u;
            }
            if (lane == 31) s_part[warp] = sum;
            __syncthreads();
            long long add = before;
            for (int w = 0; w < WARPS; ++w) {
                if (w < warp) add += s_part[w];
                before += s_part[w];
            }
            if (k < n) s_first[k] = add + sum - mine;
            __syncthreads();
        }
        if (threadIdx.x == 0) s_first[n] = before;
        __syncthreads();
        const int warps = gridDim.x * WARPS;
        if (blockIdx.x == 0)
            for (int k = threadIdx.x; k <= n; k += WARPS * 32) part.first[k] = s_first[k];
        const Deal deal(before, warps);
        if (before == 0) return;
        x0 = deal.begin(blockIdx.x * WARPS + warp), x1 = deal.begin(blockIdx.x * WARPS + warp + 1);
    } else {
        const int u = (int)blockIdx.x * WARPS + warp;
        const int2 tile = a.tile_at(u / kvh, 16);
        i = tile.x, unit = tile.y * kvh + u % kvh;   // unit = row tile * kv_heads + head
        if (i < 0 || i >= n) return;
        s = seq_work(a, i);
        if (tile.y * 16 >= s.m * a.group) return;
        x1 = s.tiles;
    }

    // Lane l knows tile base + l of the share (now) and the 32 after those (next).
    auto look = [&](long long x) {
        if (x >= x1) return Tile{-1, 0.f, 0.f, 0.f, 0};
        if constexpr (SPLIT) {
            int lo = 0, hi = n - 1;  // the last sequence with s_first <= x (empty ones have no tiles)
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_first[mid] <= x) lo = mid;
                else hi = mid - 1;
            }
            const SeqWork& w = s_seq[lo];
            const long long in = x - s_first[lo];
            const int u = (int)(in / w.tiles), kt = (int)(in - (long long)u * w.tiles);
            return tile_of<CODE>(a, w, kt, u % kvh);
        } else {
            return tile_of<CODE>(a, s, (int)x, unit % kvh);
        }
    };
    Tile now = look(x0 + lane);
    long long base = x0;

    Tile next = now;
    int into = 0;  // the stage that the next copies go to
    auto fetch = [&](long long x) {  // queue the copies of tile x; always one group
        const int k = (int)(x - base);
        const long long at = __shfl_sync(0xffffffffu, k < 32 ? now.at : next.at, k & 31);
        if (x < x1 && at >= 0) {
            const uint32_t dst = smem_u32(ring) + into * STAGE;
            const uint8_t *ks = static_cast<const uint8_t*>(a.c.k) + at, *vs = static_cast<const uint8_t*>(a.c.v) + at;
#pragma unroll
            for (int e0 = 0; e0 < KV_BLOCK * CH; e0 += 32) {
                const int e = e0 + lane, r = e / CH, c = e % CH;
                if (c * 16 < D) {
                    cp16(dst + tile_at<HDP>(r, c), ks + r * D + c * 16);
                    cp16(dst + KV_BLOCK * HDP + tile_at<HDP>(r, c), vs + r * D + c * 16);
                }
            }
        }
        cp_commit();
        into = into + 1 == STAGES ? 0 : into + 1;
    };
    if (D < HDP) {  // chunks past the head's width stay zero
        for (int st = 0; st < STAGES; ++st)
            for (int e = lane; e < 2 * KV_BLOCK * CH; e += 32) {
                const int r = e / CH % KV_BLOCK, c = e % CH;
                if (c * 16 >= D)
                    *reinterpret_cast<uint4*>(ring + st * STAGE + e / (KV_BLOCK * CH) * (KV_BLOCK * HDP) +
                                              tile_at<HDP>(r, c)) = make_uint4(0, 0, 0, 0);
            }
        __syncwarp();
    }
    R r;
    long long x = x0, u0 = 0, u1 = x1;
    // the unit that tile x belongs to: its tiles [u0, u1), sequence, head and first row
    int head = 0, r0 = 0;
    auto enter = [&] {
        if constexpr (SPLIT) {
            i = warp_last_le(n, x, [&](int k) { return s_first[k]; });
            s = s_seq[i];
            unit = (int)((x - s_first[i]) / s.tiles);
            u0 = s_first[i] + (long long)unit * s.tiles, u1 = u0 + s.tiles;
        }
        head = unit % kvh, r0 = unit / kvh * 16;
        r.load(a, s, head, r0);
    };
    // the first unit's queries before the ring fills: behind its copies they would take twice as long
    if (x < x1) enter();
#pragma unroll 1
    for (int k = 0; k < STAGES; ++k) fetch(x0 + k);
    if (SPLIT || x1 > 32) next = look(x0 + 32 + lane);
    int from_stage = 0;

    bool entered = true;
    while (x < x1) {
        if (!entered) enter();
        entered = false;
        const long long end = min(u1, x1), from = x;
        while (x < end) {
            if (x - base >= 32) {
                base += 32;
                now = next;
                next = look(base + 32 + lane);
            }
            cp_wait<STAGES - 2>();  // tiles x and x + 1 are there
            __syncwarp();
            const bool two = x + 1 < end;
            const int k0 = (int)(x - base), s1 = from_stage + 1 == STAGES ? 0 : from_stage + 1;
            const Tile d[2] = {tile_from(now, k0), k0 < 31 ? tile_from(now, k0 + 1) : tile_from(next, 0)};
            const uint8_t* const k[2] = {ring + from_stage * STAGE, ring + s1 * STAGE};
            const bool on[2] = {r.sees(d[0], a.win.sinks), two && r.sees(d[1], a.win.sinks)};
            if (on[0] || on[1]) r.tiles(d, k, on, a.win.sinks);
            __syncwarp();  // the stages are read before their next copies are queued
            fetch(x + STAGES);
            if (two) fetch(x + STAGES + 1);
            x += 1 + two;
            from_stage = two ? (s1 + 1 == STAGES ? 0 : s1 + 1) : s1;
        }
        const bool begins = from == u0, ends = end == u1;
        int slot = 2 * (blockIdx.x * WARPS + warp) + (from != x0);
        // a part that no other warp of the block has one to add to: the block's
        if (!begins && ends && warp == 0) slot = 2 * part.warps + 2 * blockIdx.x;
        if (begins && !ends && warp == WARPS - 1) slot = 2 * part.warps + 2 * blockIdx.x + 1;
        r.emit(a, s, head, r0, begins && ends ? nullptr : &part, slot);
    }
    cp_wait<0>();
    if constexpr (SPLIT) {
        __syncthreads();  // the warps' parts are visible to the block
        const Deal deal(s_first[n], gridDim.x * WARPS);
        const int w = blockIdx.x * WARPS + warp;
        const long long b0 = deal.begin(blockIdx.x * WARPS), b1 = deal.begin((blockIdx.x + 1) * WARPS);
        // The unit that the share ends in, if the block's next warp goes on with it: the warps of the block that hold parts of it, but
        // the last, share its rows out among them, so that no warp has rows of two units.
        if (x0 < x1 && u1 > x1 && x1 < b1) {
            int w0 = w, w1 = w + 1;
            while (w0 > (int)blockIdx.x * WARPS && deal.begin(w0) > u0) --w0;
            while (w1 + 1 < (int)(blockIdx.x + 1) * WARPS && deal.begin(w1 + 1) < min(u1, b1)) ++w1;
            const bool done = u0 >= b0 && u1 <= b1;
            const int to = 2 * part.warps + 2 * blockIdx.x + (u0 > b0);
            join_warp<T, HDP>(a, part, s, unit, 2 * w0 + (deal.begin(w0) < u0), 2 * (w0 + 1), w1 - w0, w - w0, done ? -1 : to);
        }
    }
}

// Adds up the blocks' parts of the units that were cut between blocks, in the order of the tiles (4 us: two dependent reads).  Block (b, row) looks at the
// border after block b's share and does the unit that it is the first to cut; a thread per element, in JOIN_Y groups
// that take the parts in turn.
constexpr int JOIN_Y = 4;
template <class T, int HDP>
__global__ void __launch_bounds__(HDP * JOIN_Y)
    kv_join_kernel(const __grid_constant__ KvAttend a, int blocks, int block_warps, void* space) {
    __shared__ float s_o[JOIN_Y][HDP], s_l[JOIN_Y], s_m[JOIN_Y];
    pdl_trigger();
    pdl_wait();
    const Partials part = partials_at<HDP>(space, blocks, blocks * block_warps);
    const int kvh = a.c.kv_heads, n = a.rows.n, b0 = blockIdx.x;
    const Deal deal(part.first[n], part.warps);
    const long long cut = deal.begin((b0 + 1) * block_warps);
    if (cut >= deal.total) return;
    const int i = warp_last_le(n, cut, [&](int k) { return part.first[k]; });
    const int row0 = a.rows.at(i), m = a.rows.at(i + 1) - row0;
    const long long first = part.first[i];
    const int units = kvh * ((m * a.group + 15) / 16);
    const long long tiles = (part.first[i + 1] - first) / units;
    const int unit = (int)((cut - first) / tiles);
    const long long u0 = first + unit * tiles;
    if (u0 == cut || deal.begin(b0 * block_warps) > u0) return;
    const int row = unit / kvh * 16 + blockIdx.y, head = unit % kvh;
    if (row >= m * a.group) return;
    const int b1 = deal.owner(u0 + tiles - 1) / block_warps, odd = deal.begin(b0 * block_warps) != u0;
    auto slot = [&](int b) { return (size_t)(2 * part.warps + 2 * b + (b == b0 ? odd : 0)) * 16 + blockIdx.y; };
    const int d = threadIdx.x, y = threadIdx.y;
    float top = -INFINITY, l = 0.f, o = 0.f;
    for (int b = b0 + y; b <= b1; b += JOIN_Y) top = fmaxf(top, __ldcg(part.ml + slot(b) * 2));
    if (d == 0) s_m[y] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < JOIN_Y; ++k) top = fmaxf(top, s_m[k]);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll 4
    for (int b = b0 + y; b <= b1; b += JOIN_Y) {
        const float away = __ldcg(part.ml + slot(b) * 2) - base, f = ex2(away);
        l += move_norm(__ldcg(part.ml + slot(b) * 2 + 1), away, f);
        o = fmaf(__ldcg(part.o + slot(b) * HDP + d), f, o);
    }
    s_o[y][d] = o;
    if (d == 0) s_l[y] = l;
    __syncthreads();
    if (y) return;
    o = l = 0.f;
#pragma unroll
    for (int k = 0; k < JOIN_Y; ++k) o += s_o[k][d], l += s_l[k];
    const bool seen = l > 0.f || l != l;
    const int query = a.query_of(row), qh = head * a.group + row - query * a.group;
    if (d < a.c.head_dim)
        static_cast<T*>(a.out)[(row0 + (long long)query) * a.out_stride + (long long)qh * a.c.head_dim + d] =
            from_f<T>(seen ? o * NORM / l : 0.f);
    if (d == 0 && a.lse)
        a.lse[(row0 + (long long)query) * a.heads + qh] = seen ? (top + NORM_LOG2 + log2f(l)) * LN2 : -INFINITY;
}

// ---------------------------------------------------------------------------
// Pieces of units, a block each (kv8_shared.cu): the block's warps take even shares of a piece's tiles and join their sums in
// shared memory.  Where units are many and short this has a quarter of kv_attend_kernel's latency: a block looks up one entry and not the
// lengths of all sequences, and nothing goes through global memory twice.  Rows at most 8: tokens as the rows of operand A.
// ---------------------------------------------------------------------------
template <class T, int HDP, bool LOW> struct PieceShape {
    static constexpr int BLOCKS = piece_blocks(HDP, LOW);
    static constexpr int STAGE = 2 * KV_BLOCK * HDP, STAGES = HDP == 256 || (HDP == 128 && LOW) ? 3 : 4;
    static constexpr int RING = PIECE_WARPS * STAGES * STAGE, SUMS = PIECE_WARPS * 16 * (HDP + 2) * 4;
    static constexpr int BYTES = RING > SUMS ? RING : SUMS;
    static_assert(BLOCKS * (BYTES + 1024) <= 227 * 1024, "shared memory");
};
template <class T, int CODE, int HDP, bool LOW, bool ALL_LOW>
__device__ __forceinline__ void piece_sums(const KvAttend& a, const PieceWork& s, int head, int r0, int x0, int x1, uint8_t* ring,
                                           const Partials& sums) {
    using P = PieceShape<T, HDP, ALL_LOW>;
    constexpr int STAGES = P::STAGES, STAGE = P::STAGE, CH = HDP / 16;
    const int lane = threadIdx.x & 31, D = a.c.head_dim;
    auto look = [&](int x) { return x < x1 ? tile_of<CODE>(a, s, x, head) : Tile{-1, 0.f, 0.f, 0.f, 0}; };
    // Lane l knows tile base + l (now) and the 32 after those (next).
    Tile now = look(x0 + lane), next = now;
    int base = x0, into = 0;
    auto fetch = [&](int x) {  // queue the copies of tile x; always one group
        const int k = x - base;
        const long long at = __shfl_sync(0xffffffffu, k < 32 ? now.at : next.at, k & 31);
        if (x < x1 && at >= 0) {
            const uint32_t dst = smem_u32(ring) + into * STAGE;
            const uint8_t *ks = static_cast<const uint8_t*>(a.c.k) + at, *vs = static_cast<const uint8_t*>(a.c.v) + at;
#pragma unroll
            for (int e0 = 0; e0 < KV_BLOCK * CH; e0 += 32) {
                const int e = e0 + lane, r = e / CH, c = e % CH;
                if (c * 16 < D) {
                    cp16(dst + tile_at<HDP>(r, c), ks + r * D + c * 16);
                    cp16(dst + KV_BLOCK * HDP + tile_at<HDP>(r, c), vs + r * D + c * 16);
                }
            }
        }
        cp_commit();
        into = into + 1 == STAGES ? 0 : into + 1;
    };
    if (D < HDP) {  // chunks past the head's width stay zero
        for (int st = 0; st < STAGES; ++st)
            for (int e = lane; e < 2 * KV_BLOCK * CH; e += 32) {
                const int r = e / CH % KV_BLOCK, c = e % CH;
                if (c * 16 >= D)
                    *reinterpret_cast<uint4*>(ring + st * STAGE + e / (KV_BLOCK * CH) * (KV_BLOCK * HDP) + tile_at<HDP>(r, c)) =
                        make_uint4(0, 0, 0, 0);
            }
        __syncwarp();
    }
#pragma unroll 1
    for (int k = 0; k < STAGES; ++k) fetch(x0 + k);
    std::conditional_t<LOW, RowsLow<T, CODE, HDP>, Rows<T, CODE, HDP>> r;
    r.load(a, s, head, r0);
    if (x1 - x0 > 32) next = look(x0 + 32 + lane);
    int from = 0;
    for (int x = x0; x < x1;) {
        if (x - base >= 32) {
            base += 32;
            now = next;
            next = look(base + 32 + lane);
        }
        cp_wait<STAGES - 2>();  // tiles x and x + 1 are there
        __syncwarp();
        const bool two = x + 1 < x1;
        const int k0 = x - base, s1 = from + 1 == STAGES ? 0 : from + 1;
        const Tile d[2] = {tile_from(now, k0), k0 < 31 ? tile_from(now, k0 + 1) : tile_from(next, 0)};
        const uint8_t* const k[2] = {ring + from * STAGE, ring + s1 * STAGE};
        const bool on[2] = {r.sees(d[0], a.win.sinks), two && r.sees(d[1], a.win.sinks)};
        if (on[0] || on[1]) r.tiles(d, k, on, a.win.sinks);
        __syncwarp();  // the stages are read before their next copies are queued
        fetch(x + STAGES);
        if (two) fetch(x + STAGES + 1);
        x += 1 + two;
        from = two ? (s1 + 1 == STAGES ? 0 : s1 + 1) : s1;
    }
    cp_wait<0>();
    __syncthreads();   // all rings have been read: the sums take their place
    r.emit(a, s, head, r0, &sums, threadIdx.x >> 5);
}

// ALL_LOW: no unit has more than 8 rows, which takes fewer registers
template <class T, int CODE, int HDP, bool ALL_LOW>
__global__ void __launch_bounds__(PIECE_WARPS * 32, (PieceShape<T, HDP, ALL_LOW>::BLOCKS))
    kv_piece_kernel(const __grid_constant__ KvAttend a, const __grid_constant__ KvPieces p) {
    using P = PieceShape<T, HDP, ALL_LOW>;
    extern __shared__ __align__(128) uint8_t ring_all[];
    // Beside the launch before, of which it reads nothing: pieces start where its blocks have ended.  That launch is an ordinary one
    // (launch_after), so the dealing launch, and all that is older, had ended before it began, and is in memory for this one as well;
    // behind a launch that begins early and waits only that one could rely on it.  Each block waits for the launch before at its end, so that whatever
    // waits for this launch waits for both.  (96 sequences in 6 groups behind up to 12,000 tokens: 103 us where this launch waits, 91 beside.)
    if (!p.beside) pdl_wait();
    pdl_trigger();
    const int b = (int)blockIdx.x, warp = threadIdx.x >> 5, kvh = a.c.kv_heads, D = a.c.head_dim;
    // Entries without pieces are before those with.  Reads that hang on others take a microsecond each: of a few entries all are read at once.
    const int total = __ldg(p.total);
    int i = -1;
    if (p.count <= 128) {
        const int lane = threadIdx.x & 31;
        int at[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) at[k] = k * 32 + lane < p.count ? __ldg(p.first + k * 32 + lane) : INT32_MAX;
#pragma unroll
        for (int k = 0; k < 4; ++k) i += __popc(__ballot_sync(0xffffffffu, at[k] <= b));
    } else {
        i = warp_last_le(p.count, b, [&](int k) { return __ldg(p.first + k); });
    }
    if (b >= total) {
        pdl_wait();
        return;
    }
    const KvEntry e = p.entries[i];
    const int in = b - e.first, unit = in / e.cuts, k = in - unit * e.cuts, head = unit % kvh, r0 = unit / kvh * 16;
    const int t0 = (int)((long long)e.s.tiles * k / e.cuts), n = (int)((long long)e.s.tiles * (k + 1) / e.cuts) - t0;
    const int x0 = t0 + n * warp / PIECE_WARPS, x1 = t0 + n * (warp + 1) / PIECE_WARPS;
    const int rows = min(16, e.s.m * a.group - r0);
    Partials sums;
    sums.o = reinterpret_cast<float*>(ring_all);
    sums.ml = sums.o + PIECE_WARPS * 16 * HDP;
    uint8_t* ring = ring_all + warp * P::STAGES * P::STAGE;
    if constexpr (ALL_LOW) {
        piece_sums<T, CODE, HDP, true, true>(a, e.s, head, r0, x0, x1, ring, sums);
    } else {
        if (rows <= 8) piece_sums<T, CODE, HDP, true, false>(a, e.s, head, r0, x0, x1, ring, sums);
        else piece_sums<T, CODE, HDP, false, false>(a, e.s, head, r0, x0, x1, ring, sums);
    }
    __syncthreads();
    // the warps' parts become the block's: 4 elements of a row to a thread
    const float2* ml = reinterpret_cast<const float2*>(sums.ml);
    for (int x = threadIdx.x; x < rows * (HDP / 4); x += PIECE_WARPS * 32) {
        const int r = x / (HDP / 4), c = x % (HDP / 4) * 4;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < PIECE_WARPS; ++w) top = fmaxf(top, ml[w * 16 + r].x);
        const float base = top == -INFINITY ? 0.f : top;
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < PIECE_WARPS; ++w) {
            const float2 y = ml[w * 16 + r];
            const float f = ex2(y.x - base);
            const float4 q = *reinterpret_cast<const float4*>(sums.o + (w * 16 + r) * HDP + c);
            l += move_norm(y.y, y.x - base, f);
            o.x = fmaf(q.x, f, o.x), o.y = fmaf(q.y, f, o.y), o.z = fmaf(q.z, f, o.z), o.w = fmaf(q.w, f, o.w);
        }
        const int row = r0 + r, query = a.query_of(row), qh = head * a.group + row - query * a.group;
        long long at = (e.s.row0 + (long long)query) * a.heads + qh;
        float* to = i < p.own ? p.o0 : p.o1;
        float2* to_ml = i < p.own ? p.ml0 : p.ml1;
        if (e.cuts > 1) at = (long long)(e.slot + in) * 16 + r, to = p.slot_o, to_ml = p.slot_ml;
        if (c < D) *reinterpret_cast<float4*>(to + at * D + c) = make_float4(o.x * NORM, o.y * NORM, o.z * NORM, o.w * NORM);
        if (c == 0) to_ml[at] = make_float2(top, l);
    }
    pdl_wait();
}

template <class T, int CODE, int HDP, bool ALL_LOW>
cudaError_t launch_pieces(const KvAttend& a, const KvPieces& p, unsigned blocks, cudaStream_t s) {
    using P = PieceShape<T, HDP, ALL_LOW>;
    const auto kernel = kv_piece_kernel<T, CODE, HDP, ALL_LOW>;
    static std::atomic<uint64_t> ready{0};
    const uint64_t bit = 1ull << (a.c.device & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, P::BYTES);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_k(kernel, dim3(blocks), dim3(PIECE_WARPS * 32), P::BYTES, s, 1, a, p);
}
template <class T, int CODE, int HDP> cudaError_t launch_pieces(const KvAttend& a, const KvPieces& p, unsigned blocks, cudaStream_t s) {
    return p.low ? launch_pieces<T, CODE, HDP, true>(a, p, blocks, s) : launch_pieces<T, CODE, HDP, false>(a, p, blocks, s);
}

template <class T, int CODE, int HDP, bool LOW>
cudaError_t launch_attend(const KvAttend& a, bool split, int sms, void* space, cudaStream_t s) {
    using S1 = Shape<T, HDP, LOW, true>;
    using S0 = Shape<T, HDP, LOW, false>;
    const int smem = split ? S1::BYTES : S0::BYTES;
    const auto kernel = split ? kv_attend_kernel<T, CODE, HDP, LOW, true> : kv_attend_kernel<T, CODE, HDP, LOW, false>;
    static std::atomic<uint64_t> ready[2];  // devices on which the kernels may use their shared memory
    const uint64_t bit = 1ull << (a.c.device & 63);
    cudaError_t e = cudaSuccess;
    if (!(ready[split].load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready[split].fetch_or(bit, std::memory_order_relaxed);
    }
    if (!split) {
        const unsigned units = (unsigned)a.tiles_of_all(16) * a.c.kv_heads;
        return launch_k(kernel, dim3((units + S0::WARPS - 1) / S0::WARPS), dim3(S0::WARPS * 32), smem, s, 1, a, space);
    }
    e = launch_k(kernel, dim3(sms), dim3(S1::WARPS * 32), smem, s, 1, a, space);
    if (e != cudaSuccess || sms < 2) return e;
    return launch_k(kv_join_kernel<T, HDP>, dim3(sms - 1, std::max(1, std::min(16, a.max_new * a.group))), dim3(HDP, JOIN_Y), 0, s, 1, a,
                    sms, S1::WARPS, space);
}
template <class T, int CODE, int HDP>
cudaError_t launch_attend(const KvAttend& a, bool split, int sms, void* space, cudaStream_t s) {
    return (long long)a.max_new * a.group <= 8 ? launch_attend<T, CODE, HDP, true>(a, split, sms, space, s)
                                               : launch_attend<T, CODE, HDP, false>(a, split, sms, space, s);
}

}  // namespace

// kv8_attn.cu is compiled once for each kind of code (kv8_attn_e4m3.cu includes it)
template <int CODE>
cudaError_t kv_launch_attend(const KvAttend& a, int dtype, bool split, int sms, void* space, cudaStream_t s) {
    const int d = a.c.head_dim;
    if (dtype == CAC_DTYPE_BF16)
        return d <= 64    ? launch_attend<bf16, CODE, 64>(a, split, sms, space, s)
               : d <= 128 ? launch_attend<bf16, CODE, 128>(a, split, sms, space, s)
                          : launch_attend<bf16, CODE, 256>(a, split, sms, space, s);
    return d <= 64    ? launch_attend<float, CODE, 64>(a, split, sms, space, s)
           : d <= 128 ? launch_attend<float, CODE, 128>(a, split, sms, space, s)
                      : launch_attend<float, CODE, 256>(a, split, sms, space, s);
}
template cudaError_t kv_launch_attend<KV8_ATTN_CODE>(const KvAttend&, int, bool, int, void*, cudaStream_t);

template <int CODE>
cudaError_t kv_launch_pieces(const KvAttend& a, const KvPieces& p, int dtype, unsigned blocks, cudaStream_t s) {
    const int d = a.c.head_dim;
    if (dtype == CAC_DTYPE_BF16)
        return d <= 64    ? launch_pieces<bf16, CODE, 64>(a, p, blocks, s)
               : d <= 128 ? launch_pieces<bf16, CODE, 128>(a, p, blocks, s)
                          : launch_pieces<bf16, CODE, 256>(a, p, blocks, s);
    return d <= 64    ? launch_pieces<float, CODE, 64>(a, p, blocks, s)
           : d <= 128 ? launch_pieces<float, CODE, 128>(a, p, blocks, s)
                      : launch_pieces<float, CODE, 256>(a, p, blocks, s);
}
template cudaError_t kv_launch_pieces<KV8_ATTN_CODE>(const KvAttend&, const KvPieces&, int, unsigned, cudaStream_t);

#if KV8_ATTN_CODE == 0
size_t kv_attend_bytes(int head_dim, int sms) {
    return head_dim <= 64 ? partial_bytes<64>(sms) : head_dim <= 128 ? partial_bytes<128>(sms) : partial_bytes<256>(sms);
}
#endif

}  // namespace cac
