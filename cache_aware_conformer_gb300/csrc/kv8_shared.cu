// Attention over the paged 8-bit K/V cache for sequences that share a prefix (include/cac_kv8.h,
// cac_kv8_attend_shared).
//
// A softmax over a sequence's tokens is a join of softmaxes over any parts of them: with a part's maximum m, its sum
// l of 2^(t - m) and its sum o of the weighted values, M = max m over the parts,
//   out = sum o 2^(m - M) / sum l 2^(m - M).
// So the tokens that all queries of a group see in the same pages are read once, with all queries of the group as rows: on the
// tensor cores of the 5th generation where these are many, together with the other tokens where they are few.  What each sequence has
// to itself is read for it, in pieces of even length, a block each; a last launch joins the parts.
//
// Measured (bf16, 8 K/V heads of 128, us; in brackets what the bytes take at a copy's rate): 64 sequences of up to 1,000 tokens behind 32,000, group
// 4, int8: 87 (19.5); launch by launch, as a profiler runs them, finding 8, dealing out 11, the shared tokens 40, the others 25, the join 11 (the
// shared tokens and the others overlap in part); 4 sequences behind 60,000: 64 (19.6); 96 sequences in 6 groups behind up to 12,000, group 8, e4m3: 91
// (21.7).  In the first, the shared tokens' kernel issues in 52 % of the cycles in which an SM is active, and its tensor cores work in 39 % of them (34 %
// of the launch); shared memory bounds it, through which a tile of 128 tokens and 256 rows brings 32 KB
// of codes in and out, 64 KB of fp16, and 260 KB as operands: about 3,100 of the 4,000 clocks that it takes.  Without the exponentials, or without
// the arithmetic of the conversion, it takes as long.
//
// What enters the tensor cores is fp16: codes exactly; for bf16 calls queries exactly after a power of two, and weights with 11 bits, three more than a
// result has; for fp32 calls both as two parts, 22 bits.  Maxima, norms and sums are fp32.  Against 64 bits the results are off by 0.0016 for bf16, its
// own rounding, and by 1.0e-6 to 2.1e-6 for fp32, where weights and sums in fp32 give 0.7e-6 to 2.4e-6 and cac_kv8_attend 0.6e-6 to 1.6e-6.
//
// What is shared is looked up on the device in each call: blocks of 16 tokens that every query of the group sees whole, in front of the
// first page of those in which the tables differ.  Nothing but the sequences' tables is compared, so a result never hangs on what
// the caller believes of them.
#include <algorithm>
#include <atomic>

#include "kv8_tc.cuh"

namespace cac {
namespace {

constexpr int PLAN_BLOCKS = 8, PLAN_THREADS = 512;   // of a group: a cluster
constexpr int LEAST_BLOCKS = 1;                      // shared blocks below this are not worth it

struct SharedCall {
    KvAttend a;                // rows, ids and window of the whole call
    const int32_t* groups;     // [n_groups + 1], NULL: one group
    int n_groups;              // at least 1
    int2* skip;                // [n]
    int32_t* group_of;         // [n] of those that share
    int4* shared;              // [n_groups]
    int32_t* group_rows;       // [n_groups + 1]
};

// One cluster for each group: which blocks its sequences share.
__global__ void __launch_bounds__(PLAN_THREADS) kv_plan_shared_kernel(const __grid_constant__ SharedCall p) {
    __shared__ int s_lo, s_hi, s_bad, s_leader, s_members, s_same;
    __shared__ int s_all[PLAN_BLOCKS];
    pdl_trigger();
    pdl_wait();
    const KvAttend& a = p.a;
    const int n = a.rows.n, g = blockIdx.x, rank = blockIdx.z, t = threadIdx.x, lane = t & 31;
    if (t == 0) s_lo = 0, s_hi = INT32_MAX, s_bad = 0, s_leader = INT32_MAX, s_members = 0, s_same = INT32_MAX;
    __syncthreads();
    auto group_at = [&](int k) { return p.groups ? p.groups[k] : k * n; };
    auto row_at = [&](int i) { return a.rows.at(i); };
    // the groups of the call: each block looks at all of them, so that all agree
    for (int k = t; k < p.n_groups; k += PLAN_THREADS) {
        const int x = group_at(k), y = group_at(k + 1);
        if (x < 0 || y < x || y > n) s_bad = 1;
    }
    __syncthreads();
    const bool fine = !s_bad;
    const int g0 = fine ? group_at(g) : 0, g1 = fine ? group_at(g + 1) : 0;
    __syncthreads();
    if (!fine && t == 0) latch_error(a.c.status, CAC_E_BOUNDS);

    // what all of the group's queries see; a sequence without queries does not matter, one that the call may not name ends the sharing
    int lo = 0, hi = INT32_MAX, members = 0, leader = INT32_MAX;
    bool bad = false;
    for (int i = g0 + t; i < g1; i += PLAN_THREADS) {
        const int r0 = row_at(i), m = row_at(i + 1) - r0, id = a.ids[i];
        if (m == 0) continue;
        if (r0 < 0 || m < 0 || r0 + (long long)m > a.rows.rows || m > a.max_new || id < 0 || id >= a.c.max_seqs) {
            bad = true;
            continue;
        }
        const int len = a.c.lens[id], first = len - m;
        if (len <= 0 || first < 0) {
            bad = true;
            continue;
        }
        lo = max(lo, a.win.low(len - 1));
        hi = min(hi, a.win.high(first, len));
        leader = min(leader, i);
        ++members;
    }
    if (members) {
        atomicMax(&s_lo, lo);
        atomicMin(&s_hi, hi);
        atomicMin(&s_leader, leader);
        atomicAdd(&s_members, members);
    }
    if (bad) s_bad = 1;
    __syncthreads();
    const int first_block = (s_lo + KV_BLOCK - 1) / KV_BLOCK;
    const bool some = fine && !s_bad && s_members >= 2 && s_hi / KV_BLOCK - first_block >= LEAST_BLOCKS;

    // Pages from that of the first block on, in front of the first one in which a table differs from the leader's: warps take the members in
    // turn.  Pages before those are not read as shared: one sequence may have released more of them than another.
    if (some) {
        const int pages = min((s_hi + a.c.page_tokens - 1) / a.c.page_tokens, a.c.max_pages);
        const int32_t* own = a.c.table + (long long)a.ids[s_leader] * a.c.max_pages;
        int same = pages;
        for (int i = s_leader + 1 + rank * (PLAN_THREADS / 32) + (t >> 5); i < g1; i += PLAN_BLOCKS * (PLAN_THREADS / 32)) {
            if (row_at(i + 1) == row_at(i)) continue;
            const int32_t* other = a.c.table + (long long)a.ids[i] * a.c.max_pages;
            if (other == own) continue;
            constexpr int GO = 8;
            for (int b = first_block * KV_BLOCK / a.c.page_tokens; b < same; b += 32 * GO) {
                int x[GO], y[GO];
#pragma unroll
                for (int u = 0; u < GO; ++u) {
                    const int k = b + u * 32 + lane;
                    x[u] = k < same ? own[k] : 0, y[u] = k < same ? other[k] : 0;
                }
                int mine = INT32_MAX;
#pragma unroll
                for (int u = GO - 1; u >= 0; --u)
                    if (x[u] != y[u]) mine = b + u * 32 + lane;
                mine = __reduce_min_sync(0xffffffffu, mine);
                if (mine < same) same = mine;   // ends the loop too
            }
        }
        if (lane == 0) atomicMin(&s_same, same);
    }
    __syncthreads();
    if (t < PLAN_BLOCKS)
        asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(dsmem_addr(&s_all[rank], t)), "r"(some ? s_same : 0) : "memory");
    cluster_sync();
    int same = s_all[0];
#pragma unroll
    for (int k = 1; k < PLAN_BLOCKS; ++k) same = min(same, s_all[k]);
    const int end_block = some ? (int)min((long long)s_hi, (long long)same * a.c.page_tokens) / KV_BLOCK : 0;
    const bool share = some && end_block - first_block >= LEAST_BLOCKS;
    const int2 range = share ? make_int2(first_block, end_block) : make_int2(0, 0);

    const int step = PLAN_BLOCKS * PLAN_THREADS, me = rank * PLAN_THREADS + t;
    for (int i = g0 + me; i < g1; i += step) p.skip[i] = range, p.group_of[i] = g;
    if (g == 0) {  // sequences of no group
        const int before = fine ? group_at(0) : n, after = fine ? group_at(p.n_groups) : n;
        for (int i = me; i < before; i += step) p.skip[i] = make_int2(0, 0);
        for (int i = after + me; i < n; i += step) p.skip[i] = make_int2(0, 0);
        for (int k = me; k <= p.n_groups; k += step) p.group_rows[k] = fine ? row_at(group_at(k)) : 0;
    }
    if (rank == 0 && t == 0) p.shared[g] = make_int4(share ? a.ids[s_leader] : 0, range.x, range.y, 0);
}

// ---------------------------------------------------------------------------
// The shared tokens of groups with many query rows, on the 5th-generation tensor cores: the roles and the mathematics of
// kv_prompt_kernel (kv8_prompt.cu), without masks, since every row sees every token.  A unit is 128 or 256 query rows of a group (row
// = query * heads of a K/V head + head) and a K/V head; its 128-token tiles are cut into pieces, one to a block, so that all SMs have
// the same number of tiles: few rows over a long prefix would leave most of them idle otherwise.  A unit that is cut leaves sums for
// kv_join_shared_kernel.
// ---------------------------------------------------------------------------
struct PrefixCall {
    KvAttend a;             // rows: the groups'
    const int4* shared;     // of each group: whose table, and the blocks [y, z)
    const int4* cut;        // of each group: first piece, pieces of each unit, first slot of units that are cut
    int groups;             // of this launch
    float* part_o;          // units in one piece: [rows][heads][head_dim]
    float2* part_ml;
    float* slot_o;          // [slot][rows of a block][head_dim] of pieces of units that are cut, and
    float2* slot_ml;        // [slot][rows of a block]
};

// Which piece is block b's
struct Piece {
    int id, head, row0, r0, rows;    // whose table; K/V head; the group's first row in the call; rows r0 .. r0 + rows - 1 of the group's
    int block0, blocks;              // of 16 tokens; 0: there is no such piece
    int slot;                        // of its results; -1: its unit is not cut
    int halves;                      // of 64 tokens
};
template <int ROWS> __device__ __forceinline__ Piece find_piece(const PrefixCall& p) {
    const KvAttend& a = p.a;
    const int kvh = a.c.kv_heads, b = (int)blockIdx.x;
    Piece q{};
    // groups without pieces are before those with
    int4 cut;
    int4 sh;
    int first0, row0, row1;
    if (p.groups <= 32) {   // all at once: reads that hang on others take a microsecond each
        const int lane = threadIdx.x & 31, at = min(lane, p.groups - 1);
        cut = p.cut[at], sh = p.shared[at], row0 = a.rows.at(at), row1 = a.rows.at(at + 1);
        first0 = __shfl_sync(0xffffffffu, cut.x, 0);
        const int g = __popc(__ballot_sync(0xffffffffu, lane < p.groups && cut.x <= b + first0)) - 1;
        cut.x = __shfl_sync(0xffffffffu, cut.x, g), cut.y = __shfl_sync(0xffffffffu, cut.y, g), cut.z = __shfl_sync(0xffffffffu, cut.z, g);
        sh.x = __shfl_sync(0xffffffffu, sh.x, g), sh.y = __shfl_sync(0xffffffffu, sh.y, g), sh.z = __shfl_sync(0xffffffffu, sh.z, g);
        row0 = __shfl_sync(0xffffffffu, row0, g), row1 = __shfl_sync(0xffffffffu, row1, g);
    } else {
        first0 = __ldg(&p.cut[0].x);
        const int g = warp_last_le(p.groups, (long long)b + first0, [&](int k) { return __ldg(&p.cut[k].x); });
        cut = p.cut[g], sh = p.shared[g], row0 = a.rows.at(g), row1 = a.rows.at(g + 1);
    }
    const int rows = (row1 - row0) * a.group, tiles = (sh.z - sh.y + 7) / 8;
    const int in = b + first0 - cut.x;
    if (cut.y == 0 || in >= (rows + ROWS - 1) / ROWS * kvh * cut.y) return q;
    const int unit = in / cut.y, k = in - unit * cut.y;
    const int t0 = (int)((long long)tiles * k / cut.y), t1 = (int)((long long)tiles * (k + 1) / cut.y);
    q.id = sh.x, q.head = unit % kvh, q.row0 = row0, q.r0 = unit / kvh * ROWS;
    q.rows = min(ROWS, rows - q.r0);
    q.block0 = sh.y + 8 * t0;
    q.blocks = min(sh.y + 8 * t1, sh.z) - q.block0;
    q.slot = cut.y > 1 ? cut.z + in : -1;
    q.halves = (q.blocks + 3) / 4;
    return q;
}

// The prompts' kernel has its tokens from L2, where other blocks' loads have brought them; here they come from memory, and a load
// into registers ahead of each piece left an SM with 12 KB on its way (a tile took 3.4 us; with three ahead, 3.8: the compiler waits for
// all of them).  So the converters have their codes brought by bulk copies, a piece of 16 tokens each, `SLOTS` ahead.
template <class T, int HDP, int TILES> struct XShape : PShape<T, HDP, TILES> {
    using P = PShape<T, HDP, TILES>;
    static constexpr int PIECE = KV_BLOCK * HDP, ROOM = (225 * 1024 - P::BYTES) / (P::CONV * (PIECE + 8));
    static constexpr int SLOTS = ROOM < 6 ? ROOM : 6, OFF_RAW = (P::OFF_BAR + 21 * 8 + 16 + 127) / 128 * 128;
    static constexpr int OFF_RAW_BAR = OFF_RAW + P::CONV * SLOTS * PIECE;
    static constexpr int XBYTES = OFF_RAW_BAR + P::CONV * SLOTS * 8 + 1024;
    static constexpr int XSMEM = XBYTES > 120 * 1024 ? XBYTES : 120 * 1024;  // one block an SM
    static_assert(SLOTS >= 2 && XSMEM <= 227 * 1024, "shared memory");
    static_assert(4 * 32 * 32 * 4 <= P::PARTS * P::TILE, "results on their way out take the place of a row tile's queries");
};

// one thread of a converged warp, the same each time
__device__ __forceinline__ bool elected() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

template <class T, int CODE, int HDP, int TILES>
__global__ void __launch_bounds__(PShape<T, HDP, TILES>::THREADS, 1) kv_prefix_kernel(const __grid_constant__ PrefixCall p) {
    using S = XShape<T, HDP, TILES>;
    constexpr int ROWS = S::NM * PT_ROWS;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);   // an offset: shared memory to the compiler too
    float* s_scale = reinterpret_cast<float*>(smem + S::OFF_SC);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);
    uint64_t *q_full = bar, *k_full = bar + 1, *k_empty = bar + 3, *v_full = bar + 5, *v_empty = bar + 7;
    uint64_t *s_full = bar + 9, *p_full = bar + 13, *o_done = bar + 17;  // s_full, p_full, o_done: [row tile][place]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 21);
    const KvAttend& a = p.a;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, D = a.c.head_dim;
    const Piece w = find_piece<ROWS>(p);   // no wait: an ordinary launch (launch_prefix)
    if (w.blocks == 0) {
        pdl_trigger();
        return;
    }
    const int R = w.r0 + w.rows, nm = __shfl_sync(0xffffffffu, w.rows > PT_ROWS ? 2 : 1, 0), halves = __shfl_sync(0xffffffffu, w.halves, 0);

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
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    bool ok = true;

    if (warp < S::SOFT) {
        // -------------------------------------------------------------- softmax: a thread per row
        const int x = warp >> 2, r = (warp & 3) * 32 + lane, row = w.r0 + x * PT_ROWS + r;
        if (x < nm) {
            const bool on = row < R;
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
                        const T* src = static_cast<const T*>(a.q) + (w.row0 + (long long)q) * a.q_stride +
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
                const int j = h >> 1;
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
                const int query = on ? a.query_of(row) : 0, qh = w.head * a.group + (on ? row - query * a.group : 0);
                const long long at = w.slot >= 0 ? (long long)w.slot * ROWS + x * PT_ROWS + r : (w.row0 + (long long)query) * a.heads + qh;
                // 32 columns at a time by way of shared memory, where the row tile's queries were: eight threads store 128 bytes of a row (a
                // row to a thread took 7 us)
                float* pad = reinterpret_cast<float*>(smem + x * S::PARTS * S::TILE) + (warp & 3) * 32 * 32;
                float* to = w.slot >= 0 ? p.slot_o : p.part_o;
#pragma unroll
                for (int c = 0; c < HDP / 32; ++c) {
                    float v[32];
                    __syncwarp();  // the loads are for a converged warp
                    tmem_ld32(col_o + c * 32, v);
                    if (S::WIDE && w.halves > S::FLUSH) {
                        float sum[32];
                        tmem_ld32(col_sum + c * 32, sum);
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] += sum[k];
                    }
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        *reinterpret_cast<float4*>(pad + lane * 32 + (k ^ (lane & 7) << 2)) =
                            make_float4(v[k] * S::NORM, v[k + 1] * S::NORM, v[k + 2] * S::NORM, v[k + 3] * S::NORM);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int of = 4 * k + (lane >> 3), e = c * 32 + (lane & 7) * 4;
                        const long long row_at = __shfl_sync(0xffffffffu, at, of);
                        const bool there = __shfl_sync(0xffffffffu, on, of);
                        if (there && e < D) *reinterpret_cast<float4*>(to + row_at * D + e) =
                                *reinterpret_cast<const float4*>(pad + of * 32 + (((lane ^ of) & 7) << 2));
                    }
                }
                if (on) (w.slot >= 0 ? p.slot_ml : p.part_ml)[at] = make_float2(m, l);
            }
        }
    } else if (warp < S::SOFT + S::CONV) {
        // -------------------------------------------------------------- converters
        // piece n: 16 tokens (block n % 8) of tile n / 16, K where n / 8 is even, else V; warp cw takes every CONV-th
        const int cw = warp - S::SOFT, pieces = (w.blocks + 7) / 8 * 16;
        const int sub = lane >> 2, c4 = lane & 3;   // token % 8 and chunk % 4 of a lane's loads
        constexpr int NL = HDP / 32;
        // Lane l knows where the warp's l-th piece of the next 32 lies, and its scales (with K: the scores need both).
        struct Spot {
            long long at;      // -1: past the end, or no page
            float ks, lv, iv;
        };
        auto look = [&](int n) {
            Spot t{-1, 1.f, -INFINITY, 0.f};  // a block that is not there: any K scale will do, its weights are 2^-inf
            const int block = (n >> 4) * 8 + (n & 7);
            if (n < pieces && block < w.blocks) {
                const int tok = (w.block0 + block) * KV_BLOCK;
                const int page = a.c.table[(long long)w.id * a.c.max_pages + tok / a.c.page_tokens];
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
        uint8_t* slots = smem + S::OFF_RAW + cw * S::SLOTS * S::PIECE;
        uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + S::OFF_RAW_BAR) + cw * S::SLOTS;
        if (lane == 0)
            for (int k = 0; k < S::SLOTS; ++k) mbar_init(raw_full + k, 1);
        fence_mbar_init();
        __syncwarp();
        auto copy = [&](int n, int slot, long long at) {   // lane 0
            if (n >= pieces) return;
            if (at < 0) {
                mbar_arrive(raw_full + slot);
                return;
            }
            mbar_expect_tx(raw_full + slot, KV_BLOCK * D);
            bulk_g2s(slots + slot * S::PIECE, static_cast<const uint8_t*>(n & 8 ? a.c.v : a.c.k) + at, KV_BLOCK * D, raw_full + slot);
        };
#pragma unroll
        for (int d = 0; d < S::SLOTS; ++d) {
            const long long at = __shfl_sync(0xffffffffu, here.at, d);
            if (lane == 0) copy(cw + S::CONV * d, d, at);
        }
        Spot then = here;
        int q = 0, slot = 0, phase = 0;  // the piece's place among the 32; its slot
        auto piece = [&](int n) {
            const float ks = __shfl_sync(0xffffffffu, here.ks, q), lv = __shfl_sync(0xffffffffu, here.lv, q),
                        iv = __shfl_sync(0xffffffffu, here.iv, q);
            const bool there = __shfl_sync(0xffffffffu, here.at, q) >= 0;
            if (q == 8) then = look(n + S::CONV * (24 + lane));  // the 32 after these: not before the first are on their way
            const int ahead = q + S::SLOTS;
            const long long ahead_at = __shfl_sync(0xffffffffu, ahead < 32 ? here.at : then.at, ahead & 31);
            if (++q == 32) {
                q = 0;
                here = then;
            }
            if (!warp_wait(raw_full + slot, phase)) return false;
            uint4 cur[NL];
            // Rows sub and sub + 8, elements of each 64: with two such parts, odd rows' other part first, so that the two rows of eight
            // threads touch all banks.
            const int odd = NL > 2 ? sub & 1 : 0;
#pragma unroll
            for (int y = 0; y < NL; ++y)
                cur[y] = there && ((y >> 1 ^ odd) * 4 + c4) * 16 < D
                             ? *reinterpret_cast<const uint4*>(slots + slot * S::PIECE + (sub + (y & 1) * 8) * D + c4 * 16 + (y >> 1 ^ odd) * 64)
                             : make_uint4(0, 0, 0, 0);
            __syncwarp();
            if (lane == 0) copy(n + S::CONV * S::SLOTS, slot, ahead_at);
            if (++slot == S::SLOTS) slot = 0, phase ^= 1;
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
                uint8_t* dst = to + (y >> 1 ^ odd) * S::PANEL + (y & 1) * 1024;
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
        int n = cw;
#pragma unroll 1
        for (; n < pieces; n += S::CONV)
            if (!piece(n)) {
                ok = false;
                break;
            }
        // after a wait that gave up: copies in flight land before the block's memory is another's
        for (int k = 0; !ok && k < S::SLOTS; ++k)
            if (!mbar_wait(raw_full + k, k < slot ? phase ^ 1 : phase)) break;
    } else {
        // -------------------------------------------------------------- MMA: a warp per row tile, which an elected thread issues for.
        // The whole warp goes round, and what the operands' addresses are made of is the same in all of its threads to the compiler too
        // (the index and the counts by a broadcast): they stay in uniform registers.  From one thread's own registers each
        // instruction took 160 clocks to issue, which was most of a tile's time.
        const int x = warp - S::SOFT - S::CONV;
        if (x < nm) {
            constexpr uint32_t qk = idesc_f16(128, PT_HALF, false), pv = idesc_f16(128, HDP, true);
            const uint64_t q0 = sdesc_k_sw128(smem + x * S::PARTS * S::TILE), k0 = sdesc_k_sw128(smem + S::OFF_K),
                           v0 = sdesc_mn_sw128(smem + S::OFF_V, S::PANEL);
            const uint32_t s0 = tmem + S::COL_S + x * 128, o0 = tmem + S::COL_O + x * HDP;
            auto scores = [&](int h) {
                if (elected()) {
                    const uint64_t kd = k0 + (((h >> 1 & 1) * S::TILE + (h & 1) * (PT_HALF * 128)) >> 4);
#pragma unroll
                    for (int part = 0; part < S::PARTS; ++part)
#pragma unroll
                        for (int k = 0; k < HDP / 16; ++k) {
                            const uint32_t step = (k >> 2) * (S::PANEL >> 4) + 2 * (k & 3);
                            mma_ss(s0 + (h & 1) * PT_HALF, q0 + part * (S::TILE >> 4) + step, kd + step, qk, part > 0 || k > 0);
                        }
                    tc_commit(s_full + 2 * x + (h & 1));
                    if (h & 1) tc_commit(k_empty + (h >> 1 & 1));
                }
                __syncwarp();
            };
            ok = warp_wait(q_full, 0) && warp_wait(k_full, 0);
            if (ok) {
                tc_fence_after();
                scores(0);
            }
            for (int h = 0; ok && h < halves; ++h) {
                const int st = h >> 1 & 1, next = h + 1;
                if (next < halves) {
                    // the next scores take the place of the weights before these: products into other accumulators need
                    // not run in order
                    if ((!(next & 1) && !warp_wait(k_full + (next >> 1 & 1), next >> 2 & 1)) ||
                        (h > 0 && !warp_wait(o_done + 2 * x + ((h - 1) & 1), (h - 1) >> 1 & 1))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    scores(next);
                }
                if ((!(h & 1) && !warp_wait(v_full + st, h >> 2 & 1)) || !warp_wait(p_full + 2 * x + (h & 1), h >> 1 & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elected()) {
                    const uint64_t vd = v0 + ((st * S::TILE + (h & 1) * (PT_HALF * 128)) >> 4);
#pragma unroll
                    for (int part = 0; part < S::PARTS; ++part)
#pragma unroll
                        for (int k = 0; k < PT_HALF / 16; ++k)
                            mma_ts(o0, s0 + (h & 1) * PT_HALF + part * 32 + 8 * k, vd + k * (2048 >> 4), pv,
                                   h % S::FLUSH > 0 || part > 0 || k > 0);
                    tc_commit(o_done + 2 * x + (h & 1));
                    if (h & 1) tc_commit(v_empty + st);
                }
                __syncwarp();
            }
        }
    }
    if (!ok) latch_error(a.c.status, CAC_E_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == S::WARPS - 1) tmem_dealloc(tmem, 512);
}

template <class T, int CODE, int HDP, int TILES> cudaError_t launch_prefix(const PrefixCall& p, unsigned blocks, cudaStream_t s) {
    using S = XShape<T, HDP, TILES>;
    const auto kernel = kv_prefix_kernel<T, CODE, HDP, TILES>;
    static std::atomic<uint64_t> ready{0};
    const uint64_t bit = 1ull << (p.a.c.device & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::XSMEM);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_after(kernel, dim3(blocks), dim3(S::THREADS), S::XSMEM, s, p);   // the pieces run beside it
}
// Row tiles of a block: one, which leaves room for more copies ahead, for a group of 128 rows, or several of half as many on average (a larger
// one among them has its tokens read once more for each 128 of its rows).
int prefix_tiles(const KvAttend& a, int dtype, int n_groups) {
    const long long rows = (long long)a.rows.rows * a.group;
    return (dtype == CAC_DTYPE_F32 && a.c.head_dim > 64) || rows <= (n_groups == 1 ? PT_ROWS : PT_ROWS / 2 * (long long)n_groups) ? 1 : 2;
}
template <class T, int CODE> cudaError_t launch_prefix(const PrefixCall& p, int tiles, unsigned blocks, cudaStream_t s) {
    if (p.a.c.head_dim <= 64) return tiles == 1 ? launch_prefix<T, CODE, 64, 1>(p, blocks, s) : launch_prefix<T, CODE, 64, 2>(p, blocks, s);
    if constexpr (sizeof(T) == 2)
        if (tiles == 2) return launch_prefix<T, CODE, 128, 2>(p, blocks, s);
    return launch_prefix<T, CODE, 128, 1>(p, blocks, s);
}

// ---------------------------------------------------------------------------
// The other tokens, and the shared ones of groups with few rows: units cut into pieces of even length (kv_piece_kernel).  One block looks
// up every sequence's work and deals it out.
// ---------------------------------------------------------------------------
// What the join needs to know of a sequence
struct __align__(16) KvJoin {
    int own_cuts, own_slot;          // pieces of a unit of its own tokens, and its first slot where these are several
    int common_cuts, common_slot;    // the same of the shared tokens
    int common_row;                  // first row of its group
    int named;                       // 0: the call may not name it, its rows are zero
    int pad[2];
};
struct DealCall {
    KvAttend a;                // the whole call's, with skip
    const int4* shared;
    const int32_t *group_rows, *group_of;
    KvEntry* entries;          // [n + n_groups]
    int32_t *first, *total;
    int4* cut;                 // [n_groups] kv_prefix_kernel's pieces: first, of each unit, first slot
    KvJoin* join;              // [n]
    int n_groups, most;        // pieces to aim at
    int prefix_rows;           // query rows of kv_prefix_kernel's units; 0: the groups are entries
    int prefix_most;           // pieces to aim at there
};
constexpr int DEAL_THREADS = 1024, LEAST_TILES = 8;

// One list of units dealt out: entry i has units(i) of tiles(i) tiles, of which each is cut into ceil(tiles / share) pieces; put(i, cuts,
// pieces before, pieces of cut units before).  The share is that of `most` even pieces, at least `least`, or up to twice
// as much where no more than `most` pieces come of it, which run at once (each begins with some us of dependent reads).  Where that many
// do not come out, because units alone are as many, longer ones are still cut: no block has more than an even share at a time.  Returns the pieces
// in all, at most the units and `most`; pieces of cut units are 2 `most` at most, since a unit of more than a share has less than twice as many
// pieces as shares.  A whole block calls it.
template <class F, class G, class P> __device__ __forceinline__ int deal_out(int count, int most, int least, F units, G tiles, P put) {
    __shared__ long long s_tiles[32];
    __shared__ int s_tries[32], s_pieces[32], s_slots[32];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    long long all = 0;
    for (int i = t; i < count; i += DEAL_THREADS) all += (long long)units(i) * tiles(i);
    for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
    __syncthreads();
    if (lane == 0) s_tiles[warp] = all;
    if (t < 32) s_tries[t] = 0;
    __syncthreads();
    all = s_tiles[lane];
    for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
    // lane k tries 1 + k / 32 of the least share
    const uint32_t aim = max(most, 1);
    const long long even = all >> 31 ? (all + aim - 1) / aim : ((uint32_t)all + aim - 1) / aim;   // 64-bit divisions take their time
    const uint32_t base = (uint32_t)min(max((long long)least, even), 1ll << 29), mine = base + (base >> 5) * lane + ((base & 31) * lane >> 5);
    int pieces = 0;
    for (int i = warp; i < count; i += 32) {
        const int u = units(i);
        if (u) pieces += u * (int)(((uint32_t)tiles(i) + mine - 1) / mine);
    }
    atomicAdd(&s_tries[lane], pieces);
    __syncthreads();
    const uint32_t fit = __ballot_sync(0xffffffffu, s_tries[lane] <= most);
    const uint32_t share = __shfl_sync(0xffffffffu, mine, fit ? __ffs(fit) - 1 : 0);
    pieces = 0;
    int slots = 0;   // before this round's entries
    for (int i0 = 0; i0 < count; i0 += DEAL_THREADS) {
        const int i = i0 + t, u = i < count ? units(i) : 0, cuts = u ? (int)(((uint32_t)tiles(i) + share - 1) / share) : 0;
        const int n = u * cuts, held = cuts > 1 ? n : 0;
        int x = n, y = held;
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, x, d), w = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) x += v, y += w;
        }
        if (lane == 31) s_pieces[warp] = x, s_slots[warp] = y;
        __syncthreads();
        int bx = s_pieces[lane], by = s_slots[lane];
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, bx, d), w = __shfl_up_sync(0xffffffffu, by, d);
            if (lane >= d) bx += v, by += w;
        }
        const int all_x = __shfl_sync(0xffffffffu, bx, 31), all_y = __shfl_sync(0xffffffffu, by, 31);
        const int px = __shfl_sync(0xffffffffu, bx, (warp + 31) & 31), py = __shfl_sync(0xffffffffu, by, (warp + 31) & 31);
        if (warp) x += px, y += py;
        if (i < count) put(i, cuts, pieces + x - n, slots + y - held);
        pieces += all_x, slots += all_y;
        __syncthreads();
    }
    return pieces;
}

__global__ void __launch_bounds__(DEAL_THREADS) kv_deal_kernel(const __grid_constant__ DealCall p) {
    __shared__ int s_units[DEAL_THREADS], s_tiles[DEAL_THREADS], s_cut[2][DEAL_THREADS];   // of the first entries, or groups
    pdl_trigger();
    pdl_wait();
    const KvAttend& a = p.a;
    const int n = a.rows.n, groups = p.n_groups, count = n + (p.prefix_rows ? 0 : groups), t = threadIdx.x, kvh = a.c.kv_heads;
    auto units_of = [&](const PieceWork& s) { return s.len > 0 && s.tiles > 0 ? (s.m * a.group + 15) / 16 * kvh : 0; };
    for (int i = t; i < count; i += DEAL_THREADS) {
        PieceWork s;
        if (i < n) {
            s = piece_work(a, i);
            p.join[i].named = s.id >= 0 && s.id < a.c.max_seqs && s.m <= a.max_new;
        } else {
            const int4 sh = p.shared[i - n];
            const int row0 = p.group_rows[i - n];
            s = PieceWork{{sh.x, sh.z * KV_BLOCK, p.group_rows[i - n + 1] - row0, row0, sh.y, 0, sh.z - sh.y}, 0, 0, true};
        }
        p.entries[i].s = s;
        if (i < DEAL_THREADS) s_units[i] = units_of(s), s_tiles[i] = s.tiles;
    }
    // What the join needs of the first sequences, and the groups' rows: read here, beside the rest
    int2 my_skip = make_int2(0, 0);
    int my_group = 0, my_row = 0;
    if (t < n) {
        my_skip = a.skip[t];
        if (my_skip.y > my_skip.x) my_group = p.group_of[t], my_row = p.group_rows[my_group];
    }
    int4 my_shared = make_int4(0, 0, 0, 0);
    int my_rows = 0;
    if (p.prefix_rows && t < groups) my_shared = p.shared[t], my_rows = p.group_rows[t + 1] - p.group_rows[t];
    __syncthreads();
    const int pieces = deal_out(
        count, p.most, LEAST_TILES, [&](int i) { return i < DEAL_THREADS ? s_units[i] : units_of(p.entries[i].s); },
        [&](int i) { return i < DEAL_THREADS ? s_tiles[i] : p.entries[i].s.tiles; },
        [&](int i, int cuts, int first, int slot) {
            KvEntry& e = p.entries[i];
            e.cuts = cuts, e.first = first, e.slot = slot, p.first[i] = first;
            if (i < n) p.join[i].own_cuts = cuts, p.join[i].own_slot = slot;
            else if (i - n < DEAL_THREADS) s_cut[0][i - n] = cuts, s_cut[1][i - n] = slot;
        });
    if (t == 0) *p.total = pieces;
    if (p.prefix_rows) {
        auto units = [&](const int4& sh, int rows) { return sh.z > sh.y ? (rows * a.group + p.prefix_rows - 1) / p.prefix_rows * kvh : 0; };
        auto tiles = [](const int4& sh) { return (sh.z - sh.y + 7) / 8; };
        auto group_units = [&](int g) { return units(p.shared[g], p.group_rows[g + 1] - p.group_rows[g]); };
        auto group_tiles = [&](int g) { return tiles(p.shared[g]); };
        __syncthreads();
        if (t < groups) s_units[t] = units(my_shared, my_rows), s_tiles[t] = tiles(my_shared);
        __syncthreads();
        deal_out(
            groups, p.prefix_most, 2, [&](int g) { return g < DEAL_THREADS ? s_units[g] : group_units(g); },
            [&](int g) { return g < DEAL_THREADS ? s_tiles[g] : group_tiles(g); },
            [&](int g, int cuts, int first, int slot) {
                p.cut[g] = make_int4(first, cuts, slot, 0);
                if (g < DEAL_THREADS) s_cut[0][g] = cuts, s_cut[1][g] = slot;
            });
    }
    __syncthreads();   // what the block has written to memory is read back below
    for (int i = t; i < n; i += DEAL_THREADS) {
        const int2 skip = i == t ? my_skip : a.skip[i];
        KvJoin& j = p.join[i];
        int cuts = 0, slot = 0, row = 0;
        if (skip.y > skip.x) {
            const int g = i == t ? my_group : p.group_of[i];
            row = i == t ? my_row : p.group_rows[g];
            if (g < DEAL_THREADS) cuts = s_cut[0][g], slot = s_cut[1][g];
            else if (p.prefix_rows) cuts = p.cut[g].y, slot = p.cut[g].z;
            else cuts = p.entries[n + g].cuts, slot = p.entries[n + g].slot;
        }
        j.common_cuts = cuts, j.common_slot = slot, j.common_row = row;
    }
}

// The parts of a group's shared tokens and of the sequence's own become the result: a team of warps for each row and head, which take the
// parts in turn.  One warp is enough where rows fill the card; 57 parts of few rows took one 15 us.
struct JoinCall {
    KvAttend a;
    const KvJoin* join;        // [n]
    KvPieces pieces;           // where the parts of entries are
    const float* slot_o;       // kv_prefix_kernel's pieces, or null: the groups are entries
    const float2* slot_ml;
    int block_rows;            // rows of its units
    int team;                  // warps: 1, 2, 4 or 8
};
// Parts of a row: `count` of them, `step` rows apart
struct PartList {
    const float* o;
    const float2* ml;
    long long at;
    int step, count;
};
constexpr int JOIN_WARPS = 8;
template <class T> __global__ void __launch_bounds__(JOIN_WARPS * 32, 4) kv_join_shared_kernel(const __grid_constant__ JoinCall p) {
    __shared__ __align__(16) float s_o[JOIN_WARPS][256];
    __shared__ float s_l[JOIN_WARPS];
    pdl_trigger();
    pdl_wait();
    const KvAttend& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x, D = a.c.head_dim, team = p.team, mate = warp & (team - 1);
    const int i = a.rows.starts ? warp_last_le(a.rows.n, row, [&](int k) { return a.rows.at(k); }) : row / a.rows.each;
    const int r0 = i < 0 ? 0 : a.rows.at(i), r1 = i < 0 ? 0 : a.rows.at(i + 1);
    const KvJoin j = p.join[max(i, 0)];
    if (row < r0 || row >= r1 || r0 < 0 || r1 > a.rows.rows) return;   // no sequence's, or of one whose rows pass the end
    // (pieces of a unit, first slot) of the own and of the shared tokens
    const int2 own = make_int2(j.named ? j.own_cuts : 0, j.own_slot), common = make_int2(j.named ? j.common_cuts : 0, j.common_slot);
    const int in_group = row - j.common_row;
    const int heads = JOIN_WARPS / team;   // of the block at a time
    for (int h0 = blockIdx.y * heads; h0 < a.heads; h0 += gridDim.y * heads) {
        const int h = min(h0 + warp / team, a.heads - 1);   // the last one more than once, alike
        const long long at = (long long)row * a.heads + h;
        const int kvh = h / a.group, hh = h - kvh * a.group;
        auto list = [&](const int2& cuts, const float* o, const float2* ml, int r, int size, const float* slot_o, const float2* slot_ml) {
            if (cuts.x <= 1) return PartList{o, ml, at, 0, cuts.x};
            const int unit = r / size * a.c.kv_heads + kvh;
            return PartList{slot_o, slot_ml, ((long long)cuts.y + (long long)unit * cuts.x) * size + r % size, size, cuts.x};
        };
        const PartList lists[2] = {
            list(own, p.pieces.o0, p.pieces.ml0, (row - r0) * a.group + hh, 16, p.pieces.slot_o, p.pieces.slot_ml),
            list(common, p.pieces.o1, p.pieces.ml1, in_group * a.group + hh, p.slot_o ? p.block_rows : 16, p.slot_o ? p.slot_o : p.pieces.slot_o,
                 p.slot_o ? p.slot_ml : p.pieces.slot_ml)};
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            for (int k = lane; k < lists[q].count; k += 32) top = fmaxf(top, lists[q].ml[lists[q].at + (long long)k * lists[q].step].x);
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float base = top == -INFINITY ? 0.f : top;
        const int e0 = lane * 4, e1 = 128 + lane * 4;
        float l = 0.f;
        float4 o[2] = {};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const PartList& x = lists[q];
            for (int k0 = mate; k0 < x.count; k0 += 32 * team) {   // lane j: part k0 + j * team
                float f = 0.f;
                if (k0 + lane * team < x.count) {
                    const float2 y = x.ml[x.at + (long long)(k0 + lane * team) * x.step];
                    f = ex2(y.x - base);
                    l += move_norm(y.y, y.x - base, f);
                }
                const int n = min(32, (x.count - k0 + team - 1) / team);
                constexpr int GO = 2;   // loads on their way at once: each takes a microsecond
                for (int j0 = 0; j0 < n; j0 += GO)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int e = b ? e1 : e0;
                        if (b && D <= 128) break;
                        float4 v[GO];
#pragma unroll
                        for (int j = 0; j < GO; ++j)
                            v[j] = j0 + j < n && e < D ? *reinterpret_cast<const float4*>(x.o + (x.at + (long long)(k0 + (j0 + j) * team) * x.step) * D + e)
                                                       : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int j = 0; j < GO; ++j) {
                            const float w = __shfl_sync(0xffffffffu, f, j0 + j);   // 0 past the last
                            o[b].x = fmaf(v[j].x, w, o[b].x), o[b].y = fmaf(v[j].y, w, o[b].y), o[b].z = fmaf(v[j].z, w, o[b].z), o[b].w = fmaf(v[j].w, w, o[b].w);
                        }
                    }
            }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (team > 1) {   // the first of a team adds the others' sums up
            __syncthreads();
            if (e0 < D) *reinterpret_cast<float4*>(&s_o[warp][e0]) = o[0];
            if (e1 < D) *reinterpret_cast<float4*>(&s_o[warp][e1]) = o[1];
            if (lane == 0) s_l[warp] = l;
            __syncthreads();
            if (mate) continue;
            for (int w = warp + 1; w < warp + team; ++w) {
                l += s_l[w];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int e = b ? e1 : e0;
                    if (e >= D) continue;
                    const float4 v = *reinterpret_cast<const float4*>(&s_o[w][e]);
                    o[b].x += v.x, o[b].y += v.y, o[b].z += v.z, o[b].w += v.w;
                }
            }
        }
        if (h0 + warp / team >= a.heads) continue;
        const bool seen = l > 0.f || l != l;
        const float inv = seen ? 1.f / l : 0.f;
        T* dst = static_cast<T*>(a.out) + row * a.out_stride + (long long)h * D;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int e = b ? e1 : e0;
            if (e >= D) continue;
            const float4 y = seen ? make_float4(o[b].x * inv, o[b].y * inv, o[b].z * inv, o[b].w * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<float4*>(dst + e) = y;
            } else {
                const __nv_bfloat162 u = __floats2bfloat162_rn(y.x, y.y), v = __floats2bfloat162_rn(y.z, y.w);
                *reinterpret_cast<uint2*>(dst + e) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
            }
        }
        if (lane == 0 && a.lse) a.lse[at] = seen ? (top + NORM_LOG2 + log2f(l)) * LN2 : -INFINITY;
    }
}

size_t up16(size_t x) { return (x + 15) & ~(size_t)15; }

// Where things lie in the workspace, each from the next multiple of 16 bytes on.
struct Space {
    size_t skip, group_of, shared, group_rows, cut, join, entries, first, total, ml0, ml1, slot_ml, prefix_ml, o0, o1, slot_o, prefix_o, bytes;
};
Space space_of(const cac_kv8& c, int n, int rows, int n_groups, int heads, int sms) {
    Space s;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t was = at;
        at += up16(bytes);
        return was;
    };
    const size_t units = (size_t)rows * heads, D = c.head_dim;
    const size_t slots = (size_t)2 * sms * piece_blocks(c.head_dim, true) * 16, prefix = c.head_dim <= 128 ? (size_t)2 * sms * 2 * PT_ROWS : 0;
    s.skip = take((size_t)n * 8), s.group_of = take((size_t)n * 4), s.shared = take((size_t)n_groups * 16);
    s.group_rows = take(((size_t)n_groups + 1) * 4), s.cut = take((size_t)n_groups * 16);
    s.join = take((size_t)n * sizeof(KvJoin));
    s.entries = take(((size_t)n + n_groups) * sizeof(KvEntry)), s.first = take(((size_t)n + n_groups) * 4), s.total = take(4);
    s.ml0 = take(units * 8), s.ml1 = take(units * 8), s.slot_ml = take(slots * 8), s.prefix_ml = take(prefix * 8);
    s.o0 = take(units * D * 4), s.o1 = take(units * D * 4), s.slot_o = take(slots * D * 4), s.prefix_o = take(prefix * D * 4);
    s.bytes = at;
    return s;
}

}  // namespace

// Whether kv_prefix_kernel reads the shared tokens, 128 rows at a time, or kv_piece_kernel, 16.
bool kv_prefix_takes(const KvAttend& a, int n_groups) {
    return a.c.head_dim <= 128 && (long long)a.rows.rows * a.group > 32ll * n_groups;
}

cudaError_t kv_attend_shared(const KvAttend& call, int dtype, const int32_t* groups, int n_groups, int sms, void* workspace,
                             cudaStream_t s) {
    const cac_kv8& c = call.c;
    const int n = call.rows.n, rows = call.rows.rows;
    const Space at = space_of(c, n, rows, n_groups, call.heads, sms);
    uint8_t* base = static_cast<uint8_t*>(workspace);
    auto place = [&](size_t x) { return static_cast<void*>(base + x); };
    const SharedCall plan{call, groups, n_groups, static_cast<int2*>(place(at.skip)), static_cast<int32_t*>(place(at.group_of)),
                          static_cast<int4*>(place(at.shared)), static_cast<int32_t*>(place(at.group_rows))};
    cudaError_t e = launch_k(kv_plan_shared_kernel, dim3(n_groups, 1, PLAN_BLOCKS), dim3(PLAN_THREADS), 0, s, PLAN_BLOCKS, plan);
    if (e != cudaSuccess) return e;

    const bool prefix = kv_prefix_takes(call, n_groups);
    KvAttend a = call;
    a.skip = plan.skip;
    const bool low = (long long)call.max_new * call.group <= 8 && (prefix || (long long)rows * call.group <= 8);
    const int most = sms * piece_blocks(c.head_dim, low), dealt = prefix ? 0 : n_groups;
    const int tiles = prefix_tiles(call, dtype, n_groups), block = tiles * PT_ROWS;
    const DealCall deal{a, plan.shared, plan.group_rows, plan.group_of, static_cast<KvEntry*>(place(at.entries)),
                        static_cast<int32_t*>(place(at.first)), static_cast<int32_t*>(place(at.total)), static_cast<int4*>(place(at.cut)),
                        static_cast<KvJoin*>(place(at.join)), n_groups, most, prefix ? block : 0, sms};
    e = launch_k(kv_deal_kernel, dim3(1), dim3(DEAL_THREADS), 0, s, 1, deal);
    if (e != cudaSuccess) return e;

    const KvPieces pieces{deal.entries, deal.first, deal.total, n + dealt, n, low, prefix,
                          static_cast<float*>(place(at.o0)), static_cast<float*>(place(at.o1)), static_cast<float*>(place(at.slot_o)),
                          static_cast<float2*>(place(at.ml0)), static_cast<float2*>(place(at.ml1)), static_cast<float2*>(place(at.slot_ml))};
    for (int g0 = 0; prefix && g0 < n_groups; g0 += TA_SEQS) {   // the groups' shared tokens
        KvAttend b = call;
        b.rows = {plan.group_rows + g0, 0, std::min(n_groups - g0, TA_SEQS), rows};
        b.ids = nullptr;
        const PrefixCall p{b, plan.shared + g0, deal.cut + g0, b.rows.n, pieces.o1, pieces.ml1, static_cast<float*>(place(at.prefix_o)),
                           static_cast<float2*>(place(at.prefix_ml))};
        const long long units = ((long long)rows * call.group / block + b.rows.n) * c.kv_heads;
        // As many blocks as there may be pieces.  A third as many units as SMs or less, all in this launch, can always be cut into one piece an SM
        // (the largest share that is tried is one and a half times the even one at least).
        const unsigned blocks = (unsigned)(n_groups <= TA_SEQS && units <= sms / 3 ? sms : units + sms);
        if (c.code == CAC_KV8_INT8)
            e = dtype == CAC_DTYPE_BF16 ? launch_prefix<bf16, CAC_KV8_INT8>(p, tiles, blocks, s) : launch_prefix<float, CAC_KV8_INT8>(p, tiles, blocks, s);
        else
            e = dtype == CAC_DTYPE_BF16 ? launch_prefix<bf16, CAC_KV8_E4M3>(p, tiles, blocks, s) : launch_prefix<float, CAC_KV8_E4M3>(p, tiles, blocks, s);
        if (e != cudaSuccess) return e;
    }
    // the others, of each sequence: as many blocks as there may be pieces
    const long long units = ((long long)rows * call.group / 16 + n) * c.kv_heads + (prefix ? 0 : ((long long)rows * call.group / 16 + n_groups) * c.kv_heads);
    const unsigned blocks = (unsigned)(units + most);
    e = c.code == CAC_KV8_INT8 ? kv_launch_pieces<CAC_KV8_INT8>(a, pieces, dtype, blocks, s)
                               : kv_launch_pieces<CAC_KV8_E4M3>(a, pieces, dtype, blocks, s);
    if (e != cudaSuccess) return e;

    const long long results = (long long)rows * call.heads;
    const int team = results > 16 * sms ? 1 : results > 8 * sms ? 2 : results > 4 * sms ? 4 : 8;
    const JoinCall join{call, deal.join, pieces, prefix ? static_cast<const float*>(place(at.prefix_o)) : nullptr,
                        static_cast<const float2*>(place(at.prefix_ml)), block, team};
    const dim3 grid(rows, std::min((call.heads * team + JOIN_WARPS - 1) / JOIN_WARPS, 64));
    return dtype == CAC_DTYPE_BF16 ? launch_k(kv_join_shared_kernel<bf16>, grid, dim3(JOIN_WARPS * 32), 0, s, 1, join)
                                   : launch_k(kv_join_shared_kernel<float>, grid, dim3(JOIN_WARPS * 32), 0, s, 1, join);
}

size_t kv_shared_bytes(const cac_kv8& c, int n, int rows, int n_groups, int heads, int sms) {
    return space_of(c, n, rows, n_groups, heads, sms).bytes;
}

}  // namespace cac
