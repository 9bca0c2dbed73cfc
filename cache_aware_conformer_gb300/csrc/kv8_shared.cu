// Attention over the paged 8-bit K/V cache for sequences that share a prefix (include/cac_kv8.h,
// cac_kv8_attend_shared).
//
// A softmax over a sequence's tokens is a join of softmaxes over any parts of them: with a part's maximum m, its sum
// l of 2^(t - m) and its sum o of the weighted values, M = max m over the parts,
//   out = sum o 2^(m - M) / sum l 2^(m - M).
// So the tokens that all queries of a group see in the same pages are read once, by one launch whose rows are all queries of the
// group; a second launch reads what each sequence has to itself, and a third joins the two.
//
// What is shared is looked up on the device in each call: blocks of 16 tokens that every query of the group sees whole, in front of the
// first page in which the tables differ.  Nothing but the sequences' tables is compared, so a result never hangs on what
// the caller believes of them.
#include <algorithm>

#include "kv8_attn.cuh"

namespace cac {
namespace {

constexpr int PLAN_BLOCKS = 8, PLAN_THREADS = 512;   // of a group: a cluster
constexpr int LEAST_BLOCKS = 1;                      // shared blocks below this are not worth it

struct SharedCall {
    KvAttend a;                // rows, ids and window of the whole call
    const int32_t* groups;     // [n_groups + 1], NULL: one group
    int n_groups;              // at least 1
    int2* skip;                // [n]
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

    // pages in front of the first one in which a table differs from the leader's: warps take the members in turn
    if (some) {
        const int pages = min((s_hi + a.c.page_tokens - 1) / a.c.page_tokens, a.c.max_pages);
        const int32_t* own = a.c.table + (long long)a.ids[s_leader] * a.c.max_pages;
        int same = pages;
        for (int i = s_leader + 1 + rank * (PLAN_THREADS / 32) + (t >> 5); i < g1; i += PLAN_BLOCKS * (PLAN_THREADS / 32)) {
            if (row_at(i + 1) == row_at(i)) continue;
            const int32_t* other = a.c.table + (long long)a.ids[i] * a.c.max_pages;
            if (other == own) continue;
            for (int b = 0; b < same; b += 128) {
                int x[4], y[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int k = b + u * 32 + lane;
                    x[u] = k < same ? own[k] : 0, y[u] = k < same ? other[k] : 0;
                }
                int mine = INT32_MAX;
#pragma unroll
                for (int u = 3; u >= 0; --u)
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
    for (int i = g0 + me; i < g1; i += step) p.skip[i] = range;
    if (g == 0) {  // sequences of no group
        const int before = fine ? group_at(0) : n, after = fine ? group_at(p.n_groups) : n;
        for (int i = me; i < before; i += step) p.skip[i] = make_int2(0, 0);
        for (int i = after + me; i < n; i += step) p.skip[i] = make_int2(0, 0);
        for (int k = me; k <= p.n_groups; k += step) p.group_rows[k] = fine ? row_at(group_at(k)) : 0;
    }
    if (rank == 0 && t == 0) p.shared[g] = make_int4(share ? a.ids[s_leader] : 0, range.x, range.y, 0);
}

// A warp for each row and head: the parts of a group's shared tokens and of the sequence's own become the result.
struct JoinCall {
    KvAttend a;
    const int2* skip;
    const float *o0, *o1;      // own, shared: [rows][heads][head_dim]
    const float2 *ml0, *ml1;
};
constexpr int JOIN_WARPS = 8;
template <class T> __global__ void __launch_bounds__(JOIN_WARPS * 32) kv_join_shared_kernel(const __grid_constant__ JoinCall p) {
    pdl_trigger();
    pdl_wait();
    const KvAttend& a = p.a;
    const int lane = threadIdx.x & 31, row = blockIdx.x, D = a.c.head_dim;
    const int i = a.rows.starts ? warp_last_le(a.rows.n, row, [&](int k) { return a.rows.at(k); }) : row / a.rows.each;
    if (i < 0) return;
    const int r0 = a.rows.at(i), r1 = a.rows.at(i + 1);
    if (row < r0 || row >= r1 || r0 < 0 || r1 > a.rows.rows) return;   // no sequence's, or of one whose rows pass the end
    const int id = a.ids[i];
    const bool named = id >= 0 && id < a.c.max_seqs && r1 - r0 <= a.max_new;
    const int2 k = p.skip[i];
    const bool two = named && k.y > k.x;
    for (int h = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5); h < a.heads; h += gridDim.y * JOIN_WARPS) {
        const long long at = (long long)row * a.heads + h;
        const float2 x = named ? p.ml0[at] : make_float2(-INFINITY, 0.f), y = two ? p.ml1[at] : make_float2(-INFINITY, 0.f);
        const float top = fmaxf(x.x, y.x), base = top == -INFINITY ? 0.f : top;
        const float fx = ex2(x.x - base), fy = ex2(y.x - base);
        const float l = move_norm(x.y, x.x - base, fx) + (two ? move_norm(y.y, y.x - base, fy) : 0.f);
        const bool seen = l > 0.f || l != l;
        const float inv = seen ? 1.f / l : 0.f;
        T* dst = static_cast<T*>(a.out) + row * a.out_stride + (long long)h * D;
        for (int e = lane * 4; e < D; e += 128) {
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            if (seen) {
                o = *reinterpret_cast<const float4*>(p.o0 + at * D + e);
                o.x *= fx, o.y *= fx, o.z *= fx, o.w *= fx;
                if (two) {
                    const float4 q = *reinterpret_cast<const float4*>(p.o1 + at * D + e);
                    o.x = fmaf(q.x, fy, o.x), o.y = fmaf(q.y, fy, o.y), o.z = fmaf(q.z, fy, o.z), o.w = fmaf(q.w, fy, o.w);
                }
                o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
            }
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<float4*>(dst + e) = o;
            } else {
                const __nv_bfloat162 u = __floats2bfloat162_rn(o.x, o.y), v = __floats2bfloat162_rn(o.z, o.w);
                *reinterpret_cast<uint2*>(dst + e) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
            }
        }
        if (lane == 0 && a.lse) a.lse[at] = seen ? (top + NORM_LOG2 + log2f(l)) * LN2 : -INFINITY;
    }
}

size_t up16(size_t x) { return (x + 15) & ~(size_t)15; }

// Where things lie in the workspace.
struct Space {
    size_t skip, shared, group_rows, split, ml0, ml1, o0, o1, bytes;
};
Space space_of(const cac_kv8& c, int n, int rows, int n_groups, int heads, int sms) {
    Space s;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t was = at;
        at += up16(bytes);
        return was;
    };
    const size_t units = (size_t)rows * heads;
    s.skip = take((size_t)n * 8), s.shared = take((size_t)n_groups * 16), s.group_rows = take(((size_t)n_groups + 1) * 4);
    s.split = take(kv_attend_bytes(c.head_dim, sms));
    s.ml0 = take(units * 8), s.ml1 = take(units * 8);
    s.o0 = take(units * c.head_dim * 4), s.o1 = take(units * c.head_dim * 4);
    s.bytes = at;
    return s;
}

}  // namespace

cudaError_t kv_attend_shared(const KvAttend& call, int dtype, const int32_t* groups, int n_groups, bool split, int sms,
                             void* workspace, cudaStream_t s) {
    const cac_kv8& c = call.c;
    const int n = call.rows.n, rows = call.rows.rows;
    const Space at = space_of(c, n, rows, n_groups, call.heads, sms);
    uint8_t* base = static_cast<uint8_t*>(workspace);
    const SharedCall plan{call, groups, n_groups, reinterpret_cast<int2*>(base + at.skip), reinterpret_cast<int4*>(base + at.shared),
                          reinterpret_cast<int32_t*>(base + at.group_rows)};
    cudaError_t e = launch_k(kv_plan_shared_kernel, dim3(n_groups, 1, PLAN_BLOCKS), dim3(PLAN_THREADS), 0, s, PLAN_BLOCKS, plan);
    if (e != cudaSuccess) return e;

    auto part = [&](const KvAttend& a, bool cut) {
        return c.code == CAC_KV8_INT8 ? kv_launch_attend<CAC_KV8_INT8>(a, dtype, cut, sms, base + at.split, s)
                                      : kv_launch_attend<CAC_KV8_E4M3>(a, dtype, cut, sms, base + at.split, s);
    };
    for (int g0 = 0; g0 < n_groups; g0 += TA_SEQS) {   // the groups' shared tokens
        KvAttend a = call;
        a.rows = {plan.group_rows + g0, 0, std::min(n_groups - g0, TA_SEQS), rows};
        a.ids = nullptr;
        a.shared = plan.shared + g0;
        a.max_new = rows;
        a.part_o = reinterpret_cast<float*>(base + at.o1), a.part_ml = reinterpret_cast<float2*>(base + at.ml1);
        if ((e = part(a, true)) != cudaSuccess) return e;
    }
    for (int i0 = 0; i0 < n; i0 += TA_SEQS) {          // the others, of each sequence
        KvAttend a = call;
        a.rows.starts = call.rows.starts ? call.rows.starts + i0 : nullptr;
        a.rows.n = std::min(n - i0, TA_SEQS);
        a.rows.base = call.rows.each * i0;
        a.ids = call.ids + i0;
        a.skip = plan.skip + i0;
        a.part_o = reinterpret_cast<float*>(base + at.o0), a.part_ml = reinterpret_cast<float2*>(base + at.ml0);
        if ((e = part(a, split)) != cudaSuccess) return e;
    }
    const JoinCall join{call, plan.skip, reinterpret_cast<const float*>(base + at.o0), reinterpret_cast<const float*>(base + at.o1),
                        reinterpret_cast<const float2*>(base + at.ml0), reinterpret_cast<const float2*>(base + at.ml1)};
    const dim3 grid(rows, std::min((call.heads + JOIN_WARPS - 1) / JOIN_WARPS, 8));
    return dtype == CAC_DTYPE_BF16 ? launch_k(kv_join_shared_kernel<bf16>, grid, dim3(JOIN_WARPS * 32), 0, s, 1, join)
                                   : launch_k(kv_join_shared_kernel<float>, grid, dim3(JOIN_WARPS * 32), 0, s, 1, join);
}

size_t kv_shared_bytes(const cac_kv8& c, int n, int rows, int n_groups, int heads, int sms) {
    return space_of(c, n, rows, n_groups, heads, sms).bytes;
}

}  // namespace cac
