// The paged 8-bit K/V cache (include/cac_kv8.h): quantising writes, reads, and
// the page operations.  Every kernel reads lengths, tables and free pages on the
// device, so the calls queue (or replay from a graph) without the host.
//
// All of it moves bytes; nothing here has arithmetic that could bound it.  The
// writers and readers take one block of 16 tokens and one head per warp, because
// a block's scale is the maximum over exactly that.
#include <algorithm>

#include "kv8.cuh"
#include "status.cuh"

namespace cac {

int kv_check_shape(const cac_kv8* c) {
    if (!c || c->n_layers < 1 || c->kv_heads < 1 || c->kv_heads > 65535 || c->head_dim < 16 || c->page_tokens < 16 ||
        c->n_pages < 1 || c->max_seqs < 1 || c->max_pages < 1)
        return CAC_E_INVAL;
    if (c->head_dim % 16 || c->head_dim > 256 || c->page_tokens % KV_BLOCK || c->page_tokens > 1024 ||
        (c->code != CAC_KV8_INT8 && c->code != CAC_KV8_E4M3))
        return CAC_E_UNSUPPORTED;
    if ((long long)c->max_pages * c->page_tokens >= (1ll << 30) || c->n_pages >= (1 << 30) || c->max_seqs >= (1 << 28))
        return CAC_E_UNSUPPORTED;
    return CAC_OK;
}

int kv_check_cache(const cac_kv8* c) {
    const int r = kv_check_shape(c);
    if (r != CAC_OK) return r;
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->table || !c->lens || !c->refs || !c->free_list ||
        !c->n_free || !c->pending || !c->work || !c->status)
        return CAC_E_INVAL;
    const uintptr_t words = reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale) |
                            reinterpret_cast<uintptr_t>(c->table) | reinterpret_cast<uintptr_t>(c->lens) |
                            reinterpret_cast<uintptr_t>(c->refs) | reinterpret_cast<uintptr_t>(c->free_list) |
                            reinterpret_cast<uintptr_t>(c->n_free) |
                            reinterpret_cast<uintptr_t>(c->work) | reinterpret_cast<uintptr_t>(c->status);
    if (((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15) || (words & 3) ||
        (reinterpret_cast<uintptr_t>(c->pending) & 7))
        return CAC_E_ALIGN;
    return CAC_OK;
}

namespace {

constexpr int PLAN_T = 1024;

__device__ __forceinline__ int pages_of(int tokens, int page_tokens) {
    return (int)(((long long)tokens + page_tokens - 1) / page_tokens);
}

// Exclusive prefix sum over the block of two counts at once, and their totals.
struct Two {
    int a, b;
};
__device__ Two block_scan(Two x, Two* total) {
    __shared__ int sa[32], sb[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int a = x.a, b = x.b;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int ua = __shfl_up_sync(0xffffffffu, a, d), ub = __shfl_up_sync(0xffffffffu, b, d);
        if (lane >= d) a += ua, b += ub;
    }
    __syncthreads();  // the arrays may still be read from an earlier call
    if (lane == 31) sa[warp] = a, sb[warp] = b;
    __syncthreads();
    int oa = 0, ob = 0, ta = 0, tb = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) oa += sa[w], ob += sb[w];
        ta += sa[w], tb += sb[w];
    }
    *total = Two{ta, tb};
    return Two{oa + a - x.a, ob + b - x.b};
}

// ---------------------------------------------------------------------------
// init
// ---------------------------------------------------------------------------
__global__ void kv_init_kernel(cac_kv8 c, long long work_ints) {
    pdl_trigger();
    pdl_wait();
    const long long t = blockIdx.x * (long long)blockDim.x + threadIdx.x, step = (long long)gridDim.x * blockDim.x;
    for (long long i = t; i < (long long)c.max_seqs * c.max_pages; i += step) c.table[i] = -1;
    for (long long i = t; i < c.max_seqs; i += step) c.lens[i] = 0, c.pending[2 * i] = 0, c.pending[2 * i + 1] = 0;
    for (long long i = t; i < c.n_pages; i += step) c.refs[i] = 0, c.free_list[i] = (int)(c.n_pages - 1 - i);
    for (long long i = t; i < work_ints; i += step) c.work[i] = 0;
    if (t == 0) *c.n_free = c.n_pages, *c.status = 0;
}

// ---------------------------------------------------------------------------
// extend.  One block decides for all sequences of the call: it needs the sum of
// what they ask before it may change anything.  Latency bounds it (a few
// dependent reads and two scans; with the kernel behind it, which copies shared pages at the memory's rate and sets the new
// blocks' scales to 0, 6.5 us for 256 sequences that ask for nothing, 11.6 with a token each and the truncate before it).
// ---------------------------------------------------------------------------
struct Want {
    int id, len, count, have, fresh;  // pages it has, pages it needs past those
    int last;                         // a last page that is not full, or -1
    bool shared, copy;                // ... that other tables name too; that has to be copied
};

__device__ __forceinline__ Want want_of(const cac_kv8& c, const KvRows& rows, const int32_t* ids, int i) {
    Want w;
    w.id = ids[i];
    w.count = rows.at(i + 1) - rows.at(i);
    w.len = c.lens[w.id];
    w.have = pages_of(w.len, c.page_tokens);
    w.fresh = pages_of(w.len + w.count, c.page_tokens) - w.have;
    w.last = -1;
    w.shared = w.copy = false;
    if (w.count > 0 && w.len % c.page_tokens) {
        w.last = c.table[(long long)w.id * c.max_pages + w.len / c.page_tokens];
        w.shared = w.last >= 0 && __ldcg(c.refs + w.last) > 1;
    }
    return w;
}

__global__ void __launch_bounds__(PLAN_T, 1) kv_extend_kernel(const cac_kv8 c, const KvRows rows, const int32_t* ids) {
    __shared__ int error, any_shared;
    __shared__ int s_place[PLAN_T], s_have[PLAN_T], s_fresh[PLAN_T], s_id[PLAN_T];
    pdl_trigger();
    pdl_wait();
    const KvWork work = kv_work(c);
    const int n = rows.n, tid = threadIdx.x;
    const long long most = (long long)c.max_pages * c.page_tokens;
    const int n_free = *c.n_free;
    if (tid == 0) error = 0, any_shared = 0;
    __syncthreads();
    Want mine{};  // entry tid, which is all of them in a call of up to PLAN_T sequences
    for (int i = tid; i < n; i += PLAN_T) {
        const int id = ids[i];
        const long long count = (long long)rows.at(i + 1) - rows.at(i);
        if (id < 0 || id >= c.max_seqs || count < 0) {
            atomicCAS(&error, 0, CAC_E_BOUNDS);
            continue;
        }
        c.pending[2 * id + 1] = i;  // its place in this call; an id listed twice finds another place there
        if (c.lens[id] + count > most) {
            atomicCAS(&error, 0, CAC_E_LIMIT);
            continue;
        }
        const Want w = want_of(c, rows, ids, i);
        if (i == tid) mine = w;
        if (w.count > 0 && w.len % c.page_tokens && w.last < 0) atomicCAS(&error, 0, CAC_E_STATE);
        if (w.shared) any_shared = 1;
    }
    auto want = [&](int i) { return i == tid ? mine : want_of(c, rows, ids, i); };
    __syncthreads();
    int failed = error;
    const bool count_shared = any_shared && !failed;
    __syncthreads();
    if (!failed)
        for (int i = tid; i < n; i += PLAN_T) {
            const Want w = want(i);
            if (c.pending[2 * w.id + 1] != i) atomicCAS(&error, 0, CAC_E_INVAL);
            if (w.shared) {  // how many of this call's sequences end in the page, and how far the longest of those fills it
                atomicAdd(work.named + w.last, 1);
                atomicMax(work.keeper + w.last, w.len % c.page_tokens);
                work.last_of[w.last] = 0;
            }
        }
    __syncthreads();
    failed = error;
    if (count_shared && !failed)
        for (int i = tid; i < n; i += PLAN_T) {  // the last of those that fill it as far
            const Want w = want(i);
            if (w.shared && __ldcg(work.keeper + w.last) == w.len % c.page_tokens) atomicMax(work.last_of + w.last, i + 1);
        }
    __syncthreads();
    // A shared page stays with one of this call's sequences that end in it when no other table names it; the others (all of
    // them, when one does) get a copy.  It stays with the longest, whose new blocks lie behind all that is copied.  Neither
    // depends on the order of the atomics.
    auto decide = [&](int i) {
        Want w = want(i);
        if (w.shared)
            w.copy = __ldcg(c.refs + w.last) > __ldcg(work.named + w.last) || __ldcg(work.last_of + w.last) != i + 1;
        return w;
    };
    long long sum = 0;
    Two total = {0, 0}, at = {0, 0};
    for (int base = 0; !failed && base < n && sum <= n_free; base += PLAN_T) {
        Want w{};
        if (base + tid < n) w = decide(base + tid);
        at = block_scan(Two{w.fresh, w.copy}, &total);
        sum += (long long)total.a + total.b;
        if (base == 0) mine = w;
    }
    if (!failed && sum > n_free) failed = CAC_E_NOMEM;  // the same for every thread
    int pages = 0, copies = 0;
    for (int base = 0; !failed && base < n; base += PLAN_T) {
        const int i = base + tid;
        Want w = mine;
        if (n > PLAN_T) {
            w = Want{};
            if (i < n) w = decide(i);
            at = block_scan(Two{w.fresh, w.copy}, &total);
        }
        // pages leave the end of the free list: first this chunk's copies, then its fresh pages
        const int top = n_free - pages - copies - 1;
        __syncthreads();
        s_fresh[tid] = 0;
        if (i < n) {
            if (w.copy) {
                const int to = c.free_list[top - at.b];
                work.copy_from[copies + at.b] = w.last;
                work.copy_to[copies + at.b] = to;
                work.copy_blocks[copies + at.b] = (w.len % c.page_tokens + KV_BLOCK - 1) / KV_BLOCK;
                c.table[(long long)w.id * c.max_pages + w.len / c.page_tokens] = to;
                c.refs[to] = 1;
            }
            const int place = top - total.b - at.a;
            int32_t* row = c.table + (long long)w.id * c.max_pages + w.have;
            if (w.fresh == 1) {
                const int page = c.free_list[place];
                row[0] = page;
                c.refs[page] = 1;
            } else {
                s_place[tid] = place, s_have[tid] = w.have, s_fresh[tid] = w.fresh, s_id[tid] = w.id;
            }
            c.pending[2 * w.id] = w.count;
            c.lens[w.id] = w.len + w.count;
        }
        __syncthreads();
        // a warp to a sequence, so that a long prompt's pages are entered 32 at a time
        for (int s = tid >> 5; s < min(PLAN_T, n - base); s += PLAN_T / 32)
            for (int k = tid & 31; k < s_fresh[s]; k += 32) {
                const int page = c.free_list[s_place[s] - k];
                c.table[(long long)s_id[s] * c.max_pages + s_have[s] + k] = page;
                c.refs[page] = 1;
            }
        pages += total.a;
        copies += total.b;
    }
    if (failed) {
        for (int i = tid; i < n; i += PLAN_T)
            if (ids[i] >= 0 && ids[i] < c.max_seqs) c.pending[2 * ids[i]] = 0;
        if (tid == 0) latch_error(c.status, failed);
    } else {
        __syncthreads();
        for (int k = tid; k < copies; k += PLAN_T) atomicSub(c.refs + work.copy_from[k], 1);
    }
    if (tid == 0) {
        work.count[0] = copies;
        if (!failed) *c.n_free = n_free - pages - copies;
    }
    if (count_shared) {  // the counters back to zero; lengths are the new ones by now, so the entry's own place is asked
        __syncthreads();
        for (int i = tid; i < n; i += PLAN_T) {
            int last = mine.last;
            bool shared = mine.shared;
            if (i != tid) {
                const int id = ids[i], count = rows.at(i + 1) - rows.at(i), len = c.lens[id] - (failed ? 0 : count);
                shared = count > 0 && len % c.page_tokens;
                last = shared ? c.table[(long long)id * c.max_pages + len / c.page_tokens] : -1;
                shared = shared && last >= 0;
            }
            if (shared) work.named[last] = 0, work.keeper[last] = 0;
        }
        for (int k = tid; k < copies; k += PLAN_T) work.named[work.copy_from[k]] = 0, work.keeper[work.copy_from[k]] = 0;
    }
}

// Whole pages, all layers: K, V and the scales of a page's first blocks.  Unit u of a copy is (layer, K or V).
__device__ __forceinline__ void copy_page(const cac_kv8& c, int from, int to, int u, int blocks) {
    const int layer = u >> 1;
    uint8_t* codes = static_cast<uint8_t*>(u & 1 ? c.v : c.k);
    float* scales = u & 1 ? c.v_scale : c.k_scale;
    const uint4* a = reinterpret_cast<const uint4*>(codes + kv_head_at(c, layer, from, 0));
    uint4* b = reinterpret_cast<uint4*>(codes + kv_head_at(c, layer, to, 0));
    const int vecs = c.kv_heads * (c.page_tokens * c.head_dim / 16);  // < 2^31: 65535 heads * 1024 * 256 / 16 = 2^30
    int i = threadIdx.x;
    for (; i + 3 * (int)blockDim.x < vecs; i += 4 * blockDim.x) {
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = __ldcs(a + i + k * blockDim.x);
#pragma unroll
        for (int k = 0; k < 4; ++k) b[i + k * blockDim.x] = x[k];
    }
    for (; i < vecs; i += blockDim.x) b[i] = a[i];
    const float* sa = scales + kv_scale_at(c, layer, from, 0);
    float* sb = scales + kv_scale_at(c, layer, to, 0);
    const int per = c.page_tokens / KV_BLOCK;
    for (int k = threadIdx.x; k < c.kv_heads * per; k += blockDim.x)
        if (k % per < blocks) sb[k] = sa[k];
}

// After an extend: the copies that it decided on, and scale 0 for every block that begins with new tokens.  A write gives such a
// block its scale; where none does, the pool's left-over scale is not taken for that of older tokens by a later write.  The new
// blocks of a sequence are dealt out to `parts` blocks of the grid.
__global__ void __launch_bounds__(256) kv_copy_kernel(const cac_kv8 c, const KvRows rows, const int32_t* ids, int parts) {
    pdl_trigger();
    pdl_wait();
    const KvWork work = kv_work(c);
    const long long units = (long long)work.count[0] * c.n_layers * 2;
    for (int u = blockIdx.x; u < rows.n * parts; u += gridDim.x) {
        const int i = u / parts, part = u - i * parts, id = ids[i], m = rows.at(i + 1) - rows.at(i);
        if (m <= 0 || id < 0 || id >= c.max_seqs) continue;
        const int2 pending = *reinterpret_cast<const int2*>(c.pending + 2 * id);
        const int len = c.lens[id];
        if (pending.x != m || pending.y != i) continue;  // the call was refused
        const int first = (len - m + KV_BLOCK - 1) / KV_BLOCK, end = (len + KV_BLOCK - 1) / KV_BLOCK;
        const int share = (end - first + parts - 1) / parts, b0 = first + part * share, n = min(share, end - b0);
        if (n <= 0) continue;
        for (long long e = threadIdx.x; e < 2ll * c.n_layers * c.kv_heads * n; e += blockDim.x) {
            const long long r = e / n;
            const int b = b0 + (int)(e - r * n), head = (int)(r % c.kv_heads), w = (int)(r / c.kv_heads);
            const int token = b * KV_BLOCK, page = c.table[(long long)id * c.max_pages + token / c.page_tokens];
            if (page < 0) continue;
            (w & 1 ? c.v_scale : c.k_scale)[kv_scale_at(c, w >> 1, page, head) + token % c.page_tokens / KV_BLOCK] = 0.f;
        }
    }
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int k = (int)(u / (c.n_layers * 2));
        copy_page(c, work.copy_from[k], work.copy_to[k], (int)(u % (c.n_layers * 2)), work.copy_blocks[k]);
    }
}

// ---------------------------------------------------------------------------
// write
// ---------------------------------------------------------------------------
constexpr int WRITE_WARPS = 8;

// Eight consecutive values as they lie in memory, and as floats
template <class T> struct Eight;
template <> struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};
template <> struct Eight<bf16> {
    uint4 a;
    __device__ __forceinline__ void load(const bf16* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = __uint_as_float(w[k] << 16);
            x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
};
__device__ __forceinline__ void store16(float* p, const float (&x)[4]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
}
__device__ __forceinline__ void store16(bf16* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

// The codes of eight finite values with |x f| rounded no further than the largest code.  For whole numbers, adding 1.5 * 2^23
// leaves the nearest one (ties to even) in the low byte: one addition where a conversion runs at a quarter of that rate.
template <int CODE> __device__ __forceinline__ uint2 encode8(const float (&x)[8], float f) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (CODE == CAC_KV8_INT8) {
            uint32_t y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = __float_as_uint(__fadd_rn(__fmul_rn(x[4 * h + k], f), 12582912.f));
            w[h] = __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
        } else {
            const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * h] * f, x[4 * h + 1] * f), __NV_SATFINITE, __NV_E4M3);
            const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * h + 2] * f, x[4 * h + 3] * f), __NV_SATFINITE, __NV_E4M3);
            w[h] = a | b << 16;
        }
    }
    return make_uint2(w[0], w[1]);
}
template <int CODE> __device__ __forceinline__ void decode8(uint2 w, float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = kv_decode<CODE>(((k < 4 ? w.x : w.y) >> (8 * (k & 3))) & 255u);
}

struct KvWrite {
    cac_kv8 c;
    KvRows rows;
    const int32_t* ids;
    const void *k, *v;
    long long k_stride, v_stride;
    int layer, blocks;
    int each;  // > 0: every sequence has this many new tokens and touches (each + 30) / 16 blocks at most
};

// Where a block of the call lies: rows [lo, hi) of it are new, the first of them row `row` of k and v; nothing to do where
// hi is 0.
struct KvPlace {
    int lo, hi, page, in_page;
    long long row;
};

// Block number b of the call belongs to the sequence i with first(i) = starts(i) / 16 + 2 i <= b < first(i + 1): m new
// tokens touch at most (m + 30) / 16 blocks, and first(i + 1) - first(i) >= m / 16 + 2, so no scan over the
// lengths is needed to deal the blocks out.  Where all counts are alike the host knows, each sequence gets as many.
__device__ __forceinline__ KvPlace place_of(const KvWrite& a, int b) {
    const cac_kv8& c = a.c;
    KvPlace p{0, 0, -1, 0, 0};
    int i, nth;
    if (a.each) {
        const int per = (a.each + 2 * KV_BLOCK - 2) / KV_BLOCK;
        i = b / per, nth = b - i * per;
    } else {
        i = warp_last_le(a.rows.n, b, [&](int s) { return a.rows.at(s) / KV_BLOCK + 2ll * s; });
        if (i < 0) return p;
        nth = b - (a.rows.at(i) / KV_BLOCK + 2 * i);
    }
    const int row0 = a.rows.at(i), m = a.rows.at(i + 1) - row0, id = a.ids[i];
    if (m == 0) return p;
    int error = 0;
    if (id < 0 || id >= c.max_seqs || row0 < 0 || m < 0 || row0 + (long long)m > a.rows.rows || nth < 0) {  // nth < 0: starts that fall
        error = CAC_E_BOUNDS;
    } else {
        const int2 pending = *reinterpret_cast<const int2*>(c.pending + 2 * id);
        const int base = c.lens[id] - m;                                     // first new token
        const int t0 = (base / KV_BLOCK + min(nth, m / KV_BLOCK + 2)) * KV_BLOCK;  // first token of the block
        if (pending.x != m || pending.y != i) {
            error = CAC_E_STATE;
        } else if (t0 < base + m) {
            p.lo = max(base - t0, 0), p.hi = min(base + m - t0, KV_BLOCK);
            p.page = c.table[(long long)id * c.max_pages + t0 / c.page_tokens];
            p.in_page = t0 % c.page_tokens;
            p.row = row0 + (long long)(t0 + p.lo - base);
        }
    }
    if (error && (threadIdx.x & 31) == 0) latch_error(c.status, error);
    return p;
}

// A warp takes a block of 16 tokens of a head at a time, BOTH: K and V of it, else one of them.  NIT = ceil(head_dim / 16)
// passes of 32 lanes x 8 values cover the block; all of a task's loads are queued before the first is used, and the
// next task's place is looked up (four dependent reads) while they are under way.
// Single tokens are bound by those reads: 3.7 us for 256 (64 wide, fp32), 4.3 for 32 (128 wide, bf16).  Prompts: 235 MB, read and written,
// in 50 us (4.7 TB/s; 35 at a plain copy's rate), where the encoding of 16 x 128 values keeps the issue slots 55 % and the
// integer pipe 49 % busy between the loads.
template <class T, int CODE, int NIT>
__global__ void __launch_bounds__(WRITE_WARPS * 32, NIT <= 8 ? 2 : 1) kv_write_kernel(const __grid_constant__ KvWrite a) {
    constexpr bool BOTH = NIT * sizeof(T) <= 16;
    constexpr int KV = BOTH ? 2 : 1;
    pdl_trigger();
    pdl_wait();
    const cac_kv8& c = a.c;
    const int lane = threadIdx.x & 31, D = c.head_dim, vec = D >> 3, per_block = (3 - KV) * c.kv_heads;
    const unsigned mul = (65536u + vec - 1) / vec;  // e / vec = e * mul >> 16 for e < 512, vec <= 32
    const long long tasks = (long long)a.blocks * per_block, step = (long long)gridDim.x * WRITE_WARPS;
    long long u = (long long)blockIdx.x * WRITE_WARPS + (threadIdx.x >> 5);
    if (u >= tasks) return;
    KvPlace p = place_of(a, (int)(u / per_block));
    for (; u < tasks; u += step) {
        const int part = (int)(u % per_block), head = part / (3 - KV);
        const bool on = p.hi > p.lo && p.page >= 0;  // a page trimmed before it was written: no query sees it
        const long long at = kv_head_at(c, a.layer, on ? p.page : 0, head) + p.in_page * D;
        const long long sc = kv_scale_at(c, a.layer, on ? p.page : 0, head) + p.in_page / KV_BLOCK;
        Eight<T> raw[KV][NIT];
        float before[KV];
#pragma unroll
        for (int w = 0; w < KV; ++w) {
            const bool v = BOTH ? w : part & 1;
            const long long stride = v ? a.v_stride : a.k_stride;
            const T* src = static_cast<const T*>(v ? a.v : a.k) + p.row * stride + (long long)head * D;
#pragma unroll
            for (int it = 0; it < NIT; ++it) {
                const int e = lane + 32 * it, row = (int)(e * mul >> 16), col = (e - row * vec) * 8;
                if (on && row >= p.lo && row < p.hi) raw[w][it].load(src + (row - p.lo) * stride + col);
            }
            before[w] = on && p.lo > 0 ? (v ? c.v_scale : c.k_scale)[sc] : 0.f;
        }
        const KvPlace next = u + step < tasks ? place_of(a, (int)((u + step) / per_block)) : p;
#pragma unroll
        for (int w = 0; w < KV; ++w) {
            const bool v = BOTH ? w : part & 1;
            uint8_t* codes = static_cast<uint8_t*>(v ? c.v : c.k) + at;
            float x[8];
            uint32_t top = 0;
#pragma unroll
            for (int it = 0; it < NIT; ++it) {
                const int row = (int)((lane + 32 * it) * mul >> 16);
                if (on && row >= p.lo && row < p.hi) {
                    raw[w][it].get(x);
#pragma unroll
                    for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
                }
            }
            top = __reduce_max_sync(0xffffffffu, top);
            const bool bad = top >= 0x7f800000u;
            if (bad) {  // the largest finite one instead
                if (lane == 0) latch_error(c.status, CAC_E_NONFINITE);
                top = 0;
#pragma unroll
                for (int it = 0; it < NIT; ++it) {
                    const int row = (int)((lane + 32 * it) * mul >> 16);
                    if (on && row >= p.lo && row < p.hi) {
                        raw[w][it].get(x);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t y = __float_as_uint(x[k]) & 0x7fffffffu;
                            if (y < 0x7f800000u) top = max(top, y);
                        }
                    }
                }
                top = __reduce_max_sync(0xffffffffu, top);
            }
            float scale = fmaxf(__uint_as_float(top) * (1.f / kv_top<CODE>()), KV_MIN_SCALE);
            if (before[w] >= scale) {
                scale = before[w];
            } else if (on && p.lo > 0) {  // the older codes at the larger scale; zeros where no write has filled the block
                const float r = before[w] / scale;
#pragma unroll 1
                for (int e = lane; e < p.lo * vec; e += 32) {
                    uint2* q = reinterpret_cast<uint2*>(codes + e * 8);
                    decode8<CODE>(*q, x);
                    *q = before[w] > 0.f ? encode8<CODE>(x, r) : make_uint2(0, 0);
                }
            }
            const float inv = 1.f / scale;
#pragma unroll
            for (int it = 0; it < NIT; ++it) {
                const int e = lane + 32 * it, row = (int)(e * mul >> 16), col = (e - row * vec) * 8;
                if (on && row >= p.lo && row < p.hi) {
                    raw[w][it].get(x);
                    if (bad) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            x[k] = x[k] != x[k] ? 0.f : fminf(fmaxf(x[k] * inv, -kv_top<CODE>()), kv_top<CODE>());
                    }
                    *reinterpret_cast<uint2*>(codes + row * D + col) = encode8<CODE>(x, bad ? 1.f : inv);
                }
            }
            if (on && lane == 0) (v ? c.v_scale : c.k_scale)[sc] = scale;
        }
        p = next;
    }
}

// ---------------------------------------------------------------------------
// read: a warp takes a few tokens of a sequence, a lane as many values at a time as make 16 bytes of output, so that
// each store of the warp is one piece of memory (16 values a lane, two or four stores apart, measured three times slower).
// 72,000 tokens: 60 us, 55 at a plain copy's rate; 256 x 16 tokens: 6.5 us.
// ---------------------------------------------------------------------------
struct KvRead {
    cac_kv8 c;
    const int32_t *ids, *first;
    void *k, *v;
    int layer, n, count, pieces, tokens;  // a sequence's pieces of `tokens` tokens
};

template <int VEC> struct Codes;
template <> struct Codes<4> { using type = uint32_t; };
template <> struct Codes<8> { using type = uint2; };

template <class T, int CODE> __global__ void __launch_bounds__(256) kv_read_kernel(const __grid_constant__ KvRead a) {
    pdl_trigger();
    pdl_wait();
    const cac_kv8& c = a.c;
    constexpr int VEC = 16 / sizeof(T);
    const int lane = threadIdx.x & 31, D = c.head_dim, vec = D / VEC, per = c.kv_heads * vec;
    const long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int i = (int)(u / a.pieces), t0 = (int)(u - (long long)i * a.pieces) * a.tokens;
    if (i >= a.n) return;
    const int id = a.ids[i], tokens = min(a.tokens, a.count - t0);
    long long at = -1, sc = 0;  // lane l: token l's first codes and scale
    if (id < 0 || id >= c.max_seqs) {
        if (lane == 0) latch_error(c.status, CAC_E_BOUNDS);
    } else if (lane < tokens) {
        const long long t = (long long)a.first[i] + t0 + lane;
        if (t >= 0 && t < c.lens[id]) {
            const int page = c.table[(long long)id * c.max_pages + t / c.page_tokens], in_page = (int)(t % c.page_tokens);
            if (page >= 0) {
                at = kv_head_at(c, a.layer, page, 0) + (long long)in_page * D;
                sc = kv_scale_at(c, a.layer, page, 0) + in_page / KV_BLOCK;
            }
        }
    }
    const long long out0 = ((long long)i * a.count + t0) * c.kv_heads * D;
    constexpr int AT_ONCE = 4;
    using Word = typename Codes<VEC>::type;
    for (int e0 = 0; e0 < tokens * per; e0 += 32 * AT_ONCE) {
        Word w[AT_ONCE][2];
        float f[AT_ONCE][2];
        long long from[AT_ONCE];
#pragma unroll
        for (int x = 0; x < AT_ONCE; ++x) {
            const int e = e0 + 32 * x + lane, t = e / per, r = e - t * per, head = r / vec;
            const long long tat = __shfl_sync(0xffffffffu, at, t & 31), tsc = __shfl_sync(0xffffffffu, sc, t & 31);
            from[x] = e < tokens * per ? tat : -1;
            if (from[x] >= 0) {
                const long long k = tat + (long long)head * c.page_tokens * D + (r - head * vec) * VEC;
                const long long s = tsc + head * (c.page_tokens / KV_BLOCK);
                if (a.k) w[x][0] = __ldcs(reinterpret_cast<const Word*>(static_cast<const uint8_t*>(c.k) + k)), f[x][0] = c.k_scale[s];
                if (a.v) w[x][1] = __ldcs(reinterpret_cast<const Word*>(static_cast<const uint8_t*>(c.v) + k)), f[x][1] = c.v_scale[s];
            }
        }
#pragma unroll
        for (int x = 0; x < AT_ONCE; ++x) {
            const int e = e0 + 32 * x + lane;
            if (e >= tokens * per) continue;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                T* dst = static_cast<T*>(v ? a.v : a.k);
                if (!dst) continue;
                float y[VEC] = {};
                if (from[x] >= 0) {
                    const uint32_t* word = reinterpret_cast<const uint32_t*>(&w[x][v]);
#pragma unroll
                    for (int k = 0; k < VEC; ++k) y[k] = kv_decode<CODE>((word[k >> 2] >> (8 * (k & 3))) & 255u) * f[x][v];
                }
                store16(dst + out0 + (long long)e * VEC, y);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// fork, truncate, trim: one block per sequence.  Chains of reads of tables and counts: 3.3 us (64 forks), 2.0 (256 truncates), 2.3 (64 trims)
// ---------------------------------------------------------------------------
constexpr int SEQ_T = 256;

// One table less names `page` (-1: none); the last one puts it on the free list.
// A whole warp calls it.
__device__ __forceinline__ void release(const cac_kv8& c, int page) {
    const bool gone = page >= 0 && atomicSub(c.refs + page, 1) == 1;
    const unsigned m = __ballot_sync(0xffffffffu, gone);
    if (!m) return;
    const int lane = threadIdx.x & 31;
    int at = 0;
    if (lane == 0) at = atomicAdd(c.n_free, __popc(m));
    at = __shfl_sync(0xffffffffu, at, 0);
    if (gone) c.free_list[at + __popc(m & ((1u << lane) - 1))] = page;
}

// Whether entry i's id stands anywhere else in ids, or at all in other (null: none)
__device__ __forceinline__ bool listed_twice(const int32_t* ids, const int32_t* other, int n, int i) {
    const int id = ids[i];
    bool hit = false;
    for (int j = threadIdx.x; j < n; j += blockDim.x) hit |= (j != i && ids[j] == id) || (other && other[j] == id);
    return __syncthreads_or(hit) != 0;
}

__global__ void __launch_bounds__(SEQ_T) kv_fork_kernel(const cac_kv8 c, int n, const int32_t* src, const int32_t* dst) {
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x, from = src[i], to = dst[i];
    if (from < 0 || from >= c.max_seqs || to < 0 || to >= c.max_seqs) {
        if (threadIdx.x == 0) latch_error(c.status, CAC_E_BOUNDS);
        return;
    }
    if (listed_twice(dst, src, n, i)) {
        if (threadIdx.x == 0) latch_error(c.status, CAC_E_INVAL);
        return;
    }
    const int len = c.lens[from], have = pages_of(len, c.page_tokens), had = pages_of(c.lens[to], c.page_tokens);
    int32_t* row = c.table + (long long)to * c.max_pages;
    const int32_t* of = c.table + (long long)from * c.max_pages;
    // A page that both name cannot reach zero here: the source names it throughout.
    for (int j0 = 0; j0 < max(have, had); j0 += SEQ_T) {
        const int j = j0 + threadIdx.x;
        const int now = j < have ? of[j] : -1;
        if (now >= 0) atomicAdd(c.refs + now, 1);
        release(c, j < had ? row[j] : -1);
        if (j < max(have, had)) row[j] = now;
    }
    __syncthreads();
    if (threadIdx.x == 0) c.lens[to] = len, c.pending[2 * to] = 0, c.pending[2 * from] = 0;
}

__global__ void __launch_bounds__(SEQ_T)
    kv_truncate_kernel(const cac_kv8 c, int n, const int32_t* ids, const int32_t* new_len, int each) {
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x, id = ids[i], asked = new_len ? new_len[i] : each;
    if (id < 0 || id >= c.max_seqs || asked < 0) {
        if (threadIdx.x == 0) latch_error(c.status, CAC_E_BOUNDS);
        return;
    }
    if (listed_twice(ids, nullptr, n, i)) {
        if (threadIdx.x == 0) latch_error(c.status, CAC_E_INVAL);
        return;
    }
    const int len = c.lens[id], to = min(asked, len), had = pages_of(len, c.page_tokens);
    int32_t* row = c.table + (long long)id * c.max_pages;
    for (int j0 = pages_of(to, c.page_tokens); j0 < had; j0 += SEQ_T) {
        const int j = j0 + threadIdx.x;
        release(c, j < had ? row[j] : -1);
        if (j < had) row[j] = -1;
    }
    __syncthreads();
    if (threadIdx.x == 0) c.lens[id] = to, c.pending[2 * id] = 0;
}

__global__ void __launch_bounds__(SEQ_T) kv_trim_kernel(const cac_kv8 c, int n, const int32_t* ids, KvWindow win) {
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x, id = ids[i];
    if (id < 0 || id >= c.max_seqs) {
        if (threadIdx.x == 0) latch_error(c.status, CAC_E_BOUNDS);
        return;
    }
    if (listed_twice(ids, nullptr, n, i)) {
        if (threadIdx.x == 0) latch_error(c.status, CAC_E_INVAL);
        return;
    }
    const int begin = pages_of(win.sinks, c.page_tokens), end = win.low(c.lens[id]) / c.page_tokens;
    int32_t* row = c.table + (long long)id * c.max_pages;
    for (int j0 = begin; j0 < end; j0 += SEQ_T) {
        const int j = j0 + threadIdx.x;
        release(c, j < end ? row[j] : -1);
        if (j < end) row[j] = -1;
    }
}

// ---------------------------------------------------------------------------
// compact.  With `used` pages in use, the moves are the k-th page in use at or
// past `used` into the k-th free page before it: as many of one as of the other.
// One block plans (eight pages a thread and round), then the moves run at the memory's rate: 5.0 us with a pool of few pages, 8.0 with
// many, of which one kernel's start and two scans are most.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(PLAN_T, 1) kv_compact_plan_kernel(const cac_kv8 c) {
    pdl_trigger();
    pdl_wait();
    const KvWork work = kv_work(c);
    const int used = c.n_pages - *c.n_free;
    int32_t *places = work.list, *movers = work.list + (c.n_pages / 2 + 1);
    int holes = 0, moves = 0;
    const int room = c.n_pages / 2 + 1;  // there are at most min(used, n_pages - used) of either
    constexpr int EACH = 8;              // consecutive pages of a thread: a scan over the block for 8,192 of them
    for (int base = 0; base < c.n_pages; base += PLAN_T * EACH) {
        const int p0 = base + threadIdx.x * EACH;
        unsigned in_use = 0;
#pragma unroll
        for (int k = 0; k < EACH; ++k) in_use |= (unsigned)(p0 + k < c.n_pages && c.refs[p0 + k] > 0) << k;
        const unsigned there = p0 >= c.n_pages ? 0u : (1u << min(EACH, c.n_pages - p0)) - 1;
        const unsigned before = p0 >= used ? 0u : (1u << min(EACH, used - p0)) - 1;  // pages before `used`
        const unsigned hole = before & there & ~in_use, mover = ~before & in_use;
        Two total;
        Two at = block_scan(Two{__popc(hole), __popc(mover)}, &total);
        at.a += holes, at.b += moves;
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            if (hole >> k & 1 && at.a < room) places[at.a++] = p0 + k;
            if (mover >> k & 1 && at.b < room) movers[at.b++] = p0 + k;
        }
        holes += total.a;
        moves += total.b;
    }
    __syncthreads();
    moves = min(min(moves, holes), room);  // equal by construction
    for (int k = threadIdx.x; k < moves; k += PLAN_T) {
        work.name[movers[k]] = places[k];
        c.refs[places[k]] = c.refs[movers[k]];
        c.refs[movers[k]] = 0;
    }
    if (threadIdx.x == 0) work.count[1] = moves, work.count[2] = used;
}

__global__ void __launch_bounds__(256) kv_compact_kernel(const cac_kv8 c) {
    pdl_trigger();
    pdl_wait();
    const KvWork work = kv_work(c);
    const int32_t *places = work.list, *movers = work.list + (c.n_pages / 2 + 1);
    const int moves = work.count[1], used = work.count[2];
    if (moves == 0) return;
    for (int k = blockIdx.x * 256 + threadIdx.x; k < c.n_pages - used; k += gridDim.x * 256) c.free_list[k] = c.n_pages - 1 - k;
    for (int s = blockIdx.x; s < c.max_seqs; s += gridDim.x) {
        int32_t* row = c.table + (long long)s * c.max_pages;
        for (int j = threadIdx.x; j < pages_of(c.lens[s], c.page_tokens); j += blockDim.x)
            if (row[j] >= used) row[j] = work.name[row[j]];
    }
    const long long units = (long long)moves * c.n_layers * 2;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int k = (int)(u / (c.n_layers * 2));
        copy_page(c, movers[k], places[k], (int)(u % (c.n_layers * 2)), c.page_tokens / KV_BLOCK);
    }
}

int launched(cudaError_t e) { return e == cudaSuccess ? CAC_OK : CAC_E_CUDA; }

// Checks that the calls over a list of sequences share.
int check_list(const cac_kv8* c, int n, const void* ids) {
    const int r = kv_check_cache(c);
    if (r != CAC_OK) return r;
    if (n < 0 || (n > 0 && !ids)) return CAC_E_INVAL;
    if (reinterpret_cast<uintptr_t>(ids) & 3) return CAC_E_ALIGN;
    return CAC_OK;
}

constexpr int COPY_BLOCKS = 152 * 8;

template <class T, int CODE, int NIT> cudaError_t launch_write(const KvWrite& a, cudaStream_t s) {
    const long long tasks = (long long)a.blocks * a.c.kv_heads * (NIT * sizeof(T) <= 16 ? 1 : 2);
    // as many blocks as the SMs hold at once (2 of each), which then take further tasks in turn
    const dim3 g((unsigned)std::min<long long>((tasks + WRITE_WARPS - 1) / WRITE_WARPS, 152 * 2)), b(WRITE_WARPS * 32);
    return launch_k(kv_write_kernel<T, CODE, NIT>, g, b, 0, s, 1, a);
}
template <class T, int CODE> cudaError_t launch_write(const KvWrite& a, cudaStream_t s) {
    if (a.c.head_dim <= 64) return launch_write<T, CODE, 4>(a, s);
    if (a.c.head_dim <= 128) return launch_write<T, CODE, 8>(a, s);
    return launch_write<T, CODE, 16>(a, s);
}

}  // namespace
}  // namespace cac

using namespace cac;

extern "C" size_t cac_kv8_work_ints(const cac_kv8* c) { return kv_check_shape(c) == CAC_OK ? kv_work_ints(*c) : 0; }

extern "C" int cac_kv8_init(const cac_kv8* c, void* stream) {
    const int r = kv_check_cache(c);
    if (r != CAC_OK) return r;
    DeviceScope dev(c->device);
    if (!dev.ok) return CAC_E_CUDA;
    return launched(launch_k(kv_init_kernel, dim3(304), dim3(256), 0, static_cast<cudaStream_t>(stream), 1, *c,
                             (long long)kv_work_ints(*c)));
}

extern "C" int cac_kv8_extend(const cac_kv8* c, int n, const int32_t* ids, const int32_t* starts, int each,
                              void* stream) {
    int r = check_list(c, n, ids);
    if (r != CAC_OK) return r;
    if ((!starts && each < 0) || n > c->max_seqs) return CAC_E_INVAL;
    if (reinterpret_cast<uintptr_t>(starts) & 3) return CAC_E_ALIGN;
    if (!starts && each > c->max_pages * c->page_tokens) return CAC_E_LIMIT;
    if (!starts && (long long)n * each > INT32_MAX) return CAC_E_LIMIT;
    if (n == 0) return CAC_OK;
    DeviceScope dev(c->device);
    if (!dev.ok) return CAC_E_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const KvRows rows{starts, each, n, INT32_MAX};
    r = launched(launch_k(kv_extend_kernel, dim3(1), dim3(PLAN_T), 0, s, 1, *c, rows, ids));
    if (r != CAC_OK) return r;
    // a long prompt's new blocks go to as many blocks of the grid as leave each sequence one
    const long long blocks = starts ? (long long)c->max_pages * (c->page_tokens / KV_BLOCK) : (each + 2 * KV_BLOCK - 2) / KV_BLOCK;
    const int parts = (int)std::max<long long>(1, std::min<long long>(COPY_BLOCKS / n, blocks));
    const long long units = (long long)n * std::max(c->n_layers * 2, parts);
    return launched(launch_k(kv_copy_kernel, dim3((unsigned)std::min<long long>(units, COPY_BLOCKS)), dim3(256), 0, s, 1, *c,
                             rows, ids, parts));
}

extern "C" int cac_kv8_write(const cac_kv8* c, int layer, int n, const int32_t* ids, const int32_t* starts, int rows,
                             const void* k, const void* v, long long k_stride, long long v_stride, int dtype,
                             void* stream) {
    const int r = check_list(c, n, ids);
    if (r != CAC_OK) return r;
    if (layer < 0 || layer >= c->n_layers || rows < 0 || n > c->max_seqs ||
        (dtype != CAC_DTYPE_F32 && dtype != CAC_DTYPE_BF16))
        return CAC_E_INVAL;
    if (n == 0 || rows == 0) return CAC_OK;
    if (!starts && rows % n) return CAC_E_INVAL;
    const long long width = (long long)c->kv_heads * c->head_dim, size = dtype == CAC_DTYPE_BF16 ? 2 : 4;
    if (!k || !v || k_stride < width || v_stride < width) return CAC_E_INVAL;
    if (((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) ||
        ((k_stride * size | v_stride * size) & 15) || (reinterpret_cast<uintptr_t>(starts) & 3))
        return CAC_E_ALIGN;
    const int each = starts ? 0 : rows / n;
    const long long blocks = each ? (long long)n * ((each + 2 * KV_BLOCK - 2) / KV_BLOCK) : (long long)rows / KV_BLOCK + 2ll * n;
    if (blocks > INT32_MAX) return CAC_E_LIMIT;
    DeviceScope dev(c->device);
    if (!dev.ok) return CAC_E_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const KvWrite a{*c, {starts, rows / n, n, rows}, ids, k, v, k_stride, v_stride, layer, (int)blocks, each};
    if (c->code == CAC_KV8_INT8)
        return launched(dtype == CAC_DTYPE_BF16 ? launch_write<bf16, CAC_KV8_INT8>(a, s)
                                                : launch_write<float, CAC_KV8_INT8>(a, s));
    return launched(dtype == CAC_DTYPE_BF16 ? launch_write<bf16, CAC_KV8_E4M3>(a, s)
                                            : launch_write<float, CAC_KV8_E4M3>(a, s));
}

extern "C" int cac_kv8_read(const cac_kv8* c, int layer, int n, const int32_t* ids, const int32_t* first, int count,
                            void* k, void* v, int dtype, void* stream) {
    const int r = check_list(c, n, ids);
    if (r != CAC_OK) return r;
    if (layer < 0 || layer >= c->n_layers || count < 0 || (dtype != CAC_DTYPE_F32 && dtype != CAC_DTYPE_BF16))
        return CAC_E_INVAL;
    if (n == 0 || count == 0 || (!k && !v)) return CAC_OK;
    if (!first) return CAC_E_INVAL;
    if (((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) ||
        (reinterpret_cast<uintptr_t>(first) & 3))
        return CAC_E_ALIGN;
    DeviceScope dev(c->device);
    if (!dev.ok) return CAC_E_CUDA;
    // a token to a warp while that leaves warps' places free (8,192 of them: 256 x 16 tokens 9.6 -> 6.5 us); four where there are
    // more, which look four tokens' places up at once (72,000 tokens: 60 us against 65)
    const int tokens = (long long)n * count <= 8192 ? 1 : 4;
    const int pieces = count / tokens + (count % tokens != 0);
    const long long blocks = ((long long)n * pieces + 7) / 8;
    if (blocks > INT32_MAX) return CAC_E_LIMIT;
    const dim3 grid((unsigned)blocks), block(256);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const KvRead a{*c, ids, first, k, v, layer, n, count, pieces, tokens};
    if (c->code == CAC_KV8_INT8)
        return launched(dtype == CAC_DTYPE_BF16
                            ? launch_k(kv_read_kernel<bf16, CAC_KV8_INT8>, grid, block, 0, s, 1, a)
                            : launch_k(kv_read_kernel<float, CAC_KV8_INT8>, grid, block, 0, s, 1, a));
    return launched(dtype == CAC_DTYPE_BF16 ? launch_k(kv_read_kernel<bf16, CAC_KV8_E4M3>, grid, block, 0, s, 1, a)
                                            : launch_k(kv_read_kernel<float, CAC_KV8_E4M3>, grid, block, 0, s, 1, a));
}

extern "C" int cac_kv8_fork(const cac_kv8* c, int n, const int32_t* src, const int32_t* dst, void* stream) {
    const int r = check_list(c, n, src);
    if (r != CAC_OK) return r;
    if (n > 0 && !dst) return CAC_E_INVAL;
    if (reinterpret_cast<uintptr_t>(dst) & 3) return CAC_E_ALIGN;
    if (n == 0) return CAC_OK;
    DeviceScope dev(c->device);
    if (!dev.ok) return CAC_E_CUDA;
    return launched(launch_k(kv_fork_kernel, dim3(n), dim3(SEQ_T), 0, static_cast<cudaStream_t>(stream), 1, *c, n, src,
                             dst));
}

extern "C" int cac_kv8_truncate(const cac_kv8* c, int n, const int32_t* ids, const int32_t* new_len, int each,
                                void* stream) {
    const int r = check_list(c, n, ids);
    if (r != CAC_OK) return r;
    if (!new_len && each < 0) return CAC_E_INVAL;
    if (reinterpret_cast<uintptr_t>(new_len) & 3) return CAC_E_ALIGN;
    if (n == 0) return CAC_OK;
    DeviceScope dev(c->device);
    if (!dev.ok) return CAC_E_CUDA;
    return launched(launch_k(kv_truncate_kernel, dim3(n), dim3(SEQ_T), 0, static_cast<cudaStream_t>(stream), 1, *c, n,
                             ids, new_len, each));
}

extern "C" int cac_kv8_trim(const cac_kv8* c, int n, const int32_t* ids, int att_left, int att_chunk, int sinks,
                            void* stream) {
    const int r = check_list(c, n, ids);
    if (r != CAC_OK) return r;
    if (att_chunk < 1 || sinks < 0) return CAC_E_INVAL;
    if (n == 0 || att_left < 0) return CAC_OK;
    DeviceScope dev(c->device);
    if (!dev.ok) return CAC_E_CUDA;
    return launched(launch_k(kv_trim_kernel, dim3(n), dim3(SEQ_T), 0, static_cast<cudaStream_t>(stream), 1, *c, n, ids,
                             KvWindow{att_left, att_chunk, sinks}));
}

extern "C" int cac_kv8_compact(const cac_kv8* c, void* stream) {
    int r = kv_check_cache(c);
    if (r != CAC_OK) return r;
    DeviceScope dev(c->device);
    if (!dev.ok) return CAC_E_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    r = launched(launch_k(kv_compact_plan_kernel, dim3(1), dim3(PLAN_T), 0, s, 1, *c));
    if (r != CAC_OK) return r;
    return launched(launch_k(kv_compact_kernel, dim3(COPY_BLOCKS), dim3(256), 0, s, 1, *c));
}

extern "C" int cac_kv8_check(const cac_kv8* c) {
    const int r = kv_check_cache(c);
    if (r != CAC_OK) return r;
    DeviceScope dev(c->device);
    if (!dev.ok || cudaDeviceSynchronize() != cudaSuccess) return CAC_E_CUDA;
    int st = 0;
    if (cudaMemcpy(&st, c->status, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return CAC_E_CUDA;
    if (st != 0 && cudaMemset(c->status, 0, 4) != cudaSuccess) return CAC_E_CUDA;
    return st;
}
