// Shared pieces of the paged 8-bit K/V cache (include/cac_kv8.h): the checked
// shape, the codes, the rows of a ragged call, and the launchers of its kernels.
#pragma once

#include <cuda_fp8.h>

#include <cfloat>

#include "cac_kv8.h"
#include "common.cuh"

namespace cac {

constexpr int KV_BLOCK = CAC_KV8_BLOCK;
constexpr float KV_MIN_SCALE = 7.888609052210118e-31f;  // 2^-100: a block of zeros or of tiny values

// ---------------------------------------------------------------------------
// codes
// ---------------------------------------------------------------------------
template <int CODE> __device__ __forceinline__ constexpr float kv_top() { return CODE == CAC_KV8_INT8 ? 127.f : 448.f; }

template <int CODE> __device__ __forceinline__ float kv_decode(uint32_t byte) {
    if constexpr (CODE == CAC_KV8_INT8) return (float)(int8_t)byte;
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
}

// ---------------------------------------------------------------------------
// rows of a ragged call: sequence i has rows starts[i] .. starts[i+1]-1, or
// base + each * i .. base + each * (i + 1) - 1 where starts is null
// ---------------------------------------------------------------------------
struct KvRows {
    const int32_t* starts;
    int each, n, rows, base = 0;
    __device__ __forceinline__ int at(int i) const { return starts ? __ldg(starts + i) : base + each * i; }
};

// The last i in [0, n) with f(i) <= x, for a function that never falls (one that does may give an i with
// f(i) > x); -1 where f(0) > x.  A whole warp calls it: 32 places are tried at once.
template <class F> __device__ __forceinline__ int warp_last_le(int n, long long x, F f) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n;  // the answer is lo - 1 or in [lo, lo + len)
    while (len > 0) {
        const int step = (len + 31) >> 5;
        const int i = lo + lane * step;
        const bool le = lane * step < len && f(i) <= x;
        const int hits = __popc(__ballot_sync(0xffffffffu, le));
        if (hits == 0) return lo - 1;
        const int first = lo + (hits - 1) * step;  // f(first) <= x
        const int end = min(lo + len, first + step);
        lo = first + 1;
        len = end - lo;
    }
    return lo - 1;
}

// ---------------------------------------------------------------------------
// layout of `work`
// ---------------------------------------------------------------------------
struct KvWork {
    int32_t *named, *keeper;    // [n_pages] zero between calls: extend's entries that end in this page; the most tokens of it that one has
    int32_t* last_of;           // in place of name: the last entry with as many, + 1
    int32_t *name, *list;       // [n_pages] compact: a moved page's new place; [2][n_pages / 2] places and their movers
    int32_t *copy_from, *copy_to;  // [max_seqs] last pages to be copied
    int32_t* copy_blocks;       // in place of list: the blocks of those that hold tokens (a copy takes a free page, so n_pages are enough)
    int32_t* count;             // [0] copies of extend, [1] moves of compact, [2] pages in use at compact
};
inline size_t kv_work_ints(const cac_kv8& c) { return (size_t)4 * c.n_pages + 2 + (size_t)2 * c.max_seqs + 16; }
__host__ __device__ inline KvWork kv_work(const cac_kv8& c) {
    KvWork w;
    w.named = c.work;
    w.keeper = w.named + c.n_pages;
    w.name = w.keeper + c.n_pages;
    w.list = w.name + c.n_pages;
    w.copy_from = w.list + c.n_pages + 2;
    w.copy_to = w.copy_from + c.max_seqs;
    w.last_of = w.name;
    w.copy_blocks = w.list;
    w.count = w.copy_to + c.max_seqs;
    return w;
}

// ---------------------------------------------------------------------------
// addresses (64-bit: a pool passes 2^31 bytes)
// ---------------------------------------------------------------------------
// codes of (layer, page, head): page_tokens rows of head_dim bytes
__host__ __device__ __forceinline__ long long kv_head_at(const cac_kv8& c, int layer, int page, int head) {
    return (((long long)layer * c.n_pages + page) * c.kv_heads + head) * c.page_tokens * c.head_dim;
}
__host__ __device__ __forceinline__ long long kv_scale_at(const cac_kv8& c, int layer, int page, int head) {
    return (((long long)layer * c.n_pages + page) * c.kv_heads + head) * (c.page_tokens / KV_BLOCK);
}

// The window of a call, and the tokens a position sees in it.
struct KvWindow {
    int left, chunk, sinks;
    __device__ __forceinline__ int begin(int p) const { return p / chunk * chunk; }  // p >= 0
    __device__ __forceinline__ int low(int p) const { return left < 0 ? 0 : max(begin(p) - left, 0); }
    __device__ __forceinline__ int high(int p, int len) const {
        const long long e = (long long)begin(p) + chunk;
        return e < len ? (int)e : len;
    }
};

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
struct KvAttend {
    cac_kv8 c;
    KvRows rows;
    KvWindow win;
    const int32_t* ids;
    const void* q;
    void* out;
    float* lse;
    long long q_stride, out_stride;
    float scale;
    int layer, heads, group, max_new;
    uint32_t group_mul;  // 2^32 / group, rounded down, + 1 (0 for a group of 1)
    const int2* skip;    // blocks [x, y) of each sequence that are read apart (kv8_shared.cu)
    // row / group of a row below 2^32: the product is the quotient or one more
    __device__ __forceinline__ int query_of(int row) const {
        if (group_mul == 0) return row;
        const int q = (int)__umulhi((uint32_t)row, group_mul);
        return q - (q * group > row);
    }

    // The query rows of a K/V head (a sequence has m * group) in tiles of `size`: sequence i's are numbers first(i) = rows before
    // it * group / size + i and on, where counts differ; m * group rows fill at most that many, first(i + 1) - first(i).
    __host__ __device__ int tiles_of_all(int size) const {
        return (int)(rows.starts ? (long long)rows.rows * group / size + rows.n
                                 : (long long)rows.n * (((long long)max_new * group + size - 1) / size));
    }
    // Sequence and tile of number b, for a whole warp; a sequence of -1 where there is none.
    __device__ __forceinline__ int2 tile_at(int b, int size) const {
        if (!rows.starts) {
            const int per = (int)(((long long)max_new * group + size - 1) / size);
            return make_int2(b / per, b % per);
        }
        const long long before = rows.at(0);
        auto first = [&](int i) { return (rows.at(i) - before) * group / size + i; };
        const int i = warp_last_le(rows.n, b, first);
        const long long y = i < 0 ? 0 : b - first(i);
        if (y < 0) {  // starts that fall
            latch_error(c.status, CAC_E_BOUNDS);
            return make_int2(-1, 0);
        }
        return make_int2(i, (int)y);
    }
};

// The device of a cache as the current one for the life of this object.
struct DeviceScope {
    int was = -1, now;
    bool ok = true;
    explicit DeviceScope(int dev) : now(dev) {
        ok = cudaGetDevice(&was) == cudaSuccess && (was == now || cudaSetDevice(now) == cudaSuccess);
        if (!ok) cudaGetLastError();
    }
    ~DeviceScope() {
        if (was >= 0 && was != now) cudaSetDevice(was);
    }
};

int sm_count(int device);                 // 0 where that cannot be told
int kv_check_shape(const cac_kv8* c);     // CAC_OK or the error of a bad shape
int kv_check_cache(const cac_kv8* c);     // shape and pointers

}  // namespace cac
