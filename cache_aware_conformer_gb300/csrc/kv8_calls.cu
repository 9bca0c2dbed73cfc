// The attention calls of the paged 8-bit K/V cache (include/cac_kv8.h): checks, and the choice of a kernel.
#include <algorithm>
#include <atomic>

#include "kv8_attn.cuh"

namespace cac {

// SMs of a device, asked for once; 0 where that fails
int sm_count(int device) {
    static std::atomic<int> known[64];
    if (device < 0 || device >= 64) return 0;
    int sms = known[device].load(std::memory_order_relaxed);
    if (sms == 0 && cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) == cudaSuccess)
        known[device].store(sms, std::memory_order_relaxed);
    return sms;
}

namespace {

// Tokens that the queries of a sequence see at most
long long longest(const cac_kv8& c, int max_new, int left, int chunk, int sinks) {
    const long long tokens = (long long)c.max_pages * c.page_tokens;
    return left < 0 ? tokens : std::min(tokens, (long long)left + 2ll * chunk + max_new + sinks + 2 * KV_BLOCK);
}

// Whether units are cut and dealt out, or a warp takes a whole one: the latter saves the deal and the join, but takes about 0.45 us
// a tile.  Measured (2 bf16 queries, windows of 220 / 450 / 900 tokens, us): 16 sequences of 8 heads 11 / 17 / 28 whole, 18 /
// 19 / 20 dealt out; 256 sequences 17 / 30 / 50 and 28 / 45 / 66; 64 of heads 128 wide 15 / 26 / 45 and 21 / 26 / 38; one of 500 tokens 21
// and 17.
bool splits(const cac_kv8& c, int n, int sms, int max_new, int left, int chunk, int sinks) {
    const long long tokens = longest(c, max_new, left, chunk, sinks);
    const long long units = (long long)n * c.kv_heads;
    const int tiles = units >= 8ll * sms ? 64 : units >= sms / 2 ? 36 : 20;
    return tokens > tiles * KV_BLOCK;
}

// CAC_OK or what is wrong with the arguments that both attention calls have
int check_attend(const cac_kv8* c, int layer, int n, const int32_t* ids, const int32_t* starts, int rows, int max_new, int heads,
                 float scale, int att_chunk, int sinks, const void* q, long long q_stride, void* out, long long out_stride,
                 float* lse, int dtype) {
    const int r = kv_check_cache(c);
    if (r != CAC_OK) return r;
    if (n < 0 || (n > 0 && !ids) || layer < 0 || layer >= c->n_layers || rows < 0 || heads < 1 || att_chunk < 1 ||
        sinks < 0 || (dtype != CAC_DTYPE_F32 && dtype != CAC_DTYPE_BF16) || !(scale - scale == 0.f))
        return CAC_E_INVAL;
    if (heads % c->kv_heads || heads > 65535) return CAC_E_INVAL;
    if (n == 0 || rows == 0) return CAC_OK;
    if ((!starts && rows % n) || (starts && max_new < 0)) return CAC_E_INVAL;
    const long long width = (long long)heads * c->head_dim, size = dtype == CAC_DTYPE_BF16 ? 2 : 4;
    if (!q || !out || q == out || q_stride < width || out_stride < width) return CAC_E_INVAL;
    const uintptr_t words = reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(starts) |
                            reinterpret_cast<uintptr_t>(lse);
    if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) ||
        ((q_stride * size | out_stride * size) & 15) || (words & 3))
        return CAC_E_ALIGN;
    return CAC_OK;
}

// Part of a call: sequences i0 .. i0 + part - 1.
KvAttend part_of(const cac_kv8& c, int layer, int n, int i0, int part, const int32_t* ids, const int32_t* starts, int rows, int most,
                 int heads, float scale, const KvWindow& win, const void* q, long long q_stride, void* out, long long out_stride,
                 float* lse) {
    const int each = rows / n, group = heads / c.kv_heads;
    KvAttend a{};
    a.c = c;
    a.rows = {starts ? starts + i0 : nullptr, each, part, rows, each * i0};
    a.win = win;
    a.ids = ids + i0;
    a.q = q, a.out = out, a.lse = lse, a.q_stride = q_stride, a.out_stride = out_stride;
    a.scale = scale, a.layer = layer, a.heads = heads, a.group = group, a.max_new = most;
    a.group_mul = group > 1 ? (uint32_t)((1ull << 32) / group) + 1 : 0u;
    return a;
}

}  // namespace
}  // namespace cac

using namespace cac;

extern "C" size_t cac_kv8_attend_workspace(const cac_kv8* c, int n, int rows, int max_new, int heads, int att_left,
                                           int att_chunk, int sinks) {
    (void)heads;
    if (kv_check_shape(c) != CAC_OK || n < 1 || rows < 1 || max_new < 0 || att_chunk < 1 || sinks < 0) return 0;
    // A call without starts has rows / n queries of each sequence, whatever max_new is; one with starts needs no more for it.
    const int most = std::max(std::max(std::min(max_new, rows), rows / n), 1);
    if (!splits(*c, n, sm_count(c->device), most, att_left, att_chunk, sinks)) return 0;
    return kv_attend_bytes(c->head_dim, sm_count(c->device));
}

extern "C" int cac_kv8_attend(const cac_kv8* c, int layer, int n, const int32_t* ids, const int32_t* starts, int rows,
                              int max_new, int heads, float scale, int att_left, int att_chunk, int sinks,
                              const void* q, long long q_stride, void* out, long long out_stride, float* lse,
                              int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const int r = check_attend(c, layer, n, ids, starts, rows, max_new, heads, scale, att_chunk, sinks, q, q_stride, out, out_stride,
                               lse, dtype);
    if (r != CAC_OK || n == 0 || rows == 0) return r;
    const int group = heads / c->kv_heads, most = starts ? std::max(std::min(max_new, rows), 1) : rows / n;
    const int sms = sm_count(c->device);
    if (sms < 1) return CAC_E_CUDA;
    const bool split = splits(*c, n, sms, most, att_left, att_chunk, sinks);
    if (split && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) ||
                  workspace_bytes < cac_kv8_attend_workspace(c, n, rows, most, heads, att_left, att_chunk, sinks)))
        return CAC_E_INVAL;
    if (((long long)rows * group / 16 + n) * c->kv_heads > INT32_MAX / 32) return CAC_E_LIMIT;
    DeviceScope dev(c->device);
    if (!dev.ok) return CAC_E_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    for (int i0 = 0; i0 < n; i0 += TA_SEQS) {
        const KvAttend a = part_of(*c, layer, n, i0, std::min(n - i0, TA_SEQS), ids, starts, rows, most, heads, scale,
                                   {att_left, att_chunk, sinks}, q, q_stride, out, out_stride, lse);
        cudaError_t e;
        if (kv_prompt_takes(a, dtype, sms, ((long long)rows * group + n - 1) / n))
            e = kv_launch_prompt(a, dtype, s);
        else
            e = c->code == CAC_KV8_INT8 ? kv_launch_attend<CAC_KV8_INT8>(a, dtype, split, sms, workspace, s)
                                        : kv_launch_attend<CAC_KV8_E4M3>(a, dtype, split, sms, workspace, s);
        if (e != cudaSuccess) return CAC_E_CUDA;
    }
    return CAC_OK;
}

extern "C" size_t cac_kv8_attend_shared_workspace(const cac_kv8* c, int n, int rows, int max_new, int n_groups, int heads,
                                                  int att_left, int att_chunk, int sinks) {
    (void)att_left;
    if (kv_check_shape(c) != CAC_OK || n < 1 || rows < 1 || max_new < 0 || n_groups < 0 || heads < 1 || att_chunk < 1 || sinks < 0)
        return 0;
    // attend's too: a call that it answers better goes to it.  Prompts always do, whose sums of both kinds would take twice what their results
    // in fp32 take (80 of 1,000 rows with 64 heads of 128: 5.2 GB).
    const int sms = sm_count(c->device);
    if (sms >= 1) {
        KvAttend a{};
        a.c = *c, a.rows.n = n;
        const long long each = ((long long)rows * (heads / c->kv_heads) + n - 1) / n;
        if (kv_prompt_takes(a, CAC_DTYPE_BF16, sms, each) && kv_prompt_takes(a, CAC_DTYPE_F32, sms, each))
            return kv_attend_bytes(c->head_dim, sms);
    }
    return std::max(kv_shared_bytes(*c, n, rows, std::max(n_groups, 1), heads, sms), kv_attend_bytes(c->head_dim, sms));
}

extern "C" int cac_kv8_attend_shared(const cac_kv8* c, int layer, int n, const int32_t* ids, const int32_t* starts, int rows,
                                     int max_new, int n_groups, const int32_t* groups, int heads, float scale, int att_left,
                                     int att_chunk, int sinks, const void* q, long long q_stride, void* out,
                                     long long out_stride, float* lse, int dtype, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    const int r = check_attend(c, layer, n, ids, starts, rows, max_new, heads, scale, att_chunk, sinks, q, q_stride, out, out_stride,
                               lse, dtype);
    if (r != CAC_OK) return r;
    if (n_groups < 0 || (n_groups > 0 && !groups) || (n_groups == 0 && groups)) return CAC_E_INVAL;
    if (reinterpret_cast<uintptr_t>(groups) & 3) return CAC_E_ALIGN;
    if (n == 0 || rows == 0) return CAC_OK;
    const int group = heads / c->kv_heads, most = starts ? std::max(std::min(max_new, rows), 1) : rows / n;
    const int sms = sm_count(c->device);
    if (sms < 1) return CAC_E_CUDA;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) ||
        workspace_bytes < cac_kv8_attend_shared_workspace(c, n, rows, most, n_groups, heads, att_left, att_chunk, sinks))
        return CAC_E_INVAL;
    if (((long long)rows * group / 16 + n) * c->kv_heads > INT32_MAX / 32 || n_groups > (1 << 28)) return CAC_E_LIMIT;
    const KvAttend a = part_of(*c, layer, n, 0, n, ids, starts, rows, most, heads, scale, {att_left, att_chunk, sinks}, q, q_stride,
                               out, out_stride, lse);
    // Two kinds of call are attend's.  Sequences with many query rows each: their products bound the call, and every row tile reads the
    // tokens anyway.  And those that have less than 70 MB to read even with nothing shared, which takes 11 us: finding out what is, the
    // parts and their join take as long; 50 MB for fp32 (where a row takes two products) with rows so few that they have no launch of their own.
    // Measured (sequences behind a prefix, own tokens up to 60; us of attend / with the prefix read once): bf16, 8 K/V heads of 128, group 4:
    // 4 sequences 67 MB 28 / 31, 132 MB 38 / 37; 8 of them 34 MB 24 / 28, 67 MB 28 / 30, 100 MB 33 / 32, 132 MB 37 / 35; 32 of them 30 MB
    // 24 / 29, 69 MB 30 / 30, 100 MB 34 / 30, 132 MB 37 / 30, 266 MB 55 / 38; 4 heads of 64, group 8: 32 sequences 34 MB 25 / 29, 67 MB 30 / 30,
    // 100 MB 36 / 31, 132 MB 42 / 34.  fp32, 4 heads of 64, group 4: 24 sequences of up to 8 queries 52 MB 40 / 40, 69 MB 45 / 41, 104 MB
    // 52 / 45; few rows, 8 heads of 64: 4 sequences 33 MB 23 / 25, 50 MB 28 / 28, 66 MB 30 / 29, 100 MB 38 / 32; 8 of them 33 MB 23 / 23, 50 MB 26 / 24,
    // 66 MB 29 / 25; 24 of them 50 MB 27 / 25, 66 MB 30 / 26; but 8 heads of 128, group 4: 8 sequences 66 MB 31 / 35, 100 MB 37 / 37.
    const long long bytes = (long long)n * c->kv_heads * longest(*c, most, att_left, att_chunk, sinks) * 2 * c->head_dim;
    const bool few = dtype == CAC_DTYPE_F32 && !kv_prefix_takes(a, std::max(n_groups, 1));
    if (bytes < (few ? 50000000 : 70000000) || kv_prompt_takes(a, dtype, sms, ((long long)rows * group + n - 1) / n))
        return cac_kv8_attend(c, layer, n, ids, starts, rows, max_new, heads, scale, att_left, att_chunk, sinks, q, q_stride, out,
                              out_stride, lse, dtype, workspace, workspace_bytes, stream);
    DeviceScope dev(c->device);
    if (!dev.ok) return CAC_E_CUDA;
    return kv_attend_shared(a, dtype, groups, std::max(n_groups, 1), sms, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? CAC_OK
               : CAC_E_CUDA;
}
