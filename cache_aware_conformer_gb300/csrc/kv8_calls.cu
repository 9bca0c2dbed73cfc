// The attention calls of the paged 8-bit K/V cache (include/cac_kv8.h): checks, and the choice of a kernel.
#include <algorithm>
#include <atomic>

#include "kv8_attn.cuh"

namespace cac {
namespace {

// SMs of a device, asked for once; 0 where that fails
int sm_count(int device) {
    static std::atomic<int> known[64];
    if (device < 0 || device >= 64) return 0;
    int sms = known[device].load(std::memory_order_relaxed);
    if (sms == 0 && cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) == cudaSuccess)
        known[device].store(sms, std::memory_order_relaxed);
    return sms;
}

// Whether units are cut and dealt out, or a warp takes a whole one: the latter saves the deal and the join, but takes about 0.45 us
// a tile.  Measured (2 bf16 queries, windows of 220 / 450 / 900 tokens, us): 16 sequences of 8 heads 11 / 17 / 28 whole, 18 /
// 19 / 20 dealt out; 256 sequences 17 / 30 / 50 and 28 / 45 / 66; 64 of heads 128 wide 15 / 26 / 45 and 21 / 26 / 38; one of 500 tokens 21
// and 17.
bool splits(const cac_kv8& c, int n, int sms, int max_new, int left, int chunk, int sinks) {
    long long tokens = (long long)c.max_pages * c.page_tokens;
    if (left >= 0) tokens = std::min(tokens, (long long)left + 2ll * chunk + max_new + sinks + 2 * KV_BLOCK);
    const long long units = (long long)n * c.kv_heads;
    const int tiles = units >= 8ll * sms ? 64 : units >= sms / 2 ? 36 : 20;
    return tokens > tiles * KV_BLOCK;
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
        const int each = rows / n, part = std::min(n - i0, TA_SEQS);
        const KvAttend a{*c, {starts ? starts + i0 : nullptr, each, part, rows, each * i0}, {att_left, att_chunk, sinks},
                         ids + i0, q, out, lse, q_stride, out_stride, scale, layer, heads, group, most,
                         group > 1 ? (uint32_t)((1ull << 32) / group) + 1 : 0u};
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
