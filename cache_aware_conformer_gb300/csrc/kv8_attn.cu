// Attention over the paged 8-bit K/V cache (include/cac_kv8.h).
//
//   t_j = scale log2(e) ks_b (q . kc_j)     kc: codes of the token, ks_b: scale of its block
//   out = sum_j 2^(t_j - m) vs_b vc_j / sum_j 2^(t_j - m),   m = max_j t_j
#include <algorithm>

#include "kv8.cuh"

namespace cac {
namespace {

constexpr int SA_WARPS = 4;

// One block per (row, head); its warps take the tokens in turn, a lane eight of
// the head's values at most.
template <class T, int CODE> __global__ void __launch_bounds__(SA_WARPS * 32)
    kv_attend_simple_kernel(const __grid_constant__ KvAttend a) {
    __shared__ float sm[SA_WARPS], sl[SA_WARPS], so[SA_WARPS][256];
    pdl_trigger();
    pdl_wait();
    const cac_kv8& c = a.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x, head = blockIdx.y;
    const int i = warp_last_le(a.rows.n, row, [&](int s) { return (long long)a.rows.at(s); });
    if (i < 0 || row >= a.rows.at(i + 1)) return;
    const int m = a.rows.at(i + 1) - a.rows.at(i), id = a.ids[i], D = c.head_dim;
    const bool fits = id >= 0 && id < c.max_seqs && m <= a.max_new;
    if (!fits && threadIdx.x == 0) latch_error(c.status, CAC_E_BOUNDS);
    const int len = fits ? c.lens[id] : 0, pos = len - m + (row - a.rows.at(i));
    const T* q = static_cast<const T*>(a.q) + row * a.q_stride + (long long)head * D;
    float qf[8], o[8] = {}, mx = -INFINITY, l = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) qf[k] = lane + 32 * k < D ? to_f(q[lane + 32 * k]) * a.scale * 1.4426950408889634f : 0.f;
    const int kvh = head / a.group;
    if (pos >= 0 && len > 0) {
        const int low = a.win.low(pos), high = a.win.high(pos, len), sink = min(a.win.sinks, low);
        for (int t = warp; t < sink + high - low; t += SA_WARPS) {
            const int j = t < sink ? t : low + t - sink;
            const int page = c.table[(long long)id * c.max_pages + j / c.page_tokens];
            if (page < 0) continue;
            const int in_page = j % c.page_tokens;
            const long long at = kv_head_at(c, a.layer, page, kvh) + (long long)in_page * D;
            const long long sc = kv_scale_at(c, a.layer, page, kvh) + in_page / KV_BLOCK;
            const uint8_t *kc = static_cast<const uint8_t*>(c.k) + at, *vc = static_cast<const uint8_t*>(c.v) + at;
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (lane + 32 * k < D) s += qf[k] * kv_decode<CODE>(kc[lane + 32 * k]);
#pragma unroll
            for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            s *= c.k_scale[sc];
            const float now = fmaxf(mx, s), f = exp2f(mx - now), p = exp2f(s - now), pv = p * c.v_scale[sc];
            l = l * f + p;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (lane + 32 * k < D) o[k] = o[k] * f + pv * kv_decode<CODE>(vc[lane + 32 * k]);
            mx = now;
        }
    }
    if (lane == 0) sm[warp] = mx, sl[warp] = l;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (lane + 32 * k < D) so[warp][lane + 32 * k] = o[k];
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < SA_WARPS; ++w) top = fmaxf(top, sm[w]);
    if (top == -INFINITY) top = 0.f;  // nothing seen
    for (int w = 0; w < SA_WARPS; ++w) sum += sl[w] * exp2f(sm[w] - top);
    T* out = static_cast<T*>(a.out) + row * a.out_stride + (long long)head * D;
    for (int d = threadIdx.x; d < D; d += blockDim.x) {
        float v = 0.f;
        for (int w = 0; w < SA_WARPS; ++w) v += so[w][d] * exp2f(sm[w] - top);
        out[d] = from_f<T>(sum != 0.f ? v / sum : 0.f);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[(long long)row * a.heads + head] = (top + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace
}  // namespace cac

using namespace cac;

extern "C" size_t cac_kv8_attend_workspace(const cac_kv8* c, int n, int rows, int max_new, int heads) {
    (void)c, (void)n, (void)rows, (void)max_new, (void)heads;
    return 0;
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
    DeviceScope dev(c->device);
    if (!dev.ok) return CAC_E_CUDA;
    KvAttend a{*c, {starts, rows / n, n, rows}, {att_left, att_chunk, sinks}, ids, q, out, lse, q_stride, out_stride,
               scale, layer, heads, heads / c->kv_heads, starts ? max_new : rows / n};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 g(rows, heads), b(SA_WARPS * 32);
    cudaError_t e;
    if (c->code == CAC_KV8_INT8)
        e = dtype == CAC_DTYPE_BF16 ? launch_k(kv_attend_simple_kernel<bf16, CAC_KV8_INT8>, g, b, 0, s, 1, a)
                                    : launch_k(kv_attend_simple_kernel<float, CAC_KV8_INT8>, g, b, 0, s, 1, a);
    else
        e = dtype == CAC_DTYPE_BF16 ? launch_k(kv_attend_simple_kernel<bf16, CAC_KV8_E4M3>, g, b, 0, s, 1, a)
                                    : launch_k(kv_attend_simple_kernel<float, CAC_KV8_E4M3>, g, b, 0, s, 1, a);
    (void)workspace, (void)workspace_bytes;
    return e == cudaSuccess ? CAC_OK : CAC_E_CUDA;
}
