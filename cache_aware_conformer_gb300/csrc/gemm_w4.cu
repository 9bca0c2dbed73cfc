// Rows times a weight matrix at 4 bits (include/cac_ops.h, cac_op_gemm_w4).
//
//   C[m][n] = sum_g scale[n][g] * (sum_{k in g} (code[n][k] - zero[n][g]) * A[m][k]) + bias[n]
//
// A warp has one row of the weights and up to ROWS rows of A; its lanes take the row's words (8 codes) in turn.
#include <algorithm>

#include "cac_ops.h"
#include "kv8.cuh"

namespace cac {
namespace {

struct W4Args {
    cac_w4 w;
    const void* a;
    const float* bias;
    void* c;
    long long a_stride, c_stride;
    int m;
};

constexpr int ROWS = 4, W4_WARPS = 8;

template <class T> __global__ void __launch_bounds__(W4_WARPS * 32) w4_kernel(const __grid_constant__ W4Args a) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, n = blockIdx.x * W4_WARPS + (threadIdx.x >> 5), m0 = blockIdx.y * ROWS;
    if (n >= a.w.n) return;
    const int K = a.w.k, groups = K / a.w.group;
    const uint32_t* row = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.w.packed) + (long long)n * (K / 2));
    const bf16* scale = static_cast<const bf16*>(a.w.scale) + (long long)n * groups;
    const uint8_t* zero = a.w.zero ? a.w.zero + (long long)n * groups : nullptr;
    float sum[ROWS] = {};
    for (int x = lane; x < K / 8; x += 32) {
        const int g = x * 8 / a.w.group;
        const uint32_t word = row[x];
        const float z = zero ? (float)zero[g] : 8.f, s = to_f(scale[g]);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (m0 + r >= a.m) break;
            const T* src = static_cast<const T*>(a.a) + (m0 + r) * a.a_stride + x * 8;
            float part = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) part = fmaf((float)(word >> (4 * j) & 15) - z, to_f(src[j]), part);
            sum[r] = fmaf(part, s, sum[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        for (int d = 16; d; d >>= 1) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], d);
        if (lane == 0 && m0 + r < a.m)
            static_cast<T*>(a.c)[(m0 + r) * a.c_stride + n] = from_f<T>(sum[r] + (a.bias ? a.bias[n] : 0.f));
    }
}

}  // namespace
}  // namespace cac

using namespace cac;

extern "C" int cac_op_gemm_w4(const cac_w4* w, int M, const void* A, long long a_stride, const float* bias, void* C,
                              long long c_stride, int dtype, void* stream) {
    if (!w || w->n < 1 || w->k < 1 || (w->group != 32 && w->group != 64 && w->group != 128) || w->k % w->group || w->device < 0 ||
        !w->packed || !w->scale || M < 1 || !A || !C || A == C || a_stride < w->k || c_stride < w->n ||
        (dtype != CAC_DTYPE_BF16 && dtype != CAC_DTYPE_F32))
        return CAC_E_INVAL;
    const int size = dtype == CAC_DTYPE_BF16 ? 2 : 4;
    if (((reinterpret_cast<uintptr_t>(w->packed) | reinterpret_cast<uintptr_t>(A)) & 15) || (a_stride * size & 15) ||
        (reinterpret_cast<uintptr_t>(w->scale) & 1) || (reinterpret_cast<uintptr_t>(bias) & 3) ||
        (reinterpret_cast<uintptr_t>(C) & (size - 1)))
        return CAC_E_ALIGN;
    DeviceScope dev(w->device);
    if (!dev.ok) return CAC_E_CUDA;
    const W4Args a{*w, A, bias, C, a_stride, c_stride, M};
    const dim3 grid((w->n + W4_WARPS - 1) / W4_WARPS, (M + ROWS - 1) / ROWS);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == CAC_DTYPE_BF16 ? launch_k(w4_kernel<bf16>, grid, dim3(W4_WARPS * 32), 0, s, 1, a)
                                                  : launch_k(w4_kernel<float>, grid, dim3(W4_WARPS * 32), 0, s, 1, a);
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? CAC_OK : CAC_E_CUDA;
}
