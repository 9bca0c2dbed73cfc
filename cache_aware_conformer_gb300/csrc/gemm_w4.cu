// Rows times a weight matrix at 4 bits (include/cac_ops.h, cac_op_gemm_w4).
//
//   C[m][n] = sum_g scale[n][g] * (sum_{k in g} (code[n][k] - zero[n][g]) * A[m][k]) + bias[n]
//
// The weights' bytes bound it: they are read once for up to 32 rows of A, which stay in shared memory.  The inner sums run on the tensor
// cores with 16 rows of weights as operand A and the rows of A as the 8 columns of operand B (mma.sync: the 128 rows of a
// tcgen05 tile would be empty but for a few, and its weights would have to pass through shared memory again).  A code less its
// zero point is exact in bf16: 128 + code is 0x4300 | code, and 128 + zero comes off in one subtraction for two.  bf16
// activations are exact too; fp32 ones enter as three bf16 parts of 8 bits each, cut off, which is all of their 24.  A group's
// sum is scaled in fp32.
//
// The order of k within a group is free as long as both operands have the same.  A thread's codes of a group lie in one
// piece of 4, 8 or 16 bytes, and the pairs that come out of a word with one mask (codes j and j + 4) are what an
// operand register holds; A is laid out to match when it is brought into shared memory, once for a block.
//
// A block has `wn` tiles of 16 rows of weights at a time and cuts their depth between 8 or 16 warps / wn; it walks over
// its tiles with a ring of asynchronous copies for each warp that runs on across them.  Where A is too wide for
// one block's shared memory, or tiles are few, a cluster of blocks cuts the depth further.  Parts are added in order.
#include <algorithm>
#include <atomic>

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
    int m, m_chunk;        // rows of A, rows of a block
    int wn;                // row tiles of a block
    int items, stages;     // row blocks, stages of a slice of the depth
};

constexpr int STAGE_K = 256, STAGE = 16 * STAGE_K / 2, STAGES = 4, PART_ROW = 20, MOST_W4_WARPS = 16;

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// codes j and j + 4 of a word less the zero point
__device__ __forceinline__ uint32_t pair_of(uint32_t word, int j, uint32_t zero) {
    return sub_bf16x2((word >> (4 * j) & 0x000f000fu) | 0x43004300u, zero);
}
__device__ __forceinline__ void w4_cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// What a row's chunk number (16 bytes of 128) is xored with, so that the fragment reads of W words touch all banks.
template <int W> __device__ __forceinline__ int swizzle(int row) { return W == 1 ? row & 7 : W == 2 ? (row & 3) << 1 : (row & 1) << 2; }

// 8 values of A as they meet the words: pairs (0, 4), (1, 5), (2, 6), (3, 7); fp32 values in three parts
template <class T> struct Octet {
    static constexpr int PARTS = sizeof(T) == 4 ? 3 : 1;
    uint4 part[PARTS];
    __device__ __forceinline__ void load(const T* src) {
        if constexpr (sizeof(T) == 2) {
            const uint4 v = *reinterpret_cast<const uint4*>(src);
            part[0] = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                                 __byte_perm(v.y, v.w, 0x7632));
        } else {
            const float4 v = reinterpret_cast<const float4*>(src)[0], u = reinterpret_cast<const float4*>(src)[1];
            const float x[8] = {v.x, u.x, v.y, u.y, v.z, u.z, v.w, u.w};
            uint32_t y[PARTS][8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float rest = x[j];
                const bool finite = fabsf(rest) < INFINITY;   // what is left of an infinity is nothing
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {
                    y[p][j] = p == 0 || finite ? __float_as_uint(rest) >> 16 : 0u;
                    rest -= __uint_as_float(y[p][j] << 16);
                }
                if (x[j] != x[j]) y[0][j] = 0x7fc0u;           // a NaN may hold all its bits in the lower half
            }
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
                part[p] = make_uint4(y[p][0] | y[p][1] << 16, y[p][2] | y[p][3] << 16, y[p][4] | y[p][5] << 16, y[p][6] | y[p][7] << 16);
        }
    }
};

// W: words (8 codes) of a thread in a group, group / 32; MT: tiles of 8 rows of A
template <class T, int W, int MT>
__global__ void __launch_bounds__(MOST_W4_WARPS * 32, 1) w4_kernel(const __grid_constant__ W4Args a) {
    constexpr int PARTS = Octet<T>::PARTS, BLOCKS = 8 / W, LOADS = 4 / W;   // groups of a stage; their scales of a thread
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, g = lane >> 2, t = lane & 3;
    const int N = a.w.n, K = a.w.k, groups = K / (32 * W);
    const int wn = warp % a.wn, wk = warp / a.wn, WK = warps / a.wn;
    const int slice_stage = blockIdx.z * a.stages;                        // first stage of this block's slice
    const int stages = min(a.stages, (K + STAGE_K - 1) / STAGE_K - slice_stage);
    const int m0 = blockIdx.y * a.m_chunk, rows = min(a.m_chunk, a.m - m0);
    uint8_t* ring = smem + warp * (STAGES * STAGE);
    uint8_t* s_a = smem + warps * (STAGES * STAGE);
    const int a_row = a.stages * STAGE_K * 2 + 64, a_plane = rows * a_row;   // + 64: eight rows' fragments touch all banks
    float* s_part = reinterpret_cast<float*>(s_a + PARTS * a.m_chunk * a_row);
    pdl_trigger();
    pdl_wait();

    // the warp's stages: wk, wk + WK, ... of each of its block's items
    int p_item = blockIdx.x, p_stage = wk, into = 0;
    if (wk >= stages) p_item = a.items;
    auto fetch = [&] {   // queue the copies of the next stage; always one group
        if (p_item < a.items) {
            const int n0 = (p_item * a.wn + wn) * 16, chunk0 = (slice_stage + p_stage) * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = j * 4 + (lane >> 3), c = lane & 7;
                if (chunk0 + c < K / 32)
                    w4_cp16(smem_u32(ring) + into * STAGE + r * 128 + ((c ^ swizzle<W>(r)) << 4),
                            static_cast<const uint8_t*>(a.w.packed) + (long long)min(n0 + r, N - 1) * (K / 2) + (chunk0 + c) * 16);
            }
            p_stage += WK;
            if (p_stage >= stages) p_stage = wk, p_item += gridDim.x;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        into = into + 1 == STAGES ? 0 : into + 1;
    };
#pragma unroll 1
    for (int k = 0; k < STAGES - 1; ++k) fetch();

    // The scales (upper half) and zero points of a stage: a thread loads some of those of its four's rows g and g + 8, number
    // x = half * BLOCKS + group at lane x % 4.
    auto scales = [&](int item, int stage, uint32_t (&v)[LOADS]) {
        const int n0 = (item * a.wn + wn) * 16;
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            const int x = t + 4 * j, half = x / BLOCKS, b = (slice_stage + stage) * BLOCKS + x % BLOCKS;
            v[j] = 8;
            if (b < groups && stage < stages && item < a.items) {
                const long long at = (long long)min(n0 + g + 8 * half, N - 1) * groups + b;
                v[j] = (uint32_t)__ldg(static_cast<const uint16_t*>(a.w.scale) + at) << 16 |
                       (a.w.zero ? (uint32_t)__ldg(a.w.zero + at) & 15u : 8u);
            }
        }
    };
    uint32_t next_scale[LOADS];
    scales(blockIdx.x, wk, next_scale);

    // A's rows of this slice
    {
        const int octets = min(a.stages * STAGE_K, K - slice_stage * STAGE_K) / 8;
        for (int e = threadIdx.x; e < rows * octets; e += blockDim.x) {
            const int m = e / octets, u = e - m * octets;
            Octet<T> o;
            o.load(static_cast<const T*>(a.a) + (m0 + m) * a.a_stride + slice_stage * STAGE_K + u * 8);
            const int in = u % (4 * W), at = u - in + (in % W) * 4 + in / W;
#pragma unroll
            for (int p = 0; p < PARTS; ++p) *reinterpret_cast<uint4*>(s_a + p * a_plane + m * a_row + at * 16) = o.part[p];
        }
    }
    __syncthreads();
    const uint8_t* a_at[MT];
#pragma unroll
    for (int y = 0; y < MT; ++y) a_at[y] = s_a + (y * 8 + g < rows ? y * 8 + g : 0) * a_row + t * 16;   // columns past the rows: any values

    int from = 0;
    int buffer = 0;
    for (int item = blockIdx.x; item < a.items; item += gridDim.x) {
        float acc[MT][4] = {};
        for (int stage = wk; stage < stages; stage += WK) {
            uint32_t now_scale[LOADS];
#pragma unroll
            for (int j = 0; j < LOADS; ++j) now_scale[j] = next_scale[j];
            if (stage + WK < stages) scales(item, stage + WK, next_scale);
            else scales(item + gridDim.x, wk, next_scale);
            asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
            __syncwarp();
            fetch();   // into the stage that was read last: all lanes are past it
            const uint8_t* at = ring + from * STAGE;
            const int left = groups - (slice_stage + stage) * BLOCKS;
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                if (b >= left) break;
                uint32_t sz[2], word[2][W];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int x = h * BLOCKS + b;
                    sz[h] = __shfl_sync(0xffffffffu, now_scale[x / 4], x % 4, 4);
                    const uint8_t* row = at + (g + 8 * h) * 128;
                    if constexpr (W == 1) {
                        word[h][0] = *reinterpret_cast<const uint32_t*>(row + ((b ^ swizzle<W>(g)) << 4) + t * 4);
                    } else if constexpr (W == 2) {
                        const uint2 v = *reinterpret_cast<const uint2*>(row + (((2 * b + (t >> 1)) ^ swizzle<W>(g)) << 4) + (t & 1) * 8);
                        word[h][0] = v.x, word[h][1] = v.y;
                    } else {
                        const uint4 v = *reinterpret_cast<const uint4*>(row + (((4 * b + t) ^ swizzle<W>(g)) << 4));
                        word[h][0] = v.x, word[h][1] = v.y, word[h][2] = v.z, word[h][3] = v.w;
                    }
                }
                const uint32_t z0 = (sz[0] & 15u) * 0x00010001u + 0x43004300u, z1 = (sz[1] & 15u) * 0x00010001u + 0x43004300u;
                const float s0 = __uint_as_float(sz[0] & 0xffff0000u), s1 = __uint_as_float(sz[1] & 0xffff0000u);
                float part[MT][4] = {};
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    uint32_t f[2][4];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        f[u][0] = pair_of(word[0][w], 2 * u, z0), f[u][1] = pair_of(word[1][w], 2 * u, z1);
                        f[u][2] = pair_of(word[0][w], 2 * u + 1, z0), f[u][3] = pair_of(word[1][w], 2 * u + 1, z1);
                    }
                    const int k = ((stage * BLOCKS + b) * W + w) * 64;
#pragma unroll
                    for (int p = PARTS - 1; p >= 0; --p)   // the small parts first
#pragma unroll
                        for (int y = 0; y < MT; ++y) {
                            const uint4 v = *reinterpret_cast<const uint4*>(a_at[y] + p * a_plane + k);
                            mma_bf16(part[y], f[0], v.x, v.y);
                            mma_bf16(part[y], f[1], v.z, v.w);
                        }
                    // fp32: sums of one word only, since the tensor cores cut sums off where fp32 rounds
                    if (sizeof(T) == 4 || w == W - 1)
#pragma unroll
                        for (int y = 0; y < MT; ++y) {
                            acc[y][0] = fmaf(part[y][0], s0, acc[y][0]), acc[y][1] = fmaf(part[y][1], s0, acc[y][1]);
                            acc[y][2] = fmaf(part[y][2], s1, acc[y][2]), acc[y][3] = fmaf(part[y][3], s1, acc[y][3]);
                            part[y][0] = part[y][1] = part[y][2] = part[y][3] = 0.f;
                        }
                }
            }
            from = from + 1 == STAGES ? 0 : from + 1;
        }
        // the warps' parts, then the blocks', in order
        float* mine = s_part + (buffer * warps + warp) * (MT * 8 * PART_ROW);
#pragma unroll
        for (int y = 0; y < MT; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) mine[(y * 8 + 2 * t + (e & 1)) * PART_ROW + g + 8 * (e >> 1)] = acc[y][e];
        __syncthreads();
        const int slices = gridDim.z, wide = a.wn * 16;
        const float* all = s_part + buffer * warps * (MT * 8 * PART_ROW);
        if (slices > 1) {   // this block's parts added up in the place of its first warps', for the others to read
            for (int e = threadIdx.x; e < rows * wide; e += blockDim.x) {
                const int m = e / wide, n = e - m * wide;
                float* at = const_cast<float*>(all) + ((n >> 4) * MT * 8 + m) * PART_ROW + (n & 15);
                float sum = *at;
                for (int k = 1; k < min(WK, stages); ++k) sum += at[k * a.wn * (MT * 8 * PART_ROW)];
                *at = sum;
            }
            cluster_sync();
        }
        const int rank = slices > 1 ? blockIdx.z : 0;
        for (int e = threadIdx.x + rank * blockDim.x; e < rows * wide; e += blockDim.x * slices) {
            const int m = e / wide, n = e - m * wide, col = item * wide + n;
            const float* at = all + ((n >> 4) * MT * 8 + m) * PART_ROW + (n & 15);
            float sum = 0.f;
            if (slices > 1) {
                for (int k = 0; k < slices; ++k) sum += ld_dsmem(at, k);
            } else {
                sum = *at;
                for (int k = 1; k < min(WK, stages); ++k) sum += at[k * a.wn * (MT * 8 * PART_ROW)];
            }
            if (col < N) static_cast<T*>(a.c)[(m0 + m) * a.c_stride + col] = from_f<T>(sum + (a.bias ? a.bias[col] : 0.f));
        }
        buffer ^= 1;
    }
    if (gridDim.z > 1) cluster_sync();   // no block ends while others read its parts
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// How a call is cut: the cheapest of the few ways there are, in stages that an SM has to go through.
struct Plan {
    int m_chunk, mt, warps, wn, slices, stages, items, blocks, smem;
};
constexpr int W4_SMEM = 226 * 1024;
bool plan_w4(int N, int K, int M, int size, int sms, Plan& best) {
    const int parts = size == 4 ? 3 : 1, all = (K + STAGE_K - 1) / STAGE_K;
    const int chunks = (M + 31) / 32;
    for (int chunk = (M + chunks - 1) / chunks; chunk >= 1; chunk /= 2) {   // fewer rows at a time where a deep A does not fit
        const int mt = chunk <= 8 ? 1 : chunk <= 16 ? 2 : 4;
        float least = 0.f;
        for (int slices = 1; slices <= 8 && slices <= all; slices *= 2) {
            const int stages = (all + slices - 1) / slices;
            if (stages * (slices - 1) >= all) continue;   // a slice would be empty
            for (int warps = 16; warps >= 8; warps /= 2) {
                const long long smem = (long long)warps * STAGES * STAGE + (long long)parts * chunk * (stages * STAGE_K * 2 + 64) +
                                       2ll * warps * mt * 8 * PART_ROW * 4;
                if (smem > W4_SMEM) continue;
                for (int wn = 1; wn <= warps; wn *= 2) {
                    const int items = (N + 16 * wn - 1) / (16 * wn), blocks = std::min(items, std::max(sms / slices, 1)), wk = warps / wn;
                    // an item costs a barrier, about 3 stages' time, with a cluster's two or three
                    const float cost = (float)((items + blocks - 1) / blocks) *
                                       ((float)((stages + wk - 1) / wk * warps) + (slices > 1 ? 8.f : 3.f));
                    if (least == 0.f || cost < least) {
                        least = cost;
                        best = {chunk, mt, warps, wn, slices, stages, items, blocks, (int)smem};
                    }
                }
            }
        }
        if (least > 0.f) return true;
    }
    return false;
}

template <class T, int W, int MT> cudaError_t launch_w4(const W4Args& a, const Plan& p, cudaStream_t s) {
    const auto kernel = w4_kernel<T, W, MT>;
    static std::atomic<uint64_t> ready{0};
    const uint64_t bit = 1ull << (a.w.device & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, W4_SMEM);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_k(kernel, dim3(p.blocks, (a.m + p.m_chunk - 1) / p.m_chunk, p.slices), dim3(p.warps * 32), p.smem, s, p.slices, a);
}
template <class T, int W> cudaError_t launch_w4(const W4Args& a, const Plan& p, cudaStream_t s) {
    return p.mt == 1 ? launch_w4<T, W, 1>(a, p, s) : p.mt == 2 ? launch_w4<T, W, 2>(a, p, s) : launch_w4<T, W, 4>(a, p, s);
}
template <class T> cudaError_t launch_w4(const W4Args& a, const Plan& p, cudaStream_t s) {
    return a.w.group == 32 ? launch_w4<T, 1>(a, p, s) : a.w.group == 64 ? launch_w4<T, 2>(a, p, s) : launch_w4<T, 4>(a, p, s);
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
    if (w->k > CAC_W4_MAX_K || w->n > INT32_MAX - 256 || M > CAC_W4_MAX_M) return CAC_E_LIMIT;
    DeviceScope dev(w->device);
    if (!dev.ok) return CAC_E_CUDA;
    const int sms = sm_count(w->device);
    Plan p;
    if (sms < 1 || !plan_w4(w->n, w->k, M, size, sms, p)) return CAC_E_CUDA;
    const W4Args a{*w, A, bias, C, a_stride, c_stride, M, p.m_chunk, p.wn, p.items, p.stages};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == CAC_DTYPE_BF16 ? launch_w4<bf16>(a, p, s) : launch_w4<float>(a, p, s);
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? CAC_OK : CAC_E_CUDA;
}
