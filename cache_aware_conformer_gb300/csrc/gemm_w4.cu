// Rows times a weight matrix at 4 bits (include/cac_ops.h, cac_op_gemm_w4).
//
//   C[m][n] = sum_g scale[n][g] * (sum_{k in g} (code[n][k] - zero[n][g]) * A[m][k]) + bias[n]
//
// The weights' bytes bound it: they are read once for up to 32 rows of A, which stay in shared memory.  The inner sums run on the tensor
// cores with 16 rows of weights as operand A and the rows of A as the 8 columns of operand B (mma.sync: the 128 rows of a
// tcgen05 tile would be empty but for a few, and its weights would have to pass through shared memory again).  A code less its
// zero point is exact in fp16, and comes out of a word with one mask and one multiply-add for two: 0x6400 | c is 1024 + c,
// 0x6400 | c << 4 is 1024 + 16 c.  Activations enter as fp16 after a power of two that brings the largest of 256 of a row under
// 2^15: bf16 ones are exact but for those 2^29 smaller than that, fp32 ones enter as hi + lo (22 bits).  A group's sum is scaled in
// fp32, and 256 products' sum by the power of two.
//
// The order of k within a group is free as long as both operands have the same.  A thread's codes of a group lie in one
// piece of 4, 8 or 16 bytes, and the pairs that come out of a word with one mask (codes j and j + 4) are what an
// operand register holds; A is laid out to match when it is brought into shared memory, once for a block.
//
// A block's 8 or 16 warps form `wn` groups; a group takes 16 rows of weights at a time and cuts their depth between its
// warps.  Each warp streams its shares through a ring of its own, a TMA copy for the codes and 4-byte copies for their scales and
// zero points, several ahead of the mathematics and across its row tiles.  Parts of a tile are handed over through
// shared memory, and each warp adds up some of a tile's results, in order, when it is done with the next tile, so that none waits: with a
// barrier of the block for each tile all warps wait for memory and compute at the same times (8192 -> 32768, one row: 45 us).
// Where A is too wide for one block's shared memory, or tiles are few, a cluster of blocks cuts the depth further and adds its parts up
// once, at the end.
//
// Beside memory it is the integer pipe that counts, which takes an instruction of a warp every other clock: 128 bytes of weights
// come from memory in 5.4 clocks of an SM, and their codes take 5 such instructions, 2.5 clocks (in bf16, whose 7 bits leave no room
// for a code that is not in the lowest place, 7).  So little else may be in the way.  Scales
// have to be asked for as early as the codes: a load that stands behind 100 KB of copies takes 2 us.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "cac_ops.h"
#include "gemm.cuh"
#include "kv8_attn.cuh"

namespace cac {
namespace {

struct W4Args {
    cac_w4 w;
    const void* a;
    const float* bias;
    void* c;
    long long a_stride, c_stride;
    int m, m_chunk;        // rows of A, rows of a block
    int wn;                // groups of a block
    int tiles, stages;     // of 16 rows of weights; stages of a slice of the depth
    int ring, turns;       // stages of a warp's ring; tiles of a group at most
};

constexpr int BOX_K = 256, BOX = 16 * BOX_K / 2;   // a copy: 16 rows of 128 bytes
constexpr int PART_ROW = 20, MOST_W4_WARPS = 16;

__device__ __forceinline__ void mma_w4(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the first product of a sum
__device__ __forceinline__ void mma_w4_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// BYTES bytes, the first `size` of them from memory
template <int BYTES> __device__ __forceinline__ void w4_cp(uint32_t dst, const void* src, int size = BYTES) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(size) : "memory");
}
// (x & MASK) | magic in one instruction, which has room for one constant: the other, 0x64006400, has to be a value that the
// compiler cannot make again for each use
__device__ __forceinline__ uint32_t magic_1024() {
    uint32_t d;
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(d));
    return d;
}
template <uint32_t MASK> __device__ __forceinline__ __half2 masked(uint32_t x, uint32_t magic) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(x), "n"(MASK), "r"(magic));
    return *reinterpret_cast<const __half2*>(&d);
}
// The eight codes of a word less the zero point, in pairs (0, 4), (1, 5), (2, 6), (3, 7).  low, high: -(1024 + z) and -(64 + z)
__device__ __forceinline__ void codes_of(uint32_t word, __half2 low, __half2 high, uint32_t magic, uint32_t (&f)[4]) {
    const __half2 part = __float2half2_rn(0.0625f);
    const uint32_t next = word >> 8;
    const __half2 y[4] = {__hadd2(masked<0x000f000fu>(word, magic), low), __hfma2(masked<0x00f000f0u>(word, magic), part, high),
                          __hadd2(masked<0x000f000fu>(next, magic), low), __hfma2(masked<0x00f000f0u>(next, magic), part, high)};
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = *reinterpret_cast<const uint32_t*>(&y[j]);
}

// The tile's row that is row g (below 8) of the operand.  Chunk c (16 bytes) of row r lies at c ^ r: with these orders the rows
// that a fragment read of W words takes at a time touch all banks.
template <int W> __device__ __forceinline__ int row_of(int g) {
    return W == 1 ? g : W == 2 ? (g & 3) << 1 | g >> 2 : g >> 1 | (g & 1) << 2;
}

// 8 values of A as they meet the words: pairs (0, 4), (1, 5), (2, 6), (3, 7), times `up`; fp32 values in two parts
template <class T> struct Octet {
    static constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
    float x[8];
    struct Raw {
        uint4 v[sizeof(T) / 2];
    };
    static __device__ __forceinline__ Raw load(const T* src, bool on) {
        Raw r;
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) r.v[k] = on ? reinterpret_cast<const uint4*>(src)[k] : make_uint4(0, 0, 0, 0);
        return r;
    }
    __device__ __forceinline__ explicit Octet(const Raw& r) {
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
            const uint32_t w[4] = {r.v[k].x, r.v[k].y, r.v[k].z, r.v[k].w};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if constexpr (sizeof(T) == 4) {
                    x[4 * k + b] = __uint_as_float(w[b]);
                } else {
                    x[2 * b] = __uint_as_float(w[b] << 16);
                    x[2 * b + 1] = __uint_as_float(w[b] & 0xffff0000u);
                }
            }
        }
    }
    __device__ __forceinline__ float largest() const {
        float y = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) y = fmaxf(y, fabsf(x[j]));
        return y;
    }
    __device__ __forceinline__ void put(uint8_t* to, int plane, float up) const {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            hi[j] = pack_half(x[j] * up, x[j + 4] * up);
            lo[j] = PARTS > 1 ? pack_rest(x[j] * up, x[j + 4] * up, hi[j]) : 0u;
        }
        *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (PARTS > 1) *reinterpret_cast<uint4*>(to + plane) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
};

// W: words (8 codes) of a thread in a group of codes, group / 32; MT: tiles of 8 rows of A; HB: boxes of a stage
template <int W, int HB> struct W4Shape {
    static constexpr int STAGE_K = HB * BOX_K, STAGE = HB * BOX;
    static constexpr int BLOCKS = HB * 8 / W;                              // groups of codes of a stage
    // Scales and zero points of a stage and row, brought as they lie in memory: in whole words, wherever they begin in one, or in one or two
    // pieces where rows are aligned to these
    static constexpr int SCALE_WORDS = BLOCKS / 2 + 1, ZERO_WORDS = (BLOCKS + 6) / 4;
    static constexpr int SCALE_PIECE = BLOCKS * 2 < 16 ? BLOCKS * 2 : 16, ZERO_PIECE = BLOCKS < 16 ? BLOCKS : 16;
    static constexpr int SCALE_ROW = (SCALE_WORDS * 4 + 15) / 16 * 16, ZERO_ROW = (ZERO_WORDS * 4 + 15) / 16 * 16;
    static constexpr int RAW = 16 * (SCALE_ROW + ZERO_ROW);
};

template <class T, int W, int MT, int HB>
__global__ void __launch_bounds__(MOST_W4_WARPS * 32, 1)
    w4_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ W4Args a) {
    using S = W4Shape<W, HB>;
    constexpr int STAGE_K = S::STAGE_K, STAGE = S::STAGE, BLOCKS = S::BLOCKS, PARTS = Octet<T>::PARTS;
    constexpr int PART = MT * 8 * PART_ROW;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    // an offset, and not a pointer made of a number: the compiler would no longer know it for shared memory
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    __shared__ uint64_t s_full[MOST_W4_WARPS * 4], s_part_full[MOST_W4_WARPS * 2], s_part_empty[MOST_W4_WARPS * 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, g = lane >> 2, t = lane & 3;
    const int N = a.w.n, K = a.w.k, groups = K / (32 * W), R = a.ring;
    const int wn = warp % a.wn, wk = warp / a.wn, WK = warps / a.wn;
    const int slice_stage = blockIdx.z * a.stages;                        // first stage of this block's slice
    const int stages = min(a.stages, (K + STAGE_K - 1) / STAGE_K - slice_stage);
    const int with = min(WK, stages);                                     // warps of a group that have stages
    const int m0 = blockIdx.y * a.m_chunk, rows = min(a.m_chunk, a.m - m0), slices = gridDim.z;
    const int tile0 = blockIdx.x * a.wn + wn, tile_step = gridDim.x * a.wn;
    uint8_t* ring = smem + warp * R * STAGE;
    uint8_t* s_a = smem + warps * R * STAGE;
    const int a_row = a.stages * STAGE_K * 2 + 64, a_plane = rows * a_row;   // + 64: eight rows' fragments touch all banks
    uint8_t* s_raw = s_a + PARTS * a.m_chunk * a_row;
    uint8_t* raw_ring = s_raw + warp * R * S::RAW;
    float* s_part = reinterpret_cast<float*>(s_raw + warps * R * S::RAW);   // [2][warps][PART]
    float* s_down = s_part + 2 * warps * PART;                            // [boxes][MT * 8]: what a row's values have to be multiplied by
    float* s_held = s_down + a.stages * HB * (MT * 8);                    // a cluster's: [turns][wn][rows][16]
    uint64_t *full = s_full + warp * 4, *part_full = s_part_full + wn * 2, *part_empty = s_part_empty + wn * 2;
    if (lane == 0) {
        for (int k = 0; k < R; ++k) mbar_init(full + k, 33);
        if (wk == 0)
            for (int k = 0; k < 2; ++k) mbar_init(part_full + k, with), mbar_init(part_empty + k, with);
    }
    fence_mbar_init();
    __syncwarp();
    pdl_trigger();
    pdl_wait();

    // the warp's stages: wk, wk + WK, ... of each of its group's tiles
    int p_tile = wk < stages ? tile0 : a.tiles, p_stage = wk, into = 0;
    bool ok = true;
    const long long scales = (long long)N * groups;
    // rows of scales and of zero points that begin with a piece
    const bool scale_even = !((reinterpret_cast<uintptr_t>(a.w.scale) | (uint32_t)(groups * 2)) & (S::SCALE_PIECE - 1));
    const bool zero_even = S::ZERO_PIECE >= 4 && !((reinterpret_cast<uintptr_t>(a.w.zero) | (uint32_t)groups) & (S::ZERO_PIECE - 1));
    auto fetch = [&] {   // queue the copies of the next stage
        if (p_tile < a.tiles) {
            if (lane == 0) {
                mbar_expect_tx(full + into, STAGE);
#pragma unroll
                for (int h = 0; h < HB; ++h)   // a box past the row's end is zeros
                    tma_load_2d(ring + into * STAGE + h * BOX, &map, (slice_stage + p_stage) * (STAGE_K / 2) + h * (BOX_K / 2),
                                p_tile * 16, full + into);
            }
            // 16 rows' scales and zero points
            const int r = lane & 15, second = lane >> 4, b0 = (slice_stage + p_stage) * BLOCKS;
            const long long at = (long long)min(p_tile * 16 + r, N - 1) * groups + b0;
            const uint32_t to = smem_u32(raw_ring) + into * S::RAW + r * S::SCALE_ROW;
            const uint16_t* scale = static_cast<const uint16_t*>(a.w.scale);
            if (scale_even) {
                constexpr int P = S::SCALE_PIECE;
                if (second * P < BLOCKS * 2 && b0 + second * (P / 2) < groups) w4_cp<P>(to + second * P, scale + at + second * (P / 2));
            } else {
#pragma unroll
                for (int k0 = 0; k0 < S::SCALE_WORDS; k0 += 2) {
                    const int k = k0 + second;
                    const long long left = (scales - (at & ~1ll)) - 2 * k;
                    if (k < S::SCALE_WORDS && left > 0) w4_cp<4>(to + 4 * k, scale + (at & ~1ll) + 2 * k, left > 1 ? 4 : 2);
                }
            }
            if (a.w.zero) {
                const uint32_t zto = smem_u32(raw_ring) + into * S::RAW + 16 * S::SCALE_ROW + r * S::ZERO_ROW;
                if (zero_even) {
                    if constexpr (S::ZERO_PIECE >= 4)
                        if (!second && b0 < groups) w4_cp<S::ZERO_PIECE>(zto, a.w.zero + at);
                } else {
#pragma unroll
                    for (int k0 = 0; k0 < S::ZERO_WORDS; k0 += 2) {
                        const int k = k0 + second;
                        const long long left = (scales - (at & ~3ll)) - 4 * k;
                        if (k < S::ZERO_WORDS && left > 0) w4_cp<4>(zto + 4 * k, a.w.zero + (at & ~3ll) + 4 * k, left < 4 ? (int)left : 4);
                    }
                }
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full + into)) : "memory");
            p_stage += WK;
            if (p_stage >= stages) p_stage = wk, p_tile += tile_step;
        }
        into = into + 1 == R ? 0 : into + 1;
    };
    for (int k = 0; k < R - 1; ++k) fetch();

    // A's rows of this slice: a warp takes 256 values of a row, GO of such at once
    {
        const int width = min(a.stages * STAGE_K, K - slice_stage * STAGE_K), boxes = stages * HB, all = rows * boxes;
        constexpr int GO = sizeof(T) == 4 ? 2 : 4;
        const T* src = static_cast<const T*>(a.a) + m0 * a.a_stride + slice_stage * STAGE_K + lane * 8;
        for (int e0 = warp; e0 < all; e0 += GO * warps) {
            typename Octet<T>::Raw raw[GO];
#pragma unroll
            for (int j = 0; j < GO; ++j) {
                const int e = e0 + j * warps, m = e / boxes, u = e - m * boxes;
                raw[j] = Octet<T>::load(src + m * a.a_stride + u * BOX_K, e < all && u * BOX_K + lane * 8 < width);
            }
#pragma unroll
            for (int j = 0; j < GO; ++j) {
                const int e = e0 + j * warps, m = e / boxes, u = e - m * boxes;
                if (e >= all) break;
                const Octet<T> o(raw[j]);
                float most = o.largest();
#pragma unroll
                for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                const float up = lift_to_half(most);
                const int in = lane % (4 * W), at = lane - in + (in % W) * 4 + in / W;
                o.put(s_a + m * a_row + u * (BOX_K * 2) + at * 16, a_plane, up);
                if (lane == 0) s_down[u * (MT * 8) + m] = 1.f / up;
            }
        }
    }
    __syncthreads();
    const uint8_t* a_at[MT];
#pragma unroll
    for (int y = 0; y < MT; ++y) a_at[y] = s_a + (y * 8 + g < rows ? y * 8 + g : 0) * a_row + t * 16;   // columns past the rows: any values

    // The parts of a tile are added up in order, some of its results by each warp.
    auto reduce = [&](int turn, int tile) {
        const int buffer = turn & 1;
        const bool there = __all_sync(0xffffffffu, mbar_wait(part_full + buffer, turn >> 1 & 1));
        const float* all = s_part + (buffer * warps + wn) * PART;
        for (int e = wk * 32 + lane; e < rows * 16; e += with * 32) {
            const int m = e >> 4, col = tile * 16 + (e & 15);
            const float* at = all + m * PART_ROW + (e & 15);
            float sum = *at;
#pragma unroll 4
            for (int k = 1; k < with; ++k) sum += at[k * a.wn * PART];
            if (!there) sum = NAN;
            if (slices > 1)
                s_held[(turn * a.wn + wn) * (rows * 16) + e] = sum;
            else if (col < N)
                static_cast<T*>(a.c)[(m0 + m) * a.c_stride + col] = from_f<T>(sum + (a.bias ? a.bias[col] : 0.f));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(part_empty + buffer);
    };
    int from = 0, phase = 0, turn = 0;
    const uint32_t magic = magic_1024();
    for (int tile = tile0; wk < stages && tile < a.tiles; tile += tile_step, ++turn) {
        float acc[MT][4] = {};
        // where in a word a row's scales and zero points begin
        const uint32_t odd[2] = {(uint32_t)min(tile * 16 + row_of<W>(g), N - 1) * (uint32_t)groups & 3u,
                                 (uint32_t)min(tile * 16 + row_of<W>(g) + 8, N - 1) * (uint32_t)groups & 3u};
        for (int stage = wk; stage < stages; stage += WK) {
            __syncwarp();   // the stage before this one has been read
            if (ok) fetch();
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(full + from, phase));
            uint8_t* raw = raw_ring + from * S::RAW;
            if ((slice_stage + stage + 1) * BLOCKS > groups) {
                // The depth ends within the stage: groups past it have scale 0 (in their words there may be anything), as A has
                // zeros there.
                __syncwarp();
                if (lane < 16) {
                    const uint32_t at = (uint32_t)min(tile * 16 + lane, N - 1) * (uint32_t)groups & 1u;
                    for (int b = groups - (slice_stage + stage) * BLOCKS; b < BLOCKS; ++b)
                        reinterpret_cast<uint16_t*>(raw + lane * S::SCALE_ROW)[at + b] = 0;
                }
                __syncwarp();
            }
            // scales and zero points of rows g and g + 8
            const uint16_t* scale_at[2];
            const uint8_t* zero_at[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                scale_at[h] = reinterpret_cast<const uint16_t*>(raw + (row_of<W>(g) + 8 * h) * S::SCALE_ROW) + (odd[h] & 1);
                zero_at[h] = raw + 16 * S::SCALE_ROW + (row_of<W>(g) + 8 * h) * S::ZERO_ROW + ((odd[h] + (slice_stage + stage) * BLOCKS) & 3);
            }
            const uint8_t* at = ring + from * STAGE + row_of<W>(g) * 128;
            const int swz = row_of<W>(g), a_stage = stage * (STAGE_K * 2);
#pragma unroll 1
            for (int hb = 0; hb < HB; ++hb) {
                float sum[MT][4] = {};
#pragma unroll
                for (int b = 0; b < 8 / W; ++b) {
                    uint32_t word[2][W];
                    float s[2];
                    __half2 z[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        s[h] = __uint_as_float((uint32_t)scale_at[h][hb * (8 / W) + b] << 16);
                        const uint32_t zz = (a.w.zero ? zero_at[h][hb * (8 / W) + b] & 15u : 8u) * 0x00100001u + 0xd400e400u;
                        z[h] = *reinterpret_cast<const __half2*>(&zz);
                        const uint8_t* row = at + hb * BOX + h * 1024;
                        if constexpr (W == 1) {
                            word[h][0] = *reinterpret_cast<const uint32_t*>(row + ((b ^ swz) << 4) + t * 4);
                        } else if constexpr (W == 2) {
                            const uint2 v = *reinterpret_cast<const uint2*>(row + (((2 * b + (t >> 1)) ^ swz) << 4) + (t & 1) * 8);
                            word[h][0] = v.x, word[h][1] = v.y;
                        } else {
                            const uint4 v = *reinterpret_cast<const uint4*>(row + (((4 * b + t) ^ swz) << 4));
                            word[h][0] = v.x, word[h][1] = v.y, word[h][2] = v.z, word[h][3] = v.w;
                        }
                    }
                    float part[MT][4];
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        uint32_t c0[4], c1[4];
                        codes_of(word[0][w], __low2half2(z[0]), __high2half2(z[0]), magic, c0);
                        codes_of(word[1][w], __low2half2(z[1]), __high2half2(z[1]), magic, c1);
                        const uint32_t f[2][4] = {{c0[0], c1[0], c0[1], c1[1]}, {c0[2], c1[2], c0[3], c1[3]}};
                        // fp32: sums of one word only, since the tensor cores cut sums off where fp32 rounds
                        constexpr bool ALONE = sizeof(T) == 4;
#pragma unroll
                        for (int p = PARTS - 1; p >= 0; --p)   // the small part first
#pragma unroll
                            for (int y = 0; y < MT; ++y) {
                                const uint4 v = *reinterpret_cast<const uint4*>(a_at[y] + p * a_plane + a_stage + hb * (BOX_K * 2) + (b * W + w) * 64);
                                if (p == PARTS - 1 && (w == 0 || ALONE)) mma_w4_first(part[y], f[0], v.x, v.y);
                                else mma_w4(part[y], f[0], v.x, v.y);
                                mma_w4(part[y], f[1], v.z, v.w);
                            }
                        if (ALONE || w == W - 1)
#pragma unroll
                            for (int y = 0; y < MT; ++y) {
                                sum[y][0] = fmaf(part[y][0], s[0], sum[y][0]), sum[y][1] = fmaf(part[y][1], s[0], sum[y][1]);
                                sum[y][2] = fmaf(part[y][2], s[1], sum[y][2]), sum[y][3] = fmaf(part[y][3], s[1], sum[y][3]);
                            }
                    }
                }
#pragma unroll
                for (int y = 0; y < MT; ++y) {
                    const float2 d = *reinterpret_cast<const float2*>(s_down + (stage * HB + hb) * (MT * 8) + y * 8 + 2 * t);
                    acc[y][0] = fmaf(sum[y][0], d.x, acc[y][0]), acc[y][1] = fmaf(sum[y][1], d.y, acc[y][1]);
                    acc[y][2] = fmaf(sum[y][2], d.x, acc[y][2]), acc[y][3] = fmaf(sum[y][3], d.y, acc[y][3]);
                }
            }
            if (++from == R) from = 0, phase ^= 1;
        }
        // Its part for the others; then what is this warp's to add up of the tile before, whose parts are there by now.
        const int buffer = turn & 1;
        if (turn > 1 && !mbar_wait(part_empty + buffer, (turn >> 1) + 1 & 1)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        float* mine = s_part + (buffer * warps + warp) * PART;
#pragma unroll
        for (int y = 0; y < MT; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                mine[(y * 8 + 2 * t + (e & 1)) * PART_ROW + row_of<W>(g) + 8 * (e >> 1)] = ok ? acc[y][e] : NAN;   // NAN: a wait gave up
        __syncwarp();
        if (lane == 0) mbar_arrive(part_full + buffer);
        if (turn > 0) reduce(turn - 1, tile - tile_step);
    }
    if (turn > 0) reduce(turn - 1, tile0 + (turn - 1) * tile_step);
    if (!ok)   // copies in flight have to land before the block's memory is another's
        for (int k = 0; k < R - 1; ++k) {
            mbar_wait(full + from, phase);
            if (++from == R) from = 0, phase ^= 1;
        }
    if (slices > 1) {
        cluster_sync();
        const int all = a.turns * a.wn * rows * 16;
        for (int e = threadIdx.x + blockIdx.z * blockDim.x; e < all; e += blockDim.x * slices) {
            const int m = (e >> 4) % rows, u = (e >> 4) / rows, tile = blockIdx.x * a.wn + u % a.wn + u / a.wn * tile_step;
            const int col = tile * 16 + (e & 15);
            if (tile >= a.tiles || col >= N) continue;
            float sum = 0.f;
            for (int k = 0; k < slices; ++k) sum += ld_dsmem(s_held + e, k);
            static_cast<T*>(a.c)[(m0 + m) * a.c_stride + col] = from_f<T>(sum + (a.bias ? a.bias[col] : 0.f));
        }
        cluster_sync();   // no block ends while others read its sums
    }
}

// How a call is cut: the cheapest of the few ways there are.
struct Plan {
    int m_chunk, mt, boxes, warps, wn, slices, stages, tiles, blocks, ring, turns, smem;
};
constexpr int W4_SMEM = 225 * 1024;
bool plan_w4(int N, int K, int M, int size, int group, int sms, const int* clusters, Plan& best) {
    const int parts = size == 4 ? 2 : 1, chunks = (M + 31) / 32, tiles = (N + 15) / 16;
    float least = 0.f;
    // fewer rows at a time where more of them leave less room for copies, or where a deep A does not fit
    for (int chunk = (M + chunks - 1) / chunks; chunk >= 8 || (chunk >= 1 && least == 0.f); chunk = chunk > 8 && chunk < 16 ? 8 : chunk / 2) {
        const int mt = chunk <= 8 ? 1 : chunk <= 16 ? 2 : 4;
        for (int boxes = 1; boxes <= 2; ++boxes) {
            const int all = (K + boxes * BOX_K - 1) / (boxes * BOX_K), blocks_of = boxes * 256 / group;
            const int raw = 16 * (((blocks_of / 2 + 1) * 4 + 15) / 16 * 16 + ((blocks_of + 6) / 4 * 4 + 15) / 16 * 16);
            for (int slices = 1; slices <= 8 && slices <= all; ++slices) {
                const int stages = (all + slices - 1) / slices;
                if (stages * (slices - 1) >= all) continue;   // a slice would be empty
                for (int warps = 16; warps >= 8; warps /= 2) {
                    for (int wn = 1; wn <= warps; wn *= 2) {
                        const int room = slices == 1 ? sms : clusters[slices], blocks = std::min((tiles + wn - 1) / wn, room), wk = warps / wn;
                        const int turns = (tiles + blocks * wn - 1) / (blocks * wn);
                        const long long fixed = 1024 + (long long)parts * chunk * (stages * boxes * BOX_K * 2 + 64) +
                                                2ll * warps * mt * 8 * PART_ROW * 4 + stages * boxes * mt * 8 * 4 +
                                                (slices > 1 ? (long long)turns * wn * chunk * 64 : 0);
                        const int ring = (int)std::min<long long>(4, (W4_SMEM - fixed) / (warps * (boxes * BOX + raw)));
                        if (ring < 2) continue;
                        // Microseconds, as fitted to 2,300 timings of every cut of 25 shapes (1 to 128 rows; the cut that it takes runs 1.01
                        // times as long as the fastest on average, 1.12 at worst).  A box is instructions, twice as slow with eight warps, which
                        // hide less of each other's latencies, and slower with less than 64 KB on their way; then come a stage's own
                        // work, a tile's, the copy of A, the rounds of blocks that several chunks of rows make, and a cluster's
                        // sums.  Without A's copy, rounds and sums, cuts were taken that ran 1.4 times as long as the fastest, 2.1 at worst.
                        const int rounds = (blocks * ((M + chunk - 1) / chunk) + room - 1) / room, steps = (stages + wk - 1) / wk;
                        const int box = 150 + blocks_of / boxes * (24 + 4 * mt) + (24 * parts + 5) * mt;
                        const float far = std::min(1.f, (float)((ring - 1) * warps * boxes * BOX) / 65536.f), few = warps == 8 ? 1.f : 0.f;
                        const float most = (float)turns * warps * steps;
                        const float cost = rounds * (most * boxes * box * 1e-3f * (0.167f + 0.156f * few + 0.032f * (1.f - far)) + most * 0.044f +
                                                     turns * 0.17f + (float)chunk * stages * boxes * parts * (0.0205f + 0.0123f * few) + 0.9f) +
                                           (slices > 1 ? 1.05f + rounds * (slices * slices * (0.0103f + 0.0009f * slices) +
                                                                           (float)turns * wn * chunk * 0.011f) : 0.f);
                        if (least == 0.f || cost < least) {
                            least = cost;
                            best = {chunk, mt, boxes, warps, wn, slices, stages, tiles, blocks, ring, turns,
                                    (int)fixed + ring * warps * (boxes * BOX + raw)};
                        }
                    }
                }
            }
        }
    }
    return least > 0.f;
}

template <class T, int W, int MT, int HB> cudaError_t launch_w4(const CUtensorMap& map, const W4Args& a, const Plan& p, cudaStream_t s) {
    const auto kernel = w4_kernel<T, W, MT, HB>;
    static std::atomic<uint64_t> ready{0};
    const uint64_t bit = 1ull << (a.w.device & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, W4_SMEM);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_k(kernel, dim3(p.blocks, (a.m + p.m_chunk - 1) / p.m_chunk, p.slices), dim3(p.warps * 32), p.smem, s, p.slices, map, a);
}
template <class T, int W, int MT> cudaError_t launch_w4(const CUtensorMap& map, const W4Args& a, const Plan& p, cudaStream_t s) {
    return p.boxes == 1 ? launch_w4<T, W, MT, 1>(map, a, p, s) : launch_w4<T, W, MT, 2>(map, a, p, s);
}
template <class T, int W> cudaError_t launch_w4(const CUtensorMap& map, const W4Args& a, const Plan& p, cudaStream_t s) {
    return p.mt == 1   ? launch_w4<T, W, 1>(map, a, p, s)
           : p.mt == 2 ? launch_w4<T, W, 2>(map, a, p, s)
                       : launch_w4<T, W, 4>(map, a, p, s);
}
template <class T> cudaError_t launch_w4(const CUtensorMap& map, const W4Args& a, const Plan& p, cudaStream_t s) {
    return a.w.group == 32   ? launch_w4<T, 1>(map, a, p, s)
           : a.w.group == 64 ? launch_w4<T, 2>(map, a, p, s)
                             : launch_w4<T, 4>(map, a, p, s);
}

// The plans of a thread's last shapes: the search takes longer than the rest of a call.
bool plan_of(int N, int K, int M, int size, int group, int device, int sms, const int* clusters, Plan& p) {
    struct Known {
        int key[6];
        Plan plan;
    };
    thread_local Known known[32] = {};
    const int key[6] = {N, K, M, size, group, device + 1};
    uint32_t h = 0;
    for (int k : key) h = h * 1000003u + (uint32_t)k;
    Known& at = known[(h ^ h >> 15) & 31];
    if (!std::equal(key, key + 6, at.key)) {
        if (!plan_w4(N, K, M, size, group, sms, clusters, at.plan)) {
            at.key[5] = 0;
            return false;
        }
        std::copy(key, key + 6, at.key);
    }
    p = at.plan;
    return true;
}

// How many clusters of 0 .. 8 blocks of one SM each the device holds at a time: not every SM has neighbours left for a cluster.
// Asked for once.
const int* clusters_of(int device, int sms) {
    static std::atomic<int> known[64];
    static int most[64][9];
    static std::mutex lock;
    if (device < 0 || device >= 64) return nullptr;
    if (!known[device].load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> hold(lock);
        const auto kernel = w4_kernel<bf16, 4, 1, 1>;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, W4_SMEM) != cudaSuccess) return nullptr;
        for (int k = 2; k <= 8; ++k) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute at;
            at.id = cudaLaunchAttributeClusterDimension;
            at.val.clusterDim.x = 1, at.val.clusterDim.y = 1, at.val.clusterDim.z = k;
            cfg.gridDim = dim3(sms, 1, k), cfg.blockDim = dim3(512), cfg.dynamicSmemBytes = W4_SMEM;
            cfg.attrs = &at, cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
                cudaGetLastError();
                n = std::max(1, sms / k / 2);
            }
            most[device][k] = n;
        }
        known[device].store(1, std::memory_order_release);
    }
    return most[device];
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
        ((reinterpret_cast<uintptr_t>(w->scale) | reinterpret_cast<uintptr_t>(w->zero) | reinterpret_cast<uintptr_t>(bias)) & 3) ||
        (reinterpret_cast<uintptr_t>(C) & (size - 1)))
        return CAC_E_ALIGN;
    if (w->k > CAC_W4_MAX_K || w->n > INT32_MAX - 256 || M > CAC_W4_MAX_M) return CAC_E_LIMIT;
    DeviceScope dev(w->device);
    if (!dev.ok) return CAC_E_CUDA;
    const int sms = sm_count(w->device);
    Plan p;
    CUtensorMap map;
    const int* clusters = sms < 1 ? nullptr : clusters_of(w->device, sms);
    if (!clusters || !plan_of(w->n, w->k, M, size, w->group, w->device, sms, clusters, p) || !make_tmap_bytes(&map, w->packed, w->k / 2, w->n, 16))
        return CAC_E_CUDA;
    const W4Args a{*w, A, bias, C, a_stride, c_stride, M, p.m_chunk, p.wn, p.tiles, p.stages, p.ring, p.turns};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == CAC_DTYPE_BF16 ? launch_w4<bf16>(map, a, p, s) : launch_w4<float>(map, a, p, s);
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? CAC_OK : CAC_E_CUDA;
}
