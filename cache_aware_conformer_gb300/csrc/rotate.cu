// Rotation of queries and keys by their position, with an optional norm for each head
// before it (include/cac_ops.h, cac_op_rotate; include/cac_kv8.h, cac_kv8_rotate).
//
// The angle of pair i at position p is p f_i.  f_i is held as a 64-bit fraction of a turn, so that p f_i modulo a
// turn is one integer product, as good at position 10^9 as at 1; its nearest quarter turn is taken off in integers, and what is left, at
// most an eighth of a turn, goes to fp32 with an error of 2^-24 of itself before sine and cosine.  These are computed
// once for a row and serve all of its heads.
//
// The work is one read and one write of q and k: memory bounds it.  A group of threads has a head: each of them two
// 16-byte pieces of it, chosen so that both elements of a pair are the thread's own (the pieces rot_dim / 2 apart, or
// next to each other); where rot_dim / 2 is no whole number of pieces the group exchanges its values
// through shared memory.  The pieces are loaded before the block looks up its positions.
//
// Measured (us; in brackets what the bytes take at a copy's rate): prompts of 22,000 rows, 40 heads of 128 bf16 with norms: 93 (67), where no pipe
// is full (issue slots 67 %) and warps wait for their loads and for the instructions before; 9,100 rows of 20 heads of 128 fp32, half of each rotated
// in pairs, at positions to 10^6: 34 (27); two rows of each of 256 sequences, 16 heads of 64 fp32: 3.3 (0.6), which are three dependent reads and
// a launch.
#include <algorithm>

#include "cac_ops.h"
#include "kv8.cuh"

namespace cac {
namespace {

constexpr int ROT_THREADS = 128, ROT_ROWS = 32;   // of a block at most

// queries or keys: blocks of their own, which have the rows and heads that keep their threads busy
struct RotSide {
    const void* in;
    void* out;
    long long in_stride, out_stride;
    const float* gain;
    int heads, block_rows, blocks;
    uint32_t heads_mul;                // 2^32 / heads, rounded down, + 1
};
struct RotArgs {
    RotSide q, k;
    const uint64_t* steps;
    const int32_t* positions;          // NULL: from the cache
    KvRows seqs;                       // the rows' sequences there
    const int32_t *ids, *lens;
    int* status;
    int max_seqs, rows;
    int head_dim, rot, lanes_log2;     // lanes of a head, a power of two
    float amplitude, eps, inv_dim;     // 1 / head_dim
};

enum { HALF_PIECES, PAIRS, HALF_ANY };

// cos and sin of p f (step: f in 2^-64 of a turn) times amp
__device__ __forceinline__ float2 turn(int p, uint64_t step, float amp) {
    const uint64_t phase = (uint64_t)(long long)p * step;
    const uint32_t t = (uint32_t)((phase + (1ull << 31)) >> 32);      // in 2^-32 of a turn
    const uint32_t quarter = (t + (1u << 29)) >> 30;
    const int rest = (int)(t - (quarter << 30));                      // -2^29 .. 2^29
    float s, c;
    sincospif((float)rest * 4.656612873077393e-10f, &s, &c);          // 2^-31: half turns
    const float a = quarter & 1 ? -s : c, b = quarter & 1 ? c : s;    // turned by quarters
    return quarter & 2 ? make_float2(-a * amp, -b * amp) : make_float2(a * amp, b * amp);
}

// Position of row r; false where it belongs to no sequence or to one that the call may not name.  A whole warp calls it.
__device__ __forceinline__ bool position(const RotArgs& a, int r, int& p) {
    if (a.positions) {
        p = a.positions[r];
        return true;
    }
    int i;
    if (a.seqs.starts) {
        i = warp_last_le(a.seqs.n, r, [&](int k) { return a.seqs.at(k); });
        if (i < 0) return false;
    } else {
        i = r / a.seqs.each;
    }
    const int first = a.seqs.at(i), end = a.seqs.at(i + 1);
    if (r < first || r >= end) return false;
    const int id = a.ids[i];
    if (first < 0 || end > a.rows || id < 0 || id >= a.max_seqs) {
        latch_error(a.status, CAC_E_BOUNDS);
        return false;
    }
    p = a.lens[id] - (end - r);
    return true;
}

template <class T> struct Piece {
    static constexpr int N = 16 / sizeof(T);
};
template <class T> __device__ __forceinline__ void unpack(const uint4& u, float (&x)[16 / sizeof(T)]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        if constexpr (sizeof(T) == 4) {
            x[b] = __uint_as_float(w[b]);
        } else {
            x[2 * b] = __uint_as_float(w[b] << 16);
            x[2 * b + 1] = __uint_as_float(w[b] & 0xffff0000u);
        }
    }
}
template <class T> __device__ __forceinline__ uint4 pack(const float (&x)[16 / sizeof(T)]) {
    uint32_t w[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        if constexpr (sizeof(T) == 4) {
            w[b] = __float_as_uint(x[b]);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * b], x[2 * b + 1]);
            w[b] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// two products, or sums of products, in one instruction
__device__ __forceinline__ float2 mul_two(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma_two(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\t"
        "mov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
// sum over a group of 2^log2 lanes
__device__ __forceinline__ float group_sum(float x, int log2) {
    for (int d = 1 << log2 >> 1; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

template <class T, int HOW>
__global__ void __launch_bounds__(ROT_THREADS, 8) rotate_kernel(const __grid_constant__ RotArgs a) {
    constexpr int N = Piece<T>::N;
    extern __shared__ __align__(16) float2 s_turn[];   // [block_rows][turns of a row], then the exchange
    __shared__ int s_pos[ROT_ROWS], s_there[ROT_ROWS];
    pdl_trigger();
    pdl_wait();
    const bool keys = (int)blockIdx.x >= a.q.blocks;
    const RotSide s = keys ? a.k : a.q;
    const int D = a.head_dim, R = a.rot, half = R >> 1, pieces = D / N;
    const int row0 = ((int)blockIdx.x - (keys ? a.q.blocks : 0)) * s.block_rows, rows = min(s.block_rows, a.rows - row0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int l = threadIdx.x & ((1 << a.lanes_log2) - 1);           // the thread's place in its head's group
    const int stride = (int)(gridDim.y * blockDim.x) >> a.lanes_log2, units = rows * s.heads;   // units: a row's head
    const int rounds = (units - ((int)(blockIdx.y * blockDim.x + warp * 32) >> a.lanes_log2) + stride - 1) / stride;
    if ((int)(blockIdx.y * blockDim.x) >> a.lanes_log2 >= units) return;

    // the thread's two pieces
    int c0, c1;
    bool turned = false;                                             // HALF_PIECES: c0 holds a, c1 holds b
    if constexpr (HOW == HALF_PIECES) {
        const int h = half / N;
        turned = l < h;
        c0 = turned ? l : 2 * h + 2 * (l - h);
        c1 = turned ? l + h : c0 + 1;
    } else {
        c0 = 2 * l, c1 = 2 * l + 1;
    }
    const bool mine = c0 < pieces;
    // A thread's own pairs are N in a row, l N and on: two cosines and two sines to 16 bytes, neighbours' next to each other
    const int owners = (half + N - 1) / N, row_turns = HOW == HALF_ANY ? half : owners * N;

    auto row_of = [&](int u) {   // u / heads: units of a block are below 2^21, where the product is the quotient or one more
        const int r = s.heads == 1 ? u : (int)__umulhi((uint32_t)u, s.heads_mul);
        return r - (r * s.heads > u);
    };
    uint4 in[2] = {};
    auto load = [&](int u) {
        if (u < units && mine) {
            const int r = row_of(u);
            const T* src = static_cast<const T*>(s.in) + (long long)(row0 + r) * s.in_stride + (u - r * s.heads) * D;
            in[0] = *reinterpret_cast<const uint4*>(src + c0 * N);
            in[1] = *reinterpret_cast<const uint4*>(src + c1 * N);
        }
    };
    int u = (int)(blockIdx.y * blockDim.x + threadIdx.x) >> a.lanes_log2;
    load(u);

    for (int r = warp; r < rows; r += warps) {
        int p = 0;
        const bool there = position(a, row0 + r, p);
        if (lane == 0) s_pos[r] = p, s_there[r] = there;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < rows * half; e += blockDim.x) {
        const int r = e / half, i = e - r * half;
        const float2 cs = turn(s_pos[r], a.steps[i], a.amplitude);
        if constexpr (HOW == HALF_ANY) {
            s_turn[r * row_turns + i] = cs;
        } else {
            float* to = reinterpret_cast<float*>(s_turn + r * row_turns) + ((i % N >> 1) * owners + i / N) * 4 + (i & 1);
            to[0] = cs.x, to[2] = cs.y;
        }
    }
    float gain[2][N];
    if (s.gain && mine)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < N; ++j) gain[b][j] = __ldg(s.gain + (b ? c1 : c0) * N + j);
    __syncthreads();

    // whole warps go round together: the groups' sums are shuffles
    for (int k = 0; k < rounds; ++k, u += stride) {
        const bool on = u < units && mine;
        const int r = on ? row_of(u) : 0, head = on ? u - r * s.heads : 0;
        float x[2][N];
        unpack<T>(in[0], x[0]);
        unpack<T>(in[1], x[1]);
        const bool store = on && s_there[r];
        load(u + stride);
        if (s.gain) {
            float2 two = make_float2(0.f, 0.f);
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < N; j += 2) two = fma_two(make_float2(x[b][j], x[b][j + 1]), make_float2(x[b][j], x[b][j + 1]), two);
            float sum = group_sum(on ? two.x + two.y : 0.f, a.lanes_log2);
            // squares of values over 2^60 or so leave fp32: such a head is brought down by 2^80 first (and its eps with it)
            const bool huge = !(sum < 1.3e36f);
            float eps = a.eps;
            if (__any_sync(0xffffffffu, huge)) {
                float again = 0.f;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        if (huge) x[b][j] *= 8.271806125530277e-25f;
                        again = fmaf(x[b][j], x[b][j], again);
                    }
                again = group_sum(on ? again : 0.f, a.lanes_log2);
                if (huge) sum = again, eps = 0.f;
            }
            // The approximate root (2 units in the last place) and one step of Newton's method; beside an infinity finite elements become 0, and
            // the step would make a NaN of the root's 0.
            const float mean = sum * a.inv_dim + eps, y = rsqrtf(mean);
            const float inv = mean < INFINITY ? fmaf(y, 0.5f * fmaf(-mean * y, y, 1.f), y) : y;
            if (mine)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < N; j += 2) {
                        const float2 y = mul_two(make_float2(x[b][j], x[b][j + 1]),
                                                 mul_two(make_float2(inv, inv), make_float2(gain[b][j], gain[b][j + 1])));
                        x[b][j] = y.x, x[b][j + 1] = y.y;
                    }
        }
        const float2* t = s_turn + r * row_turns;
        if constexpr (HOW == HALF_ANY) {
            // the head's values in shared memory, a group's own piece of it
            float* ex = reinterpret_cast<float*>(s_turn + ((s.block_rows * row_turns + 1) & ~1)) +
                        (threadIdx.x >> a.lanes_log2) * (2 * N << a.lanes_log2);
            __syncwarp();
            if (on)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < N; ++j) ex[(b ? c1 : c0) * N + j] = x[b][j];
            __syncwarp();
            if (on)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const int e = (b ? c1 : c0) * N + j;
                        if (e < half) {
                            const float2 cs = t[e];
                            x[b][j] = x[b][j] * cs.x - ex[e + half] * cs.y;
                        } else if (e < R) {
                            const float2 cs = t[e - half];
                            x[b][j] = ex[e - half] * cs.y + x[b][j] * cs.x;
                        }
                    }
        } else if (HOW == HALF_PIECES ? turned : l < owners) {
            const float4* own = reinterpret_cast<const float4*>(t) + l;
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                const float4 cs = own[j / 2 * owners];
                const float2 c = make_float2(cs.x, cs.y), sn = make_float2(cs.z, cs.w);
                if constexpr (HOW == HALF_PIECES) {
                    const float2 p = make_float2(x[0][j], x[0][j + 1]), q = make_float2(x[1][j], x[1][j + 1]);
                    const float2 y = fma_two(p, c, mul_two(make_float2(-q.x, -q.y), sn)), z = fma_two(p, sn, mul_two(q, c));
                    x[0][j] = y.x, x[0][j + 1] = y.y, x[1][j] = z.x, x[1][j + 1] = z.y;
                } else {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int i = j + b;
                        if (l * N + i < half) {
                            float &p = x[i / (N / 2)][2 * i % N], &q = x[i / (N / 2)][2 * i % N + 1];
                            const float was = p;
                            p = was * (b ? c.y : c.x) - q * (b ? sn.y : sn.x);
                            q = was * (b ? sn.y : sn.x) + q * (b ? c.y : c.x);
                        }
                    }
                }
            }
        }
        if (store) {
            T* dst = static_cast<T*>(s.out) + (long long)(row0 + r) * s.out_stride + head * D;
            *reinterpret_cast<uint4*>(dst + c0 * N) = pack<T>(x[0]);
            *reinterpret_cast<uint4*>(dst + c1 * N) = pack<T>(x[1]);
        }
    }
}

template <class T> cudaError_t launch_rotate(const RotArgs& a, int layout, dim3 grid, int threads, cudaStream_t s) {
    constexpr int N = Piece<T>::N;
    const int half = a.rot / 2, rows = std::max(a.q.block_rows, a.k.block_rows);
    const size_t turns = (size_t)rows * ((half + N - 1) / N * N) * 8;
    if (layout == CAC_ROTARY_PAIRS) return launch_k(rotate_kernel<T, PAIRS>, grid, dim3(threads), turns, s, 1, a);
    if (half % N == 0) return launch_k(rotate_kernel<T, HALF_PIECES>, grid, dim3(threads), turns, s, 1, a);
    return launch_k(rotate_kernel<T, HALF_ANY>, grid, dim3(threads), turns + (size_t)threads * 2 * N * 4, s, 1, a);
}

int rotate(const cac_rotary* r, RotArgs& a, int heads, int kv_heads, void* stream) {
    if (a.rows >= 1 << 30) return CAC_E_LIMIT;   // blocks of both sides are counted in 31 bits
    const int sms = sm_count(r->device);
    if (sms < 1) return CAC_E_CUDA;
    const int D = r->head_dim, N = r->dtype == CAC_DTYPE_BF16 ? 8 : 4;
    a.steps = r->steps;
    a.q.gain = r->q_gain, a.k.gain = r->k_gain;
    a.head_dim = D, a.rot = r->rot_dim;
    a.amplitude = r->amplitude, a.eps = r->eps, a.inv_dim = 1.f / (float)D;
    a.lanes_log2 = 0;
    while (2 << a.lanes_log2 < D / N) ++a.lanes_log2;                // an even number of pieces: D is a multiple of 16
    // A block has rows enough for some rounds of its threads, since it begins with 4 us of dependent reads and sines (three rows of 40
    // heads: 117 us for 22,000 rows), but not so many that SMs stay empty, and no more than 36 KB of sines; the heads of few rows are dealt
    // out over several blocks.
    const int room = std::max(1, std::min(ROT_ROWS, 36 * 1024 / std::max((a.rot / 2 + N) * 8, 1)));
    int threads = 32;
    long long most = 0;
    for (RotSide* s : {&a.q, &a.k}) {
        s->heads = s == &a.q ? heads : kv_heads;
        s->heads_mul = s->heads > 1 ? (uint32_t)((1ull << 32) / s->heads) + 1 : 0u;
        const long long items = (long long)s->heads << a.lanes_log2; // threads' work of a row
        if (items == 0) {
            s->block_rows = 1, s->blocks = 0;
            continue;
        }
        s->block_rows = (int)std::max(1ll, std::min({(long long)room, a.rows / (sms * 4ll), (10ll * ROT_THREADS + items - 1) / items}));
        s->blocks = (a.rows + s->block_rows - 1) / s->block_rows;
        most = std::max(most, items * s->block_rows);
        threads = std::max(threads, (int)std::min<long long>(ROT_THREADS, (items * s->block_rows + 31) / 32 * 32));
    }
    const unsigned blocks = (unsigned)a.q.blocks + (unsigned)a.k.blocks;
    const unsigned split = blocks >= 2u * sms ? 1u : (unsigned)((most + threads - 1) / threads);
    DeviceScope dev(r->device);
    if (!dev.ok) return CAC_E_CUDA;
    const dim3 grid(blocks, split);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = r->dtype == CAC_DTYPE_BF16 ? launch_rotate<bf16>(a, r->layout, grid, threads, s)
                                                     : launch_rotate<float>(a, r->layout, grid, threads, s);
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? CAC_OK : CAC_E_CUDA;
}

// CAC_OK or what is wrong with the rotation, or with one side of the call
int check(const cac_rotary* r) {
    if (!r) return CAC_E_INVAL;
    if (r->head_dim < 16 || r->head_dim > 256 || r->head_dim % 16 || r->rot_dim < 0 || r->rot_dim > r->head_dim || r->rot_dim % 2 ||
        (r->layout != CAC_ROTARY_HALF && r->layout != CAC_ROTARY_PAIRS) ||
        (r->dtype != CAC_DTYPE_BF16 && r->dtype != CAC_DTYPE_F32) || r->device < 0 || !(r->amplitude - r->amplitude == 0.f) ||
        !(r->eps >= 1e-20f && r->eps - r->eps == 0.f) || (r->rot_dim && !r->steps))
        return CAC_E_INVAL;
    if ((reinterpret_cast<uintptr_t>(r->steps) & 7) ||
        ((reinterpret_cast<uintptr_t>(r->q_gain) | reinterpret_cast<uintptr_t>(r->k_gain)) & 15))
        return CAC_E_ALIGN;
    return CAC_OK;
}
int check(const cac_rotary* r, int heads, const RotSide& s) {
    if (heads == 0) return CAC_OK;
    const long long width = (long long)heads * r->head_dim, size = r->dtype == CAC_DTYPE_BF16 ? 2 : 4;
    if (!s.in || !s.out || s.in_stride < width || s.out_stride < width || (s.in == s.out && s.in_stride != s.out_stride))
        return CAC_E_INVAL;
    if (((reinterpret_cast<uintptr_t>(s.in) | reinterpret_cast<uintptr_t>(s.out)) & 15) ||
        ((s.in_stride * size | s.out_stride * size) & 15))
        return CAC_E_ALIGN;
    return CAC_OK;
}

}  // namespace
}  // namespace cac

using namespace cac;

extern "C" int cac_op_rotary_steps(int rot_dim, double base, int scaling, double factor, double original, double low,
                                   double high, uint64_t* steps) {
    if (rot_dim < 0 || rot_dim % 2 || rot_dim > 256 || !(base > 1.0) || !(factor >= 1.0) || base > 1e300 || factor > 1e300 ||
        scaling < CAC_ROTARY_NONE || scaling > CAC_ROTARY_RAMP || (rot_dim && !steps) ||
        (scaling == CAC_ROTARY_BASE && rot_dim == 2) || (scaling == CAC_ROTARY_RAMP && (!(original > 0.0) || !(high > low) || !(low >= -1e300))))
        return CAC_E_INVAL;
    const double two_pi = 6.283185307179586476925286766559;
    if (scaling == CAC_ROTARY_BASE && rot_dim > 2) base *= pow(factor, (double)rot_dim / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / rot_dim);
        if (scaling == CAC_ROTARY_LINEAR) f /= factor;
        if (scaling == CAC_ROTARY_RAMP) {
            const double r = std::min(std::max((original * f / two_pi - low) / (high - low), 0.0), 1.0);
            f *= r + (1.0 - r) / factor;
        }
        steps[i] = (uint64_t)rint(ldexp(f / two_pi, 64));  // under 2^62: f is 1 at most
    }
    return CAC_OK;
}

extern "C" int cac_op_rotate(const cac_rotary* r, int rows, const int32_t* positions, int heads, const void* q,
                             long long q_stride, void* q_out, long long q_out_stride, int kv_heads, const void* k,
                             long long k_stride, void* k_out, long long k_out_stride, void* stream) {
    int e = check(r);
    if (e != CAC_OK) return e;
    if (rows < 0 || heads < 0 || kv_heads < 0 || heads > 65535 || kv_heads > 65535 || (rows > 0 && !positions)) return CAC_E_INVAL;
    if (reinterpret_cast<uintptr_t>(positions) & 3) return CAC_E_ALIGN;
    RotArgs a{};
    a.q = {q, q_out, q_stride, q_out_stride}, a.k = {k, k_out, k_stride, k_out_stride};
    if (rows == 0 || heads + kv_heads == 0) return CAC_OK;
    if ((e = check(r, heads, a.q)) != CAC_OK || (e = check(r, kv_heads, a.k)) != CAC_OK) return e;
    a.positions = positions;
    a.rows = rows;
    return rotate(r, a, heads, kv_heads, stream);
}

extern "C" int cac_kv8_rotate(const cac_kv8* c, const cac_rotary* r, int n, const int32_t* ids, const int32_t* starts, int rows,
                              int heads, const void* q, long long q_stride, void* q_out, long long q_out_stride, const void* k,
                              long long k_stride, void* k_out, long long k_out_stride, void* stream) {
    int e = kv_check_cache(c);
    if (e != CAC_OK || (e = check(r)) != CAC_OK) return e;
    if (n < 0 || (n > 0 && !ids) || rows < 0 || heads < 0 || r->head_dim != c->head_dim || r->device != c->device) return CAC_E_INVAL;
    const int kv_heads = k || k_out ? c->kv_heads : 0;
    if (heads > 65535) return CAC_E_INVAL;
    if ((reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(starts)) & 3) return CAC_E_ALIGN;
    if (n == 0 || rows == 0 || heads + kv_heads == 0) return CAC_OK;
    if (!starts && rows % n) return CAC_E_INVAL;
    RotArgs a{};
    a.q = {q, q_out, q_stride, q_out_stride}, a.k = {k, k_out, k_stride, k_out_stride};
    if ((e = check(r, heads, a.q)) != CAC_OK || (e = check(r, kv_heads, a.k)) != CAC_OK) return e;
    a.seqs = {starts, rows / n, n, rows};
    a.ids = ids, a.lens = c->lens, a.status = c->status, a.max_seqs = c->max_seqs;
    a.rows = rows;
    return rotate(r, a, heads, kv_heads, stream);
}
