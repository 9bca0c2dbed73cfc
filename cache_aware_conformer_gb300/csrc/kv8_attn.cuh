// What the attention kernels over the 8-bit cache share: the codes in fp16, and what a sequence of a call asks for.
#pragma once

#include "kv8.cuh"

namespace cac {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// A row's norm is a sum of weight / V scale.  The weights are held times 2^lift and reach 2^15 at most, a scale is between 2^-100 (a
// block of zeros) and 2^121, so the norm is held times 2^-(lift + 4): one seen token leaves at least 2^-125, whose reciprocal is
// a number too, and the sum over zero values stays within fp32's range (where lift is 7 and every weight is at its highest, up
// to 2^24 tokens).
__host__ __device__ constexpr float norm_factor(int lift) { return 1.f / (float)(1ll << (lift + 4)); }
constexpr float NORM_LOG2 = 4.f;  // log2 of what the norm lacks when the lift is taken off the maximum

// ---------------------------------------------------------------------------
// codes to fp16, exactly: the four bytes of a word as two pairs.  For e4m3 the conversion instruction (its bits moved into place by
// hand, which no NaN could come out of, took 249 us where this takes 216 in 128 windows of 4,096 tokens); so whoever reads
// codes that no write may have filled puts zeros in their place.
// ---------------------------------------------------------------------------
template <int CODE> __device__ __forceinline__ void half4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (CODE == CAC_KV8_INT8) {
        w ^= 0x80808080u;  // u = code + 128; 0x6400 | u is 1024 + u
        uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));  // - 1152
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
    } else {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    }
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// what the rounding in pack_half left over, rounded
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return pack_half(a - f.x, b - f.y);
}
// The power of two that brings a row's largest value between 2^14 and 2^15, as far as fp32's exponents go
__device__ __forceinline__ float lift_to_half(float amax) {
    return __uint_as_float((uint32_t)min(268 - (int)(__float_as_uint(amax) >> 23), 254) << 23);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A token's part of the norm, weight / V scale, may be large where its weight is under the smallest float: its V block is then far
// smaller than the largest one, a block of zeros beside ordinary values above all.  The norms' parts of blocks whose log2 scale is
// under FAR are therefore exponentials of their own, and a norm that moves to another maximum does so in two steps where one factor
// would be 0.  Results are exact this way for scales up to 2^75 beside any; next to larger ones, tokens of blocks 2^115 times
// smaller start to be lost.
constexpr float FAR = -40.f;
// l times r = 2^d
__device__ __forceinline__ float move_norm(float l, float d, float r) {
    if (d > -100.f) return l * r;
    const float half = ex2(0.5f * d);
    return l * half * half;
}

// What a sequence of the call asks for.
struct SeqWork {
    int id, len, m, row0;      // len 0: nothing is seen
    int lot, skt, tiles;       // its window's first block, the sink blocks before it, blocks in all (at least 1)
};
__device__ __forceinline__ SeqWork seq_work(const KvAttend& a, int i) {
    SeqWork s;
    s.row0 = a.rows.at(i);
    s.m = a.rows.at(i + 1) - s.row0;
    s.id = a.ids[i];
    s.len = 0, s.lot = 0, s.skt = 0, s.tiles = 1;
    const bool rows_ok = s.m >= 0 && s.row0 >= 0 && s.row0 + (long long)s.m <= a.rows.rows;
    if (!rows_ok) s.m = 0;
    if (s.id >= 0 && s.id < a.c.max_seqs && s.m <= a.max_new && rows_ok) {
        s.len = a.c.lens[s.id];
    } else {
        latch_error(a.c.status, CAC_E_BOUNDS);
    }
    if (s.len > 0 && s.m > 0) {
        const int low = a.win.low(max(s.len - s.m, 0)), high = a.win.high(s.len - 1, s.len);
        s.lot = low / KV_BLOCK;
        s.skt = min((min(a.win.sinks, high) + KV_BLOCK - 1) / KV_BLOCK, s.lot);
        s.tiles = s.skt + (high + KV_BLOCK - 1) / KV_BLOCK - s.lot;
    }
    return s;
}

constexpr int TA_SEQS = 512;     // sequences of one launch of kv8_attn.cu's kernels

// kv8_attn.cu: few query rows to a K/V head.  split: units may be cut, with workspace of kv_attend_bytes
template <int CODE>
cudaError_t kv_launch_attend(const KvAttend& a, int dtype, bool split, int sms, void* space, cudaStream_t s);
extern template cudaError_t kv_launch_attend<CAC_KV8_INT8>(const KvAttend&, int, bool, int, void*, cudaStream_t);
extern template cudaError_t kv_launch_attend<CAC_KV8_E4M3>(const KvAttend&, int, bool, int, void*, cudaStream_t);
size_t kv_attend_bytes(int head_dim, int sms);
// kv8_prompt.cu
// whether it takes a call whose sequences have `rows` query rows to a K/V head on average
bool kv_prompt_takes(const KvAttend& a, int dtype, int sms, long long rows);
cudaError_t kv_launch_prompt(const KvAttend& a, int dtype, cudaStream_t s);

}  // namespace cac
