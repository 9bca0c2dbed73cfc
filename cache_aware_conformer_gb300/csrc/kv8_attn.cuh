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
    __device__ __forceinline__ int block(int kt) const { return kt < skt ? kt : lot + kt - skt; }
};
__device__ __forceinline__ SeqWork seq_work(const KvAttend& a, int i) {
    SeqWork s;
    s.row0 = a.rows.at(i);
    s.m = a.rows.at(i + 1) - s.row0;
    s.len = 0, s.lot = 0, s.skt = 0, s.tiles = 1;
    s.id = a.ids[i];
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
// The tokens that a row's query sees.
struct RowSeen {
    int low, high;
};
__device__ __forceinline__ RowSeen row_seen(const KvAttend& a, const SeqWork& s, int row) {
    const int p = s.len - s.m + a.query_of(row);
    const bool on = row < s.m * a.group && p >= 0 && s.len > 0;
    return {on ? a.win.low(p) : 0, on ? a.win.high(p, s.len) : 0};
}

// Of a call that reads some blocks apart (kv8_shared.cu): a sequence's work without those, which may leave it no blocks, or the work on those, as
// rows of several sequences.  A type of its own: the other calls do without the tests (windows of 4,095 tokens took 0.7 % longer with them).
struct PieceWork : SeqWork {
    int gap0, gap;             // from block gap0 on, gap blocks are left out
    bool whole;                // the rows all see all of the blocks
    __device__ __forceinline__ int block(int kt) const {
        if (kt < skt) return kt;
        const int b = lot + kt - skt;
        return b < gap0 ? b : b + gap;
    }
};
__device__ __forceinline__ PieceWork piece_work(const KvAttend& a, int i) {
    PieceWork s{seq_work(a, i), 0, 0, false};
    if (s.len > 0 && s.m > 0) {
        const int2 k = a.skip[i];
        s.gap0 = k.x, s.gap = k.y - k.x;
        s.tiles -= s.gap;
    }
    return s;
}
__device__ __forceinline__ RowSeen row_seen(const KvAttend& a, const PieceWork& s, int row) {
    if (s.whole) return {s.lot * KV_BLOCK, s.len};
    return row_seen(a, static_cast<const SeqWork&>(s), row);
}

constexpr int TA_SEQS = 512;     // sequences of one launch of kv8_attn.cu's kernels

// kv8_attn.cu: few query rows to a K/V head.  split: units may be cut, with workspace of kv_attend_bytes
template <int CODE>
cudaError_t kv_launch_attend(const KvAttend& a, int dtype, bool split, int sms, void* space, cudaStream_t s);
extern template cudaError_t kv_launch_attend<CAC_KV8_INT8>(const KvAttend&, int, bool, int, void*, cudaStream_t);
extern template cudaError_t kv_launch_attend<CAC_KV8_E4M3>(const KvAttend&, int, bool, int, void*, cudaStream_t);
size_t kv_attend_bytes(int head_dim, int sms);
// Units of a call cut into pieces, a block each (kv8_shared.cu): an entry is a sequence or a group of them, its units are its K/V heads and
// tiles of 16 query rows.
struct KvEntry {
    PieceWork s;
    int cuts;              // pieces of each unit; 0: the entry has none
    int first, slot;       // its first piece, and slot of its results where it is cut
};
struct KvPieces {
    const KvEntry* entries;
    const int32_t* first;  // [count] the entries' again
    const int32_t* total;  // pieces in all
    int count, own;        // entries; those from own on go to o1, ml1
    bool low;              // no unit has more than 8 rows
    bool beside;           // runs beside the launch before it (kv8_attn.cu says what that one has to be)
    float *o0, *o1, *slot_o;       // [rows][heads][head_dim]; [slot][16][head_dim]: sums times the norm's factor
    float2 *ml0, *ml1, *slot_ml;   // their maxima and norms
};
constexpr int PIECE_WARPS = 4;
// blocks of an SM that take pieces at once; low: of units of 8 rows at most
constexpr int piece_blocks(int head_dim, bool low) { return head_dim <= 64 ? (low ? 5 : 3) : head_dim <= 128 ? (low ? 4 : 3) : 1; }
template <int CODE>
cudaError_t kv_launch_pieces(const KvAttend& a, const KvPieces& p, int dtype, unsigned blocks, cudaStream_t s);
extern template cudaError_t kv_launch_pieces<CAC_KV8_INT8>(const KvAttend&, const KvPieces&, int, unsigned, cudaStream_t);
extern template cudaError_t kv_launch_pieces<CAC_KV8_E4M3>(const KvAttend&, const KvPieces&, int, unsigned, cudaStream_t);
// kv8_prompt.cu
// whether it takes a call whose sequences have `rows` query rows to a K/V head on average
bool kv_prompt_takes(const KvAttend& a, int dtype, int sms, long long rows);
cudaError_t kv_launch_prompt(const KvAttend& a, int dtype, cudaStream_t s);
// kv8_shared.cu: a.rows and a.ids are the whole call's; workspace of kv_shared_bytes
bool kv_prefix_takes(const KvAttend& a, int n_groups);   // whether the shared tokens have a launch of their own
cudaError_t kv_attend_shared(const KvAttend& a, int dtype, const int32_t* groups, int n_groups, int sms, void* workspace, cudaStream_t s);
size_t kv_shared_bytes(const cac_kv8& c, int n, int rows, int n_groups, int heads, int sms);

}  // namespace cac
