// Shared by the scored attention kernels and the row-scaled FP8 cache: how a
// score is capped and biased, which keys a query sees, and the format's scale
// bytes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "mma_sync.cuh"
#include "pkv_internal.cuh"
#include "pkv_ptx.cuh"

namespace pkv {

// Scale bytes of the row-scaled FP8 cache: e + 127 for e in [-100, 120] (448 *
// 2^120 is above the largest float; below 2^-100 a row's codes lose bits
// instead, so that 2^e and 2^-e stay normal numbers with room for sums).
constexpr int kMinScaleByte = 27, kMaxScaleByte = 247;

// 2^e of a scale byte.
__device__ __forceinline__ float row_scale(unsigned char b) { return __uint_as_float((uint32_t)b << 23); }

// Four E4M3 codes (bytes 0 .. 3 of c) as floats; exact.
__device__ __forceinline__ void e4m3x4_to_float(uint32_t c, float *x) {
    uint32_t lo, hi;
    e4m3x4_to_f16(c, lo, hi);
    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    x[0] = p.x, x[1] = p.y, x[2] = q.x, x[3] = q.y;
}

// What a call asks of its scores.
struct ScoreArgs {
    float scale;                  // multiplies q.k
    float softcap;                // > 0: x <- softcap * tanh(x / softcap)
    const float *slopes;          // [num_heads] or nullptr: x <- x - slope * |p - t|
    int window;                   // > 0: only keys with p - t < window
    const int32_t *prefix_lens;   // [num_seqs] or nullptr: keys t < prefix_len are seen whatever p
    const int32_t *key_starts;    // [queries] or nullptr: keys t < key_start are not seen
};

// The keys that a query sees: [first, pre) and [lo, hi), the first empty where
// the two would meet or overlap (then it is part of the second).
struct KeyRange {
    int first, pre, lo, hi;
    __device__ __forceinline__ bool sees(int t) const { return (t >= lo && t < hi) || (t >= first && t < pre); }
    __device__ __forceinline__ bool meets(int a, int b) const {  // some key of [a, b) is seen
        return (max(a, lo) < min(b, hi)) || (max(a, first) < min(b, pre));
    }
};

// ks: the query's first key, pre: the sequence's prefix, both clamped; p0 .. p1:
// the position (a query) or positions (a block of queries, the union of their
// keys), p1 < len.
__device__ __forceinline__ KeyRange key_range(int ks, int pre, int window, int p0, int p1) {
    KeyRange r;
    r.first = ks;
    r.pre = pre;
    r.lo = max(ks, window > 0 ? max(p0, 0) - window + 1 : 0);  // (before the context's first token every key is within reach)
    r.hi = p1 + 1;
    if (r.lo >= r.hi) {  // no key at or before p1
        r.lo = ks;
        r.hi = max(ks, pre);
        r.pre = ks;
    } else if (pre >= r.lo) {
        r.lo = ks;
        r.hi = max(r.hi, pre);
        r.pre = ks;
    }
    return r;
}

__device__ __forceinline__ int key_start_of(const ScoreArgs &s, int64_t query) {
    return s.key_starts ? max(0, s.key_starts[query]) : 0;
}
__device__ __forceinline__ int prefix_of(const ScoreArgs &s, int seq, int len) {
    return s.prefix_lens ? min(max(0, s.prefix_lens[seq]), len) : 0;
}

// Caps above kWideCap (in base 2; 50 in base e) take tanh of small z by its series, so that a wide cap costs the scores that
// are far below it no accuracy: tanh z = z (1 - z^2/3 + 2 z^4/15 - 17 z^6/315), off by 3.3e-7 of it at kTanhSmall.
constexpr float kWideCap = 73.f, kTanhSmall = 0.25f;
constexpr double kTanhSeries[4] = {1.0, -1.0 / 3.0, 2.0 / 15.0, -17.0 / 315.0};

// Beyond this a cap changes no score below 1e12 by 1e-4, and larger ones are further apart than that: none is applied, which
// keeps the factors made of it within float32's range.
constexpr float kNoCap = 1e20f;

// A host-side constant as float, kept finite (0 times it stays 0).
inline float finite_float(double x) { return (float)(x > 3e38 ? 3e38 : x < -3e38 ? -3e38 : x); }

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

namespace scored {

// 3-D view of a bf16 cache, one box for both 64-column halves of some rows: [half][row][128 B].
inline bool make_slab_map(CUtensorMap *map, const void *base, int64_t rows, int D, int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {64u, (cuuint64_t)rows, (cuuint64_t)(D / 64)};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, 128u};
    cuuint32_t box[3] = {64u, (cuuint32_t)box_rows, (cuuint32_t)(D / 64)};
    cuuint32_t estr[3] = {1u, 1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kGMax = 8;  // query heads per KV head

// A call's arguments, shared by every kernel of it.
struct Args {
    void *out;
    const void *q;
    const void *k_cache, *v_cache;
    const unsigned char *k_scales, *v_scales;  // row-scaled FP8 cache
    const int32_t *block_tables, *seq_lens;
    const int32_t *q_starts;  // nullptr: one query per sequence
    int num_seqs, num_q, max_q_len, num_heads, num_kv_heads, group, block_size, max_blocks, num_blocks, max_seq_len;
    ScoreArgs s;
    unsigned int *err;
};

// Laid-out tiles are counted in 32-bit integers: a batch that could have more takes a launch for each part of it.
constexpr int64_t kMaxTiles = INT32_MAX / 2;

// What a context can hold: the caller's limit, or what the block table addresses.
inline int64_t longest_context(const Args &a) {
    return std::min<int64_t>(a.max_seq_len, (int64_t)a.max_blocks * a.block_size);
}

// The call for sequences [s0, s0 + n) of a's.
inline Args part_of(const Args &a, int head_dim, int s0, int n) {
    Args p = a;
    p.num_seqs = n;
    p.block_tables += (int64_t)s0 * a.max_blocks;
    p.seq_lens += s0;
    if (a.s.prefix_lens) p.s.prefix_lens += s0;
    if (a.q_starts) {  // rows of queries, and their first keys, count over the whole batch
        p.q_starts += s0;
    } else {
        const int64_t at = (int64_t)s0 * a.num_heads * head_dim * 2;  // (bf16)
        p.out = static_cast<char *>(a.out) + at;
        p.q = static_cast<const char *>(a.q) + at;
        p.num_q = n;
        if (a.s.key_starts) p.s.key_starts += s0;
    }
    return p;
}

// Checks that the calls share; *empty: valid, and nothing to do.
pkv_status check(const Args &a, int head_dim, int dtype, bool fp8, bool *empty);

// One query per sequence over bf16 or row-scaled FP8 caches (scored_decode.cu).
size_t decode_workspace(int64_t num_seqs, int num_heads, int head_dim);
bool decode_fits(const Args &a);  // one sequence's longest context can be counted
pkv_status run_decode(const Args &a, int head_dim, void *workspace, cudaStream_t st);

// Several queries per sequence on the tensor cores (scored_rows.cu).
size_t rows_workspace(int head_dim);
pkv_status run_rows(const Args &a, int head_dim, void *workspace, size_t workspace_bytes, cudaStream_t st);

}  // namespace scored
}  // namespace pkv
