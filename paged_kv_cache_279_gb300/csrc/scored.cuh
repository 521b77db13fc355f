// Shared by the scored attention kernels and the row-scaled FP8 cache: how a
// score is capped and biased, which keys a query sees, and the format's scale
// bytes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

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
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
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

// The keys that the query at position p of a context of len tokens sees:
// [first, pre) and [lo, hi), the first empty where the two would meet or
// overlap (then it is part of the second).
struct KeyRange {
    int first, pre, lo, hi;
    __device__ __forceinline__ bool sees(int t) const { return (t >= lo && t < hi) || (t >= first && t < pre); }
    __device__ __forceinline__ bool meets(int a, int b) const {  // some key of [a, b) is seen
        return (max(a, lo) < min(b, hi)) || (max(a, first) < min(b, pre));
    }
};

__device__ __forceinline__ KeyRange key_range(const ScoreArgs &s, int seq, int64_t query, int p, int len) {
    KeyRange r;
    const int ks = s.key_starts ? max(0, s.key_starts[query]) : 0;
    const int pre = s.prefix_lens ? min(max(0, s.prefix_lens[seq]), len) : 0;
    r.lo = max(ks, s.window > 0 ? p - s.window + 1 : 0);
    r.hi = p + 1;  // p < len
    r.first = ks;
    r.pre = pre;
    if (r.lo >= r.hi) {  // no key at or before p
        r.lo = r.first;
        r.hi = max(r.first, pre);
        r.pre = r.first;
    } else if (pre >= r.lo) {
        r.lo = min(r.lo, r.first);
        r.hi = max(r.hi, pre);
        r.pre = r.first;
    }
    return r;
}

}  // namespace pkv
