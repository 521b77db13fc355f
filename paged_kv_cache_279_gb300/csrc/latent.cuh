// Shared by the latent attention translation units: the arguments of a call and
// the rules of its lengths.
#pragma once

#include <stdint.h>

#include "pkv_internal.cuh"

namespace pkv {
namespace latent {

constexpr int kRope = PKV_LATENT_ROPE_DIM;

struct Args {
    void *out;               // [T][H][V]
    const void *q;           // [T][H][V + kRope]
    const void *cache;       // [NB][B][V + kRope]
    const int32_t *tables;   // [S][maxb]
    const int32_t *lens;     // [S]
    const int32_t *q_starts; // [S + 1]; NULL: one query a sequence
    unsigned char *ws;
    unsigned int *err;
    int S, T, H, V, B, bshift, maxb, NB, max_q, max_len;
    int rows;                // most query rows of a sequence, at most T * H
    int whole;               // > 0: no context is cut, share id is row tile id % whole of sequence id / whole
    uint32_t hmul;           // x / H = x * hmul >> hshift for x < 2^31
    int hshift;
    int once;                // the cache's rows are the first to leave L2
    float scale_log2;        // scale * log2(e)
};

// The context and queries of sequence s: L tokens, n queries whose first is
// row q0, query i at position L - n0 + i with n0 the entries q_starts give it.
// Lengths outside [0, cap] are clamped, bad query starts leave n = 0, and more
// than max_q queries are cut; each is reported by the caller that asks for it.
struct Seq {
    int L, q0, n, n0;
    bool flagged;
};
__host__ __device__ __forceinline__ Seq sequence(const Args &a, int s) {
    Seq r;
    const int len = a.lens[s];
    const int cap = (int)min((int64_t)a.max_len, (int64_t)a.maxb * a.B);
    r.L = max(0, min(len, cap));
    r.flagged = len != r.L;
    if (!a.q_starts) {
        r.q0 = s, r.n = r.n0 = 1;
        return r;
    }
    const int b = a.q_starts[s], e = a.q_starts[s + 1];
    if (b < 0 || e < b || e > a.T) {
        r.q0 = 0, r.n = r.n0 = 0;
        r.flagged = true;
        return r;
    }
    r.q0 = b, r.n0 = e - b, r.n = min(r.n0, a.max_q);
    if (r.n != r.n0 || r.n0 > r.L) r.flagged = true;
    return r;
}

// x / H, 0 <= x < 2^31: with l = ceil(log2 H), hmul = floor(2^(31 + l) / H) + 1 passes 2^(31 + l) / H by at most 2^l / H.
__host__ __device__ __forceinline__ int by_heads(const Args &a, int x) { return (int)((uint64_t)(uint32_t)x * a.hmul >> a.hshift); }

// bf16 on the tensor cores: workspace of a call, and the call, its arguments checked.  run_mma: row tiles of up to
// 64 rows; run_pair: of 128.
size_t mma_workspace(int64_t T, int H, int V);
pkv_status run_mma(const Args &a, cudaStream_t st);
size_t pair_workspace(int V);
pkv_status run_pair(const Args &a, cudaStream_t st);

}  // namespace latent
}  // namespace pkv
