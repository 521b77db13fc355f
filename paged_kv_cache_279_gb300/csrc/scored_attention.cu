// Scored attention over the paged cache: attention whose scores are capped by
// a tanh or biased by distance and whose keys are limited by a window, a
// document's start and an always visible prefix (scored.cuh has the rules).
//   * scored_simt_kernel -- decode, one CTA per (sequence, kv head, 512-token
//     partition) on CUDA cores over float32 caches, float32 arithmetic with expf
//     and tanhf; scored_reduce_kernel merges the partitions.
//
// With x_t the score of a seen key, the running state of a row is (M, l, o) with
// M = max_t x_t, l = sum e^(x_t - M), o = sum e^(x_t - M) v_t; states merge by
// rescaling to the larger M, and the result is o / l (zeros when nothing is seen).
#include <algorithm>
#include <climits>
#include <cmath>

#include "pkv_internal.cuh"
#include "scored.cuh"

namespace pkv {

pkv_status append_new_tokens(const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                             const int32_t *block_tables, const int32_t *seq_lens, int num_seqs, int num_kv_heads,
                             int head_dim, int block_size, int max_blocks_per_seq, int num_blocks, int max_seq_len,
                             int dtype, cudaStream_t st);

namespace scored {

constexpr int kPartition = 512;  // tokens per CTA of the CUDA-core kernel

struct SimtArgs : Args {
    float *part_o;   // [seqs][Hq][parts][D]
    float *part_ml;  // [seqs][Hq][parts][2]
    int parts;
};

// The context length of a sequence: what is addressable of it.
__device__ __forceinline__ int context_len(const Args &a, int seq, bool report) {
    const int raw = a.seq_lens[seq], len = raw < 0 ? 0 : min(raw, min(a.max_seq_len, a.max_blocks * a.block_size));
    if (report && raw != len) flag_error(a.err, PKV_DEVERR_SEQ_LEN);
    return len;
}

// N (2 or 4) consecutive elements of a cache row.
template <int N>
__device__ __forceinline__ void load_cached(const float *p, float (&x)[N]) {
    if constexpr (N == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        x[0] = v.x, x[1] = v.y;
    }
}

// A warp takes eight tokens at once: four lanes share a token's K row (16-byte pieces in turn) for the scores of all heads,
// and every lane owns D / 32 consecutive entries of the output.  Loads of sixteen rows are in flight; with a token at a
// time, four sequences of up to 100 tokens took 15 us instead of 6.
template <int D>
__global__ void __launch_bounds__(128) scored_simt_kernel(const SimtArgs a) {
    constexpr int NW = 4, E = D / 32, C = D / 16;  // C: 4-element pieces of a K row per lane
    __shared__ float so[NW][kGMax * D], sm[NW][kGMax], sl[NW][kGMax];
    __shared__ float4 sq[kGMax * D / 4];
    grid_dependency_wait();
    grid_launch_dependents();
    const int seq = blockIdx.x, kvh = blockIdx.y, part = blockIdx.z, G = a.group, B = a.block_size;
    const int len = context_len(a, seq, kvh == 0 && part == 0 && threadIdx.x == 0), pos = len - 1;
    const int t0 = part * kPartition, t1 = min(len, t0 + kPartition);
    if (part > 0 && t0 >= len) return;
    const KeyRange kr = key_range(key_start_of(a.s, seq), prefix_of(a.s, seq, len), a.s.window, pos, pos);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, piece = lane & 3;

    const float *qb = static_cast<const float *>(a.q) + ((int64_t)seq * a.num_heads + kvh * G) * D;
    for (int i = threadIdx.x; i < G * D; i += 128) reinterpret_cast<float *>(sq)[i] = qb[i];
    float o[kGMax][E], m[kGMax], l[kGMax], slope[kGMax];
#pragma unroll
    for (int g = 0; g < kGMax; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
        slope[g] = a.s.slopes && g < G ? a.s.slopes[kvh * G + g] : 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) o[g][j] = 0.f;
    }
    __syncthreads();
    const int32_t *bt = a.block_tables + (int64_t)seq * a.max_blocks;
    for (int base = t0 + 8 * warp; base < t1; base += 8 * NW) {
        if (!kr.meets(base, min(base + 8, t1))) continue;
        const int t = base + (lane >> 2);
        int64_t row = -1;  // of this lane's token
        if (t < t1 && kr.sees(t)) {
            const int lb = t / B, blk = bt[lb];
            if (blk >= 0 && blk < a.num_blocks) row = ((int64_t)blk * a.num_kv_heads + kvh) * B + (t - lb * B);
            else if (piece == 0) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
        }
        float kf[C][4], vf[8][E];
        if (row >= 0) {
#pragma unroll
            for (int c = 0; c < C; ++c) load_cached(static_cast<const float *>(a.k_cache) + row * D + 16 * c + 4 * piece, kf[c]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = __shfl_sync(0xffffffffu, row, 4 * i);
            if (r >= 0) {
                load_cached(static_cast<const float *>(a.v_cache) + r * D + E * lane, vf[i]);
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j) vf[i][j] = 0.f;
            }
        }
        const float away = (float)abs(pos - t);
#pragma unroll
        for (int g = 0; g < kGMax; ++g) {
            if (g >= G) break;
            float x = 0.f;
            if (row >= 0) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float4 qv = sq[(g * D + 16 * c) / 4 + piece];
                    x = fmaf(qv.x, kf[c][0], fmaf(qv.y, kf[c][1], fmaf(qv.z, kf[c][2], fmaf(qv.w, kf[c][3], x))));
                }
            }
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            x *= a.s.scale;
            if (a.s.softcap > 0.f) x = a.s.softcap * tanhf(x / a.s.softcap);
            x -= slope[g] * away;
            if (row < 0) x = -INFINITY;
            float mx = x;
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
            const float mn = fmaxf(m[g], mx);
            if (mn != m[g]) {
                const float al = expf(m[g] - mn);
                l[g] *= al;
#pragma unroll
                for (int j = 0; j < E; ++j) o[g][j] *= al;
                m[g] = mn;
            }
            const float p = x == -INFINITY ? 0.f : expf(x - mn);  // (a key that is not seen, or one whose score is -infinity)
            l[g] += p;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float w = __shfl_sync(0xffffffffu, p, 4 * i);
#pragma unroll
                for (int j = 0; j < E; ++j) o[g][j] = fmaf(w, vf[i][j], o[g][j]);
            }
        }
    }
#pragma unroll
    for (int g = 0; g < kGMax; ++g) {
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], sh);
    }
#pragma unroll
    for (int g = 0; g < kGMax; ++g) {
#pragma unroll
        for (int j = 0; j < E; ++j) so[warp][g * D + E * lane + j] = o[g][j];
        if (lane == 0) {
            sm[warp][g] = m[g];
            sl[warp][g] = l[g];
        }
    }
    __syncthreads();
    const bool whole = len <= kPartition;
    for (int i = threadIdx.x; i < G * D; i += 128) {
        const int g = i / D, d = i % D;
        float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) M = fmaxf(M, sm[k][g]);
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            if (sl[k][g] == 0.f) continue;  // a warp that saw nothing
            const float c = sm[k][g] == M ? 1.f : expf(sm[k][g] - M);
            O = fmaf(c, so[k][g * D + d], O);
            L = fmaf(c, sl[k][g], L);
        }
        const int64_t row = (int64_t)seq * a.num_heads + kvh * G + g;
        if (whole) {
            static_cast<float *>(a.out)[row * D + d] = L != 0.f ? O / L : 0.f;
        } else {
            const int64_t p = row * a.parts + part;
            a.part_o[p * D + d] = O;
            if (d == 0) {
                a.part_ml[2 * p] = M;
                a.part_ml[2 * p + 1] = L;
            }
        }
    }
}

// One warp per (sequence, head): the partitions' states, merged in order.
template <int D>
__global__ void __launch_bounds__(128) scored_reduce_kernel(const SimtArgs a) {
    constexpr int E = D / 32;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)a.num_seqs * a.num_heads) return;
    const int len = context_len(a, (int)(row / a.num_heads), false);
    if (len <= kPartition) return;
    const int n = (len + kPartition - 1) / kPartition;
    const float *ml = a.part_ml + row * a.parts * 2, *po = a.part_o + row * a.parts * D + lane;
    float M = -INFINITY, L = 0.f, o[E];
    for (int j = 0; j < n; ++j) M = fmaxf(M, ml[2 * j]);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int j = 0; j < n; ++j) {
        if (ml[2 * j + 1] == 0.f) continue;
        const float c = ml[2 * j] == M ? 1.f : expf(ml[2 * j] - M);
        L = fmaf(c, ml[2 * j + 1], L);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(c, po[(int64_t)j * D + 32 * e], o[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) static_cast<float *>(a.out)[row * D + lane + 32 * e] = L != 0.f ? o[e] / L : 0.f;
}

static size_t simt_workspace(int64_t seqs, int64_t heads, int64_t D, int64_t max_seq_len) {
    const int64_t parts = (max_seq_len + kPartition - 1) / kPartition;
    if ((double)seqs * heads * parts * (D * 4 + 8) > 4e18) return SIZE_MAX;  // (no device holds it: refused)
    return parts <= 1 ? 0 : round256((size_t)(seqs * heads * parts * D * 4)) + round256((size_t)(seqs * heads * parts * 8));
}

// What a call of a type needs.
static size_t decode_need(int64_t seqs, int heads, int head_dim, int max_seq_len, int dtype) {
    return dtype == PKV_F32 ? simt_workspace(seqs, heads, head_dim, max_seq_len) : decode_workspace(seqs, heads, head_dim);
}

static int simt_parts(const Args &a) { return std::max(1, (int)(((int64_t)a.max_seq_len + kPartition - 1) / kPartition)); }
static bool simt_fits(const Args &a) { return a.num_kv_heads <= 65535 && simt_parts(a) <= 65535; }

template <int D>
static pkv_status run_simt(const Args &args, void *workspace, cudaStream_t st) {
    SimtArgs a{};
    static_cast<Args &>(a) = args;
    a.parts = simt_parts(a);
    if (a.parts > 1) {
        a.part_o = static_cast<float *>(workspace);
        a.part_ml = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) +
                                              round256((size_t)a.num_seqs * a.num_heads * a.parts * D * 4));
    }
    const dim3 grid((unsigned)a.num_seqs, (unsigned)a.num_kv_heads, (unsigned)a.parts);
    pkv_status rc = launch_pdl(scored_simt_kernel<D>, grid, dim3(128), 0, st, a);
    if (rc == PKV_OK && a.parts > 1)
        rc = launch_pdl(scored_reduce_kernel<D>, dim3((unsigned)(((int64_t)a.num_seqs * a.num_heads + 3) / 4)), dim3(128), 0, st, a);
    return rc;
}

// max_seq_len 0: no context holds a token, and every row is zeros.
__global__ void __launch_bounds__(256) scored_zero_kernel(const Args a, int64_t chunks) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t i = i0; i < chunks; i += step) static_cast<uint4 *>(a.out)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int64_t s = i0; s < a.num_seqs; s += step) context_len(a, (int)s, true);
}

// A valid call, its new tokens stored first: nothing is stored by one that is refused.
static pkv_status decode(const Args &a, int head_dim, int dtype, const void *k_new, const void *v_new, void *workspace, size_t bytes,
                         cudaStream_t st) {
    if (!(dtype == PKV_F32 ? simt_fits(a) : decode_fits(a))) return PKV_ERR_UNSUPPORTED;
    const size_t need = a.max_seq_len > 0 ? decode_need(a.num_seqs, a.num_heads, head_dim, a.max_seq_len, dtype) : 0;
    if (need > 0 && (!workspace || bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))) return PKV_ERR_INVALID;
    if (k_new) {
        const pkv_status rc = append_new_tokens(k_new, v_new, const_cast<void *>(a.k_cache), const_cast<void *>(a.v_cache),
                                                a.block_tables, a.seq_lens, a.num_seqs, a.num_kv_heads, head_dim, a.block_size,
                                                a.max_blocks, a.num_blocks, a.max_seq_len, dtype, st);
        if (rc != PKV_OK) return rc;
    }
    if (dtype == PKV_F32) return head_dim == 128 ? run_simt<128>(a, workspace, st) : run_simt<64>(a, workspace, st);
    if (a.max_seq_len > 0) return run_decode(a, head_dim, workspace, st);
    const int64_t chunks = (int64_t)a.num_seqs * a.num_heads * head_dim / 8;
    return launch_pdl(scored_zero_kernel, dim3((unsigned)std::min<int64_t>((chunks + 255) / 256, 65536)), dim3(256), 0, st, a, chunks);
}

pkv_status check(const Args &a, int head_dim, int dtype, bool fp8, bool *empty) {
    *empty = false;
    if (a.num_seqs < 0 || a.num_q < 0 || a.num_heads < 1 || a.num_kv_heads < 1 || a.max_blocks < 1 || a.num_blocks < 1 ||
        a.max_seq_len < 0 || a.max_q_len < 0 || !std::isfinite(a.s.scale) || !std::isfinite(a.s.softcap) ||
        a.s.softcap < 0.f || a.s.window < 0)
        return PKV_ERR_INVALID;
    if (a.num_heads % a.num_kv_heads != 0) return PKV_ERR_INVALID;
    if (dtype != PKV_F32 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (a.block_size != 16 && a.block_size != 32 && (fp8 || a.block_size != 8)) return PKV_ERR_UNSUPPORTED;
    if (a.num_heads / a.num_kv_heads > kGMax) return PKV_ERR_UNSUPPORTED;
    if (a.num_seqs == 0 || a.num_q == 0) {
        *empty = true;
        return PKV_OK;
    }
    if (!a.out || !a.q || !a.k_cache || !a.v_cache || !a.block_tables || !a.seq_lens) return PKV_ERR_INVALID;
    if (!aligned16(a.out) || !aligned16(a.q) || !aligned16(a.k_cache) || !aligned16(a.v_cache)) return PKV_ERR_INVALID;
    if (fp8 && (!a.k_scales || !a.v_scales || !aligned16(a.k_scales) || !aligned16(a.v_scales))) return PKV_ERR_INVALID;
    // TMA row coordinates are 32-bit, positions too
    if (((int64_t)a.num_blocks + 1) * a.num_kv_heads * a.block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    if ((int64_t)a.max_blocks * a.block_size > INT32_MAX) return PKV_ERR_INVALID;
    return PKV_OK;
}

}  // namespace scored
}  // namespace pkv

using namespace pkv;

PKV_API size_t paged_attention_decode_scored_workspace_size(int num_seqs, int num_heads, int head_dim, int max_seq_len) {
    if (num_seqs <= 0 || num_heads <= 0 || head_dim <= 0 || max_seq_len <= 0) return 0;
    // whatever the type: the tensor-core kernel's and the CUDA-core kernel's (float32)
    return std::max(scored::decode_need(num_seqs, num_heads, head_dim, max_seq_len, PKV_F32),
                    scored::decode_need(num_seqs, num_heads, head_dim, max_seq_len, PKV_BF16));
}

PKV_API size_t paged_attention_decode_scored_workspace_size_for(int num_seqs, int num_heads, int head_dim, int max_seq_len,
                                                                int dtype) {
    if (num_seqs <= 0 || num_heads <= 0 || head_dim <= 0 || max_seq_len <= 0) return 0;
    if (dtype != PKV_F32 && dtype != PKV_BF16) return 0;
    return scored::decode_need(num_seqs, num_heads, head_dim, max_seq_len, dtype);
}

PKV_API size_t paged_attention_multi_token_scored_workspace_size(int num_q_tokens, int num_heads, int head_dim,
                                                                 int max_seq_len) {
    if (num_q_tokens <= 0 || num_heads <= 0 || head_dim <= 0 || max_seq_len <= 0) return 0;
    if (head_dim != 64 && head_dim != 128) return 0;
    return scored::rows_workspace(head_dim);
}

PKV_API pkv_status paged_attention_decode_scored(void *out, const void *q, const void *k_new, const void *v_new,
                                                 void *k_cache, void *v_cache, const int32_t *block_tables,
                                                 const int32_t *seq_lens, int num_seqs, int num_heads, int num_kv_heads,
                                                 int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                                                 int max_seq_len, float scale, float softcap, const float *alibi_slopes,
                                                 int window, const int32_t *prefix_lens, const int32_t *key_starts,
                                                 void *workspace, size_t workspace_bytes, int dtype, void *stream) {
    scored::Args a{};
    a.out = out, a.q = q, a.k_cache = k_cache, a.v_cache = v_cache;
    a.block_tables = block_tables, a.seq_lens = seq_lens;
    a.num_seqs = a.num_q = num_seqs, a.num_heads = num_heads, a.num_kv_heads = num_kv_heads;
    a.group = num_kv_heads > 0 ? num_heads / num_kv_heads : 0;
    a.block_size = block_size, a.max_blocks = max_blocks_per_seq, a.num_blocks = num_blocks, a.max_seq_len = max_seq_len;
    a.max_q_len = 1;
    a.s = ScoreArgs{scale, softcap, alibi_slopes, window, prefix_lens, key_starts};
    bool empty;
    const pkv_status rc = scored::check(a, head_dim, dtype, false, &empty);
    if (rc != PKV_OK || empty) return rc;
    if ((k_new == nullptr) != (v_new == nullptr) || !aligned16(k_new) || !aligned16(v_new)) return PKV_ERR_INVALID;
    if (k_new && max_seq_len < 1) return PKV_ERR_INVALID;  // every context holds at least its new token
    a.err = device_error_word();
    return scored::decode(a, head_dim, dtype, k_new, v_new, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

PKV_API pkv_status paged_attention_decode_scored_fp8_rows(
    void *out, const void *q, const void *k_cache, const void *v_cache, const void *k_scales, const void *v_scales,
    const int32_t *block_tables, const int32_t *seq_lens, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
    int block_size, int max_blocks_per_seq, int num_blocks, int max_seq_len, float scale, float softcap,
    const float *alibi_slopes, int window, const int32_t *prefix_lens, const int32_t *key_starts, void *workspace,
    size_t workspace_bytes, void *stream) {
    scored::Args a{};
    a.out = out, a.q = q, a.k_cache = k_cache, a.v_cache = v_cache;
    a.k_scales = static_cast<const unsigned char *>(k_scales), a.v_scales = static_cast<const unsigned char *>(v_scales);
    a.block_tables = block_tables, a.seq_lens = seq_lens;
    a.num_seqs = a.num_q = num_seqs, a.num_heads = num_heads, a.num_kv_heads = num_kv_heads;
    a.group = num_kv_heads > 0 ? num_heads / num_kv_heads : 0;
    a.block_size = block_size, a.max_blocks = max_blocks_per_seq, a.num_blocks = num_blocks, a.max_seq_len = max_seq_len;
    a.max_q_len = 1;
    a.s = ScoreArgs{scale, softcap, alibi_slopes, window, prefix_lens, key_starts};
    bool empty;
    const pkv_status rc = scored::check(a, head_dim, PKV_BF16, true, &empty);
    if (rc != PKV_OK || empty) return rc;
    a.err = device_error_word();
    return scored::decode(a, head_dim, PKV_BF16, nullptr, nullptr, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

PKV_API pkv_status paged_attention_multi_token_scored(
    void *out, const void *q, const void *k_cache, const void *v_cache, const int32_t *block_tables,
    const int32_t *seq_lens, const int32_t *q_starts, int num_seqs, int num_q_tokens, int num_heads, int num_kv_heads,
    int head_dim, int block_size, int max_blocks_per_seq, int num_blocks, int max_q_len, int max_seq_len, float scale,
    float softcap, const float *alibi_slopes, int window, const int32_t *prefix_lens, const int32_t *key_starts,
    void *workspace, size_t workspace_bytes, void *stream) {
    scored::Args a{};
    a.out = out, a.q = q, a.k_cache = k_cache, a.v_cache = v_cache;
    a.block_tables = block_tables, a.seq_lens = seq_lens, a.q_starts = q_starts;
    a.num_seqs = num_seqs, a.num_q = num_q_tokens, a.num_heads = num_heads, a.num_kv_heads = num_kv_heads;
    a.group = num_kv_heads > 0 ? num_heads / num_kv_heads : 0;
    a.block_size = block_size, a.max_blocks = max_blocks_per_seq, a.num_blocks = num_blocks, a.max_seq_len = max_seq_len;
    a.max_q_len = max_q_len;
    a.s = ScoreArgs{scale, softcap, alibi_slopes, window, prefix_lens, key_starts};
    bool empty;
    const pkv_status rc = scored::check(a, head_dim, PKV_BF16, false, &empty);
    if (rc != PKV_OK || empty) return rc;
    if (!q_starts || max_q_len < 1 || max_seq_len < 1) return PKV_ERR_INVALID;
    a.err = device_error_word();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return scored::run_rows(a, head_dim, workspace, workspace_bytes, st);
}
