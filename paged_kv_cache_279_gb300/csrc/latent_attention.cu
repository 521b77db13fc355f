// Attention over a paged cache of latent rows: arguments, workspace sizes and the
// CUDA-core kernel.
//
// A token's cache row c_t = [latent | rotated key part] serves every query head as
// its key, and its latent part as its value:
//     out = sum_t softmax_t(scale * q . c_t) latent_t
// (the absorbed form: the projections from the latent to a head's keys and values
// are folded into the query and into what reads the output).
//
// bf16 runs on the tensor cores (latent_mma.cu).
//
// latent_simt_kernel: float32.  A warp takes kRW heads of
// one query and every eighth batch of kTok tokens of a run of the context; its
// lanes hold the heads' queries, the running output and the rows of the batch in
// registers, split over the row's entries, so each row is read from memory once a
// warp in 16-byte loads and used for kRW heads.  The kRW * kTok sums over the lanes
// are formed by exchanging halves (16 shuffles for 16 sums, not 80).  Nothing is shared
// between queries: each reads its context once for every kRW heads.  Bound by
// float32 arithmetic: (2 V + 64) FMAs a head and token.  4 sequences of up to 100
// tokens, 4 heads: 8.7 us, of which four dependent loads (length, block, row, and the
// query's) are half.
#include <cmath>

#include "latent.cuh"
#include "pkv_ptx.cuh"

namespace pkv {
namespace latent {

namespace {

constexpr int kRW = 4;     // heads of a warp
constexpr int kTok = 4;    // tokens of a step
constexpr int kWarps = 8;  // of a CTA: the same heads, different tokens

constexpr int kPairRows = 64;  // a sequence's query rows above which pairs of CTAs take them (bf16)

// How the tokens of a call are split over CTAs: `parts` runs of `run` tokens.
struct Split {
    int parts, run;
};
// Parts that fill the GPU with one CTA an SM (what their registers allow).
inline int most_parts(int64_t T, int H) {
    const int64_t items = T * ((H + kRW - 1) / kRW);
    const int64_t want = items < 1 ? 1 : (152 + items - 1) / items;
    return (int)(want > 64 ? 64 : want);
}
inline Split split_of(int64_t T, int H, int max_len) {
    // no run shorter than 128 tokens: its partial results cost as much as its rows
    int64_t parts = ((int64_t)max_len + 127) / 128;
    if (parts > most_parts(T, H)) parts = most_parts(T, H);
    if (parts < 1) parts = 1;
    Split s;
    s.run = (int)(((max_len + parts - 1) / parts + 15) / 16 * 16);
    if (s.run < 16) s.run = 16;
    s.parts = (int)(((int64_t)max_len + s.run - 1) / s.run);
    if (s.parts < 1) s.parts = 1;
    return s;
}

__device__ __forceinline__ void load4(const float *p, float *x) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load2(const float *p, float *x) {
    const float2 v = *reinterpret_cast<const float2 *>(p);
    x[0] = v.x, x[1] = v.y;
}

// Entry e of a lane's share of a row: lanes hold runs of 4 entries, 128 apart.
__device__ __forceinline__ int entry(int lane, int e) { return (e >> 2) * 128 + 4 * lane + (e & 3); }

// Partial results of one (query row, part): V sums, then the maximum (base 2) and
// the sum of weights.
__host__ __device__ inline int64_t partial_floats(int V) { return V + 4; }

// The sequence that query row `tok` belongs to: the last with q_starts[s] <= tok.
__device__ __forceinline__ int sequence_of(const Args &a, int tok) {
    if (!a.q_starts) return tok;
    int lo = 0, hi = a.S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.q_starts[mid] <= tok) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <int V>
__global__ void __launch_bounds__(kWarps * 32) latent_simt_kernel(const __grid_constant__ Args a, Split sp) {
    constexpr int NV = V / 32;       // entries of the latent part a lane holds
    constexpr int D = V + kRope;
    __shared__ float sh_o[kWarps][V];
    __shared__ float sh_m[kWarps], sh_l[kWarps];
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hg = (a.H + kRW - 1) / kRW;
    const int tok = blockIdx.x / hg, h0 = (blockIdx.x - tok * hg) * kRW, part = blockIdx.y;
    const int nh = min(kRW, a.H - h0);
    if (part == 0 && threadIdx.x == 0)
        for (int64_t k = blockIdx.x; k < a.S; k += gridDim.x)
            if (sequence(a, (int)k).flagged) flag_error(a.err, PKV_DEVERR_SEQ_LEN);
    const int s = sequence_of(a, tok);
    const Seq sq = sequence(a, s);
    const int i = tok - sq.q0;
    if (i < 0 || i >= sq.n) return;
    const int end = max(0, min(sq.L - sq.n0 + i + 1, sq.L));  // tokens this query sees
    const int t0 = part * sp.run, t1 = min(end, t0 + sp.run);
    if (t0 >= end && part > 0) return;  // parts past the end are not merged either

    float q[kRW][NV + 2], o[kRW][NV], m[kRW], l[kRW];
    const float *qb = (const float *)a.q + ((int64_t)tok * a.H + h0) * D;
#pragma unroll
    for (int r = 0; r < kRW; ++r) {
        const float *qr = qb + (int64_t)(r < nh ? r : 0) * D;
#pragma unroll
        for (int j = 0; j < NV / 4; ++j) load4(qr + j * 128 + 4 * lane, &q[r][4 * j]);
        load2(qr + V + 2 * lane, &q[r][NV]);
#pragma unroll
        for (int e = 0; e < NV + 2; ++e) q[r][e] *= a.scale_log2;
#pragma unroll
        for (int e = 0; e < NV; ++e) o[r][e] = 0.f;
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
    const int32_t *table = a.tables + (int64_t)s * a.maxb;
    const float *cache = (const float *)a.cache;
    for (int t = t0 + warp * kTok; t < t1; t += kWarps * kTok) {
        float c[kTok][NV + 2];
        bool ok[kTok];
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            ok[k] = t + k < t1;
            int64_t row = 0;
            if (ok[k]) {
                const int blk = table[(t + k) >> a.bshift];
                if ((unsigned)blk >= (unsigned)a.NB) {
                    ok[k] = false;
                    if (lane == 0) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                } else {
                    row = ((int64_t)blk << a.bshift) + ((t + k) & (a.B - 1));
                }
            }
#pragma unroll
            for (int e = 0; e < NV + 2; ++e) c[k][e] = 0.f;
            if (ok[k]) {
                const float *cr = cache + row * D;
#pragma unroll
                for (int j = 0; j < NV / 4; ++j) load4(cr + j * 128 + 4 * lane, &c[k][4 * j]);
                load2(cr + V + 2 * lane, &c[k][NV]);
            }
        }
        // 16 sums over the lanes, by halves: after the step over lane bit 4, 3, 2, 1
        // a lane holds 8, 4, 2, 1 of them; the last step completes it
        float v[kRW * kTok];
#pragma unroll
        for (int r = 0; r < kRW; ++r)
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                float x = 0.f;
#pragma unroll
                for (int e = 0; e < NV + 2; ++e) x = fmaf(q[r][e], c[k][e], x);
                v[r * kTok + k] = x;
            }
#pragma unroll
        for (int w = 8, bit = 16; w >= 1; w >>= 1, bit >>= 1) {
            const bool up = lane & bit;
#pragma unroll
            for (int j = 0; j < w; ++j) {
                const float keep = up ? v[j + w] : v[j], give = up ? v[j] : v[j + w];
                v[j] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
            }
        }
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
        // the sum of (r, k) lies in lanes 2 (4 r + k) and the next
#pragma unroll
        for (int r = 0; r < kRW; ++r) {
            float x[kTok], top = m[r];
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                x[k] = __shfl_sync(0xffffffffu, v[0], 2 * (r * kTok + k));
                if (!ok[k]) x[k] = -INFINITY;
                top = fmaxf(top, x[k]);
            }
            const float ref = top == -INFINITY ? 0.f : top;
            const float f = exp2f(m[r] - ref);
            m[r] = top;
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                x[k] = exp2f(x[k] - ref);
                sum += x[k];
            }
            l[r] = l[r] * f + sum;
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                float y = o[r][e] * f;
#pragma unroll
                for (int k = 0; k < kTok; ++k) y = fmaf(x[k], c[k][e], y);
                o[r][e] = y;
            }
        }
    }
    // join the warps, head by head
    const bool final = sp.parts == 1 || end <= sp.run;
    for (int r = 0; r < nh; ++r) {
        float lr = 0.f, mr = -INFINITY;
#pragma unroll
        for (int rr = 0; rr < kRW; ++rr)
            if (rr == r) {
                lr = l[rr], mr = m[rr];
#pragma unroll
                for (int e = 0; e < NV; ++e) sh_o[warp][entry(lane, e)] = o[rr][e];
            }
        if (lane == 0) sh_m[warp] = mr, sh_l[warp] = lr;
        __syncthreads();
        float top = -INFINITY, f[kWarps], sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh_m[w]);
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            f[w] = exp2f(sh_m[w] - ref);
            sum += sh_l[w] * f[w];
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t orow = (int64_t)tok * a.H + h0 + r;
        float *pr = (float *)a.ws + (orow * sp.parts + part) * partial_floats(V);
        for (int e = threadIdx.x; e < V; e += kWarps * 32) {
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) x += sh_o[w][e] * f[w];
            // a query that sees nothing has sum 0 and gets zeros
            if (final) ((float *)a.out)[orow * V + e] = sum == 0.f ? 0.f : x * inv;
            else pr[e] = x;
        }
        if (!final && threadIdx.x == 0) pr[V] = top, pr[V + 1] = sum;
        __syncthreads();
    }
}

// One CTA a (query, head): the parts of its context, in order.
__global__ void __launch_bounds__(128) latent_join_kernel(const __grid_constant__ Args a, Split sp) {
    grid_dependency_wait();
    const int tok = blockIdx.x / a.H;
    const int s = sequence_of(a, tok);
    const Seq sq = sequence(a, s);
    const int i = tok - sq.q0;
    if (i < 0 || i >= sq.n) return;
    const int end = max(0, min(sq.L - sq.n0 + i + 1, sq.L));
    if (end <= sp.run) return;  // one part: stored by the first kernel
    const int parts = (end + sp.run - 1) / sp.run;
    const float *p = (const float *)a.ws + (int64_t)blockIdx.x * sp.parts * partial_floats(a.V);
    float top = -INFINITY;
    for (int k = 0; k < parts; ++k) top = fmaxf(top, p[k * partial_floats(a.V) + a.V]);
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int k = 0; k < parts; ++k) sum += p[k * partial_floats(a.V) + a.V + 1] * exp2f(p[k * partial_floats(a.V) + a.V] - ref);
    for (int e = threadIdx.x; e < a.V; e += 128) {
        float x = 0.f;
        for (int k = 0; k < parts; ++k) x += p[k * partial_floats(a.V) + e] * exp2f(p[k * partial_floats(a.V) + a.V] - ref);
        ((float *)a.out)[(int64_t)blockIdx.x * a.V + e] = sum == 0.f ? 0.f : x / sum;
    }
}

// Grows with the longest context in one step, from nothing: a call may bound that by its block tables.
size_t simt_workspace(int64_t T, int H, int V, int max_len) {
    const int parts = most_parts(T, H);
    return parts == 1 || max_len <= 128 ? 0 : round256((size_t)T * H * parts * partial_floats(V) * sizeof(float));
}

// Zeros for every query, and the flags of bad lengths and starts: nothing is in sight.
__global__ void __launch_bounds__(256) latent_zero_kernel(const __grid_constant__ Args a) {
    grid_dependency_wait();
    for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
        const Seq q = sequence(a, s);
        if (q.flagged && threadIdx.x == 0) flag_error(a.err, PKV_DEVERR_SEQ_LEN);
        uint4 *o = reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.out + (int64_t)q.q0 * a.H * a.V);
        for (int64_t i = threadIdx.x; i < (int64_t)q.n * a.H * a.V / 8; i += 256) o[i] = make_uint4(0, 0, 0, 0);
    }
}

pkv_status run_simt(const Args &a, cudaStream_t st) {
    const Split sp = split_of(a.T, a.H, a.max_len);
    const int64_t items = (int64_t)a.T * ((a.H + kRW - 1) / kRW);
    const dim3 grid((unsigned)items, (unsigned)sp.parts);
    const pkv_status rc = a.V == 512 ? launch_pdl(latent_simt_kernel<512>, grid, dim3(kWarps * 32), 0, st, a, sp)
                                     : launch_pdl(latent_simt_kernel<256>, grid, dim3(kWarps * 32), 0, st, a, sp);
    if (rc != PKV_OK || sp.parts == 1) return rc;
    return launch_pdl(latent_join_kernel, dim3((unsigned)(a.T * a.H)), dim3(128), 0, st, a, sp);
}

size_t workspace(int64_t T, int H, int V, int max_len, int dtype) {
    if (max_len < 1) return 0;
    if (dtype == PKV_F32) return simt_workspace(T, H, V, max_len);
    const size_t one = mma_workspace(T, H, V), two = T * H > kPairRows ? pair_workspace(V) : 0;
    return one > two ? one : two;
}

bool known_shape(int H, int V) { return H >= 1 && H <= 128 && (V == 256 || V == 512); }

pkv_status run(Args &a, float scale, size_t ws_bytes, int dtype, void *stream) {
    if (a.S < 0 || a.T < 0 || a.H < 1 || a.V < 1 || a.B < 1 || a.maxb < 1 || a.NB < 1 || a.max_len < 0 || a.max_q < 1)
        return PKV_ERR_INVALID;
    a.scale_log2 = scale * 1.4426950408889634f;
    if (!std::isfinite(a.scale_log2)) return PKV_ERR_INVALID;
    if (dtype != PKV_F32 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (!known_shape(a.H, a.V)) return PKV_ERR_UNSUPPORTED;
    if (a.B != 8 && a.B != 16 && a.B != 32 && a.B != 64) return PKV_ERR_UNSUPPORTED;
    if (a.S == 0 || a.T == 0) return PKV_OK;
    // positions, cache rows, query rows and sequences of 31 bits, with room for a tile (or the sequences of a block's threads)
    // past the last
    if ((int64_t)a.maxb * a.B > 0x7ffff000ll) return PKV_ERR_INVALID;
    if ((int64_t)a.NB * a.B > 0x7fffffffll) return PKV_ERR_UNSUPPORTED;
    if ((int64_t)a.T * a.H > 0x7ffff000ll || a.S > 0x7ffff000) return PKV_ERR_UNSUPPORTED;
    if (!a.out || !a.q || !a.cache || !a.tables || !a.lens) return PKV_ERR_INVALID;
    if (!aligned16(a.out) || !aligned16(a.q) || !aligned16(a.cache)) return PKV_ERR_INVALID;
    a.max_len = (int)((int64_t)a.max_len < (int64_t)a.maxb * a.B ? a.max_len : (int64_t)a.maxb * a.B);
    a.rows = (a.q_starts ? (a.max_q < a.T ? a.max_q : a.T) : 1) * a.H;
    a.bshift = a.B == 8 ? 3 : a.B == 16 ? 4 : a.B == 32 ? 5 : 6;
    int l = 0;
    while (1 << l < a.H) ++l;
    a.hshift = 31 + l;
    a.hmul = (uint32_t)(((1ull << a.hshift) / (unsigned)a.H) + 1);
    a.err = device_error_word();
    const size_t need = workspace(a.T, a.H, a.V, a.max_len, dtype);
    if (need && (!a.ws || (reinterpret_cast<uintptr_t>(a.ws) & 255u) || ws_bytes < need)) return PKV_ERR_INVALID;
    if (dtype == PKV_F32) return run_simt(a, (cudaStream_t)stream);
    if (a.max_len == 0) {  // contexts without a token
        const unsigned grid = a.S < 1024 ? (unsigned)a.S : 1024u;
        return launch_pdl(latent_zero_kernel, dim3(grid), dim3(256), 0, (cudaStream_t)stream, a);
    }
    return a.rows > kPairRows ? run_pair(a, (cudaStream_t)stream) : run_mma(a, (cudaStream_t)stream);
}

}  // namespace

}  // namespace latent
}  // namespace pkv

using namespace pkv;

PKV_API size_t paged_latent_attention_workspace_size(int num_q_tokens, int num_heads, int latent_dim, int max_seq_len, int dtype) {
    if (num_q_tokens < 1 || max_seq_len < 1 || !latent::known_shape(num_heads, latent_dim)) return 0;
    if (dtype != PKV_F32 && dtype != PKV_BF16) return 0;
    return latent::workspace(num_q_tokens, num_heads, latent_dim, max_seq_len, dtype);
}

PKV_API pkv_status paged_latent_attention_decode(void *out, const void *q, const void *cache, const int32_t *block_tables,
                                                 const int32_t *seq_lens, int num_seqs, int num_heads, int latent_dim,
                                                 int block_size, int max_blocks_per_seq, int num_blocks, int max_seq_len,
                                                 float scale, void *workspace, size_t workspace_bytes, int dtype,
                                                 void *stream) {
    latent::Args a{};
    a.out = out, a.q = q, a.cache = cache, a.tables = block_tables, a.lens = seq_lens;
    a.S = a.T = num_seqs, a.H = num_heads, a.V = latent_dim, a.B = block_size, a.maxb = max_blocks_per_seq, a.NB = num_blocks;
    a.max_q = 1, a.max_len = max_seq_len;
    a.ws = (unsigned char *)workspace;
    return latent::run(a, scale, workspace_bytes, dtype, stream);
}

PKV_API pkv_status paged_latent_attention_multi_token(void *out, const void *q, const void *cache, const int32_t *block_tables,
                                                      const int32_t *seq_lens, const int32_t *q_starts, int num_seqs,
                                                      int num_q_tokens, int num_heads, int latent_dim, int block_size,
                                                      int max_blocks_per_seq, int num_blocks, int max_q_len, int max_seq_len,
                                                      float scale, void *workspace, size_t workspace_bytes, int dtype,
                                                      void *stream) {
    if (num_seqs > 0 && num_q_tokens > 0 && !q_starts) return PKV_ERR_INVALID;
    latent::Args a{};
    a.out = out, a.q = q, a.cache = cache, a.tables = block_tables, a.lens = seq_lens, a.q_starts = q_starts;
    a.S = num_seqs, a.T = num_q_tokens, a.H = num_heads, a.V = latent_dim, a.B = block_size, a.maxb = max_blocks_per_seq;
    a.NB = num_blocks, a.max_q = max_q_len, a.max_len = max_seq_len;
    a.ws = (unsigned char *)workspace;
    return latent::run(a, scale, workspace_bytes, dtype, stream);
}
