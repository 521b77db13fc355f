// Scored decode attention (one query per sequence) over bf16 and row-scaled FP8
// caches.  Bound by HBM: 16 tokens x <= 8 query heads x head_dim per KV head is
// G flop a byte, a few percent of even the legacy tensor path, so the
// contractions run on mma.sync and the work is to stream the cache.
//
// All (sequence, KV head) segments are laid end to end as one list of tiles (16
// tokens, FP8: 32), only those that the query sees: the tiles of the always
// visible prefix, then those from the window's or document's start.  Each
// segment stands behind kLead empty tiles, a charge for its fixed costs, and
// every warp of a grid that fills the machine takes an equal share of the list.
// A warp streams its tiles through its own ring of TMA boxes, so no warp waits
// for another; block ids are resolved 32 tiles at a time, one per lane, ahead of
// the stream.  A segment cut by a share's border leaves partial states (o, m,
// l), one per warp, which a second kernel merges.
//
//     S^T = K Q^T  (tokens x heads, m16n8k16)      x = cap and bias of S, base 2
//     O^T += V^T P^T, P = 2^(x - m)                running m, l per head
// Row-scaled FP8: codes widen to f16 (exact); the first product is taken heads x
// tokens, so that the weights come out in the layout the second one takes and a
// lane deals with one head.  (E4M3 operands of mma.sync, the query as a sum of
// two, were no faster: 920 instructions a tile against 720.)  A key's scale 2^ke
// multiplies its scores.  A value's scale 2^ve goes into the weight, w = 2^(x +
// ve - m + 14) with m the maximum of x + ve, so that w <= 2^14 uses f16's range
// whatever the scales are; l sums w 2^-ve, and out = o / l as before.  Scales below
// 2^-80 (zero rows: 2^-100) count as that in m: an addend of l is then at most 2^94,
// and no number of keys takes l out of float32's range.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "mma_sync.cuh"
#include "pkv_internal.cuh"
#include "scored.cuh"

namespace pkv {
namespace scored {
namespace {

constexpr int kNW = 4, kNS = 2;   // warps per CTA, ring stages per warp
constexpr int kMaxWarps = 2048;   // partial slots in the workspace: two per warp
constexpr int kMaxSeqs = 8192;    // of a launch: their tiles' table is in shared memory

template <int D, bool F8>
struct Tile {
    static constexpr int kTok = F8 ? 32 : 16;
    static constexpr int kLead = F8 ? 2 : 3;  // empty tiles in front of a segment
    static constexpr int kMinShare = F8 ? 8 : 16;  // tiles (256 tokens), less where every segment is shorter
    static constexpr int kKV = kTok * D * (F8 ? 1 : 2);
    static constexpr int kStage = 2 * kKV;
    static constexpr int kScales = F8 ? 2 * kTok : 0;  // per stage: K scales, V scales
};

struct DecodeArgs : Args {
    float k1;        // no cap: scale * log2 e; cap: 2 * scale / softcap * log2 e (the exponent of e^2z)
    float c2;        // softcap * log2 e, 0: no cap
    float *part_o;   // [2 warps][G][D]
    float *part_ml;  // [2 warps][G][2]
    int2 *segs;      // [S * Hkv]: (first warp, parts); parts 0: nothing to merge, -1: no key seen
    int bshift;
};

template <int D, bool F8>
struct Smem {
    int ring, scales, bars, prefix, total;
    __host__ __device__ explicit Smem(int num_seqs) {
        ring = 0;
        scales = kNW * kNS * Tile<D, F8>::kStage;
        bars = scales + kNW * kNS * Tile<D, F8>::kScales;
        prefix = bars + kNW * kNS * 8;
        total = prefix + (num_seqs + 1) * 4 + 1024;  // + alignment slack
    }
};

// What a segment's tiles are: context tile i is key tile pt0 + i (i < np), else mt0 + i - np.
struct SegTiles {
    KeyRange r;
    int len, pt0, np, mt0, n;
};

template <int TT>
__device__ __forceinline__ SegTiles seg_tiles(const DecodeArgs &a, int s, int raw, int pre, int ks) {
    const int cap = min(a.max_seq_len, a.max_blocks << a.bshift);
    SegTiles x;
    x.len = raw < 0 ? 0 : min(raw, cap);
    x.r = key_range(max(0, ks), min(max(0, pre), x.len), a.s.window, x.len - 1, x.len - 1);
    x.mt0 = x.r.lo / TT;
    const int nm = x.r.hi > x.r.lo ? (x.r.hi + TT - 1) / TT - x.mt0 : 0;
    x.pt0 = x.r.first / TT;
    int pe = x.r.pre > x.r.first ? (x.r.pre + TT - 1) / TT : x.pt0;
    if (nm > 0) pe = min(pe, x.mt0);
    x.np = max(0, pe - x.pt0);
    x.n = x.np + nm;
    return x;
}
template <int TT>
__device__ __forceinline__ SegTiles load_seg(const DecodeArgs &a, int s) {
    const int raw = a.seq_lens[s];
    const int pre = a.s.prefix_lens ? a.s.prefix_lens[s] : 0, ks = a.s.key_starts ? a.s.key_starts[s] : 0;
    return seg_tiles<TT>(a, s, raw, pre, ks);
}

constexpr float kLeastExp = -80.f;  // of a value's scale in a row-scaled reference

// l 2^d, d <= 0, also where 2^d is below float32's range (l: up to 2^125, where V rows of the least scale came first).
__device__ __forceinline__ float lower_sum(float l, float d) {
    return l * ex2_approx(fmaxf(d, -100.f)) * ex2_approx(fminf(d + 100.f, 0.f));
}

__device__ __forceinline__ uint32_t range_bits(int a, int b) {  // bits [a, b) of 32, any integers
    a = max(a, 0);
    b = min(b, 32);
    return a >= b ? 0u : (b == 32 ? 0xffffffffu : (1u << b) - 1u) & ~((1u << a) - 1u);
}

// One tile as a lane holds it ahead of the stream.
struct Slot {
    int y0, y1;     // cache rows of its (up to two) boxes, -1: none
    uint32_t mask;  // tokens that are seen
    int t0;         // first token
};

// Running state of a warp: O of heads 2tq and 2tq + 1, sixteen head_dim rows per
// fragment (which ones: see entry()); m and l of the same heads (bf16) or of head
// g (FP8, in [0]).
template <int D>
struct Acc {
    float m[2], l[2];
    float o[D / 16][4];
    __device__ __forceinline__ void reset() {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
    __device__ __forceinline__ void scale(float a0, float a1) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            o[i][0] *= a0;
            o[i][1] *= a1;
            o[i][2] *= a0;
            o[i][3] *= a1;
        }
    }
};

// The queries as MMA operand, and what their scores need: of heads 2tq, 2tq + 1
// (bf16) or of head g (FP8, in [0]).
template <int D>
struct Query {
    uint32_t b[D / 16][2];
    float f[2];             // factor of the raw products
    float slope[2];         // slope * log2 e
};

template <int D, bool F8>
__device__ __forceinline__ void load_query(const DecodeArgs &a, int seq, int kvh, int lane, Query<D> &q) {
    const int g = lane >> 2, t = lane & 3, h0 = kvh * a.group;
    const __nv_bfloat16 *row = static_cast<const __nv_bfloat16 *>(a.q) + ((int64_t)seq * a.num_heads + h0 + g) * D;
    q.f[0] = q.f[1] = a.k1;
    if constexpr (!F8) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            q.b[k][0] = g < a.group ? *reinterpret_cast<const uint32_t *>(row + 16 * k + 2 * t) : 0u;
            q.b[k][1] = g < a.group ? *reinterpret_cast<const uint32_t *>(row + 16 * k + 8 + 2 * t) : 0u;
        }
    } else {
        // entries 16c + 4t .. + 3, the order in which the keys' codes come; times a power of two that takes the head's largest
        // |q| into [2^14, 2^15) (exact: 8 significant bits)
        uint2 w[D / 16];
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            w[c] = g < a.group ? *reinterpret_cast<const uint2 *>(row + 16 * c + 4 * t) : make_uint2(0u, 0u);
            amax = fmaxf(amax, fmaxf(fmaxf(fabsf(bf16x2_lo(w[c].x)), fabsf(bf16x2_hi(w[c].x))),
                                     fmaxf(fabsf(bf16x2_lo(w[c].y)), fabsf(bf16x2_hi(w[c].y)))));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int fe = min(253, max(1, 268 - (int)((__float_as_uint(amax) >> 23) & 0xffu)));
        const float f = __uint_as_float((uint32_t)fe << 23);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            q.b[c][0] = pack_f16x2(bf16x2_lo(w[c].x) * f, bf16x2_hi(w[c].x) * f);
            q.b[c][1] = pack_f16x2(bf16x2_lo(w[c].y) * f, bf16x2_hi(w[c].y) * f);
        }
        q.f[0] *= __uint_as_float((uint32_t)(254 - fe) << 23);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int h = F8 ? g : 2 * t + j;
        q.slope[j] = a.s.slopes && h < a.group && (!F8 || j == 0) ? a.s.slopes[h0 + h] * 1.44269504f : 0.f;
    }
}

// c tanh z, y = 2 z log2 e: c - 2 c / (1 + e^2z), good to 2^-21 of c.
__device__ __forceinline__ float cap_score(float y, float c2) {
    return c2 - 2.f * c2 * rcp_approx(1.f + ex2_approx(y));
}
// The same with the series for small z.
__device__ __noinline__ float cap_score_wide(float y, float c2) {
    const float z = y * 0.34657359f, u = z * z;
    constexpr float s1 = (float)kTanhSeries[1], s2 = (float)kTanhSeries[2], s3 = (float)kTanhSeries[3];
    return fabsf(z) < kTanhSmall ? c2 * (z * fmaf(fmaf(fmaf(s3, u, s2), u, s1), u, 1.f)) : cap_score(y, c2);
}

// Raw product -> score in base 2: `f` the head's factor, away = p - t.
__device__ __forceinline__ float score(float s, float f, float c2, float slope, float away) {
    float x = s * f;
    if (c2 > 0.f) x = c2 > kWideCap ? cap_score_wide(x, c2) : cap_score(x, c2);
    return fmaf(-slope, away, x);
}

// New maxima of both heads over a tile's scores (N values of each head in every
// lane of its column); the state moves to them.  Returns the references.
template <int D, int N>
__device__ __forceinline__ void move_to(Acc<D> &acc, const float (&x)[N][2], float (&ref)[2]) {
    float mx[2] = {x[0][0], x[0][1]};
#pragma unroll
    for (int i = 1; i < N; ++i) {
        mx[0] = fmaxf(mx[0], x[i][0]);
        mx[1] = fmaxf(mx[1], x[i][1]);
    }
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) {
        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], sh));
        mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], sh));
    }
    const float n0 = fmaxf(acc.m[0], mx[0]), n1 = fmaxf(acc.m[1], mx[1]);
    ref[0] = n0 == -INFINITY ? 0.f : n0;
    ref[1] = n1 == -INFINITY ? 0.f : n1;
    // the maxima rarely move once a few tiles are in
    if (__any_sync(0xffffffffu, n0 != acc.m[0] || n1 != acc.m[1])) {
        const float a0 = ex2_approx(acc.m[0] - ref[0]), a1 = ex2_approx(acc.m[1] - ref[1]);
        acc.l[0] *= a0;
        acc.l[1] *= a1;
        acc.scale(a0, a1);
    }
    acc.m[0] = n0;
    acc.m[1] = n1;
}

// One bf16 tile: K at sk, V at sv, 128-byte swizzled halves [half][16 rows].
template <int D>
__device__ __forceinline__ void attend_bf16(const DecodeArgs &a, unsigned char *sk, unsigned char *sv, const Slot &t, int pos,
                                            const Query<D> &q, Acc<D> &acc, int lane) {
    constexpr int kHalf = 16 * 128;
    const uint32_t ok = t.mask;
    if (ok != 0xffffu) {  // tokens that are not seen may hold anything: a zero weight must meet a zero
#pragma unroll 1
        for (int e = lane; e < D / 64 * 16 * 8; e += 32) {
            const int r = (e >> 3) & 15;
            if (!((ok >> r) & 1u)) *reinterpret_cast<uint4 *>(sv + (e >> 7) * kHalf + r * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
    }
    const int r0 = lane >> 2, lj = lane >> 3, lr = lane & 7;
    const int ktok = lr + 8 * (lj & 1), vtok = lr + 8 * (lj >> 1);
    const uint32_t krow = smem_u32(sk) + ktok * 128, vrow = smem_u32(sv) + vtok * 128;
    float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        uint32_t x0, x1, x2, x3;
        ldmatrix_x4(krow + (k >> 2) * kHalf + (((2 * (k & 3) + (lj >> 1)) ^ lr) << 4), x0, x1, x2, x3);
        mma_bf16_16816(sc, x0, x1, x2, x3, q.b[k][0], q.b[k][1]);
    }
    float x[2][2], ref[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int tok = r0 + 8 * i;
        const bool seen = (ok >> tok) & 1u;
        const float away = (float)(pos - t.t0 - tok);  // p >= t: no key past the query's position
#pragma unroll
        for (int j = 0; j < 2; ++j) x[i][j] = seen ? score(sc[2 * i + j], q.f[j], a.c2, q.slope[j], away) : -INFINITY;
    }
    move_to<D>(acc, x, ref);
    // the sums use the same rounded weights as the numerator
    const uint32_t p0 = pack_bf16x2(ex2_approx(x[0][0] - ref[0]), ex2_approx(x[0][1] - ref[1]));
    const uint32_t p1 = pack_bf16x2(ex2_approx(x[1][0] - ref[0]), ex2_approx(x[1][1] - ref[1]));
    acc.l[0] += bf16x2_lo(p0) + bf16x2_lo(p1);
    acc.l[1] += bf16x2_hi(p0) + bf16x2_hi(p1);
    const uint32_t b0 = movmatrix_trans(p0), b1 = movmatrix_trans(p1);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        uint32_t x0, x1, x2, x3;
        ldmatrix_x4_trans(vrow + (i >> 2) * kHalf + (((2 * (i & 3) + (lj & 1)) ^ lr) << 4), x0, x1, x2, x3);
        mma_bf16_16816(acc.o[i], x0, x1, x2, x3, b0, b1);
    }
}

// 16-byte chunk c of row r of a code tile (128-byte rows: 128-byte swizzle; 64-byte rows: 64-byte swizzle).
template <int D>
__device__ __forceinline__ uint32_t code_chunk(int r, int c) {
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// One FP8 tile: codes of 32 tokens, K at sk, V at sv; scale bytes at ss (K, then V).
template <int D>
__device__ __forceinline__ void attend_fp8(const DecodeArgs &a, unsigned char *sk, unsigned char *sv, const unsigned char *ss,
                                           const Slot &t, int pos, const Query<D> &q, Acc<D> &acc, int lane) {
    const uint32_t ok = t.mask;
    if (ok != 0xffffffffu) {
#pragma unroll 1
        for (int e = lane; e < 32 * D / 16; e += 32) {
            const int r = e / (D / 16);
            if (!((ok >> r) & 1u)) *reinterpret_cast<uint4 *>(sv + r * D + (e % (D / 16)) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
    }
    const int g = lane >> 2, tq = lane & 3, lr = lane & 7;
    const uint32_t ska = smem_u32(sk), sva = smem_u32(sv);
    const bool full = ok == 0xffffffffu;
    // 16 tokens at a time: all 32 at once (720 instructions) were slower where pieces are short (64 sequences: 36 us, so 35)
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        // S (heads x tokens): row g head g, columns 2tq, 2tq + 1 of eight tokens each
        float sc[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; k += 4) {  // four 16-byte chunks of eight token rows at once
                uint32_t x[4];
                ldmatrix_x4(ska + code_chunk<D>(16 * h + 8 * n + lr, k + (lane >> 3)), x[0], x[1], x[2], x[3]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t b0, b1;
                    e4m3x4_to_f16(x[c], b0, b1);
                    mma_f16_8816(sc[n], q.b[k + c][0], q.b[k + c][1], b0, b1);
                }
            }
        }
        // head g, tokens 8n + 2tq + i: scores xs, and x with the value's exponent
        const float b0 = -q.slope[0] * (float)(pos - t.t0 - 16 * h - 2 * tq);  // p >= t: no key past the query's position
        const uint32_t okh = ok >> (16 * h);
        float x[2][2], xs[2][2], mx = -INFINITY;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const uint32_t kb = *reinterpret_cast<const uint16_t *>(ss + 16 * h + 8 * n + 2 * tq);
            const uint32_t vb = *reinterpret_cast<const uint16_t *>(ss + 32 + 16 * h + 8 * n + 2 * tq);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float kf = __uint_as_float(i ? (kb & 0xff00u) << 15 : (kb & 0xffu) << 23);
                const float ve = __uint_as_float(0x4b000000u | (i ? vb >> 8 : vb & 0xffu)) - 8388735.f;  // 2^23 + byte, less 2^23 + 127
                float s = sc[n][i] * (q.f[0] * kf);
                if (a.c2 > 0.f) s = a.c2 > kWideCap ? cap_score_wide(s, a.c2) : cap_score(s, a.c2);
                if (a.s.slopes) s += fmaf(q.slope[0], (float)(8 * n + i), b0);
                if (!full && !((okh >> (8 * n + 2 * tq + i)) & 1u)) s = -INFINITY;
                xs[n][i] = s;
                x[n][i] = s + ve;
                if (!full && s == -INFINITY) x[n][i] = -INFINITY;  // the scale of a token that is not seen may be anything
                mx = fmaxf(mx, s + fmaxf(ve, kLeastExp));
            }
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float top = fmaxf(acc.m[0], mx), ref = top == -INFINITY ? 0.f : top;
        if (__any_sync(0xffffffffu, top != acc.m[0])) {
            const float f = ex2_approx(acc.m[0] - ref);
            acc.l[0] = lower_sum(acc.l[0], acc.m[0] - ref);
            acc.scale(__shfl_sync(0xffffffffu, f, 8 * tq), __shfl_sync(0xffffffffu, f, 8 * tq + 4));
        }
        acc.m[0] = top;
        const float up = 14.f - ref;  // weights up to 2^14
        uint32_t p[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            p[n] = pack_f16x2(ex2_approx(x[n][0] + up), ex2_approx(x[n][1] + up));
            acc.l[0] += ex2_approx(xs[n][0] + up) + ex2_approx(xs[n][1] + up);  // w 2^-ve
        }
        // V^T fragments from token rows: lane (g, tq) reads D / 8 consecutive entries of tokens 2tq, 2tq + 1, 2tq + 8, 2tq + 9
        // and pairs two tokens' bytes; fragment i holds entries D/8 g + 2i (rows g) and + 1 (rows g + 8)
        constexpr int W = D / 32;  // 32-bit words of a lane's entries
        uint32_t v[4][W];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int tok = 16 * h + 2 * tq + (r & 1) + 8 * (r >> 1);
            if constexpr (D == 128) {
                const float4 c = lds128(sva + code_chunk<D>(tok, g));
                v[r][0] = __float_as_uint(c.x), v[r][1] = __float_as_uint(c.y);
                v[r][2] = __float_as_uint(c.z), v[r][3] = __float_as_uint(c.w);
            } else {
                const uint32_t at = sva + code_chunk<D>(tok, g >> 1) + (g & 1) * 8;
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[r][0]), "=r"(v[r][1]) : "r"(at));
            }
        }
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int u = 0; u < 2; ++u) {  // entries 4w + 2u, 4w + 2u + 1
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16(__byte_perm(v[0][w], v[1][w], u ? 0x7362 : 0x5140), a0, a1);
                e4m3x4_to_f16(__byte_perm(v[2][w], v[3][w], u ? 0x7362 : 0x5140), a2, a3);
                mma_f16_16816(acc.o[2 * w + u], a0, a1, a2, a3, p[0], p[1]);
            }
    }
}

__device__ __forceinline__ bool wait_tile(uint64_t *bar, uint32_t parity) {
    uint32_t i = 0;
#pragma unroll 1
    while (!mbar_try_wait(bar, parity))
        if (++i == kWaitLimit) return false;
    return true;
}

// head_dim entry of acc.o[i][j] (rows g for j < 2, g + 8 above)
template <int D, bool F8>
__device__ __forceinline__ int entry(int i, int g, int j) {
    return F8 ? D / 8 * g + 2 * i + (j >> 1) : 16 * i + g + 8 * (j >> 1);
}

template <int D, bool F8>
__global__ void __launch_bounds__(kNW * 32, 3)
scored_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ DecodeArgs a) {
    using T_ = Tile<D, F8>;
    constexpr int TT = T_::kTok;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const Smem<D, F8> L(a.num_seqs);
    int *prefix = reinterpret_cast<int *>(smem + L.prefix);
    __shared__ int warp_sums[kNW], carry, seg_max;
    grid_launch_dependents();
    const int S = a.num_seqs, Hkv = a.num_kv_heads, B = a.block_size;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // Laid-out tiles before each sequence.  This reads lengths, prefixes and starts only, which no kernel of the library
    // writes, so it may run under the previous kernel's tail; so may the block ids' loads below.
    if (threadIdx.x == 0) {
        prefix[0] = carry = seg_max = 0;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
    }
    __syncthreads();
    int my_max = 0;
#pragma unroll 1
    for (int base = 0; base < S; base += kNW * 32) {
        const int s = base + threadIdx.x;
        int v = 0;
        if (s < S) {
            const int raw = a.seq_lens[s];
            const int pre = a.s.prefix_lens ? a.s.prefix_lens[s] : 0, ks = a.s.key_starts ? a.s.key_starts[s] : 0;
            const SegTiles x = seg_tiles<TT>(a, s, raw, pre, ks);
            if (raw != x.len && blockIdx.x == 0) flag_error(a.err, PKV_DEVERR_SEQ_LEN);
            v = x.n > 0 ? x.n + T_::kLead : 0;
            my_max = max(my_max, v);
            v *= Hkv;
        }
        int x = v;
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, sh);
            if (lane >= sh) x += y;
        }
        if (lane == 31) warp_sums[warp] = x;
        __syncthreads();
        int before = carry;
        for (int k = 0; k < warp; ++k) before += warp_sums[k];
        if (s < S) prefix[s + 1] = before + x;
        __syncthreads();
        if (threadIdx.x == kNW * 32 - 1) carry = before + x;
        __syncthreads();
    }
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) my_max = max(my_max, __shfl_xor_sync(0xffffffffu, my_max, sh));
    if (lane == 0) atomicMax(&seg_max, my_max);
    unsigned char *ring = smem + warp * kNS * T_::kStage;
    unsigned char *scales = smem + L.scales + warp * kNS * T_::kScales;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L.bars) + warp * kNS;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kNS; ++i) mbar_init(&bars[i], F8 ? 5 : 1);  // the expected bytes, four lanes' scale bytes
        fence_barrier_init();
    }
    __syncthreads();

    const int64_t T = prefix[S];
    const int64_t warps = (int64_t)gridDim.x * kNW;
    const int64_t min_share = max(1, min(T_::kMinShare, seg_max));
    const int64_t parts = max((int64_t)1, min(warps, T / min_share));
    const int64_t gw = (int64_t)blockIdx.x * kNW + warp;
    const int lo = gw < parts ? (int)(gw * T / parts) : 0, hi = gw < parts ? (int)((gw + 1) * T / parts) : 0;

    auto seq_of = [&](int t) {  // the sequence that holds laid-out tile t: largest with prefix[seq] <= t
        int x = 0, y = S;
#pragma unroll 1
        while (y - x > 1) {
            const int mid = (x + y) >> 1;
            if (prefix[mid] <= t) x = mid; else y = mid;
        }
        return x;
    };
    // this lane's tile of the 32 from `t` on
    auto resolve = [&](int t) {
        Slot k{-1, -1, 0u, 0};
        t += lane;
        if (t >= hi) return k;
        const int s = seq_of(t);
        const int n = (prefix[s + 1] - prefix[s]) / Hkv, in = t - prefix[s], kvh = in / n, i = in - kvh * n - T_::kLead;
        if (i < 0) return k;
        const SegTiles x = load_seg<TT>(a, s);
        k.t0 = (i < x.np ? x.pt0 + i : x.mt0 + i - x.np) * TT;
        k.mask = range_bits(x.r.lo - k.t0, x.r.hi - k.t0) | range_bits(x.r.first - k.t0, x.r.pre - k.t0);
        if (TT == 16) k.mask &= 0xffffu;
        const int boxh = min(B, TT);
        const int32_t *bt = a.block_tables + (int64_t)s * a.max_blocks;
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
            const int tok = k.t0 + sb * boxh;
            if (sb * boxh >= TT) break;
            const uint32_t mine = range_bits(sb * boxh, (sb + 1) * boxh);
            if (!(k.mask & mine)) continue;  // no token of the box is seen: not read
            int blk = bt[tok >> a.bshift];
            if (blk < 0 || blk >= a.num_blocks) {
                flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                k.mask &= ~mine;
                continue;
            }
            const int y = (int)(((int64_t)blk * Hkv + kvh) * B + (tok & (B - 1)));
            if (sb == 0) k.y0 = y; else k.y1 = y;
        }
        return k;
    };
    Slot cur{-1, -1, 0u, 0}, nxt{-1, -1, 0u, 0};
    if (lo < hi) {
        cur = resolve(lo);
        nxt = resolve(lo + 32);
    }
    grid_dependency_wait();
    // sequences that see nothing have no tile: their rows are zeroed by the merge
#pragma unroll 1
    for (int s = blockIdx.x; s < S; s += gridDim.x)
        if (prefix[s + 1] == prefix[s])
#pragma unroll 1
            for (int h = threadIdx.x; h < Hkv; h += kNW * 32) a.segs[(int64_t)s * Hkv + h] = make_int2(0, -1);
    if (lo >= hi) return;

    const int boxh = min(B, TT);
    // Issue tile k of the share (held by lane k % 32 of `from`) into its stage.
    auto issue = [&](const Slot &from, int k, bool wrote) {
        const int buf = k % kNS;
        const int y0 = __shfl_sync(0xffffffffu, from.y0, k & 31), y1 = __shfl_sync(0xffffffffu, from.y1, k & 31);
        const uint32_t dk = smem_u32(ring + buf * T_::kStage), dv = dk + T_::kKV, b = smem_u32(&bars[buf]);
        const int n = (y0 >= 0) + (y1 >= 0);
        if (lane == 0) {
            if (wrote) fence_proxy_async();  // rows of the stage zeroed by plain stores: the copies come after them
            mbar_arrive_expect_tx(&bars[buf], (uint32_t)(n * boxh) * (F8 ? 2u * D : 4u * D));
        }
        __syncwarp();
        // As few copies as the scattered blocks allow: an SM starts one TMA copy in some 50 cycles, whatever its size (with
        // the scale bytes as bulk copies of their own, eight copies a tile, 8 x 16000 FP8 tokens took 58 us).
        if constexpr (F8) {
            // lanes 0 - 3: (box, codes of K / V) by TMA; 4 - 7: their scale bytes by cp.async, which arrive on the barrier too
            const int sb = (lane >> 1) & 1, isv = lane & 1, y = sb ? y1 : y0;
            if (lane < 4) {
                if (y >= 0) tma_load_2d((isv ? dv : dk) + (uint32_t)(sb * boxh) * D, isv ? &tm_v : &tm_k, b, 0, y);
            } else if (lane < 8) {
                if (y >= 0)
#pragma unroll 1
                    for (int c = 0; c < boxh; c += 16)
                        cp_async16(smem_u32(scales + buf * T_::kScales) + isv * TT + sb * boxh + c, (isv ? a.v_scales : a.k_scales) + y + c);
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(b) : "memory");
            }
        } else if (D == 128 && boxh == 16) {
            if (lane < 2 && y0 >= 0) tma_load_3d(lane ? dv : dk, lane ? &tm_v : &tm_k, b, 0, y0, 0);  // both halves in one box
        } else {
            // lanes: (box, half, K / V)
            constexpr int H = D / 64;
            const int sb = lane / (2 * H), h = (lane >> 1) % H, y = sb ? y1 : y0;
            if (lane < 4 * H && y >= 0)
                tma_load_2d(((lane & 1) ? dv : dk) + h * (16 * 128) + sb * boxh * 128, (lane & 1) ? &tm_v : &tm_k, b, h * 64, y);
        }
    };
    const int ntiles = hi - lo;
#pragma unroll
    for (int k = 0; k < kNS; ++k)
        if (k < ntiles) issue(cur, k, false);

    int seq = seq_of(lo), kvh, seg0, segn;  // the segment being attended, its laid-out start and tiles
    auto locate = [&](int t) {
        segn = (prefix[seq + 1] - prefix[seq]) / Hkv;
        kvh = (t - prefix[seq]) / segn;
        seg0 = prefix[seq] + kvh * segn;
    };
    locate(lo);
    Query<D> q, qn;
    load_query<D, F8>(a, seq, kvh, lane, q);
    bool dead = false;
    Acc<D> acc;
#pragma unroll 1
    for (int k = 0; k < ntiles;) {
        // one piece: the segment's tiles in this share
        const int pa = lo + k, pb = min(hi, seg0 + segn), kend = pb - lo;
        const int this_seq = seq, this_kvh = kvh, s0 = seg0, s1 = seg0 + segn;
        const int raw = a.seq_lens[seq];
        const int pos = min(raw, min(a.max_seq_len, a.max_blocks << a.bshift)) - 1;  // it has tiles: the length is positive
        if (kend < ntiles) {  // the next piece's queries, while this one runs
            if (++kvh == Hkv) {
                kvh = 0;
                do { ++seq; } while (prefix[seq + 1] == prefix[seq]);
            }
            locate(pb);
            load_query<D, F8>(a, seq, kvh, lane, qn);
        }
        acc.reset();
#pragma unroll 1
        for (; k < kend; ++k) {
            const int buf = k % kNS;
            if (!dead && !wait_tile(&bars[buf], (uint32_t)((k / kNS) & 1))) {
                if (lane == 0) flag_error(a.err, PKV_DEVERR_TIMEOUT);
                dead = true;
                // no copy is issued any more; those in flight land before the CTA's shared memory is another's
#pragma unroll 1
                for (int j = k; j < min(ntiles, k + kNS); ++j) wait_tile(&bars[j % kNS], (uint32_t)((j / kNS) & 1));
            }
            Slot t;
            t.mask = __shfl_sync(0xffffffffu, cur.mask, k & 31);
            t.t0 = __shfl_sync(0xffffffffu, cur.t0, k & 31);
            unsigned char *sk = ring + buf * T_::kStage;
            if (t.mask != 0u && !dead) {
                if constexpr (F8) attend_fp8<D>(a, sk, sk + T_::kKV, scales + buf * T_::kScales, t, pos, q, acc, lane);
                else attend_bf16<D>(a, sk, sk + T_::kKV, t, pos, q, acc, lane);
            }
            __syncwarp();
            if (k + kNS < ntiles && !dead) issue(((k + kNS) & 31) < kNS ? nxt : cur, k + kNS, t.mask != (TT == 32 ? 0xffffffffu : 0xffffu));
            if ((k & 31) == 31) {
                cur = nxt;
                nxt = resolve(lo + k + 33);
            }
        }
        // ---- the piece's result ----
        const int g = lane >> 2, tq = lane & 3, G = a.group;
        if constexpr (F8) {  // head g's, over its four lanes; then to the lanes of its column
            acc.l[0] += __shfl_xor_sync(0xffffffffu, acc.l[0], 1);
            acc.l[0] += __shfl_xor_sync(0xffffffffu, acc.l[0], 2);
            const float l = acc.l[0], m = acc.m[0];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                acc.l[j] = __shfl_sync(0xffffffffu, l, 8 * tq + 4 * j);
                acc.m[j] = __shfl_sync(0xffffffffu, m, 8 * tq + 4 * j);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int sh = 4; sh < 32; sh <<= 1) acc.l[j] += __shfl_xor_sync(0xffffffffu, acc.l[j], sh);
        }
        const bool whole = pa <= s0 + T_::kLead && pb == s1;  // every real tile
        const int64_t w0 = share_owner(s0 + T_::kLead, T, parts);  // the warp with the segment's first real tile
        if (gw == w0 && lane == 0)
            a.segs[(int64_t)this_seq * Hkv + this_kvh] = make_int2((int)w0, whole ? 0 : (int)(share_owner(s1 - 1, T, parts) - w0) + 1);
        if (gw >= w0) {  // a share that ends inside the lead tiles holds none of the segment
            const float inv[2] = {acc.l[0] != 0.f ? 1.f / acc.l[0] : 0.f, acc.l[1] != 0.f ? 1.f / acc.l[1] : 0.f};
            const int64_t slot = 2 * gw + (gw == w0 ? 1 : 0);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int h = 2 * tq + (j & 1), d = entry<D, F8>(i, g, j);
                    if (h >= G) continue;
                    if (whole)
                        static_cast<__nv_bfloat16 *>(a.out)[((int64_t)this_seq * a.num_heads + this_kvh * G + h) * D + d] =
                            __float2bfloat16_rn(acc.o[i][j] * inv[j & 1]);
                    else
                        a.part_o[(slot * G + h) * D + d] = acc.o[i][j];
                }
            if (!whole && g == 0)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (2 * tq + j < G)
                        reinterpret_cast<float2 *>(a.part_ml)[slot * G + 2 * tq + j] =
                            make_float2(dead ? __int_as_float(0x7fc00000) : acc.m[j], acc.l[j]);
        }
        q = qn;
    }
}

// One warp per (sequence, query head): the partial states of a segment that was
// cut, merged in order (part 0 is its first warp's last piece, part j the first
// piece of warp w0 + j); zero rows where no key is seen.
template <int D, bool F8>
__global__ void __launch_bounds__(128) scored_decode_merge_kernel(const __grid_constant__ DecodeArgs a) {
    // Not earlier: the next call's CTAs would take their places while this kernel's wait beside the attention kernel's last
    // ones, and end up two on some SMs (8 x 16000 tokens FP8: 58 -> 71 us).
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)a.num_seqs * a.num_heads) return;
    const int lane = threadIdx.x & 31, G = a.group;
    const int64_t s = row / a.num_heads;
    const int h = (int)(row - s * a.num_heads);
    const int2 seg = a.segs[s * a.num_kv_heads + h / G];
    if (seg.y == 0) return;
    constexpr int E = D / 32;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + row * D + E * lane;
    float o[E], M = -INFINITY, L = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    auto slot = [&](int j) { return ((int64_t)(2 * (seg.x + j) + (j == 0 ? 1 : 0)) * G + h % G); };
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml);
    constexpr int U = 8;  // parts whose rows are loaded together
    for (int j0 = 0; j0 < seg.y; j0 += U) {
        float2 x[U];
        float v[U][E], mx = M;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = slot(min(j0 + u, seg.y - 1));
            x[u] = j0 + u < seg.y ? ml[at] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] = a.part_o[at * D + E * lane + e];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) mx = fmaxf(mx, x[u].x);
        const float f = M == -INFINITY ? 0.f : ex2_approx(M - mx);
        L = F8 ? lower_sum(L, M - mx) : L * f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= f;
        M = mx;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float w = x[u].x == -INFINITY ? 0.f : ex2_approx(x[u].x - M);
            if (j0 + u >= seg.y) continue;
            L += F8 ? lower_sum(x[u].y, x[u].x - M) : x[u].y * w;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = w != 0.f ? fmaf(w, v[u][e], o[e]) : o[e];
        }
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    uint32_t p[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) p[e / 2] = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) reinterpret_cast<uint32_t *>(out)[e] = p[e];
}

struct WsLayout {
    size_t o, ml, segs, total;
    WsLayout(int64_t num_segs, int G, int D) {
        o = 0;
        ml = round256((size_t)2 * kMaxWarps * G * D * 4);
        segs = ml + round256((size_t)2 * kMaxWarps * G * 8);
        total = segs + round256((size_t)num_segs * 8);
    }
};

// Code rows: 2-D view [blocks * Hkv * B][D] bytes, box D x min(B, 32) rows, swizzled by the row's width.
bool make_code_map(CUtensorMap *map, const void *base, int64_t rows, int D, int boxh) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)D};
    cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)boxh};
    cuuint32_t estr[2] = {1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool F8>
pkv_status launch(const DecodeArgs &a, cudaStream_t st) {
    static bool done[128] = {};
    auto kern = scored_decode_kernel<D, F8>;
    if (!ensure_smem(kern, Smem<D, F8>(kMaxSeqs).total, done)) return PKV_ERR_CUDA;
    const int smem = Smem<D, F8>(a.num_seqs).total;
    // CTAs per SM, asked once per shared-memory size in a row (the devices of a process are alike): (size << 8) | CTAs
    static std::atomic<int64_t> known{0};
    int64_t k = known.load(std::memory_order_relaxed);
    if ((k >> 8) != smem) {
        int per = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, kNW * 32, smem) != cudaSuccess || per < 1)
            return PKV_ERR_CUDA;
        known.store(k = ((int64_t)smem << 8) | per, std::memory_order_relaxed);
    }
    const int per_sm = (int)(k & 255);
    const int grid = std::min(sm_count() * per_sm, kMaxWarps / kNW);
    if (grid < 1) return PKV_ERR_CUDA;
    CUtensorMap mk, mv;
    const int64_t rows = (int64_t)a.num_blocks * a.num_kv_heads * a.block_size;
    const int boxh = std::min(a.block_size, Tile<D, F8>::kTok);
    if (F8 ? !make_code_map(&mk, a.k_cache, rows, D, boxh) || !make_code_map(&mv, a.v_cache, rows, D, boxh)
        : D == 128 && boxh == 16
            ? !make_slab_map(&mk, a.k_cache, rows, D, boxh) || !make_slab_map(&mv, a.v_cache, rows, D, boxh)
            : !make_cache_map(&mk, a.k_cache, rows, D, boxh) || !make_cache_map(&mv, a.v_cache, rows, D, boxh))
        return PKV_ERR_CUDA;
    pkv_status rc = launch_pdl(kern, dim3((unsigned)grid), dim3(kNW * 32), smem, st, mk, mv, a);
    if (rc == PKV_OK)
        rc = launch_pdl(scored_decode_merge_kernel<D, F8>, dim3((unsigned)(((int64_t)a.num_seqs * a.num_heads + 3) / 4)), dim3(128),
                        0, st, a);
    return rc;
}

}  // namespace

size_t decode_workspace(int64_t num_seqs, int num_heads, int head_dim) {
    // for any grouping: G <= 8 heads a KV head, at most num_heads segments a sequence
    return WsLayout(std::min<int64_t>(num_seqs, kMaxSeqs) * num_heads, std::min(num_heads, kGMax), head_dim).total;
}

static int64_t seqs_per_launch(const Args &a) {
    return std::min<int64_t>(kMaxSeqs, kMaxTiles / (a.num_kv_heads * ((longest_context(a) + 15) / 16 + 4)));
}

bool decode_fits(const Args &a) { return seqs_per_launch(a) >= 1; }

pkv_status run_decode(const Args &args, int head_dim, void *workspace, cudaStream_t st) {
    DecodeArgs a{};
    static_cast<Args &>(a) = args;
    if (a.s.softcap > kNoCap) a.s.softcap = 0.f;
    const bool fp8 = a.k_scales != nullptr;
    const int64_t most = seqs_per_launch(a);
    const double log2e = 1.4426950408889634;
    a.c2 = finite_float(a.s.softcap * log2e);
    a.k1 = finite_float(a.s.softcap > 0.f ? 2.0 * a.s.scale / a.s.softcap * log2e : a.s.scale * log2e);
    a.bshift = a.block_size == 8 ? 3 : a.block_size == 16 ? 4 : 5;
    const WsLayout lay(std::min<int64_t>(a.num_seqs, most) * a.num_kv_heads, a.group, head_dim);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    a.part_o = reinterpret_cast<float *>(ws + lay.o);
    a.part_ml = reinterpret_cast<float *>(ws + lay.ml);
    a.segs = reinterpret_cast<int2 *>(ws + lay.segs);
    const ScoreArgs score = a.s;
    pkv_status rc = PKV_OK;
    for (int64_t s0 = 0; s0 < args.num_seqs && rc == PKV_OK; s0 += most) {  // (a part begins when the one before is through)
        static_cast<Args &>(a) = part_of(args, head_dim, (int)s0, (int)std::min<int64_t>(most, args.num_seqs - s0));
        a.s.softcap = score.softcap;
        if (fp8) rc = head_dim == 128 ? launch<128, true>(a, st) : launch<64, true>(a, st);
        else rc = head_dim == 128 ? launch<128, false>(a, st) : launch<64, false>(a, st);
    }
    return rc;
}

}  // namespace scored
}  // namespace pkv
