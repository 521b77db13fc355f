// Scored attention of several queries per sequence (prefill, chunks of one,
// verification of drafted tokens) on the 5th-generation tensor cores.
//
// Per KV head, the query heads of consecutive queries form rows that meet the
// same 128-key tiles of the paged cache:
//     S = Q K^T (M 128 rows, N 128 keys, K head_dim)      scores, in tensor memory
//     P = 2^(y(S) - m)                                     y: the score in base 2, capped and biased
//     O += P V  (M 128, N head_dim, K 128 keys)
// with a running reference m and sum l per row; m moves (and O is rescaled)
// only when a tile's maximum passes it by more than 2^8.
//
// A context is a set of at most 256 rows (two groups of 128: paired) or, where
// no sequence has more than 128, of at most 128 rows whose tiles the two groups
// take in turn (alternating; their states are merged at the context's end).
// Its tiles are those that some row sees: the tiles of the always visible
// prefix, then those from the first row's window or document to the last row's
// position.  All contexts are laid end to end, each behind kCharge virtual
// tiles that stand for its fixed costs, and every CTA (one per SM) takes an
// equal share.  A context cut by a share's border leaves partial states (o, m,
// l) in the workspace, which a second kernel merges; no CTA waits for another.
//
// Warps: 0-7 and 8-15 two softmax groups (two threads per row = TMEM lane, one
// for each half of a tile's keys), 16 the MMA issuer, 17 / 18 the producers of
// K / V tiles (one TMA box per block and column half, or per block), 19 the
// scheduler, which walks the share and publishes one descriptor per piece of a
// context.  While one group works on
// its scores the tensor cores run the other's products: the issue order is
// P V (group 0), Q K^T (0, next tile), P V (1), Q K^T (1, next tile).
// Tensor memory: S of group g at columns 128 g (P overwrites its first half as
// bf16 pairs), O at 256 + g * head_dim.  A row's S being complete implies that
// every earlier product of the issuing thread is, P V of its group included, so
// a rescale of O needs no wait of its own.
// Every wait is bounded; one that gives up flags PKV_DEVERR_TIMEOUT.
#include <algorithm>
#include <climits>
#include <cmath>

#include "pkv_internal.cuh"
#include "scored.cuh"

namespace pkv {
namespace scored {
namespace {

constexpr int kTok = 128;   // keys per tile
constexpr int kRows = 128;  // rows of a softmax group
constexpr int kHalf = kTok / 2;      // a softmax thread's keys of a tile
constexpr int kGroupWarps = 8;       // two halves of four warps
constexpr int kThreads = 640;
constexpr int kMmaWarp = 16, kKWarp = 17, kVWarp = 18, kSchedWarp = 19;
constexpr int kDescs = 6;  // piece descriptors in flight
constexpr int kRecs = 8;  // tile records (more than the K producer can be ahead of the softmax)
constexpr int kCharge = 2;   // virtual tiles of a context
constexpr int kMinShare = kCharge + 1;
constexpr float kRescale = 8.f;
constexpr float kMaxC2 = 73.f;  // softcap * log2 e up to which capped scores take a fixed reference (cap 50)
constexpr uint32_t kTmemCols = 512, kOBase = 256;
constexpr int kMaxCtas = 160;   // partial slots in the workspace: two per CTA
constexpr int kMergeRows = 32;  // rows per CTA of the merge kernel
enum Kind { kPlain = 0, kCap = 1, kBias = 2, kCapBias = 3 };

struct RowsArgs : Args {
    float k1;       // plain, biased: scale * log2 e; capped: scale / softcap
    float c2;       // capped: softcap * log2 e
    float m0;       // capped: the reference
    float near[4], far[6];  // capped: c2 tanh(k1 s) = s * sum near[i] s^2i for |k1 s| <= kTanhNear (far: kTanhFar)
    float *part_o;  // [2 kMaxCtas][D][256]: columns of 256 rows
    float *part_ml; // [2 kMaxCtas][256][2]
    int4 *merges;   // [kMaxCtas]: (parts, first query row, rows, kv head) of the context begun and cut in that share
    int bshift, per_ctx, scan_w;  // log2 block size, queries per context, lanes per sequence in the scan
};

struct Piece {
    int ntiles;  // 0: no more
    int i0;      // first tile within the context
    int np, pt0, mt0;   // context tile i is key tile pt0 + i (i < np) or mt0 + i - np
    int seq, kvh, row0, nrows, pos0, pre;
    int ks0, cpre, lo, hi;  // the context's keys: [ks0, cpre) and [lo, hi) (KeyRange)
    int slot;                 // partial slot, -1: the whole context
    int jf[2], jl[2];         // group g takes the tiles jf .. jl (none: jl < jf); alternating: those of its parity
};

// A tile's record, written by the K producer.
struct TileRec {
    int t0;        // first key
    uint32_t bad;  // bits of blocks with an invalid id (their keys are masked)
    int whole;     // every key is seen by some row: no V row has to be zeroed
    int pad;
};

__device__ __forceinline__ int key_tile(const Piece &p, int j) {
    const int i = p.i0 + j;
    return i < p.np ? p.pt0 + i : p.mt0 + i - p.np;
}
template <bool ALT>
__device__ __forceinline__ bool has_rows(const Piece &p, int g) { return ALT || p.nrows > g * kRows; }
template <int D, bool ALT>
struct Layout {
    static constexpr int H = D / 64;
    static constexpr int kQTile = H * kRows * 128;
    static constexpr int kQBytes = (ALT ? 1 : 2) * kQTile;
    static constexpr int kTile = H * kTok * 128;  // K or V of one tile
    static constexpr int NK = D == 128 ? 2 : 4;
    static constexpr int NV = D == 128 ? (ALT ? 3 : 2) : 4;
    static constexpr int q = 0;
    static constexpr int kring = q + kQBytes;
    static constexpr int vring = kring + NK * kTile;
    static constexpr int xch = vring + NV * kTile;        // float [2][2 groups][2 halves][kRows]: maxima of even / odd tiles
    static constexpr int fin_ml = xch + 8 * kRows * 4;    // float2 [2 groups][2 halves][kRows]: (m, l) at a piece's end
    static constexpr int desc = fin_ml + 4 * kRows * 8;
    static constexpr int recs = (desc + kDescs * (int)sizeof(Piece) + 15) & ~15;
    static constexpr int bars = recs + kRecs * (int)sizeof(TileRec);
    static constexpr int kBars = 2 * NK + 2 * NV + 6 * 2 + 2 * kDescs + 1 + 8;
    static constexpr int misc = bars + kBars * 8;  // TMEM address, scan scratch
    static constexpr int total = misc + 128;
    static_assert(total <= 227 * 1024, "shared memory per CTA");
};

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0u;
}

__device__ __forceinline__ bool wait_or_flag(uint64_t *bar, uint32_t parity, bool &dead, unsigned int *err) {
    if (dead) return false;
    if (mbar_wait_bounded(bar, parity)) return true;
    flag_error(err, PKV_DEVERR_TIMEOUT);
    dead = true;
    return false;
}

// ---------------------------------------------------------------------------
// Contexts
// ---------------------------------------------------------------------------
struct Seq {
    int q0, Q, L, pre;
};

// Sequence s; bad descriptions count as no queries (flagged by the CTA that reports).
__device__ __forceinline__ Seq load_seq(const RowsArgs &a, int s, bool report) {
    const int cap = min(a.max_seq_len, a.max_blocks * a.block_size);
    Seq x;
    x.q0 = a.q_starts[s];
    const int q1 = a.q_starts[s + 1];
    const int raw = a.seq_lens[s];
    const int pre = a.s.prefix_lens ? a.s.prefix_lens[s] : 0;
    x.L = raw < 0 ? 0 : min(raw, cap);
    x.pre = min(max(0, pre), x.L);
    x.Q = q1 - x.q0;
    if (x.q0 < 0 || q1 < x.q0 || q1 > a.num_q) {
        if (report) flag_error(a.err, PKV_DEVERR_SEQ_LEN);
        x.q0 = x.Q = 0;
        return x;
    }
    if (report && (raw != x.L || x.Q > a.max_q_len || x.Q > x.L)) flag_error(a.err, PKV_DEVERR_SEQ_LEN);
    x.Q = min(x.Q, a.max_q_len);  // further queries are not attended
    return x;
}

struct CtxTiles {
    KeyRange r;
    int ks0, pt0, np, mt0, n;
};

// Tiles of query block b of a sequence.  Positions count from the sequence's
// real query count: row i sits at L - Qall + i (Qall before the max_q_len cut).
__device__ __forceinline__ CtxTiles ctx_tiles(const RowsArgs &a, const Seq &x, int pos_first, int b) {
    CtxTiles c;
    const int i0 = b * a.per_ctx, i1 = min(x.Q, i0 + a.per_ctx) - 1;
    c.ks0 = key_start_of(a.s, x.q0 + i0);
    c.r = key_range(c.ks0, x.pre, a.s.window, pos_first + i0, pos_first + i1);
    c.mt0 = c.r.lo / kTok;
    const int nm = c.r.hi > c.r.lo ? (c.r.hi + kTok - 1) / kTok - c.mt0 : 0;
    c.pt0 = c.r.first / kTok;
    int pe = c.r.pre > c.r.first ? (c.r.pre + kTok - 1) / kTok : c.pt0;
    if (nm > 0) pe = min(pe, c.mt0);
    c.np = max(0, pe - c.pt0);
    c.n = c.np + nm;
    return c;
}

__device__ __forceinline__ int first_pos(const RowsArgs &a, const Seq &x, int s) {
    return x.Q > 0 ? x.L - (a.q_starts[s + 1] - a.q_starts[s]) : 0;
}

__device__ __forceinline__ int laid_out(int n) { return n > 0 ? n + kCharge : 0; }

__host__ __device__ __forceinline__ int64_t split_parts(int64_t T, int64_t ctas) {
    const int64_t by_size = T / kMinShare > 1 ? T / kMinShare : 1;
    return ctas < by_size ? ctas : by_size;
}

// ---------------------------------------------------------------------------
// Softmax step
// ---------------------------------------------------------------------------
__device__ __forceinline__ void st16u(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}

__device__ __forceinline__ void ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void st8u(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// tanh z / z as polynomials in z^2: least squares of the error of tanh, reweighted towards its largest (Lawson's method),
// in 64 bits.  |z| <= 0.75: off by at most 3.7e-6; |z| <= 1.25: 2.4e-6 -- of the cap, so 2e-4 of a score at a cap of 50,
// where the weight's rounding to bf16 is worth 2e-3 to 4e-3.
constexpr float kTanhNear = 0.75f, kTanhFar = 1.25f;
constexpr double kTanh3[4] = {0.9999556008, -0.3322276376, 0.1257709249, -0.03377828486};
constexpr double kTanh5[6] = {0.9999746925, -0.3328393216, 0.1305362538, -0.04692675917, 0.01253202075, -0.001682072195};

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// bits [a, b) of a 32-bit word, a and b taken from any integers
__device__ __forceinline__ uint32_t bit_range(int a, int b) {
    a = max(a, 0);
    b = min(b, 32);
    if (a >= b) return 0u;
    return (b == 32 ? 0xffffffffu : (1u << b) - 1u) & ~((1u << a) - 1u);
}

struct RowState {
    float m, l;    // reference and sum
    int p;         // position
    KeyRange r;
    float slope2;  // slope * log2 e
};

// Maximum over N values, four chains of three-input maxima; ABS: of their magnitudes.
template <bool ABS, int N>
__device__ __forceinline__ float max_of(const float (&s)[N]) {
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = ABS ? fabsf(s[i]) : s[i];
#pragma unroll
        for (int k = i + 4; k + 4 < N; k += 8)
            m[i] = ABS ? fmax3(m[i], fabsf(s[k]), fabsf(s[k + 4])) : fmax3(m[i], s[k], s[k + 4]);
        if (N % 8 == 0) m[i] = fmaxf(m[i], ABS ? fabsf(s[N - 4 + i]) : s[N - 4 + i]);
    }
    return fmaxf(fmax3(m[0], m[1], m[2]), m[3]);
}

// The 32 keys from t on that the row sees, as bits.
__device__ __forceinline__ uint32_t seen32(const KeyRange &r, int t, uint32_t bad, int bshift, int word) {
    uint32_t m = bit_range(r.lo - t, r.hi - t) | bit_range(r.first - t, r.pre - t);
    if (bad) {
        const int per = 32 >> bshift;  // blocks of the word
        for (int b = 0; b < per; ++b)
            if ((bad >> (word * per + b)) & 1u) m &= ~bit_range(b << bshift, (b + 1) << bshift);
    }
    return m;
}

// Raw products -> scores in base 2 plus nm: c tanh(z) + nm, z = k1 s.  For |z| small in the whole warp an odd polynomial
// (the cap's factors folded in on the host) on the FMA pipe, two keys an instruction: the exponential is then the only
// special function of a score.  The FMA pipe is what bounds capped scores, hence the shortest polynomial for the usual
// sizes.  cap_near computes that one whatever the sizes and cap_far does the rest again where cap_near does not hold.
template <int N>
__device__ __forceinline__ void cap_near(float (&s)[N], const RowsArgs &a, uint64_t nm2) {
    const uint64_t q0 = f32x2(a.near[0], a.near[0]), q1 = f32x2(a.near[1], a.near[1]);
    const uint64_t q2 = f32x2(a.near[2], a.near[2]), q3 = f32x2(a.near[3], a.near[3]);
#pragma unroll
    for (int k = 0; k < N; k += 2) {
        const uint64_t x = f32x2(s[k], s[k + 1]), u = mul_f32x2(x, x);
        const uint64_t y = fma_f32x2(fma_f32x2(fma_f32x2(q3, u, q2), u, q1), u, q0);
        f32x2_split(fma_f32x2(x, y, nm2), s[k], s[k + 1]);
    }
}

template <int N>
__device__ __forceinline__ void cap_far(float (&s)[N], const RowsArgs &a, float nm, float top) {
    if (!__any_sync(0xffffffffu, top > kTanhFar)) {
        const uint64_t nm2 = f32x2(nm, nm);
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            const uint64_t x = f32x2(s[k], s[k + 1]), u = mul_f32x2(x, x);
            uint64_t y = f32x2(a.far[5], a.far[5]);
#pragma unroll
            for (int i = 4; i >= 0; --i) y = fma_f32x2(y, u, f32x2(a.far[i], a.far[i]));
            f32x2_split(fma_f32x2(x, y, nm2), s[k], s[k + 1]);
        }
    } else {
        // tanh z = 1 - 2 / (1 + e^2z), good to 2^-21
        const float z2 = 2.f * 1.44269504f * a.k1;
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] = (a.c2 + nm) - (2.f * a.c2) * rcp_approx(1.f + ex2_approx(s[k] * z2));
    }
}

__device__ __forceinline__ void cap32(float (&s)[32], const RowsArgs &a) {
    const float top = max_of<true>(s) * fabsf(a.k1);
    if (!__any_sync(0xffffffffu, top > kTanhNear)) cap_near(s, a, 0ull);
    else cap_far(s, a, 0.f, top);
}

// Capped: the weights of 16 keys of S at sp (loaded in s) to P at `to`, their sum to ls; w: the keys that are seen.
__device__ __forceinline__ void cap_weights16(float (&s)[16], uint32_t sp, uint32_t to, const RowsArgs &a, float nm, uint64_t nm2,
                                              bool full, uint32_t w, uint64_t (&ls)[2]) {
    const float top = max_of<true>(s) * fabsf(a.k1);
    cap_near(s, a, nm2);
    if (__any_sync(0xffffffffu, top > kTanhNear)) {
        ld16(sp, s);
        tc::wait_ld();
        cap_far(s, a, nm, top);
    }
    if (!full) {
#pragma unroll
        for (int k = 0; k < 16; ++k) s[k] = (w >> k) & 1u ? s[k] : -INFINITY;
    }
    uint32_t pk[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float e0 = ex2_approx(s[2 * k]), e1 = ex2_approx(s[2 * k + 1]);
        pk[k] = pack_bf16x2(e0, e1);
        ls[k & 1] = add_f32x2(ls[k & 1], f32x2(e0, e1));
    }
    st8u(to, pk);
}

// Weights 2^(f s + nm) of 32 keys to P (bf16 pairs) at `to`, their sum to ls.
__device__ __forceinline__ void weights32(const float (&s)[32], float f, float nm, uint32_t to, uint64_t (&ls)[2]) {
    const uint64_t f2 = f32x2(f, f), nm2 = f32x2(nm, nm);
    uint32_t pk[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        float a0, a1;
        f32x2_split(fma_f32x2(f32x2(s[2 * k], s[2 * k + 1]), f2, nm2), a0, a1);
        const float e0 = ex2_approx(a0), e1 = ex2_approx(a1);
        pk[k] = pack_bf16x2(e0, e1);
        ls[k & 1] = add_f32x2(ls[k & 1], f32x2(e0, e1));
    }
    st16u(to, pk);
}

// One tile of one row's half (64 keys): 32 keys at a time in loops that are not
// unrolled -- unrolled code of 128 keys ran at the pace of its instruction
// fetches (6 to 10 cycles an instruction).  S (raw products) at sp, P (bf16
// pairs) back over the half's first 32 columns, always behind the reads.  t0:
// the half's first key; bad: bits of its blocks with an invalid id; beyond: some
// row may see keys past its position (a prefix).  Returns with `move` set when O
// has to be scaled by `alpha` before the tile's product.
//
// A first pass finds the maximum, meet() gives the row's (both halves weigh by
// the same reference); scores that are biased or masked are written back over S
// by it, in base 2 (plain ones stay raw: the exponential's FMA scales them).
// Capped scores without a bias need neither: they lie within +-c2, and up to
// kMaxC2 a fixed reference c2 / 4 keeps weights within 2^-(5/4 c2) .. 2^(3/4 c2)
// (cap 50: 2^-90 .. 2^54), far from the ends of float32's and bf16's range for
// sums over 2^20 keys of V entries between 2^-36 and 2^53.
template <int KIND, typename Meet>
__device__ __forceinline__ void softmax_half(uint32_t sp, int t0, uint32_t bad, const RowsArgs &a, bool beyond,
                                             RowState &st, bool &move, float &alpha, Meet meet) {
    const bool mine = ((t0 >= st.r.lo && t0 + kHalf <= st.r.hi) || (t0 >= st.r.first && t0 + kHalf <= st.r.pre)) && bad == 0u;
    const bool full = __all_sync(0xffffffffu, mine);
    move = false;
    alpha = 1.f;
    uint64_t ls[2] = {0ull, 0ull};
    if constexpr (KIND == kCap) {
        // every score lies within +-c2: one reference does for all tiles (and every part of a context); 16 keys are loaded
        // while 16 are worked on
        const float nm = -st.m;
        const uint64_t nm2 = f32x2(nm, nm);
        float x0[16], x1[16];
        ld16(sp, x0);
#pragma unroll 1
        for (int c = 0; c < kHalf; c += 32) {
            const uint32_t w = full ? 0u : seen32(st.r, t0 + c, bad, a.bshift, c / 32);
            tc::wait_ld();
            ld16(sp + c + 16, x1);
            cap_weights16(x0, sp + c, sp + c / 2, a, nm, nm2, full, w, ls);
            tc::wait_ld();
            if (c + 32 < kHalf) ld16(sp + c + 32, x0);
            cap_weights16(x1, sp + c + 16, sp + c / 2 + 8, a, nm, nm2, full, w >> 16, ls);
        }
        float x, y;
        f32x2_split(add_f32x2(ls[0], ls[1]), x, y);
        st.l += x + y;
        tc::wait_st();
        return;
    }
    const bool stored = KIND != kPlain || !full;
    float mt = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < kHalf / 32; ++c) {
        float s[32];
        tc::ld32(sp + 32 * c, s);
        tc::wait_ld();
        const int t = t0 + 32 * c;
        if constexpr (KIND == kCapBias) cap32(s, a);
        if constexpr (KIND == kBias || KIND == kCapBias) {
            const float f = KIND == kBias ? a.k1 : 1.f, d0 = (float)(st.p - t);
            if (beyond) {
#pragma unroll
                for (int k = 0; k < 32; ++k) s[k] = fmaf(-st.slope2, fabsf(d0 - (float)k), s[k] * f);
            } else {
                // -slope (p - t - k): one FMA for the pair's bias, one for the score
                const uint64_t f2 = f32x2(f, f), b0 = f32x2(-st.slope2 * d0, -st.slope2 * d0), sl = f32x2(st.slope2, st.slope2);
#pragma unroll
                for (int k = 0; k < 32; k += 2)
                    f32x2_split(fma_f32x2(f32x2(s[k], s[k + 1]), f2, fma_f32x2(sl, f32x2((float)k, (float)(k + 1)), b0)), s[k],
                                s[k + 1]);
            }
        }
        if (!full) {
            const uint32_t w = seen32(st.r, t, bad, a.bshift, c);
#pragma unroll
            for (int k = 0; k < 32; ++k) s[k] = (w >> k) & 1u ? s[k] : -INFINITY;
        }
        mt = fmaxf(mt, max_of<false>(s));
        if (stored) tc::st32(sp + 32 * c, s);
    }
    if (stored) tc::wait_st();
    if (KIND == kPlain) mt *= a.k1;
    mt = meet(mt);
    if (mt != -INFINITY) {
        if (st.m == -INFINITY) {
            st.m = mt;  // nothing summed yet
        } else if (mt > st.m + kRescale) {
            alpha = ex2_approx(st.m - mt);
            st.m = mt;
            st.l *= alpha;
            move = true;
        }
    }
    const float nm = st.m == -INFINITY ? 0.f : -st.m, f = KIND == kPlain ? a.k1 : 1.f;
#pragma unroll 1
    for (int c = 0; c < kHalf / 32; ++c) {
        float s[32];
        tc::ld32(sp + 32 * c, s);
        tc::wait_ld();
        weights32(s, f, nm, sp + 16 * c, ls);
    }
    float x, y;
    f32x2_split(add_f32x2(ls[0], ls[1]), x, y);
    st.l += x + y;
    tc::wait_st();
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <int D, int KIND, bool ALT>
__global__ void __launch_bounds__(kThreads, 1)
scored_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ RowsArgs a) {
    using L = Layout<D, ALT>;
    constexpr int H = L::H, NK = L::NK, NV = L::NV;
    extern __shared__ __align__(1024) unsigned char smem[];
    Piece *descs = reinterpret_cast<Piece *>(smem + L::desc);
    TileRec *recs = reinterpret_cast<TileRec *>(smem + L::recs);
    float *xch = reinterpret_cast<float *>(smem + L::xch);
    float2 *fin_ml = reinterpret_cast<float2 *>(smem + L::fin_ml);
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + L::bars), *k_empty = k_full + NK;
    uint64_t *v_full = k_empty + NK, *v_empty = v_full + NV;
    uint64_t *s_full = v_empty + NV, *p_full = s_full + 2;      // per group
    uint64_t *q_ready = p_full + 2, *o_last = q_ready + 2, *o_free = o_last + 2;
    uint64_t *desc_full = o_free + 2, *desc_empty = desc_full + kDescs, *fin = desc_empty + kDescs;
    uint64_t *xch_full = fin + 1;   // per group: its rows' m and l of a piece are in xch
    uint64_t *pair = xch_full + 2;  // [2][4]: both halves of 32 rows have posted
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::misc);
    int *scratch = reinterpret_cast<int *>(smem + L::misc + 16);  // [20] warp sums, carry, found sequence, its start
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int Hkv = a.num_kv_heads, G = a.group, B = a.block_size;

    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if ((smem_u32(smem) & 1023u) != 0u) {  // swizzled tiles need it; never expected
        if (threadIdx.x == 0) flag_error(a.err, PKV_DEVERR_TIMEOUT);
        return;
    }

    // ---- scan: laid-out tiles of every sequence; scan_w lanes share one ----
    const int W = a.scan_w, per_pass = kThreads / W, sub = threadIdx.x % W;
    auto seq_total = [&](int s, bool report) {
        int t = 0;
        if (s < a.num_seqs) {
            const Seq x = load_seq(a, s, report && sub == 0);
            const int fp = first_pos(a, x, s), nb = (x.Q + a.per_ctx - 1) / a.per_ctx;
            for (int b = sub; b < nb; b += W) t += laid_out(ctx_tiles(a, x, fp, b).n);
        }
        for (int sh = 1; sh < W; sh <<= 1) t += __shfl_xor_sync(0xffffffffu, t, sh);
        return t * Hkv;
    };
    int T = 0, my_s0 = 0, my_s1 = 0;
    int64_t parts = 1;
    int start = 0, v = 0;  // this thread's sequence of the last pass: its laid-out start and tiles
    // the total, then the sequence that holds this share's start (from registers when one pass covers every sequence)
    for (int round = 0; round < (a.num_seqs > per_pass ? 2 : 1); ++round) {
        if (threadIdx.x == 0) scratch[20] = 0;
        __syncthreads();
        for (int base = 0; base < a.num_seqs; base += per_pass) {
            const int s = base + threadIdx.x / W;
            const int total = seq_total(s, round == 0 && blockIdx.x == 0);
            v = sub == 0 ? total : 0;
            int x = v;
#pragma unroll
            for (int sh = 1; sh < 32; sh <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, sh);
                if (lane >= sh) x += y;
            }
            if (lane == 31) scratch[warp] = x;
            __syncthreads();
            int before = scratch[20];
            for (int w = 0; w < warp; ++w) before += scratch[w];
            const int end = before + x;
            start = end - v;
            if (round == 1 && v > 0 && my_s0 >= start && my_s0 < end) {
                scratch[21] = s;
                scratch[22] = start;
            }
            __syncthreads();
            if (threadIdx.x == kThreads - 1) scratch[20] = end;
            __syncthreads();
        }
        if (round == 0) {
            T = scratch[20];
            parts = split_parts(T, gridDim.x);
            __syncthreads();  // every thread has the total before the next round clears it
            if (threadIdx.x == 0) a.merges[blockIdx.x] = make_int4(0, 0, 0, 0);
            if (T == 0 || blockIdx.x >= parts) return;
            my_s0 = (int)((int64_t)blockIdx.x * T / parts);
            my_s1 = (int)(((int64_t)blockIdx.x + 1) * T / parts);
        }
    }
    const int s0 = my_s0, s1 = my_s1;
    if (a.num_seqs <= per_pass && v > 0 && s0 >= start && s0 < start + v) {
        scratch[21] = threadIdx.x / W;
        scratch[22] = start;
    }

    if (threadIdx.x == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], kGroupWarps);
            mbar_init(&q_ready[i], kGroupWarps);
            mbar_init(&o_last[i], 1);
            mbar_init(&o_free[i], ALT ? 2 * kGroupWarps : kGroupWarps);
            mbar_init(&xch_full[i], kGroupWarps);
        }
        for (int i = 0; i < kDescs; ++i) {
            mbar_init(&desc_full[i], 1);
            mbar_init(&desc_empty[i], 2 * kGroupWarps + 3);  // softmax warps, producers, MMA
        }
        for (int i = 0; i < 8; ++i) mbar_init(&pair[i], 2);
        mbar_init(fin, 1);
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t q_s = smem_u32(smem + L::q), k_s = smem_u32(smem + L::kring), v_s = smem_u32(smem + L::vring);

    if (warp >= 2 * kGroupWarps) {
        bool dead = false;
        if (warp == kSchedWarp) {
            // ======================= scheduler =======================
            int s = scratch[21];
            int t = s0;                 // next laid-out tile of the share
            int seq_start = scratch[22];  // laid-out start of sequence s
            int p = 0;
            while (t < s1 && !dead) {
                const Seq x = load_seq(a, s, false);
                const int fp = first_pos(a, x, s), nb = (x.Q + a.per_ctx - 1) / a.per_ctx;
                int per_kvh = 0;
                for (int b = lane; b < nb; b += 32) per_kvh += laid_out(ctx_tiles(a, x, fp, b).n);
#pragma unroll
                for (int sh = 16; sh > 0; sh >>= 1) per_kvh += __shfl_xor_sync(0xffffffffu, per_kvh, sh);
                for (int kvh = per_kvh > 0 ? (t - seq_start) / per_kvh : Hkv; kvh < Hkv && t < s1 && !dead; ++kvh) {
                    int pos = seq_start + kvh * per_kvh;  // laid-out start of block b0
                    for (int b0 = 0; b0 < nb && t < s1 && !dead; b0 += 32) {
                        CtxTiles c{};
                        if (b0 + lane < nb) c = ctx_tiles(a, x, fp, b0 + lane);
                        int end = laid_out(c.n);
#pragma unroll
                        for (int sh = 1; sh < 32; sh <<= 1) {
                            const int y = __shfl_up_sync(0xffffffffu, end, sh);
                            if (lane >= sh) end += y;
                        }
                        end += pos;
                        const int begin = end - laid_out(c.n);
                        // this lane's context: its real tiles [i0, i1) in the share
                        const int i0 = max(0, max(s0, begin) - begin - kCharge), i1 = min(s1, end) - begin - kCharge;
                        const bool mine = c.n > 0 && begin < s1 && end > s0 && i1 > i0;
                        for (uint32_t todo = __ballot_sync(0xffffffffu, mine); todo && !dead; todo &= todo - 1) {
                            const int d = p % kDescs;
                            if (lane == 0 && p >= kDescs)
                                wait_or_flag(&desc_empty[d], (uint32_t)((p / kDescs - 1) & 1), dead, a.err);
                            dead = __shfl_sync(0xffffffffu, dead, 0);
                            if (lane == __ffs(todo) - 1 && !dead) {
                                Piece pc;
                                pc.ntiles = i1 - i0;
                                pc.i0 = i0;
                                pc.np = c.np;
                                pc.pt0 = c.pt0;
                                pc.mt0 = c.mt0;
                                pc.seq = s;
                                pc.kvh = kvh;
                                const int q0 = (b0 + lane) * a.per_ctx;
                                pc.row0 = x.q0 + q0;
                                const int nq = min(x.Q - q0, a.per_ctx);
                                pc.nrows = nq * G;
                                pc.pos0 = fp + q0;
                                pc.ks0 = c.ks0;
                                pc.pre = x.pre;
                                pc.cpre = c.r.pre;
                                pc.lo = c.r.lo;
                                pc.hi = c.r.hi;
                                const bool begins = begin + kCharge >= s0, ends = end <= s1;
                                pc.slot = begins && ends ? -1 : 2 * (int)blockIdx.x + (begins ? 1 : 0);
                                if (begins && !ends)
                                    // the shares that hold the rest
                                    a.merges[blockIdx.x] = make_int4(
                                        (int)share_owner(end - 1, T, parts) - (int)blockIdx.x + 1, pc.row0, pc.nrows, kvh);
                                for (int g = 0; g < 2; ++g) {
                                    pc.jf[g] = ALT ? g : 0;
                                    pc.jl[g] = pc.ntiles - 1;
                                    if (ALT) continue;
                                    // tiles at either end that none of the group's rows can see a key of
                                    const int qa = min(nq - 1, g * kRows / G), qb = min(nq - 1, (g * kRows + kRows - 1) / G);
                                    const int glo = a.s.window > 0 ? pc.pos0 + qa - a.s.window + 1 : 0, ghi = pc.pos0 + qb + 1;
                                    auto idle = [&](int j) {
                                        const int t0 = key_tile(pc, j) * kTok;
                                        return t0 >= pc.pre && (t0 >= ghi || t0 + kTok <= glo);
                                    };
                                    if (pc.nrows <= g * kRows) pc.jl[g] = -1;
                                    while (pc.jl[g] >= 0 && idle(pc.jl[g])) --pc.jl[g];
                                    while (pc.jf[g] <= pc.jl[g] && idle(pc.jf[g])) ++pc.jf[g];
                                }
                                descs[d] = pc;
                                mbar_arrive(&desc_full[d]);
                            }
                            __syncwarp();
                            ++p;
                        }
                        pos = __shfl_sync(0xffffffffu, end, 31);
                        t = max(t, min(s1, pos));
                    }
                }
                seq_start += per_kvh * Hkv;
                t = max(t, min(s1, seq_start));
                ++s;
                if (s >= a.num_seqs) break;
            }
            if (lane == 0 && !dead) {
                const int d = p % kDescs;
                if (p >= kDescs) wait_or_flag(&desc_empty[d], (uint32_t)((p / kDescs - 1) & 1), dead, a.err);
                if (!dead) {
                    descs[d].ntiles = 0;
                    mbar_arrive(&desc_full[d]);
                }
            }
        } else if (warp == kKWarp || warp == kVWarp) {
            // ======================= producers =======================
            const bool isk = warp == kKWarp;
            const int N = isk ? NK : NV;
            uint64_t *full = isk ? k_full : v_full, *empty = isk ? k_empty : v_empty;
            const int bpt = kTok >> a.bshift;  // blocks per tile, at most 16
            int tau = 0;
            for (int p = 0; !dead; ++p) {
                const int d = p % kDescs;
                if (!wait_or_flag(&desc_full[d], (uint32_t)((p / kDescs) & 1), dead, a.err)) break;
                const Piece &pc = descs[d];
                const int n = pc.ntiles;
                if (n == 0) break;
                const int32_t *bt = a.block_tables + (int64_t)pc.seq * a.max_blocks;
                const KeyRange r{pc.ks0, pc.cpre, pc.lo, pc.hi};
                const int kvh = pc.kvh;
                // this lane's block of a tile: its id, INT_MIN where no row sees a key of it
                auto block_id = [&](int j) {
                    if (j >= n || lane >= bpt) return (int)INT_MIN;
                    const int t = key_tile(pc, j) * kTok + (lane << a.bshift);
                    return r.meets(t, t + B) ? (int)bt[t >> a.bshift] | (bt[t >> a.bshift] == INT_MIN ? 1 : 0) : INT_MIN;
                };
                int next = block_id(0);
                for (int j = 0; j < n; ++j, ++tau) {
                    const int st = tau % N;
                    const int id = next;
                    next = block_id(j + 1);
                    if (tau >= N && lane == 0) wait_or_flag(&empty[st], (uint32_t)((tau / N - 1) & 1), dead, a.err);
                    dead = __shfl_sync(0xffffffffu, dead, 0);
                    if (dead) break;
                    const bool live = id != INT_MIN, bad = live && (id < 0 || id >= a.num_blocks);
                    const uint32_t nlive = (uint32_t)__popc(__ballot_sync(0xffffffffu, live)), badm = __ballot_sync(0xffffffffu, bad);
                    if (lane == 0) {
                        if (isk) {
                            const int t0 = key_tile(pc, j) * kTok;
                            TileRec rec;
                            rec.t0 = t0;
                            rec.bad = badm;
                            rec.whole = badm == 0u && ((t0 >= r.lo && t0 + kTok <= r.hi) || (t0 >= r.first && t0 + kTok <= r.pre));
                            rec.pad = 0;
                            recs[tau % kRecs] = rec;
                            if (badm) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                        }
                        mbar_arrive_expect_tx(&full[st], nlive * (uint32_t)(H * 128) << a.bshift);
                    }
                    __syncwarp();
                    // an invalid id is read as block 0, its keys masked
                    const int y = live ? (int)(((int64_t)(bad ? 0 : id) * Hkv + kvh) * B) : -1;
                    if (isk) {
                        const uint32_t dst = k_s + st * L::kTile;
                        const int jb = lane / H, h = lane % H;
                        const int yb = __shfl_sync(0xffffffffu, y, jb);
                        if (jb < bpt && yb >= 0)
                            tma_load_2d(dst + h * (kTok * 128) + ((jb << a.bshift) * 128), &tm_k, smem_u32(&full[st]), h * 64, yb);
                    } else if (live) {
                        tma_load_3d(v_s + st * L::kTile + ((lane << a.bshift) * (H * 128)), &tm_v, smem_u32(&full[st]), 0, y, 0);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&desc_empty[d]);
            }
            // copies in flight (only after a timeout) land before the CTA exits
            if (lane == 0 && dead)
                for (int k = max(0, tau - N); k < tau; ++k) mbar_wait_bounded(&full[k % N], (uint32_t)((k / N) & 1));
        } else {
            // ======================= MMA issuer =======================
            // The whole warp walks (uniform registers), one elected lane issues.
            constexpr uint32_t idesc_qk = tc::instr_desc(kTok, false), idesc_pv = tc::instr_desc(D, true);
            const uint32_t pv_lbo = (uint32_t)(B * 128), pv_sbo = B >= 16 ? 1024u : (uint32_t)(H * B * 128);
            const bool leader = elect_one();
            const uint64_t qd0 = tc::smem_desc(q_s, 16, 1024), kd0 = tc::smem_desc(k_s, 16, 1024);
            const uint64_t vd0 = tc::smem_desc(v_s, pv_lbo, pv_sbo);
            // 16 keys of V further: inside a block of 32 every second step, else a block (B = 8: two)
            const uint32_t odd = B == 32 ? 16 * 128 >> 4 : (uint32_t)(H * 16 * 128) >> 4, two = (uint32_t)(2 * H * 16 * 128) >> 4;
            int tau = 0;
            int pend[2] = {-1, -1};             // tile whose P V the group still owes
            bool fresh[2] = {false, false};     // ... and it starts the piece's O
            bool owe_free[2] = {false, false};  // the previous piece's O may still be being read
            bool had[2] = {false, false};       // the previous piece had rows of the group
            int npv[2] = {0, 0}, nof[2] = {0, 0}, nqr[2] = {0, 0};  // phases passed: p_full, o_free, q_ready
            // the owed product; `closing`: and the end of the piece, everything issued: its softmax may read O
            auto finish = [&](int g, bool closing) {
                const int v = pend[g];
                if (v >= 0 && !dead) {
                    wait_or_flag(&p_full[g], (uint32_t)(npv[g] & 1), dead, a.err);
                    wait_or_flag(&v_full[v % NV], (uint32_t)((v / NV) & 1), dead, a.err);
                    if (fresh[g] && owe_free[g]) {
                        wait_or_flag(&o_free[g], (uint32_t)(nof[g] & 1), dead, a.err);
                        ++nof[g];
                        owe_free[g] = false;
                    }
                    if (dead) return;
                    tc::fence_after();
                    const uint64_t vd = vd0 + (uint64_t)((uint32_t)(v % NV) * (uint32_t)(L::kTile >> 4));
                    const uint32_t acc = fresh[g] ? 0u : 1u;
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < kTok / 16; ++k)
                            tc::mma_ts(tmem + kOBase + (uint32_t)g * D,
                                       tmem + (uint32_t)(g * kTok + (k < kHalf / 16 ? 8 * k : kHalf + 8 * k - kHalf / 2)),
                                       vd + (uint64_t)((uint32_t)(k >> 1) * two + (uint32_t)(k & 1) * odd), idesc_pv,
                                       k == 0 ? acc : 1u);
                        if (ALT) tc::commit(&v_empty[v % NV]);
                    }
                    __syncwarp();
                    ++npv[g];
                    pend[g] = -1;
                }
                if (!closing || !had[g]) return;
                if (owe_free[g]) {  // no product of the piece waited for it
                    wait_or_flag(&o_free[g], (uint32_t)(nof[g] & 1), dead, a.err);
                    ++nof[g];
                }
                owe_free[g] = true;
                if (leader) tc::commit(&o_last[g]);
                __syncwarp();
            };
            for (int p = 0; !dead; ++p) {
                const int d = p % kDescs;
                if (!wait_or_flag(&desc_full[d], (uint32_t)((p / kDescs) & 1), dead, a.err)) break;
                const int n = descs[d].ntiles, nrows = descs[d].nrows;
                if (n == 0) break;
                const int jf[2] = {descs[d].jf[0], descs[d].jf[1]}, jl[2] = {descs[d].jl[0], descs[d].jl[1]};
                bool started[2] = {false, false};
                for (int j = 0; j < n && !dead; ++j, ++tau) {
                    const int st = tau % NK;
                    bool open = j == 0 && p > 0;  // the previous piece is still to be closed
                    if (open && !mbar_test_wait(&k_full[st], (uint32_t)((tau / NK) & 1))) {
                        finish(0, true);  // rather than wait for this piece's keys first
                        finish(1, true);
                        open = false;
                    }
                    wait_or_flag(&k_full[st], (uint32_t)((tau / NK) & 1), dead, a.err);
                    const uint64_t kd = kd0 + (uint64_t)((uint32_t)st * (uint32_t)(L::kTile >> 4));
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const bool act = ALT ? (j & 1) == g : (j >= jf[g] && j <= jl[g]);
                        if (open || (j > 0 && (!ALT || act))) finish(g, open);
                        if (j == 0) {
                            had[g] = ALT || nrows > g * kRows;
                            if (had[g] && (!ALT || g == 0)) wait_or_flag(&q_ready[g], (uint32_t)(nqr[g]++ & 1), dead, a.err);
                        }
                        if (!act || dead) continue;
                        tc::fence_after();
                        const uint64_t qd = qd0 + (uint64_t)(ALT ? 0 : g * (L::kQTile >> 4));
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                const uint64_t off = (uint64_t)(((k >> 2) * (kTok * 128) + (k & 3) * 32) >> 4);
                                tc::mma(tmem + (uint32_t)g * kTok, qd + off, kd + off, idesc_qk, k > 0 ? 1u : 0u);
                            }
                            tc::commit(&s_full[g]);
                        }
                        __syncwarp();
                        pend[g] = tau;
                        fresh[g] = !started[g];
                        started[g] = true;
                    }
                    if (dead) break;
                    if (leader) tc::commit(&k_empty[st]);
                    if (!ALT && tau > 0) {  // both groups' products with the previous tile's V are issued
                        wait_or_flag(&v_full[(tau - 1) % NV], (uint32_t)(((tau - 1) / NV) & 1), dead, a.err);
                        if (leader) tc::commit(&v_empty[(tau - 1) % NV]);
                    }
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(&desc_empty[d]);
            }
            if (!dead) {
                finish(0, true);
                finish(1, true);
            }
            // every product has completed before the tensor memory is freed
            if (leader) tc::commit(fin);
            __syncwarp();
            mbar_wait_bounded(fin, 0u);
        }
    } else {
        // ======================= softmax =======================
        const int g = warp >> 3, hf = (warp >> 2) & 1, wq = warp & 3;
        const int rr = wq * 32 + lane;                // TMEM lane
        const int cr = ALT ? rr : g * kRows + rr;     // row of the context
        const uint32_t trow = tmem + ((uint32_t)(wq * 32) << 16);
        const uint32_t sp = trow + (uint32_t)(g * kTok + hf * kHalf);
        bool dead = false;
        int ns = 0;     // tiles of this group so far
        int npl = 0;    // pieces with rows of this group so far
        int nmeet = 0;  // meetings of the halves so far
        int tau0 = 0;
        // both halves of the warp's rows have come here
        auto meet_barrier = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&pair[g * 4 + wq]);
            wait_or_flag(&pair[g * 4 + wq], (uint32_t)(nmeet & 1), dead, a.err);
            ++nmeet;
        };
        auto slot = [&](int n, int h) -> float & { return xch[((n & 1) * 4 + g * 2 + h) * kRows + rr]; };
        auto copy_q = [&](const Piece &pc) {  // this thread's half of its row
            const bool live = cr < pc.nrows;
            const int row = pc.row0 + (live ? cr / G : 0), head = pc.kvh * G + cr % G;
            const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) + ((int64_t)row * a.num_heads + head) * D;
            const uint32_t base = q_s + (ALT ? 0u : (uint32_t)g * L::kQTile) + rr * 128;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const int k = hf * (D / 16) + i;
                const uint32_t dst = base + (k >> 3) * (kRows * 128) + (((k & 7) ^ (rr & 7)) << 4);
                if (live) cp_async16(dst, src + k * 8);
                else asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(dst), "r"(0u) : "memory");
            }
        };
        auto q_done = [&]() {
            cp_async_wait_all();
            fence_proxy_async();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_ready[ALT ? 0 : g]);
        };
        for (int p = 0; !dead; ++p) {
            const int d = p % kDescs;
            if (!wait_or_flag(&desc_full[d], (uint32_t)((p / kDescs) & 1), dead, a.err)) break;
            const Piece &pc = descs[d];
            const int n = pc.ntiles;
            if (n == 0) break;
            if (p == 0 && (ALT ? g == 0 : has_rows<ALT>(pc, g))) {
                copy_q(pc);
                q_done();
            }
            const bool live = cr < pc.nrows;
            // warps without rows only pass the barriers; the other rows of a warp with some go by the last query's keys,
            // so that they keep no tile from the path without masks
            const bool live_warp = (ALT ? 0 : g * kRows) + wq * 32 < pc.nrows;
            const int qi = min(cr, pc.nrows - 1) / G;
            const int64_t qrow = pc.row0 + qi;
            RowState st;
            st.m = KIND == kCap ? a.m0 : -INFINITY;
            st.l = 0.f;
            st.p = pc.pos0 + qi;
            st.r = key_range(max(pc.ks0, key_start_of(a.s, qrow)), pc.pre, a.s.window, st.p, st.p);
            st.slope2 = 0.f;
            if constexpr (KIND == kBias || KIND == kCapBias)
                st.slope2 = a.s.slopes ? a.s.slopes[pc.kvh * G + cr % G] * 1.44269504f : 0.f;
            // the next piece's queries, once this group's Q is free
            bool copied = false;
            auto next_q = [&]() {
                const int dn = (p + 1) % kDescs;
                if (!wait_or_flag(&desc_full[dn], (uint32_t)(((p + 1) / kDescs) & 1), dead, a.err)) return;
                const Piece &nx = descs[dn];
                if (nx.ntiles > 0 && has_rows<ALT>(nx, g)) {
                    copy_q(nx);
                    copied = true;
                }
            };
            const int jf = pc.jf[g], jl = pc.jl[g], pre = pc.pre;
            bool any = false;
            for (int j = jf; j <= jl; j += ALT ? 2 : 1) {
                const int tau = tau0 + j;
                wait_or_flag(&s_full[g], (uint32_t)(ns & 1), dead, a.err);
                if (dead) break;
                tc::fence_after();
                const TileRec rec = recs[tau % kRecs];
                const int t0 = rec.t0;
                const uint32_t bad = rec.bad;
                if (j == jl) next_q();  // every Q K^T on this Q has completed (ALT: the group of the piece's last tile copies)
                // V rows of keys that no row sees hold stale values, or none were loaded: zero weights must meet zeros
                if (!rec.whole) {
                    wait_or_flag(&v_full[tau % NV], (uint32_t)((tau / NV) & 1), dead, a.err);
                    const KeyRange r{pc.ks0, pc.cpre, pc.lo, pc.hi};
                    const uint32_t vb = v_s + (uint32_t)(tau % NV) * L::kTile;
                    for (int e = hf * kRows + rr; e < kTok * H * 8; e += 2 * kRows) {
                        const int key = (e >> 3) % kTok, h = e / (kTok * 8), chk = e & 7;
                        if (r.sees(t0 + key) && !((bad >> (key >> a.bshift)) & 1u)) continue;
                        const uint32_t row = vb + (key >> a.bshift) * (H * 128 << a.bshift) + h * (128 << a.bshift) +
                                             (key & (B - 1)) * 128;
                        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(row + chk * 16), "r"(0u) : "memory");
                    }
                    fence_proxy_async();
                }
                bool move = false;
                float alpha = 1.f;
                if (live_warp) {
                    softmax_half<KIND>(sp, t0 + hf * kHalf, bad >> (hf * (kHalf >> a.bshift)), a, t0 < pre, st, move, alpha, [&](float mt) {
                                           slot(ns, hf) = mt;
                                           meet_barrier();
                                           return fmaxf(mt, slot(ns, hf ^ 1));
                                       });
                }
                if (__any_sync(0xffffffffu, move)) {  // in both halves' warps alike: each takes half of the columns
                    const uint32_t ob = trow + kOBase + (uint32_t)(g * D + hf * (D / 2));
#pragma unroll 1
                    for (int c = 0; c < D / 64; ++c) {
                        float o[32];
                        tc::ld32(ob + c * 32, o);
                        tc::wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] *= alpha;
                        tc::st32(ob + c * 32, o);
                    }
                    tc::wait_st();
                }
                any = true;
                ++ns;
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[g]);
                if (copied) {  // after this tile's weights: Q for the next piece
                    q_done();
                    copied = false;
                }
            }
            if (dead) break;
            tau0 += n;
            // ---- the piece's result: the sums of a row's halves (ALT: and groups) meet, each thread writes its columns ----
            const int64_t orow = (qrow * a.num_heads + pc.kvh * G + cr % G) * D;
            if (ALT || has_rows<ALT>(pc, g)) {
                wait_or_flag(&o_last[g], (uint32_t)(npl & 1), dead, a.err);
                if (ALT) wait_or_flag(&o_last[g ^ 1], (uint32_t)(npl & 1), dead, a.err);
                tc::fence_after();
                // overwritten only after the next piece's products, which wait for all these reads (o_free)
                if (!any) st.m = -INFINITY;  // O holds nothing
                fin_ml[(g * 2 + hf) * kRows + rr] = make_float2(st.m, st.l);
                if constexpr (ALT) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&xch_full[g]);
                    wait_or_flag(&xch_full[0], (uint32_t)(npl & 1), dead, a.err);
                    wait_or_flag(&xch_full[1], (uint32_t)(npl & 1), dead, a.err);
                } else {
                    meet_barrier();
                }
                ++npl;
                if (dead) break;
                const float l_own = st.l + fin_ml[(g * 2 + (hf ^ 1)) * kRows + rr].y;
                float M = st.m, Ls = l_own, wm = 1.f, wo = 0.f;
                if constexpr (ALT) {
                    const float2 x0 = fin_ml[((g ^ 1) * 2) * kRows + rr], x1 = fin_ml[((g ^ 1) * 2 + 1) * kRows + rr];
                    M = fmaxf(st.m, x0.x);
                    wm = st.m == -INFINITY ? 0.f : ex2_approx(st.m - M);
                    wo = x0.x == -INFINITY ? 0.f : ex2_approx(x0.x - M);
                    Ls = l_own * wm + (x0.y + x1.y) * wo;
                } else if (st.m == -INFINITY) {
                    wm = 0.f;
                }
                const float inv = Ls != 0.f ? 1.f / Ls : 0.f;
                if (live_warp) {
                    constexpr int kCols = ALT ? D / 4 : D / 2;
                    const int col0 = (ALT ? g * 2 + hf : hf) * kCols;
#pragma unroll 1
                    for (int c = col0; c < col0 + kCols; c += 16) {
                        float o[16], x[16];
                        ld16(trow + kOBase + (uint32_t)(g * D + c), o);
                        if (ALT) ld16(trow + kOBase + (uint32_t)((g ^ 1) * D + c), x);
                        tc::wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) {  // a state without keys may hold anything
                            o[k] = wm != 0.f ? o[k] * wm : 0.f;
                            if (ALT && wo != 0.f) o[k] = fmaf(x[k], wo, o[k]);
                        }
                        if (!live) continue;
                        if (pc.slot < 0) {
                            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + orow + c);
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                dst[k] = make_uint4(pack_bf16x2(o[8 * k] * inv, o[8 * k + 1] * inv),
                                                    pack_bf16x2(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                                    pack_bf16x2(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                                                    pack_bf16x2(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
                        } else {
                            float *dst = a.part_o + ((int64_t)pc.slot * D + c) * (2 * kRows) + cr;
#pragma unroll
                            for (int k = 0; k < 16; ++k) dst[k * (2 * kRows)] = o[k];
                        }
                    }
                    if (live && pc.slot >= 0 && hf == 0 && (!ALT || g == 0))
                        reinterpret_cast<float2 *>(a.part_ml)[(int64_t)pc.slot * (2 * kRows) + cr] = make_float2(M, Ls);
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&o_free[g]);
                    if (ALT) mbar_arrive(&o_free[g ^ 1]);
                }
            }
            // No tile of this group in the piece: its Q was never read.  The next one is announced only now, after the MMA
            // thread has passed this piece's announcement (o_last), or there was none.
            if (!ALT && jl < jf) {
                next_q();
                if (copied) q_done();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&desc_empty[d]);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// The states of contexts cut by shares' borders, merged: CTA (c, k) takes rows
// 32 k .. of the context that share c begins and does not end; lanes are rows,
// the four warps quarters of the columns.  Part 0 is that share's last piece
// (slot 2 c + 1), part j the first piece of share c + j (slot 2 (c + j)).  The
// CTAs behind those zero the rows of contexts that see nothing (CTA = sequence).
template <int D>
__global__ void __launch_bounds__(128) scored_rows_merge_kernel(const __grid_constant__ RowsArgs a, int ctas) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int kPer = 2 * kRows / kMergeRows;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out);
    if ((int)blockIdx.x >= ctas * kPer) {
        const int s = blockIdx.x - ctas * kPer;
        const Seq x = load_seq(a, s, false);
        const int fp = first_pos(a, x, s), nb = (x.Q + a.per_ctx - 1) / a.per_ctx;
        for (int b = threadIdx.x; b < nb; b += 128) {
            if (ctx_tiles(a, x, fp, b).n > 0) continue;
            const int64_t q0 = x.q0 + (int64_t)b * a.per_ctx, n = min(x.Q - b * a.per_ctx, a.per_ctx);
            uint4 *row = reinterpret_cast<uint4 *>(out + q0 * a.num_heads * D);
            for (int64_t i = 0; i < n * a.num_heads * (D / 8); ++i) row[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    const int c = blockIdx.x / kPer, k = blockIdx.x % kPer;
    const int4 m = a.merges[c];
    const int lane = threadIdx.x & 31, cr = k * kMergeRows + lane;
    if (cr >= m.z || m.x == 0) return;
    constexpr int E = D / 4;
    const int col = (threadIdx.x >> 5) * E;
    auto slot = [&](int j) { return (int64_t)(j == 0 ? 2 * c + 1 : 2 * (c + j)); };
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml);
    float M = -INFINITY;
    for (int j = 0; j < m.x; ++j) M = fmaxf(M, ml[slot(j) * (2 * kRows) + cr].x);
    float L = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int j = 0; j < m.x; ++j) {
        const float2 x = ml[slot(j) * (2 * kRows) + cr];
        const float w = x.x == -INFINITY ? 0.f : ex2_approx(x.x - M);
        L += x.y * w;
        const float *src = a.part_o + (slot(j) * D + col) * (2 * kRows) + cr;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += w * src[(int64_t)e * (2 * kRows)];
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    uint4 *dst = reinterpret_cast<uint4 *>(out + ((int64_t)(m.y + cr / a.group) * a.num_heads + m.w * a.group + cr % a.group) * D + col);
#pragma unroll
    for (int e = 0; e < E / 8; ++e)
        dst[e] = make_uint4(pack_bf16x2(o[8 * e] * inv, o[8 * e + 1] * inv), pack_bf16x2(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                            pack_bf16x2(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                            pack_bf16x2(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
}

struct WsLayout {
    size_t o, ml, merges, total;
    explicit WsLayout(int D) {
        o = 0;
        ml = round256((size_t)2 * kMaxCtas * D * 2 * kRows * 4);
        merges = ml + round256((size_t)2 * kMaxCtas * 2 * kRows * 8);
        total = merges + round256((size_t)kMaxCtas * 16);
    }
};

template <int D, int KIND, bool ALT>
pkv_status launch(const RowsArgs &a, cudaStream_t st) {
    constexpr int smem = Layout<D, ALT>::total;
    static bool done[128] = {};
    auto kern = scored_rows_kernel<D, KIND, ALT>;
    if (!ensure_smem(kern, smem, done)) return PKV_ERR_CUDA;
    CUtensorMap mk, mv;
    const int64_t rows = (int64_t)a.num_blocks * a.num_kv_heads * a.block_size;
    if (!make_cache_map(&mk, a.k_cache, rows, D, a.block_size) || !make_slab_map(&mv, a.v_cache, rows, D, a.block_size))
        return PKV_ERR_CUDA;
    const int ctas = std::min(sm_count(), kMaxCtas);
    if (ctas < 1) return PKV_ERR_CUDA;
    pkv_status rc = launch_pdl(kern, dim3((unsigned)ctas), dim3(kThreads), smem, st, mk, mv, a);
    if (rc == PKV_OK)
        rc = launch_pdl(scored_rows_merge_kernel<D>, dim3((unsigned)(ctas * (2 * kRows / kMergeRows) + a.num_seqs)), dim3(128),
                        0, st, a, ctas);
    return rc;
}

template <int D, bool ALT>
pkv_status launch_kind(const RowsArgs &a, cudaStream_t st) {
    // a plain score's maximum is found before the scaling, which needs a positive scale
    const bool bias = a.s.slopes != nullptr;
    if (a.s.softcap > 0.f) return bias || a.c2 > kMaxC2 ? launch<D, kCapBias, ALT>(a, st) : launch<D, kCap, ALT>(a, st);
    return bias || !(a.s.scale > 0.f) ? launch<D, kBias, ALT>(a, st) : launch<D, kPlain, ALT>(a, st);
}

}  // namespace

size_t rows_workspace(int head_dim) { return WsLayout(head_dim).total; }

pkv_status run_rows(const Args &args, int head_dim, void *workspace, size_t workspace_bytes, cudaStream_t st) {
    const WsLayout lay(head_dim);
    if (!workspace || workspace_bytes < lay.total || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return PKV_ERR_INVALID;
    RowsArgs a{};
    static_cast<Args &>(a) = args;
    // the alternating form where no sequence has more rows than one group
    const bool alt = (int64_t)a.max_q_len * a.group <= kRows;
    a.per_ctx = (alt ? kRows : 2 * kRows) / a.group;
    a.bshift = a.block_size == 8 ? 3 : a.block_size == 16 ? 4 : 5;
    const int64_t blocks = ((int64_t)a.max_q_len + a.per_ctx - 1) / a.per_ctx;
    a.scan_w = 1;
    while (a.scan_w < 32 && a.scan_w < blocks) a.scan_w *= 2;
    // laid-out tiles are counted in 32-bit integers
    if ((int64_t)a.num_seqs * a.num_kv_heads > INT32_MAX / 2 / (blocks * ((a.max_seq_len + kTok - 1) / kTok + 1 + kCharge)))
        return PKV_ERR_UNSUPPORTED;
    const double log2e = 1.4426950408889634;
    a.k1 = a.s.softcap > 0.f ? (float)((double)a.s.scale / a.s.softcap) : (float)(a.s.scale * log2e);
    a.c2 = (float)(a.s.softcap * log2e);
    a.m0 = 0.25f * a.c2;
    double f = a.s.softcap * log2e * a.k1;
    for (int i = 0; i < 6; ++i, f *= (double)a.k1 * a.k1) {
        a.far[i] = (float)(kTanh5[i] * f);
        if (i < 4) a.near[i] = (float)(kTanh3[i] * f);
    }
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    a.part_o = reinterpret_cast<float *>(ws + lay.o);
    a.part_ml = reinterpret_cast<float *>(ws + lay.ml);
    a.merges = reinterpret_cast<int4 *>(ws + lay.merges);
    if (head_dim == 128) return alt ? launch_kind<128, true>(a, st) : launch_kind<128, false>(a, st);
    return alt ? launch_kind<64, true>(a, st) : launch_kind<64, false>(a, st);
}

}  // namespace scored
}  // namespace pkv
