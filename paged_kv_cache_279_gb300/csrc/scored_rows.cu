// Scored attention of several queries per sequence (prefill, chunks of one,
// verification of drafted tokens) on the 5th-generation tensor cores.
//
// Per KV head, the query heads of consecutive queries form up to 128 rows that
// meet the same 128-key tiles of the paged cache:
//     S = Q K^T (M 128 rows, N 128 keys, K head_dim)      scores, in tensor memory
//     P = 2^(y(S) - m)                                     y: the score in base 2, capped and biased
//     O += P V  (M 128, N head_dim, K 128 keys)
// with a reference m and a sum l per row.  m is the first 32 keys' maximum, rounded
// up to an integer, and moves only where a score passes it by more than kJump: what
// was summed is then scaled by a power of two, which rounds nothing.
//
// A context is one such set of rows and the tiles that some row sees: those of
// the always visible prefix, then those from the first row's window or document
// to the last row's position.  All contexts are laid end to end, each behind
// kCharge virtual tiles that stand for its fixed costs, and every CTA (one per
// SM) takes an equal share.  A context cut by a share's border leaves partial
// states (o, m, l) in the workspace, which a second kernel merges; no CTA waits
// for another.
//
// What bounds it is the softmax step between the two products (issue slots, the FMA
// pipe, instruction fetches and latency), so three tiles are in flight per SM: three
// S buffers, three sets of four warps (a thread per row = TMEM lane), tile t with set
// t % 3, one O.  Two chains of 128 x 128 tiles with an O each left the tensor cores
// idle between them (8 x 512 queries of 4096: 311 us; this form 252 to 274 us, with
// the tensor pipe 47 % and the issue slots 57 % busy, at the board's power limit in a
// long run).  What costs most is code size: the loops over a tile are
// rolled and their rare parts loops of their own; unrolled by two they took 6 to 13 %
// longer.
//
// Warps: 0-11 the softmax sets, 12-15 the epilogue (reads O at a context's end
// while the sets go on), 16 the issuer of Q K^T and 21 that of P V (one warp for
// both products was the bottleneck: 317 us, with two 283), 17 / 18 the producers of
// K (a column half each) and 19 of V (one TMA box per block), 20 the scheduler,
// which walks the share, publishes one descriptor per piece of a context and loads
// its queries (one box per column half).
// Infinities and NaN in V: P V multiplies them by the zero weights of rows that do not see
// their key, and 0 times infinity is NaN.  Nothing guards against that at first.  The epilogue
// looks at what it reads of O, and a CTA that met an infinity or NaN walks its share a second
// time, carefully: in tiles that not every row sees whole, the sets take infinities and NaN
// out of V, and the epilogue adds them to the rows that see their keys.  O may also have passed
// float32's range by itself (weights up to 2^kJump, under a cap 2^54, on very large V): in the
// second walk the references follow every score, so weights are at most 1.  The look costs 1 of
// 57 us (64 x 5 queries) and of 177 (prompts of documents); reading every such tile's V for them at
// once would cost each of them some 100 instructions a thread.  The second walk is code of its own
// (as a flag in the same code it took 2 to 3 % more).
//
// Tensor memory: S at columns 128 (t % 3) (P overwrites its first half as bf16
// pairs), O at 384.
// Every wait is bounded; one that gives up flags PKV_DEVERR_TIMEOUT.
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "pkv_internal.cuh"
#include "scored.cuh"

namespace pkv {
namespace scored {
namespace {

constexpr int kTok = 128;   // keys per tile
constexpr int kRows = 128;  // rows of a context
constexpr int kSets = 3;    // softmax sets and S buffers
constexpr int kEpiWarp = 4 * kSets, kMmaWarp = 16, kKWarp = 17, kVWarp = 19, kSchedWarp = 20, kPvWarp = 21;
constexpr int kThreads = 22 * 32;
constexpr int kDescs = 6;   // piece descriptors in flight
constexpr int kRecs = 8;    // tile records (more than the K producers can be ahead of the softmax)
constexpr int kCharge = 1;  // virtual tiles of a context (prompts of documents: 1: 170 us, 2: 180, 3: 194)
constexpr int kMinShare = kCharge + 1;
constexpr float kJump = 32.f;  // a row's reference moves where a score passes it by more (weights stay below 2^kJump)
constexpr float kMaxC2 = kWideCap;  // softcap * log2 e up to which capped scores take a fixed reference (cap 50)
constexpr uint32_t kTmemCols = 512, kOBase = kSets * kTok;
constexpr int kMaxCtas = 160;   // partial slots in the workspace: two per CTA
constexpr int kMergeRows = 32;  // rows per CTA of the merge kernel

enum Kind { kPlain = 0, kCap = 1, kBias = 2, kCapBias = 3 };

struct RowsArgs : Args {
    float k1;       // plain, biased: scale * log2 e; capped: scale / softcap
    float c2;       // capped: softcap * log2 e
    float m0;       // capped: the reference
    float near[4];  // capped: c2 tanh(k1 s) = s * sum near[i] s^2i for |k1 s| <= near_max (kTanhNear; wide caps: kTanhSmall)
    float near_max;
    float *part_o;  // [2 kMaxCtas][D][kRows]: columns of rows
    float *part_ml; // [2 kMaxCtas][kRows][2]
    int4 *merges;   // [kMaxCtas]: (parts, first query row, rows, kv head) of the context begun and cut in that share
    int bshift, per_ctx, scan_w;  // log2 block size, queries per context, lanes per sequence in the scan
};

struct Piece {
    int ntiles;  // 0: no more
    int i0;      // first tile within the context
    int np, pt0, mt0;   // context tile i is key tile pt0 + i (i < np) or mt0 + i - np
    int seq, kvh, row0, nq, nrows, pos0, pre;
    int ks0, cpre, lo, hi;  // the context's keys: [ks0, cpre) and [lo, hi) (KeyRange)
    int fks, flo, fhi;      // keys that every row sees: [flo, fhi) and [fks, pre)
    int slot;               // partial slot, -1: the whole context
};

// A tile's record, written by the first K producer.
struct TileRec {
    int t0;        // first key
    uint32_t bad;  // bits of blocks with an invalid id (their keys are masked)
    int whole;     // every key is seen by some row: no V row has to be zeroed
    int full;      // every key is seen by every row
};

template <int D>
struct Layout {
    static constexpr int H = D / 64;
    static constexpr int kQTile = H * kRows * 128;
    static constexpr int kTile = H * kTok * 128;  // K or V of one tile
    static constexpr int NK = D == 128 ? 2 : 4;
    static constexpr int NV = D == 128 ? 2 : 4;
    static constexpr int q = 0;                         // two tiles of queries
    static constexpr int kring = q + 2 * kQTile;
    static constexpr int vring = kring + NK * kTile;
    static constexpr int fin_ml = vring + NV * kTile;   // float2 [2][kSets][kRows]: (m, l) of a piece's rows, pieces in turn
    static constexpr int mref = fin_ml + 2 * kSets * kRows * 8;  // float [kRows]: the rows' reference after the latest tile
    // float [4][kRows]: the first tile's, pieces in turn (three would do: the tile that last reads piece p - 3's is the third
    // before piece p's first at the latest, and done when that one begins)
    static constexpr int start = mref + kRows * 4;
    static constexpr int desc = start + 4 * kRows * 4;
    static constexpr int recs = (desc + kDescs * (int)sizeof(Piece) + 15) & ~15;
    static constexpr int bars = recs + kRecs * (int)sizeof(TileRec);
    static constexpr int kBars = 2 * NK + 2 * NV + 3 * kSets + 4 * kSets + 4 + 2 + 4 + 16 + 2 * kDescs + 2;
    static constexpr int misc = bars + kBars * 8;       // TMEM address, scan scratch
    static constexpr int redo = misc + 124;             // an output was infinite or NaN
    static constexpr int fin_bad = misc + 128;          // [2][4 kSets]: per warp, V entries taken out of a piece's tiles
    static constexpr int total = fin_bad + 2 * 4 * kSets * 4;
    static_assert(total <= 227 * 1024, "shared memory per CTA");
};

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0u;
}

__device__ __forceinline__ void mbar_inval(uint64_t *bar) {
    asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void prefetch_l1(const void *p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// Waits are many and rarely long: kept to a few instructions, and one that gives up sets `dead` (then no other waits), which
// the kernel's end reports.
__device__ __forceinline__ bool drain(uint64_t *bar, uint32_t parity) {
    uint32_t i = 0;
#pragma unroll 1
    while (!mbar_try_wait(bar, parity))
        if (++i == kWaitLimit) return false;
    return true;
}
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, bool &dead) {
    if (!dead) dead = !drain(bar, parity);
    return !dead;
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

// The T laid-out tiles cut into equal shares, share c = [floor(c T / n), floor((c + 1) T / n)), in 32-bit steps
// (T = each * n + rest).
struct Shares {
    int n, each, rest;
    __device__ __forceinline__ Shares(int T, int ctas) {
        n = min(ctas, max(T / kMinShare, 1));
        each = T / n;
        rest = T - each * n;
    }
    __device__ __forceinline__ int begin(int c) const { return c * each + (int)((uint32_t)(c * rest) / (uint32_t)n); }
    __device__ __forceinline__ int owner(int t) const {  // the share that holds tile t
        int c = min(n - 1, t / each);
#pragma unroll 1
        while (begin(c) > t) --c;
        return c;
    }
};

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

__device__ __forceinline__ void ld4(uint32_t taddr, float (&v)[4]) {
    uint32_t r[4];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void st4(uint32_t taddr, const float (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(__float_as_uint(v[0])),
                 "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3]))
                 : "memory");
}

// tanh z / z as a polynomial in z^2: least squares of the error of tanh, reweighted towards its largest (Lawson's method),
// in 64 bits.  |z| <= 0.75: off by at most 3.7e-6 of the cap, so 2e-4 of a score at a cap of 50, where the weight's
// rounding to bf16 is worth 2e-3 to 4e-3.
constexpr float kTanhNear = 0.75f;
constexpr double kTanh3[4] = {0.9999556008, -0.3322276376, 0.1257709249, -0.03377828486};

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// bits [a, b) of a 32-bit word, a and b taken from any integers (shl gives 0 from 32 on)
__device__ __forceinline__ uint32_t bits_from(int a) {
    uint32_t m;
    asm("shl.b32 %0, %1, %2;" : "=r"(m) : "r"(0xffffffffu), "r"(max(a, 0)));
    return m;
}
__device__ __forceinline__ uint32_t bit_range(int a, int b) { return bits_from(a) & ~bits_from(b); }

struct RowState {
    float m, l;    // reference and sum
    int p;         // position
    KeyRange r;
    float slope2;  // slope * log2 e
};

constexpr int kStep = 32;  // keys a step

// Maximum over a step's values, four chains of three-input maxima; ABS: of their magnitudes.
template <bool ABS>
__device__ __forceinline__ float max_of(const float (&s)[kStep]) {
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = ABS ? fabsf(s[i]) : s[i];
#pragma unroll
        for (int k = i + 4; k + 4 < kStep; k += 8)
            m[i] = ABS ? fmax3(m[i], fabsf(s[k]), fabsf(s[k + 4])) : fmax3(m[i], s[k], s[k + 4]);
        m[i] = fmaxf(m[i], ABS ? fabsf(s[kStep - 4 + i]) : s[kStep - 4 + i]);
    }
    return fmaxf(fmax3(m[0], m[1], m[2]), m[3]);
}

__device__ __forceinline__ void ld_s(uint32_t taddr, float (&v)[kStep]) {
    tc::ld32(taddr, v);
    tc::wait_ld();
}

// The keys of step c of the tile at t0 that the row sees, as bits.
__device__ __forceinline__ uint32_t seen_bits(const KeyRange &r, int t0, uint32_t bad, int bshift, int c) {
    const int t = t0 + kStep * c;
    uint32_t w = bit_range(r.lo - t, r.hi - t);
    if (r.pre > t) w |= bit_range(r.first - t, r.pre - t);
    if (bad) {
#pragma unroll
        for (int i = 0; i < kStep; i += 8)
            if ((bad >> ((kStep * c + i) >> bshift)) & 1u) w &= ~(0xffu << i);
    }
    return w;
}

__device__ __forceinline__ void mask_s(float (&s)[kStep], uint32_t w, float hidden = -INFINITY) {
#pragma unroll
    for (int k = 0; k < kStep; ++k) s[k] = (w >> k) & 1u ? s[k] : hidden;
}

__device__ __forceinline__ void no_weights(uint32_t to) {
    const uint32_t z[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < kStep / 2; i += 8) st8u(to + i, z);
}

// Raw products of kStep keys (at sp) -> scores in base 2 plus nm: c tanh(z) + nm, z = k1 s.  For |z| small in the whole warp
// an odd polynomial (the cap's factors folded in on the host) on the FMA pipe, two keys an instruction: the exponential is
// then the only special function of a score.  Else, in a loop to keep the code short,
// tanh z = 1 - 2 / (1 + e^2z), good to 2^-21; the scores go back over S.  Under a wide cap
// (WIDE: there may be one) small z take the series there too: what other rows reach must not
// cost them accuracy.
__device__ __forceinline__ void cap_near(float (&s)[kStep], const RowsArgs &a, uint64_t nm2) {
    const uint64_t q0 = f32x2(a.near[0], a.near[0]), q1 = f32x2(a.near[1], a.near[1]);
    const uint64_t q2 = f32x2(a.near[2], a.near[2]), q3 = f32x2(a.near[3], a.near[3]);
#pragma unroll
    for (int k = 0; k < kStep; k += 2) {
        const uint64_t x = f32x2(s[k], s[k + 1]), u = mul_f32x2(x, x);
        const uint64_t y = fma_f32x2(fma_f32x2(fma_f32x2(q3, u, q2), u, q1), u, q0);
        f32x2_split(fma_f32x2(x, y, nm2), s[k], s[k + 1]);
    }
}

template <bool WIDE>
__device__ __forceinline__ void cap_far(float (&s)[kStep], uint32_t sp, const RowsArgs &a, float nm) {
    const float z2 = 2.f * 1.44269504f * a.k1, small = WIDE && a.c2 > kWideCap ? kTanhSmall : 0.f;
    constexpr float s1 = (float)kTanhSeries[1], s2 = (float)kTanhSeries[2], s3 = (float)kTanhSeries[3];
#pragma unroll 1
    for (int i = 0; i < kStep / 4; ++i) {
        float x[4];
        ld4(sp + 4 * i, x);
        tc::wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float far = (a.c2 + nm) - (2.f * a.c2) * rcp_approx(1.f + ex2_approx(x[k] * z2));
            if constexpr (WIDE) {
                const float z = x[k] * a.k1, u = z * z;
                x[k] = fabsf(z) < small ? fmaf(a.c2 * z, fmaf(fmaf(fmaf(s3, u, s2), u, s1), u, 1.f), nm) : far;
            } else {
                x[k] = far;
            }
        }
        st4(sp + 4 * i, x);
    }
    tc::wait_st();
    ld_s(sp, s);
}

template <bool WIDE>
__device__ __forceinline__ void cap_s(float (&s)[kStep], uint32_t sp, const RowsArgs &a, float nm, uint64_t nm2) {
    const float top = max_of<true>(s) * fabsf(a.k1);
    cap_near(s, a, nm2);
    if (__builtin_expect(__any_sync(0xffffffffu, top > a.near_max), 0)) cap_far<WIDE>(s, sp, a, nm);
}

// Raw products of kStep keys at sp, the first `ahead` keys before the row's position -> scores in base 2 plus nm.  beyond: keys
// past the position may be seen.
template <int KIND>
__device__ __forceinline__ void scores(float (&s)[kStep], uint32_t sp, int ahead, float slope2, bool beyond, const RowsArgs &a, float nm,
                                       bool full, uint32_t w) {
    ld_s(sp, s);
    if constexpr (KIND == kCapBias) {
        if (!full) mask_s(s, w, 0.f);  // what is hidden has no say in how the others are capped
        cap_s<true>(s, sp, a, 0.f, 0ull);
    }
    const float f = KIND == kCapBias ? 1.f : a.k1;
    const uint64_t f2 = f32x2(f, f), nm2 = f32x2(nm, nm);
    if constexpr (KIND == kPlain) {
#pragma unroll
        for (int k = 0; k < kStep; k += 2) f32x2_split(fma_f32x2(f32x2(s[k], s[k + 1]), f2, nm2), s[k], s[k + 1]);
    } else {
        // -slope |ahead - k|, linear unless the position is inside: one FMA for the pair's bias, one for the score
        const float sl = beyond && ahead <= 0 ? -slope2 : slope2, b = fmaf(-sl, (float)ahead, nm);
        if (__builtin_expect(beyond && __any_sync(0xffffffffu, ahead > 0 && ahead < kStep - 1), 0)) {
            if (KIND == kCapBias) {  // capped scores over S
#pragma unroll
                for (int i = 0; i < kStep; i += 4) st4(sp + i, reinterpret_cast<const float(&)[4]>(s[i]));
                tc::wait_st();
            }
#pragma unroll 1
            for (int i = 0; i < kStep / 4; ++i) {
                float x[4];
                ld4(sp + 4 * i, x);
                tc::wait_ld();
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = fmaf(-slope2, fabsf((float)(ahead - 4 * i - k)), fmaf(x[k], f, nm));
                st4(sp + 4 * i, x);
            }
            tc::wait_st();
            ld_s(sp, s);
            return;
        }
        const uint64_t b2 = f32x2(b, b), sl2 = f32x2(sl, sl);
#pragma unroll
        for (int k = 0; k < kStep; k += 2)
            f32x2_split(fma_f32x2(f32x2(s[k], s[k + 1]), f2, fma_f32x2(sl2, f32x2((float)k, (float)(k + 1)), b2)), s[k], s[k + 1]);
    }
}

// a += low half, b += high half of a pair of bf16 (mixed adds: 2 % of the call less than widening first).
__device__ __forceinline__ void add_bf16x2(float &a, float &b, uint32_t v) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tadd.f32.bf16 %0, lo, %0;\n\tadd.f32.bf16 %1, hi, %1;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(v));
}

// Weights 2^s of kStep keys to P (bf16 pairs) at `to`, the sum of the rounded ones to ls: a row that one key dominates gets its
// value exactly.
__device__ __forceinline__ void weights(const float (&s)[kStep], uint32_t to, uint64_t (&ls)[2]) {
#pragma unroll
    for (int i = 0; i < kStep; i += 16) {
        float lf[4];
        f32x2_split(ls[0], lf[0], lf[1]);
        f32x2_split(ls[1], lf[2], lf[3]);
        uint32_t pk[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            pk[k] = pack_bf16x2(ex2_approx(s[i + 2 * k]), ex2_approx(s[i + 2 * k + 1]));
            add_bf16x2(lf[2 * (k & 1)], lf[2 * (k & 1) + 1], pk[k]);
        }
        st8u(to + i / 2, pk);
        ls[0] = f32x2(lf[0], lf[1]);
        ls[1] = f32x2(lf[2], lf[3]);
    }
}

// The rows' reference over the tiles of a piece, handed from tile to tile.
struct Chain {
    float *mref;        // this row's after the tile before
    float *start;       // this row's reference as the piece's first tile began
    uint64_t *started;  // that is known
    uint32_t start_parity;
    uint64_t *before;   // the tile before has left its reference (nullptr: the CTA's first tile)
    uint64_t *mine;     // this tile has
    uint64_t *done;     // the tile before's product is complete
    uint32_t parity;    // of both
    bool first;         // the piece's first tile
    bool begun;         // this set has had a tile of the piece: its state has a reference
};

// The first 16 n weights at `to` times f, a power of two.
__device__ __forceinline__ void rescale_weights(uint32_t to, int n, float f) {
    tc::wait_st();
#pragma unroll 1
    for (int c = 0; c < 2 * n; ++c) {
        float w[4];
        ld4(to + 4 * c, w);
        tc::wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t u = __float_as_uint(w[k]);
            w[k] = __uint_as_float(pack_bf16x2(__uint_as_float(u << 16) * f, __uint_as_float(u & 0xffff0000u) * f));
        }
        st4(to + 4 * c, w);
    }
}

// One tile of one row, 32 keys at a time in loops that are not unrolled: more code
// than that ran at the pace of its instruction fetches (all 128 keys unrolled: 6 to 10
// cycles an instruction), and 16 keys at a time wait longer for their own results
// (prompts of documents: 203 us, with 32 176 us).  S (raw products) at sp, P (bf16
// pairs) back over its first 64 columns, always behind the reads.  beyond: some row
// may see keys past its position (a prefix).  Steps that no row of the warp sees are
// skipped.
//
// One pass: a score goes straight to its weight 2^(y - m).  m is the reference that
// this set's tile before left, for its first tile of a piece the one that the piece's
// first tile found in its first step, the maximum of the keys seen there.  Where a score
// passes m by more than kJump, m moves to it, and the tile's earlier weights are
// scaled.  At the end the tile before's final reference is awaited and the larger
// of the two taken: this tile's weights or O (complete up to the tile before) are
// rescaled where theirs was another.  Rounded up to integers, references seldom
// differ, and scaling is exact.
//
// Capped scores without a bias need none of this: they lie within +-c2, and up to
// kMaxC2 a fixed reference c2 / 4 keeps weights within 2^-(5/4 c2) .. 2^(3/4 c2)
// (cap 50: 2^-90 .. 2^54), far from the ends of float32's and bf16's range for
// sums over 2^20 keys of V entries between 2^-36 and 2^53 (larger ones: the second walk).
//
// CLOSE: the reference follows every score that passes it (the second walk).
template <int D, int KIND, bool CLOSE>
__device__ __forceinline__ void softmax_tile(uint32_t sp, uint32_t op, const TileRec &rec, const RowsArgs &a, bool beyond,
                                             RowState &st, const Chain &ch, int lane, bool &dead) {
    const int t0 = rec.t0;
    const bool full = rec.full != 0;
    uint64_t ls[2] = {0ull, 0ull};
    float x[kStep];
    if constexpr (KIND == kCap) {
        const float nm = -st.m;
        const uint64_t nm2 = f32x2(nm, nm);
        // (a loop for tiles that every row sees whole: the shorter, the faster)
        if (full) {
#pragma unroll 1
            for (int c = 0; c < kTok / kStep; ++c) {
                ld_s(sp + kStep * c, x);
                cap_s<false>(x, sp + kStep * c, a, nm, nm2);
                weights(x, sp + kStep / 2 * c, ls);
            }
        } else {
#pragma unroll 1
            for (int c = 0; c < kTok / kStep; ++c) {
                const uint32_t w = seen_bits(st.r, t0, rec.bad, a.bshift, c);
                if (!__any_sync(0xffffffffu, w != 0u)) {
                    no_weights(sp + kStep / 2 * c);
                    continue;
                }
                ld_s(sp + kStep * c, x);
                mask_s(x, w, 0.f);  // what is hidden has no say in how the others are capped
                cap_s<false>(x, sp + kStep * c, a, nm, nm2);
                mask_s(x, w);
                weights(x, sp + kStep / 2 * c, ls);
            }
        }
    } else {
        constexpr float jump = CLOSE ? 0.f : kJump;
        // what a tile begins with depends on no other's pace, so results do not either
        float m = -INFINITY;
        bool unknown = ch.first;
        if (ch.begun) {
            m = st.m;
        } else if (!ch.first) {
            wait_for(ch.started, ch.start_parity, dead);
            m = *ch.start;
        }
        auto publish = [&] {
            *ch.start = m;
            __syncwarp();
            if (lane == 0) mbar_arrive(ch.started);
            unknown = false;
        };
        float nm = m == -INFINITY ? 0.f : -m, top = m == -INFINITY ? -INFINITY : jump;
#pragma unroll 1
        for (int c = 0; c < kTok / kStep; ++c) {
            uint32_t w = 0xffffffffu;
            if (!full) {
                w = seen_bits(st.r, t0, rec.bad, a.bshift, c);
                if (!__any_sync(0xffffffffu, w != 0u)) {
                    no_weights(sp + kStep / 2 * c);
                    continue;
                }
            }
            scores<KIND>(x, sp + kStep * c, st.p - t0 - kStep * c, st.slope2, beyond, a, nm, full, w);
            if (!full) mask_s(x, w);
            const float mc = max_of<false>(x);
            if (__builtin_expect(__any_sync(0xffffffffu, mc > top), 0)) {
                const float up = mc > top ? ceilf(mc) : 0.f;  // relative to the reference so far
                const float f = m == -INFINITY ? 1.f : ex2_approx(-up);  // (no weight so far but 0)
                if (__any_sync(0xffffffffu, f != 1.f)) rescale_weights(sp, kStep / 16 * c, f);
                ls[0] = mul_f32x2(ls[0], f32x2(f, f));
                ls[1] = mul_f32x2(ls[1], f32x2(f, f));
#pragma unroll
                for (int k = 0; k < kStep; ++k) x[k] -= up;
                if (mc > top) {
                    m = up - nm;
                    nm = -m;
                    top = jump;
                }
                if (unknown) publish();
            }
            weights(x, sp + kStep / 2 * c, ls);
        }
        if (unknown) publish();
        // the tile before's reference
        if (ch.before) wait_for(ch.before, ch.parity, dead);
        const float old = ch.first ? -INFINITY : *ch.mref, mf = fmaxf(old, m);
        *ch.mref = mf;
        __syncwarp();
        if (lane == 0) mbar_arrive(ch.mine);
        const float f = m == -INFINITY || m == mf ? 1.f : ex2_approx(m - mf);
        if (__any_sync(0xffffffffu, f != 1.f)) {
            rescale_weights(sp, kTok / 16, f);
            ls[0] = mul_f32x2(ls[0], f32x2(f, f));
            ls[1] = mul_f32x2(ls[1], f32x2(f, f));
        }
        if (st.m != mf) {
            st.l = st.m == -INFINITY ? st.l : st.l * ex2_approx(st.m - mf);
            st.m = mf;
        }
        const bool move = old != -INFINITY && mf != old;
        if (__any_sync(0xffffffffu, move)) {
            wait_for(ch.done, ch.parity, dead);
            tc::fence_after();
            const float alpha = move ? ex2_approx(old - mf) : 1.f;
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
                float o[16];
                ld16(op + c * 16, o);
                tc::wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] *= alpha;
                st16u(op + c * 16, reinterpret_cast<const uint32_t(&)[16]>(o));
            }
        }
    }
    float l0, l1;
    f32x2_split(add_f32x2(ls[0], ls[1]), l0, l1);
    st.l += l0 + l1;
    tc::wait_st();
}

// ---------------------------------------------------------------------------
// Infinities and NaN in V
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool odd_lo(uint32_t v) { return (v & 0x7f80u) == 0x7f80u; }
__device__ __forceinline__ bool odd_hi(uint32_t v) { return (v & 0x7f800000u) == 0x7f800000u; }

// Zeroes the infinities and NaN of the V row at `row` (halves `half` bytes apart); true where there were some.
template <int H>
__device__ __noinline__ bool clean_row(uint32_t row, uint32_t half, int lane) {
    bool any = false;
#pragma unroll 1
    for (int i = 0; i < 8 * H; ++i) {
        const uint32_t at = row + (uint32_t)(i >> 3) * half + (uint32_t)((i + lane) & 7) * 16;
        const float4 f = lds128(at);
        uint32_t v[4] = {__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(f.z), __float_as_uint(f.w)};
        bool odd = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            odd = odd || odd_lo(v[k]) || odd_hi(v[k]);
            if (odd_lo(v[k])) v[k] &= 0xffff0000u;
            if (odd_hi(v[k])) v[k] &= 0xffffu;
        }
        if (odd)
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
        any = any || odd;
    }
    return any;
}

// Adds the infinities and NaN of V to the O of the rows (of this warp; a lane's sees r) that see their keys, over the tiles
// of a piece from which the sets took them.  op: O of the warp's rows.  A row none of whose outputs is finite any more is
// done, which bounds the time where everything is NaN.
template <int D>
__device__ __noinline__ void add_odd_values(const RowsArgs &a, const Piece &pc, const KeyRange r, uint32_t op, int lane) {
    const int32_t *bt = a.block_tables + (int64_t)pc.seq * a.max_blocks;
    const int B = a.block_size;
    bool done = false;
#pragma unroll 1
    for (int i = pc.i0; i < pc.i0 + pc.ntiles; ++i) {
        const int t0 = (i < pc.np ? pc.pt0 + i : pc.mt0 + i - pc.np) * kTok;
        if ((t0 >= pc.flo && t0 + kTok <= pc.fhi) || (t0 >= pc.fks && t0 + kTok <= pc.pre)) continue;  // every row sees it
#pragma unroll 1
        for (int c = 0; c < kTok; c += 32) {
            // a lane a key: its V row, and whether it holds any
            const int t = t0 + c + lane;
            const KeyRange cr{pc.ks0, pc.cpre, pc.lo, pc.hi};
            int64_t row = -1;
            bool odd = false;
            if (cr.sees(t)) {
                const int blk = bt[t >> a.bshift];
                if (blk >= 0 && blk < a.num_blocks) row = ((int64_t)blk * a.num_kv_heads + pc.kvh) * B + (t & (B - 1));
            }
            if (row >= 0) {
                const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.v_cache) + row * D);
#pragma unroll 4
                for (int k = 0; k < D / 8; ++k) {
                    const uint4 x = v[k];
                    odd = odd || odd_lo(x.x) || odd_hi(x.x) || odd_lo(x.y) || odd_hi(x.y) || odd_lo(x.z) || odd_hi(x.z) ||
                          odd_lo(x.w) || odd_hi(x.w);
                }
            }
#pragma unroll 1
            for (uint32_t todo = __ballot_sync(0xffffffffu, odd); todo; todo &= todo - 1) {
                const int k = __ffs(todo) - 1;
                const bool mine = !done && r.sees(t0 + c + k);
                if (!__any_sync(0xffffffffu, mine)) continue;
                const uint32_t *v = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(a.v_cache) +
                                                                       __shfl_sync(0xffffffffu, row, k) * D);
                bool finite = false;
#pragma unroll 1
                for (int d = 0; d < D; d += 16) {
                    uint32_t x[8];
                    bool some = false;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        x[j] = v[d / 2 + j];
                        some = some || odd_lo(x[j]) || odd_hi(x[j]);
                    }
                    finite = finite || !some;
                    if (!some) continue;  // (the same in every lane)
                    float o[16];
                    ld16(op + (uint32_t)d, o);
                    tc::wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (mine && odd_lo(x[j])) o[2 * j] += bf16x2_lo(x[j]);
                        if (mine && odd_hi(x[j])) o[2 * j + 1] += bf16x2_hi(x[j]);
                        finite = finite || fabsf(o[2 * j]) < INFINITY || fabsf(o[2 * j + 1]) < INFINITY;
                    }
                    st16u(op + (uint32_t)d, reinterpret_cast<const uint32_t(&)[16]>(o));
                    tc::wait_st();
                }
                done = done || !finite;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <int D, int KIND>
__global__ void __launch_bounds__(kThreads, 1)
scored_rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ RowsArgs a) {
    using L = Layout<D>;
    constexpr int H = L::H, NK = L::NK, NV = L::NV;
    extern __shared__ __align__(1024) unsigned char smem[];
    Piece *descs = reinterpret_cast<Piece *>(smem + L::desc);
    TileRec *recs = reinterpret_cast<TileRec *>(smem + L::recs);
    float2 *fin_ml = reinterpret_cast<float2 *>(smem + L::fin_ml);
    float *mref = reinterpret_cast<float *>(smem + L::mref);
    float *start_ref = reinterpret_cast<float *>(smem + L::start);
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + L::bars), *k_empty = k_full + NK;
    uint64_t *v_full = k_empty + NK, *v_empty = v_full + NV;
    uint64_t *s_full = v_empty + NV, *p_full = s_full + kSets, *o_done = p_full + kSets;  // per set
    uint64_t *m_full = o_done + kSets;                                                   // [set][4]: per warp
    uint64_t *q_full = m_full + 4 * kSets, *q_empty = q_full + 2;                        // per query tile
    uint64_t *o_last = q_empty + 2, *o_free = o_last + 1;
    uint64_t *fin_full = o_free + 1, *fin_empty = fin_full + 2;                          // pieces in turn
    uint64_t *started = fin_empty + 2;                                                   // [piece % 4][4]: per warp
    uint64_t *desc_full = started + 16, *desc_empty = desc_full + kDescs, *all_done = desc_empty + kDescs;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::misc);
    int *scratch = reinterpret_cast<int *>(smem + L::misc + 16);  // [22] warp sums, carry, found sequence, its start
    volatile int *redo = reinterpret_cast<int *>(smem + L::redo), *fin_bad = reinterpret_cast<int *>(smem + L::fin_bad);
    constexpr int kCarry = kThreads / 32, kFound = kCarry + 1, kStart = kCarry + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int Hkv = a.num_kv_heads, G = a.group, B = a.block_size;

    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_q)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
    }
    if ((smem_u32(smem) & 1023u) != 0u) {  // swizzled tiles need it; never expected
        if (threadIdx.x == 0) flag_error(a.err, PKV_DEVERR_TIMEOUT);
        return;
    }

    // ---- scan: laid-out tiles of every sequence; scan_w lanes share one (of 640 threads: whole groups of lanes) ----
    const int W = a.scan_w, per_pass = 640 / W, sub = threadIdx.x % W;
    auto seq_total = [&](int s, bool report) {
        int t = 0;
        if (s < a.num_seqs) {
            const Seq x = load_seq(a, s, report && sub == 0);
            const int fp = first_pos(a, x, s), nb = (x.Q + a.per_ctx - 1) / a.per_ctx;
#pragma unroll 1
            for (int b = sub; b < nb; b += W) t += laid_out(ctx_tiles(a, x, fp, b).n);
        }
#pragma unroll 1
        for (int sh = 1; sh < W; sh <<= 1) t += __shfl_xor_sync(0xffffffffu, t, sh);
        return t * Hkv;
    };
    int T = 0, my_s0 = 0, my_s1 = 0;
    Shares shares(0, 1);
    int start = 0, v = 0;  // this thread's sequence of the last pass: its laid-out start and tiles
    // the total, then the sequence that holds this share's start (from registers when one pass covers every sequence)
#pragma unroll 1
    for (int round = 0; round < (a.num_seqs > per_pass ? 2 : 1); ++round) {
        if (threadIdx.x == 0) scratch[kCarry] = 0;
        __syncthreads();
#pragma unroll 1
        for (int base = 0; base < a.num_seqs; base += per_pass) {
            const int s = threadIdx.x < 640 ? base + threadIdx.x / W : a.num_seqs;
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
            const int before = scratch[kCarry] + (int)__reduce_add_sync(0xffffffffu, lane < warp ? (unsigned)scratch[lane] : 0u);
            const int end = before + x;
            start = end - v;
            if (round == 1 && v > 0 && my_s0 >= start && my_s0 < end) {
                scratch[kFound] = s;
                scratch[kStart] = start;
            }
            __syncthreads();
            if (threadIdx.x == kThreads - 1) scratch[kCarry] = end;
            __syncthreads();
        }
        if (round == 0) {
            T = scratch[kCarry];
            shares = Shares(T, gridDim.x);
            __syncthreads();  // every thread has the total before the next round clears it
            // So far only lengths, starts and prefixes were read, which no kernel of the library writes: this may run under
            // the previous kernel's tail.  What follows may not.
            grid_dependency_wait();
            grid_launch_dependents();
            if (threadIdx.x == 0) a.merges[blockIdx.x] = make_int4(0, 0, 0, 0);
            if (T == 0 || (int)blockIdx.x >= shares.n) return;
            my_s0 = shares.begin(blockIdx.x);
            my_s1 = shares.begin(blockIdx.x + 1);
        }
    }
    const int s0 = my_s0, s1 = my_s1;
    if (a.num_seqs <= per_pass && v > 0 && s0 >= start && s0 < start + v) {
        scratch[kFound] = threadIdx.x / W;
        scratch[kStart] = start;
    }

    // rows of the query tiles that no box fills: what they hold must not differ from run to run
    for (int i = a.per_ctx * G * 8 + threadIdx.x; i < kRows * 8; i += kThreads)
        for (int t = 0; t < 2 * H; ++t) *reinterpret_cast<uint4 *>(smem + L::q + t * (kRows * 128) + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async();
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    bool dead = false;
    auto walk = [&](auto again) {
        constexpr bool careful = decltype(again)::value;
        if (threadIdx.x == 0) {
            *redo = 0;
            if (careful)
#pragma unroll 1
                for (int i = 0; i < L::kBars; ++i) mbar_inval(&k_full[i]);
#pragma unroll 1
            for (int i = 0; i < NK; ++i) {
                mbar_init(&k_full[i], H);
                mbar_init(&k_empty[i], 1);
            }
#pragma unroll 1
            for (int i = 0; i < NV; ++i) {
                mbar_init(&v_full[i], 1);
                mbar_init(&v_empty[i], 1);
            }
#pragma unroll 1
            for (int i = 0; i < kSets; ++i) {
                mbar_init(&s_full[i], 1);
                mbar_init(&p_full[i], 4);
                mbar_init(&o_done[i], 1);
            }
#pragma unroll 1
            for (int i = 0; i < 4 * kSets; ++i) mbar_init(&m_full[i], 1);
#pragma unroll 1
            for (int i = 0; i < 16; ++i) mbar_init(&started[i], 1);
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                mbar_init(&q_full[i], 1);
                mbar_init(&q_empty[i], 1);
                mbar_init(&fin_full[i], 4 * kSets);
                mbar_init(&fin_empty[i], 4);
            }
            mbar_init(o_last, 1);
            mbar_init(o_free, 4);
#pragma unroll 1
            for (int i = 0; i < kDescs; ++i) {
                mbar_init(&desc_full[i], 1);
                mbar_init(&desc_empty[i], 4 * kSets + 4 + 2 + H + 1);  // softmax, epilogue, MMA, producers
            }
            mbar_init(&all_done[0], 1);
            mbar_init(&all_done[1], 1);
            fence_barrier_init();
        }
        tc::fence_before();
        __syncthreads();
        tc::fence_after();
        const uint32_t tmem = *tmem_slot;
        const uint32_t q_s = smem_u32(smem + L::q), k_s = smem_u32(smem + L::kring), v_s = smem_u32(smem + L::vring);

        if (warp == kSchedWarp) {
            // ======================= scheduler =======================
            int s = scratch[kFound];
            int t = s0;                     // next laid-out tile of the share
            int seq_start = scratch[kStart];  // laid-out start of sequence s
            int p = 0;
            while (t < s1 && !dead) {
                const Seq x = load_seq(a, s, false);
                const int fp = first_pos(a, x, s), nb = (x.Q + a.per_ctx - 1) / a.per_ctx;
                int per_kvh = 0;
#pragma unroll 1
                for (int b = lane; b < nb; b += 32) per_kvh += laid_out(ctx_tiles(a, x, fp, b).n);
#pragma unroll
                for (int sh = 16; sh > 0; sh >>= 1) per_kvh += __shfl_xor_sync(0xffffffffu, per_kvh, sh);
#pragma unroll 1
                for (int kvh = per_kvh > 0 ? (t - seq_start) / per_kvh : Hkv; kvh < Hkv && t < s1 && !dead; ++kvh) {
                    int pos = seq_start + kvh * per_kvh;  // laid-out start of block b0
#pragma unroll 1
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
#pragma unroll 1
                        for (uint32_t todo = __ballot_sync(0xffffffffu, mine); todo && !dead; todo &= todo - 1) {
                            const int d = p % kDescs;
                            if (lane == 0 && p >= kDescs)
                                wait_for(&desc_empty[d], (uint32_t)((p / kDescs - 1) & 1), dead);
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
                                pc.nq = nq;
                                pc.nrows = nq * G;
                                pc.pos0 = fp + q0;
                                pc.pre = x.pre;
                                pc.ks0 = c.ks0;
                                pc.cpre = c.r.pre;
                                pc.lo = c.r.lo;
                                pc.hi = c.r.hi;
                                // what the last row's document or window leaves, up to the first row's position
                                pc.fks = max(c.ks0, key_start_of(a.s, pc.row0 + nq - 1));
                                pc.flo = max(pc.fks, a.s.window > 0 ? max(pc.pos0 + nq, 1) - a.s.window : 0);
                                pc.fhi = pc.pos0 + 1;
                                const bool begins = begin + kCharge >= s0, ends = end <= s1;
                                pc.slot = begins && ends ? -1 : 2 * (int)blockIdx.x + (begins ? 1 : 0);
                                if (begins && !ends)  // the shares that hold the rest
                                    a.merges[blockIdx.x] = make_int4(shares.owner(end - 1) - (int)blockIdx.x + 1, pc.row0,
                                                                     pc.nrows, kvh);
                                descs[d] = pc;
                                mbar_arrive(&desc_full[d]);
                                // the rows' loads at the piece's start
                                if (a.s.key_starts)
#pragma unroll 1
                                    for (int i = 0; i < nq; i += 32) prefetch_l1(a.s.key_starts + pc.row0 + i);
                                // its queries: per_ctx queries of the KV head's G heads, one box per column half
                                const int qb = p & 1;
                                if (p >= 2) wait_for(&q_empty[qb], (uint32_t)((p / 2 - 1) & 1), dead);
                                if (!dead) {
                                    mbar_arrive_expect_tx(&q_full[qb], (uint32_t)(H * a.per_ctx * G * 128));
#pragma unroll
                                    for (int h = 0; h < H; ++h)
                                        tma_load_3d(q_s + (uint32_t)(qb * L::kQTile + h * (kRows * 128)), &tm_q, smem_u32(&q_full[qb]),
                                                    h * 64, kvh * G, pc.row0);
                                }
                            }
                            dead = __any_sync(0xffffffffu, dead);
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
                if (p >= kDescs) wait_for(&desc_empty[d], (uint32_t)((p / kDescs - 1) & 1), dead);
                if (!dead) {
                    descs[d].ntiles = 0;
                    mbar_arrive(&desc_full[d]);
                }
            }
            // queries in flight (only after a timeout) land before the CTA exits
            if (dead && lane == 0)
#pragma unroll 1
                for (int k = max(0, p - 2); k < p; ++k) drain(&q_full[k & 1], (uint32_t)((k >> 1) & 1));
        } else if (warp == kVWarp || (warp >= kKWarp && warp < kKWarp + H)) {
            // ======================= producers =======================
            const bool isk = warp != kVWarp;
            const int half = warp - kKWarp;  // K: column half
            const int N = isk ? NK : NV;
            uint64_t *full = isk ? k_full : v_full, *empty = isk ? k_empty : v_empty;
            const int bpt = kTok >> a.bshift;  // blocks per tile, at most 16
            int tau = 0;
#pragma unroll 1
            for (int p = 0; !dead; ++p) {
                const int d = p % kDescs;
                if (!wait_for(&desc_full[d], (uint32_t)((p / kDescs) & 1), dead)) break;
                const Piece &pc = descs[d];
                const int n = pc.ntiles;
                if (n == 0) break;
                const int32_t *bt = a.block_tables + (int64_t)pc.seq * a.max_blocks;
                const KeyRange r{pc.ks0, pc.cpre, pc.lo, pc.hi};
                const int kvh = pc.kvh, flo = pc.flo, fhi = pc.fhi, fks = pc.fks, pre = pc.pre;
                const int i1 = pc.i0 + n, np = pc.np, pt0 = pc.pt0, mt0 = pc.mt0;
                // the latest keys first: with a bias by distance the largest scores come first, and the rows' reference seldom moves
                auto first_key = [&](int j) {
                    const int i = i1 - 1 - j;
                    return (i < np ? pt0 + i : mt0 + i - np) * kTok;
                };
                // this lane's block of a tile: its id, INT_MIN where no row sees a key of it
                auto block_id = [&](int j) {
                    if (j >= n || lane >= bpt) return (int)INT_MIN;
                    const int t = first_key(j) + (lane << a.bshift);
                    if (!r.meets(t, t + B)) return (int)INT_MIN;
                    return max((int)bt[t >> a.bshift], INT_MIN + 1);
                };
                int next = block_id(0);
#pragma unroll 1
                for (int j = 0; j < n; ++j, ++tau) {
                    const int st = tau % N;
                    const int id = next;
                    next = block_id(j + 1);
                    if (tau >= N) wait_for(&empty[st], (uint32_t)((tau / N - 1) & 1), dead);
                    if (__any_sync(0xffffffffu, dead)) {
                        dead = true;
                        break;
                    }
                    const bool live = id != INT_MIN, bad = live && (id < 0 || id >= a.num_blocks);
                    const uint32_t nlive = (uint32_t)__popc(__ballot_sync(0xffffffffu, live)), badm = __ballot_sync(0xffffffffu, bad);
                    if (lane == 0) {
                        if (isk && half == 0) {
                            const int t0 = first_key(j);
                            TileRec rec;
                            rec.t0 = t0;
                            rec.bad = badm;
                            rec.whole = badm == 0u && ((t0 >= r.lo && t0 + kTok <= r.hi) || (t0 >= r.first && t0 + kTok <= r.pre));
                            rec.full = badm == 0u && ((t0 >= flo && t0 + kTok <= fhi) || (t0 >= fks && t0 + kTok <= pre));
                            recs[tau % kRecs] = rec;
                            if (badm) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                        }
                        mbar_arrive_expect_tx(&full[st], nlive * (uint32_t)((isk ? 1 : H) * 128) << a.bshift);
                    }
                    __syncwarp();
                    // an invalid id is read as block 0, its keys masked
                    if (live) {
                        const int y = (int)(((int64_t)(bad ? 0 : id) * Hkv + kvh) * B);
                        if (isk)
                            tma_load_2d(k_s + st * L::kTile + half * (kTok * 128) + ((lane << a.bshift) * 128), &tm_k, smem_u32(&full[st]),
                                        half * 64, y);
                        else
                            tma_load_3d(v_s + st * L::kTile + ((lane << a.bshift) * (H * 128)), &tm_v, smem_u32(&full[st]), 0, y, 0);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&desc_empty[d]);
            }
            // copies in flight (only after a timeout) land before the CTA exits
            if (lane == 0 && dead)
#pragma unroll 1
                for (int k = max(0, tau - N); k < tau; ++k) drain(&full[k % N], (uint32_t)((k / N) & 1));
        } else if (warp == kMmaWarp) {
            // ======================= Q K^T issuer =======================
            // Both issuers walk as whole warps (uniform registers) and one elected lane issues.
            constexpr uint32_t idesc = tc::instr_desc(kTok, false);
            const bool leader = elect_one();
            const uint64_t qd0 = tc::smem_desc(q_s, 16, 1024), kd0 = tc::smem_desc(k_s, 16, 1024);
            int st = 0, sb = 0;            // K stage, S buffer
            uint32_t kph = 0, sph = 1;     // their phases (a buffer's first use waits for nothing)
            int d = 0, p = 0, tau = 0;
            uint32_t dph = 0;
#pragma unroll 1
            for (;; ++p) {
                wait_for(&desc_full[d], dph, dead);
                const int n = dead ? 0 : descs[d].ntiles;
                if (n == 0) break;
                tau += n;
                wait_for(&q_full[p & 1], (uint32_t)((p >> 1) & 1), dead);
                const uint64_t qd = qd0 + (uint64_t)((uint32_t)(p & 1) * (uint32_t)(L::kQTile >> 4));
#pragma unroll 1
                for (int j = 0; j < n; ++j) {
                    wait_for(&k_full[st], kph, dead);
                    wait_for(&o_done[sb], sph, dead);  // the P V that read the buffer before
                    if (dead) break;
                    tc::fence_after();
                    const uint64_t kd = kd0 + (uint64_t)((uint32_t)st * (uint32_t)(L::kTile >> 4));
                    if (leader) {
#pragma unroll 1  // (the shorter code leaves more of the instruction cache to the softmax)
                        for (int k = 0; k < D / 16; ++k) {
                            const uint64_t off = (uint64_t)(((k >> 2) * (kTok * 128) + (k & 3) * 32) >> 4);
                            tc::mma(tmem + (uint32_t)sb * kTok, qd + off, kd + off, idesc, k > 0 ? 1u : 0u);
                        }
                        tc::commit(&s_full[sb]);
                        tc::commit(&k_empty[st]);
                        if (j + 1 == n) tc::commit(&q_empty[p & 1]);
                    }
                    __syncwarp();
                    if (++st == NK) st = 0, kph ^= 1u;
                    if (++sb == kSets) sb = 0, sph ^= 1u;
                }
                if (lane == 0) mbar_arrive(&desc_empty[d]);
                if (++d == kDescs) d = 0, dph ^= 1u;
            }
            if (lane == 0) scratch[0] = tau, scratch[1] = p;
            if (leader) tc::commit(&all_done[0]);
            __syncwarp();
            drain(&all_done[0], 0u);
        } else if (warp == kPvWarp) {
            // ======================= P V issuer =======================
            constexpr uint32_t idesc = tc::instr_desc(D, true);
            const uint32_t pv_lbo = (uint32_t)(B * 128), pv_sbo = B >= 16 ? 1024u : (uint32_t)(H * B * 128);
            const bool leader = elect_one();
            const uint64_t vd0 = tc::smem_desc(v_s, pv_lbo, pv_sbo);
            // 16 keys of V further: inside a block of 32 every second step, else a block (B = 8: two)
            const uint32_t odd = B == 32 ? 16 * 128 >> 4 : (uint32_t)(H * 16 * 128) >> 4, two = (uint32_t)(2 * H * 16 * 128) >> 4;
            int st = 0, sb = 0;
            uint32_t vph = 0, sph = 0;
            int d = 0;
            uint32_t dph = 0;
#pragma unroll 1
            for (int p = 0;; ++p) {
                wait_for(&desc_full[d], dph, dead);
                const int n = dead ? 0 : descs[d].ntiles;
                if (n == 0) break;
                if (p > 0) wait_for(o_free, (uint32_t)((p - 1) & 1), dead);  // the piece before's O has been read
#pragma unroll 1
                for (int j = 0; j < n; ++j) {
                    wait_for(&v_full[st], vph, dead);
                    wait_for(&p_full[sb], sph, dead);
                    if (dead) break;
                    tc::fence_after();
                    const uint64_t vd = vd0 + (uint64_t)((uint32_t)st * (uint32_t)(L::kTile >> 4));
                    if (leader) {
#pragma unroll 1  // (the shorter code leaves more of the instruction cache to the softmax)
                        for (int k = 0; k < kTok / 16; ++k)
                            tc::mma_ts(tmem + kOBase, tmem + (uint32_t)(sb * kTok + 8 * k),
                                       vd + (uint64_t)((uint32_t)(k >> 1) * two + (uint32_t)(k & 1) * odd), idesc, j > 0 || k > 0 ? 1u : 0u);
                        tc::commit(&o_done[sb]);
                        tc::commit(&v_empty[st]);
                        if (j + 1 == n) tc::commit(o_last);
                    }
                    __syncwarp();
                    if (++st == NV) st = 0, vph ^= 1u;
                    if (++sb == kSets) sb = 0, sph ^= 1u;
                }
                if (lane == 0) mbar_arrive(&desc_empty[d]);
                if (++d == kDescs) d = 0, dph ^= 1u;
            }
            // every product has completed before the tensor memory is freed
            if (leader) tc::commit(&all_done[1]);
            __syncwarp();
            drain(&all_done[1], 0u);
        } else if (warp < kEpiWarp) {
            // ======================= softmax =======================
            constexpr int K = careful && KIND == kCap ? kCapBias : KIND;  // (a moving reference)
            const int set = warp >> 2, wq = warp & 3;
            const int rr = wq * 32 + lane;  // TMEM lane and row of the context
            const int rq = rr / G, rh = rr - rq * G;  // its query and head
            const uint32_t trow = tmem + ((uint32_t)(wq * 32) << 16);
            const uint32_t sp = trow + (uint32_t)(set * kTok), op = trow + kOBase;
            const int prev = set == 0 ? kSets - 1 : set - 1;  // the set of the tile before
            int tau0 = 0;
#pragma unroll 1
            for (int p = 0; !dead; ++p) {
                const int d = p % kDescs;
                if (!wait_for(&desc_full[d], (uint32_t)((p / kDescs) & 1), dead)) break;
                const Piece &pc = descs[d];
                const int n = pc.ntiles, pre = pc.pre;
                if (n == 0) break;
                // warps without rows only pass the barriers; the other rows of a warp with some go by the last query's keys
                const bool live_warp = wq * 32 < pc.nrows;
                const int qi = min(rq, pc.nq - 1);
                RowState st;
                st.m = K == kCap ? a.m0 : -INFINITY;
                st.l = 0.f;
                st.p = pc.pos0 + qi;
                st.r = key_range(max(pc.ks0, key_start_of(a.s, (int64_t)pc.row0 + qi)), pre, a.s.window, st.p, st.p);
                st.slope2 = 0.f;
                if constexpr (K == kBias || K == kCapBias)
                    st.slope2 = a.s.slopes ? a.s.slopes[pc.kvh * G + rh] * 1.44269504f : 0.f;
                const KeyRange cr{pc.ks0, pc.cpre, pc.lo, pc.hi};
                bool any = false, taken = false;
                int j = set - tau0 % kSets;
                if (j < 0) j += kSets;
#pragma unroll 1
                for (; j < n; j += kSets) {
                    const int tau = tau0 + j, turn = tau / kSets;
                    wait_for(&s_full[set], (uint32_t)(turn & 1), dead);
                    if (dead) break;
                    tc::fence_after();
                    const TileRec rec = recs[tau % kRecs];
                    // the tile before's barriers have come round as often as this one's, one time less for the first set
                    const int bturn = set == 0 ? turn - 1 : turn;
                    Chain ch;
                    ch.mref = mref + rr;
                    ch.start = start_ref + (p & 3) * kRows + rr;
                    ch.started = &started[(p & 3) * 4 + wq];
                    ch.start_parity = (uint32_t)((p >> 2) & 1);
                    ch.begun = any;
                    ch.before = tau > 0 ? &m_full[prev * 4 + wq] : nullptr;
                    ch.mine = &m_full[set * 4 + wq];
                    ch.done = &o_done[prev];
                    ch.parity = (uint32_t)(bturn & 1);
                    ch.first = j == 0;
                    if (live_warp) {
                        softmax_tile<D, K, careful>(sp, op, rec, a, rec.t0 < pre, st, ch, lane, dead);
                    } else if (K != kCap) {
                        if (ch.before) wait_for(ch.before, ch.parity, dead);
                        __syncwarp();
                        if (lane == 0) {
                            if (ch.first) mbar_arrive(ch.started);
                            mbar_arrive(ch.mine);
                        }
                    }
                    // V rows of keys that no row sees hold stale values, or none were loaded: zero weights must meet zeros
                    if (!rec.whole || (careful && !rec.full)) {
                        // A parity tells a stage's use from the one before it only, and P V is known to be complete up to tile
                        // tau - kSets: the stage's use before has to be over first (it does not wait for this tile).
                        const int st_v = tau % NV, used = tau - NV;
                        if (NV < kSets && used >= 0) wait_for(&o_done[used % kSets], (uint32_t)((used / kSets) & 1), dead);
                        wait_for(&v_full[st_v], (uint32_t)((tau / NV) & 1), dead);
                        const uint32_t row = v_s + (uint32_t)st_v * L::kTile + (rr >> a.bshift) * (H * 128 << a.bshift) +
                                             (rr & (B - 1)) * 128;
                        if (!cr.sees(rec.t0 + rr) || ((rec.bad >> (rr >> a.bshift)) & 1u)) {  // a thread per key
#pragma unroll 4
                            for (int i = 0; i < 8 * H; ++i)
                                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(row + (i >> 3) * (128 << a.bshift) +
                                                                                           ((i + lane) & 7) * 16),
                                             "r"(0u)
                                             : "memory");
                        } else if (careful && !rec.full) {
                            taken = clean_row<H>(row, 128 << a.bshift, lane) || taken;
                        }
                        fence_proxy_async();
                    }
                    any = true;
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[set]);
                }
                if (dead) break;
                tau0 += n;
                // the piece's reference and sum of this set's tiles, for the epilogue
                const int f = p & 1;
                if (p >= 2) wait_for(&fin_empty[f], (uint32_t)((p / 2 - 1) & 1), dead);
                fin_ml[(f * kSets + set) * kRows + rr] = make_float2(any ? st.m : -INFINITY, st.l);
                if (careful) taken = __any_sync(0xffffffffu, taken);
                __syncwarp();
                if (lane == 0) {
                    if (careful) fin_bad[f * 4 * kSets + warp] = taken;
                    mbar_arrive(&fin_full[f]);
                    mbar_arrive(&desc_empty[d]);
                }
            }
        } else if (warp < kEpiWarp + 4) {
            // ======================= epilogue =======================
            const int wq = warp & 3, rr = wq * 32 + lane;
            const int64_t rel = ((int64_t)(rr / G) * a.num_heads + rr % G) * D;
            const uint32_t op = tmem + ((uint32_t)(wq * 32) << 16) + kOBase;
#pragma unroll 1
            for (int p = 0; !dead; ++p) {
                const int d = p % kDescs, f = p & 1;
                if (!wait_for(&desc_full[d], (uint32_t)((p / kDescs) & 1), dead)) break;
                const Piece &pc = descs[d];
                if (pc.ntiles == 0) break;
                const int nrows = pc.nrows, slot = pc.slot;
                const int64_t orow = ((int64_t)pc.row0 * a.num_heads + pc.kvh * G) * D + rel;
                wait_for(&fin_full[f], (uint32_t)((p >> 1) & 1), dead);
                float2 x[kSets];
#pragma unroll
                for (int i = 0; i < kSets; ++i) x[i] = fin_ml[(f * kSets + i) * kRows + rr];
                const bool taken = careful && __any_sync(0xffffffffu, lane < 4 * kSets && fin_bad[f * 4 * kSets + lane] != 0);
                __syncwarp();
                if (lane == 0) mbar_arrive(&fin_empty[f]);
                float M = x[0].x, l = 0.f;
#pragma unroll
                for (int i = 1; i < kSets; ++i) M = fmaxf(M, x[i].x);
#pragma unroll
                for (int i = 0; i < kSets; ++i)  // (a set without a tile: l = 0)
                    l += x[i].x == -INFINITY || x[i].x == M ? x[i].y : x[i].y * ex2_approx(x[i].x - M);
                const float inv = l != 0.f ? 1.f / l : 0.f;
                wait_for(o_last, (uint32_t)(p & 1), dead);
                if (dead) break;
                tc::fence_after();
                const bool live = rr < nrows;
                if (taken && wq * 32 < nrows) {
                    const int qi = min(rr / G, pc.nq - 1), pos = pc.pos0 + qi;
                    add_odd_values<D>(a, pc, key_range(max(pc.ks0, key_start_of(a.s, (int64_t)pc.row0 + qi)), pc.pre, a.s.window, pos, pos),
                                      op, lane);
                }
                // Every row of the product meets every V entry, so any row tells whether a column did: the warps share the columns.
                uint64_t odd[2] = {0ull, 0ull};  // NaN once an output is infinite or NaN
                int look = wq * 16;
                if (wq * 32 < nrows) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float o[16];
                        ld16(op + (uint32_t)c, o);
                        tc::wait_ld();
                        if (c == look) {
                            look += (nrows + 31) / 32 * 16;
#pragma unroll
                            for (int k = 0; k < 16; k += 2) odd[(k >> 1) & 1] = fma_f32x2(f32x2(o[k], o[k + 1]), 0ull, odd[(k >> 1) & 1]);
                        }
                        if (slot < 0) {
                            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + orow + c);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint4 v = make_uint4(pack_bf16x2(o[8 * k] * inv, o[8 * k + 1] * inv),
                                                           pack_bf16x2(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                                           pack_bf16x2(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                                                           pack_bf16x2(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
                                if (live) dst[k] = v;
                            }
                        } else {
                            float *dst = a.part_o + ((int64_t)slot * D + c) * kRows + rr;
#pragma unroll
                            for (int k = 0; k < 16; ++k) dst[k * kRows] = o[k];
                        }
                    }
                    if (slot >= 0) reinterpret_cast<float2 *>(a.part_ml)[(int64_t)slot * kRows + rr] = make_float2(M, l);
                }
                float odd0, odd1;
                f32x2_split(add_f32x2(odd[0], odd[1]), odd0, odd1);
                if (live && odd0 + odd1 != 0.f) *redo = 1;
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_free);
                __syncwarp();
                if (lane == 0) mbar_arrive(&desc_empty[d]);
            }
        }
        tc::fence_before();
        const bool gave_up = __syncthreads_or(dead);
        tc::fence_after();
        return gave_up || careful || *redo == 0;
    };
    if (!walk(std::false_type{})) {
        // The barriers start anew: the issuers' last arrivals that no one has waited for come first.
        if (threadIdx.x == 0) {
            const int tau = scratch[0], p = scratch[1];
#pragma unroll 1
            for (int k = max(0, tau - NK); k < tau; ++k) wait_for(&k_empty[k % NK], (uint32_t)((k / NK) & 1), dead);
#pragma unroll 1
            for (int k = max(0, tau - NV); k < tau; ++k) wait_for(&v_empty[k % NV], (uint32_t)((k / NV) & 1), dead);
#pragma unroll 1
            for (int k = max(0, tau - kSets); k < tau; ++k) wait_for(&o_done[k % kSets], (uint32_t)((k / kSets) & 1), dead);
#pragma unroll 1
            for (int k = max(0, p - 2); k < p; ++k) wait_for(&q_empty[k & 1], (uint32_t)((k >> 1) & 1), dead);
        }
        if (!__syncthreads_or(dead)) walk(std::true_type{});
    }
    if (dead) flag_error(a.err, PKV_DEVERR_TIMEOUT);
    if (warp == kMmaWarp) {
        const uint32_t tmem = *tmem_slot;
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// The states of contexts cut by shares' borders, merged: CTA (c, k) takes rows
// 32 k .. of the context that share c begins and does not end; lanes are rows,
// the four warps quarters of the columns.  Part 0 is that share's last piece
// (slot 2 c + 1), part j the first piece of share c + j (slot 2 (c + j)).  The
// CTAs behind those, `empties` for each sequence, zero the rows of contexts that see
// nothing (4000 queries of 32 heads: 41 us a call, by one CTA 524, by one thread a context 1067).
template <int D>
__global__ void __launch_bounds__(128) scored_rows_merge_kernel(const __grid_constant__ RowsArgs a, int ctas, int empties) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int kPer = kRows / kMergeRows;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out);
    if ((int)blockIdx.x >= ctas * kPer) {
        const int e = blockIdx.x - ctas * kPer, s = e / empties, lane = threadIdx.x & 31;
        const Seq x = load_seq(a, s, false);
        const int fp = first_pos(a, x, s), nb = (x.Q + a.per_ctx - 1) / a.per_ctx;
        // a lane a block, the sequence's warps in turn; a warp writes the rows of its empty ones
        const int warps = 4 * empties;
        for (int b0 = e % empties * 4 + (threadIdx.x >> 5); b0 < nb; b0 += 32 * warps) {
            const int own = b0 + lane * warps;
            const bool empty = own < nb && ctx_tiles(a, x, fp, own).n == 0;
            for (uint32_t todo = __ballot_sync(0xffffffffu, empty); todo; todo &= todo - 1) {
                const int b = b0 + (__ffs(todo) - 1) * warps;
                const int64_t q0 = x.q0 + (int64_t)b * a.per_ctx, n = min(x.Q - b * a.per_ctx, a.per_ctx);
                uint4 *row = reinterpret_cast<uint4 *>(out + q0 * a.num_heads * D);
                for (int64_t i = lane; i < n * a.num_heads * (D / 8); i += 32) row[i] = make_uint4(0u, 0u, 0u, 0u);
            }
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
    for (int j = 0; j < m.x; ++j) M = fmaxf(M, ml[slot(j) * kRows + cr].x);
    float L = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int j = 0; j < m.x; ++j) {
        const float2 x = ml[slot(j) * kRows + cr];
        const float w = x.x == -INFINITY ? 0.f : ex2_approx(x.x - M);
        L += x.y * w;
        const float *src = a.part_o + (slot(j) * D + col) * kRows + cr;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += w * src[e * kRows];
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
        ml = round256((size_t)2 * kMaxCtas * D * kRows * 4);
        merges = ml + round256((size_t)2 * kMaxCtas * kRows * 8);
        total = merges + round256((size_t)kMaxCtas * 16);
    }
};

// The queries of G heads of per_ctx tokens as one box per column half: dims (head_dim, heads, tokens), a row per (token, head).
bool make_query_map(CUtensorMap *map, const RowsArgs &a, int D) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.num_heads, (cuuint64_t)a.num_q};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.num_heads * D * 2};
    cuuint32_t box[3] = {64u, (cuuint32_t)a.group, (cuuint32_t)a.per_ctx};
    cuuint32_t estr[3] = {1u, 1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int KIND>
pkv_status launch(const RowsArgs &a, cudaStream_t st) {
    constexpr int smem = Layout<D>::total;
    static bool done[128] = {};
    auto kern = scored_rows_kernel<D, KIND>;
    if (!ensure_smem(kern, smem, done)) return PKV_ERR_CUDA;
    CUtensorMap mq, mk, mv;
    const int64_t rows = (int64_t)a.num_blocks * a.num_kv_heads * a.block_size;
    if (!make_query_map(&mq, a, D) || !make_cache_map(&mk, a.k_cache, rows, D, a.block_size) ||
        !make_slab_map(&mv, a.v_cache, rows, D, a.block_size))
        return PKV_ERR_CUDA;
    const int ctas = std::min(sm_count(), kMaxCtas);
    if (ctas < 1) return PKV_ERR_CUDA;
    const int blocks = (std::min(a.max_q_len, a.num_q) - 1) / a.per_ctx + 1;
    const int empties = std::max(1, std::min((blocks + 3) / 4, ctas / a.num_seqs));
    pkv_status rc = launch_pdl(kern, dim3((unsigned)ctas), dim3(kThreads), smem, st, mq, mk, mv, a);
    if (rc == PKV_OK)
        rc = launch_pdl(scored_rows_merge_kernel<D>, dim3((unsigned)(ctas * (kRows / kMergeRows) + a.num_seqs * empties)), dim3(128),
                        0, st, a, ctas, empties);
    return rc;
}

template <int D>
pkv_status launch_kind(const RowsArgs &a, cudaStream_t st) {
    const bool bias = a.s.slopes != nullptr;
    if (a.s.softcap > 0.f) return bias || a.c2 > kMaxC2 ? launch<D, kCapBias>(a, st) : launch<D, kCap>(a, st);
    return bias ? launch<D, kBias>(a, st) : launch<D, kPlain>(a, st);
}

}  // namespace

size_t rows_workspace(int head_dim) { return WsLayout(head_dim).total; }

pkv_status run_rows(const Args &args, int head_dim, void *workspace, size_t workspace_bytes, cudaStream_t st) {
    const WsLayout lay(head_dim);
    if (!workspace || workspace_bytes < lay.total || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return PKV_ERR_INVALID;
    RowsArgs a{};
    static_cast<Args &>(a) = args;
    if (a.s.softcap > kNoCap) a.s.softcap = 0.f;
    a.per_ctx = kRows / a.group;
    a.bshift = a.block_size == 8 ? 3 : a.block_size == 16 ? 4 : 5;
    const int64_t blocks = ((int64_t)std::min(a.max_q_len, a.num_q) + a.per_ctx - 1) / a.per_ctx;
    a.scan_w = 1;
    while (a.scan_w < 32 && a.scan_w < blocks) a.scan_w *= 2;
    // (the number of all queries is no bound of a part's contexts: query ranges may overlap)
    const int64_t most = kMaxTiles / (a.num_kv_heads * ((longest_context(a) + kTok - 1) / kTok + 1 + kCharge)) / blocks;
    if (most < 1) return PKV_ERR_UNSUPPORTED;
    const double log2e = 1.4426950408889634;
    a.k1 = finite_float(a.s.softcap > 0.f ? (double)a.s.scale / a.s.softcap : a.s.scale * log2e);
    a.c2 = finite_float(a.s.softcap * log2e);
    a.m0 = 0.25f * a.c2;
    if (a.s.softcap > 0.f) {
        a.k1 = std::min(std::max(a.k1, -1e38f), 1e38f);  // 2 log2 e k1 stays finite: no score of 0 becomes NaN
        double f = a.s.softcap * log2e * a.k1;
        const bool wide = a.c2 > kWideCap;
        a.near_max = wide ? kTanhSmall : kTanhNear;
        bool folds = true;  // the cap's factors folded into the coefficients are normal numbers
        for (int i = 0; i < 4; ++i, f *= (double)a.k1 * a.k1) {
            const double x = (wide ? kTanhSeries : kTanh3)[i] * f;
            folds = folds && std::fabs(x) > 1e-37 && std::fabs(x) < 1e37;
            a.near[i] = (float)(folds ? x : 0.0);
        }
        if (!folds) {  // a scale far from the cap's: c2 k1 s where |z| < 2^-12 (off by 2^-25 of it), the others as large ones
            a.near[0] = finite_float(a.s.softcap * log2e * a.k1);
            a.near[1] = a.near[2] = a.near[3] = 0.f;
            a.near_max = a.k1 == 0.f || std::fabs(a.k1) > 1e-22f ? 0x1p-12f : -1.f;  // (-1: s^2 would pass float32's range)
        }
    }
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    a.part_o = reinterpret_cast<float *>(ws + lay.o);
    a.part_ml = reinterpret_cast<float *>(ws + lay.ml);
    a.merges = reinterpret_cast<int4 *>(ws + lay.merges);
    const float softcap = a.s.softcap;
    pkv_status rc = PKV_OK;
    for (int64_t s0 = 0; s0 < args.num_seqs && rc == PKV_OK; s0 += most) {  // (a part begins when the one before is through)
        static_cast<Args &>(a) = part_of(args, head_dim, (int)s0, (int)std::min<int64_t>(most, args.num_seqs - s0));
        a.s.softcap = softcap;
        rc = head_dim == 128 ? launch_kind<128>(a, st) : launch_kind<64>(a, st);
    }
    return rc;
}

}  // namespace scored
}  // namespace pkv
