// Shared by the tensor-core kernels of latent attention: tcgen05 pieces, the walk over
// contexts in equal shares, and the location of a share's first tile.
#pragma once

#include "latent.cuh"
#include "pkv_ptx.cuh"

namespace pkv {
namespace latent {

constexpr int kDescs = 4;      // pieces in flight between the warps of a CTA
constexpr int kHead = 2;       // tiles that a context's start and end are worth
constexpr float kSlack = 8.f;  // log2 of how far a weight may pass 1 before its row's reference moves

// kind::f16 instruction descriptor: bf16 operands, float32 accumulators.
__host__ __device__ constexpr uint32_t idesc(int m, int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// A bounded wait by a whole warp, the part that is seldom reached (out of line: the kernels' speed is their
// instruction cache's); true: it gave up, or some other warp of the CTA had.
static __device__ __noinline__ bool wait_on(uint64_t *bar, uint32_t parity, int *dead, unsigned int *err) {
    bool ok = false;
    for (uint32_t i = 0; i < kWaitLimit && !ok; ++i) {
        ok = mbar_try_wait(bar, parity);
        if ((i & 255u) == 255u && *(volatile int *)dead) break;
    }
    if (!__any_sync(0xffffffffu, !ok)) return false;
    *(volatile int *)dead = 1;
    flag_error(err, PKV_DEVERR_TIMEOUT);
    return true;
}

// Maximum of three that is NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Whether one of eight bf16 entries is an infinity or NaN.
__device__ __forceinline__ bool not_finite(const uint4 &y) {
    const uint32_t z[4] = {y.x, y.y, y.z, y.w};
    bool found = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) found |= (z[i] & 0x7f80u) == 0x7f80u || (z[i] & 0x7f800000u) == 0x7f800000u;
    return found;
}

// Barrier of the softmax warps (their THREADS), alone and with a vote.
template <int THREADS>
__device__ __forceinline__ void softmax_sync() {
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(THREADS) : "memory");
}
template <int THREADS>
__device__ __forceinline__ bool softmax_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "n"(THREADS)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void ld_16x256b(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

__device__ __forceinline__ void ld_16x256b(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}

__device__ __forceinline__ void ld_16x256b(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}

__device__ __forceinline__ void ld_32x32b(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}

__device__ __forceinline__ void ld_32x32b(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}

__device__ __forceinline__ void st_32x32b(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}

__device__ __forceinline__ void st_32x32b(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]) : "memory");
}

// What L2 is told of the cache's rows.
__device__ __forceinline__ uint64_t row_policy(const Args &a) {
    uint64_t p;
    if (a.once) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}

// 8 rows of the cache from `row` on, on their way into L2.
template <int V>
__device__ __forceinline__ void prefetch_rows(const Args &a, int row) {
    constexpr int kRow = (V + kRope) * 2;
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                     __cvta_generic_to_global((const unsigned char *)a.cache + (int64_t)row * kRow)),
                 "r"(8 * kRow)
                 : "memory");
}

// One share's part of a context.
struct Piece {
    int tiles;     // 0: no more pieces
    int t0, end;   // first token of the first tile; tokens that some row of the row tile sees
    int row0, rows;
    int lim0;      // tokens that row r sees: lim0 + (qh0 + r) / H
    int qh0;
    int seq;
    int out;       // 0: the whole context; 1: its first tiles; 2: later ones
};

// The walk over contexts (sequence, row tile): row tile k of a sequence is rows
// [k N, k N + N) of its n H query rows.  Its last row's query sees
//     p0 + 1 + floor(min(k N + N - 1, n H - 1) / H)  tokens, p0 = L - n0 the first query's position,
// A context counts kHead tiles more than it has, at its start: what its queries' load and the
// storing of its output take.  Its tiles are, but for the last row tile, floor((k + c) / m) with m = TOK H / N and
// c = floor((N - 1 + H (p0 + TOK)) / N): where N divides TOK, sums over k have a closed form.
// ONE: a sequence's rows are one row tile at most (N rows hold any, as the transposed kernel's do); N need not divide TOK.
template <int N, int TOK, bool ONE>
struct Walk {
    int s, k, R;           // sequence, row tile, row tiles of the sequence
    int L, q0, nH, p0, k0; // k0: first row tile with a query that sees a token
    bool flagged;
    __host__ __device__ __forceinline__ void open(const Args &a, int seq) {
        s = seq;
        const Seq q = sequence(a, seq);
        flagged = q.flagged;
        L = q.L, q0 = q.q0, nH = q.n * a.H, p0 = q.L - q.n0;
        R = (nH + N - 1) / N;
        const int blind = max(0, min(q.n, -p0));  // queries in front of the context
        k0 = L == 0 ? R : (int)((int64_t)blind * a.H / N);
        if (blind == q.n) k0 = R;
        k = k0;
    }
    __host__ __device__ __forceinline__ int end(const Args &a, int kk) const {  // tokens row tile kk sees
        if (!a.q_starts) return L;
        const int last = min((kk + 1) * N, nH) - 1;
        return min(L, p0 + 1 + by_heads(a, last));
    }
    __host__ __device__ __forceinline__ int tiles(const Args &a, int kk) const { return (end(a, kk) + TOK - 1) / TOK; }
    // tiles, heads included, of row tiles k0 .. kk - 1, kk < R
    __host__ __device__ __forceinline__ int64_t before(const Args &a, int kk) const {
        static_assert(!ONE && TOK % N == 0 && (N & (N - 1)) == 0, "the closed form");
        if (kk <= k0) return 0;
        constexpr int kPer = TOK / N;
        const int64_t x = N - 1 + (int64_t)a.H * (p0 + TOK), c = (x - (x & (N - 1))) / N;  // floor: p0 may be below -TOK
        return G(a, kk + c, kPer) - G(a, k0 + c, kPer) + (int64_t)kHead * (kk - k0);
    }
    static __host__ __device__ __forceinline__ int64_t G(const Args &a, int64_t x, int per) {  // sum of floor(j / m), j < x, m = per H
        const int64_t y = x / per, m = (int64_t)per * a.H;
        const int64_t q = (uint64_t)y < (1ull << 31) ? by_heads(a, (int)y) : y / a.H;
        return m * (q * (q - 1) / 2) + q * (x - q * m);
    }
    __host__ __device__ __forceinline__ int64_t total(const Args &a) const {
        if (k0 >= R) return 0;
        if constexpr (ONE) return tiles(a, 0) + kHead;
        else return before(a, R - 1) + tiles(a, R - 1) + kHead;
    }
    // The row tile that tile `off` of the sequence, heads included, falls in; off then counts from its start.
    __host__ __device__ __forceinline__ void find(const Args &a, int64_t &off) {
        k = k0;
        if constexpr (!ONE) {
            int hi = R;  // the last k with before(k) <= off
            while (hi - k > 1) {
                const int mid = (k + hi) >> 1;
                if (before(a, mid) <= off) k = mid;
                else hi = mid;
            }
            off -= before(a, k);
        }
    }
};

// A CTA's (or CTA pair's) share of all contexts' tiles laid end to end, heads included: `parts` equal shares at
// most, this one from tile `off` of context (w.s, w.k) on, `left` tiles.
template <int N, int TOK, bool ONE>
struct Share {
    Walk<N, TOK, ONE> w;
    int64_t off, left, last, total;
    int parts;
    bool over;   // the context of w has been handed out
    bool blind;  // some sequence s with s mod `most` = id has queries that see nothing

    int after;  // tiles of the last piece's context behind it

    // The next piece of the share, false if there is none.
    __device__ __forceinline__ bool take(const Args &a, Piece &pc) {
        while (left > 0) {
            if (over) {
                if (++w.k >= w.R) do {
                    if (w.s + 1 >= a.S) return false;  // lengths that changed under the call
                    w.open(a, w.s + 1);
                } while (w.k0 >= w.R);
                off = 0;
            }
            over = true;
            // of the context's kHead + nt tiles, `n` from `off` on are this share's
            const int nt = w.tiles(a, w.k);
            const int n = (int)min((int64_t)nt + kHead - off, left);
            const int i0 = max(0, (int)off - kHead), i1 = max(0, (int)off + n - kHead);
            left -= n;
            if (i1 == i0) continue;
            pc.tiles = i1 - i0;
            pc.t0 = i0 * TOK;
            pc.end = w.end(a, w.k);
            pc.qh0 = w.k * N;
            pc.row0 = w.q0 * a.H + pc.qh0;
            pc.rows = min(N, w.nH - pc.qh0);
            pc.lim0 = w.p0 + 1;
            pc.seq = w.s;
            pc.out = pc.tiles == nt ? 0 : i0 == 0 ? 1 : 2;
            after = nt - i1;
            return true;
        }
        return false;
    }
    // How many shares, from this one (`id`) on, hold parts of the context that begins here and is cut, once the last
    // piece is taken: it ends `after` tiles behind the share.
    __device__ __forceinline__ int reach(int id) const { return (int)(share_owner(last + after - 1, total, parts) - id) + 1; }
};

// Zeros for a sequence's queries that see nothing, but for those in a row tile with others; by thread `me` of `threads`.
template <int N, int TOK, bool ONE>
__device__ __forceinline__ void zero_blind(const Args &a, const Walk<N, TOK, ONE> &w, int me, int threads) {
    const int64_t vecs = min((int64_t)w.k0 * N, (int64_t)w.nH) * (a.V / 8);
    uint4 *o = reinterpret_cast<uint4 *>((unsigned char *)a.out + (int64_t)w.q0 * a.H * a.V * 2);
    for (int64_t i = me; i < vecs; i += threads) o[i] = make_uint4(0, 0, 0, 0);
}

// Share `id` of at most `most`: each of the block's `threads` threads sums the tiles of a run of sequences, and
// the one whose run holds the share's first tile finds it.  By the whole block; `scratch`: 1 KB of shared memory,
// free after the block's next barrier.
template <int N, int TOK, bool ONE>
__device__ __forceinline__ Share<N, TOK, ONE> locate(const Args &a, float *scratch, int id, int most, int threads) {
    int64_t *scan = reinterpret_cast<int64_t *>(scratch);  // the warps' totals; then where the share begins
    Walk<N, TOK, ONE> &begin = *reinterpret_cast<Walk<N, TOK, ONE> *>(scan + 18);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int run = (a.S + threads - 1) / threads;
    const int sb = min(a.S, (int)threadIdx.x * run), se = min(a.S, sb + run);
    int64_t mine = 0;
    bool blind = false;
    Share<N, TOK, ONE> r;
    Walk<N, TOK, ONE> &w = r.w;
    if (a.whole) {
        const int s = id / a.whole, k = id - s * a.whole;
        r.off = r.left = r.last = r.total = r.parts = 0;
        r.over = r.blind = false;
        if (s >= a.S) return r;
        w.open(a, s);
        if (k == 0) {
            if (w.flagged && threadIdx.x == 0) flag_error(a.err, PKV_DEVERR_SEQ_LEN);
            zero_blind(a, w, threadIdx.x, threads);
        }
        w.k = k;
        if (k >= w.k0 && k < w.R) r.left = w.tiles(a, k) + kHead;
        return r;
    }
    for (int s = sb; s < se; ++s) {
        w.open(a, s);
        mine += w.total(a);
        if ((w.flagged || w.k0 > 0) && s % most == id) {
            if (w.flagged) flag_error(a.err, PKV_DEVERR_SEQ_LEN);
            blind |= w.k0 > 0;
        }
    }
    int64_t incl = mine;
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    r.blind = __syncthreads_or(blind);
    int64_t base = 0, total = 0;
    for (int i = 0; i < threads / 32; ++i) {
        if (i < warp) base += scan[i];
        total += scan[i];
    }
    const int64_t excl = base + incl - mine;
    // The least share grows with the root of a context's tiles: what a context's pieces cost to join grows with their
    // number (16000 tokens alone: 23.0 us with shares of 2 tiles, 18.7 with 4; two of 600 to 1500: 10.8 and 11.6).
    const int least = max(2, (int)sqrtf((float)total / (16.f * (float)a.S)));
    int parts = total >= (int64_t)most * least ? most : (int)total / least;
    if (parts < 1) parts = 1;
    int64_t first = 0, last = 0;
    if (id < parts && total < (1 << 24)) {  // 32-bit division is a fifth of the time (id < 256)
        first = (uint32_t)id * (uint32_t)total / (uint32_t)parts;
        last = (uint32_t)(id + 1) * (uint32_t)total / (uint32_t)parts;
    } else if (id < parts) {
        first = (int64_t)id * total / parts;
        last = (int64_t)(id + 1) * total / parts;
    }
    if (first < last && first >= excl && first < excl + mine) {
        int64_t off = first - excl;
        for (int s = sb; run > 1; ++s) {
            w.open(a, s);
            const int64_t t = w.total(a);
            if (off < t || s + 1 >= se) break;
            off -= t;
        }
        w.find(a, off);
        begin = w;
        scan[16] = off;
    }
    __syncthreads();
    r.w = begin;
    r.off = scan[16], r.left = last - first, r.last = last, r.total = total, r.parts = parts, r.over = false;
    return r;
}

// What is left for the join of a context that is cut: first row, rows, pieces (one in each of as many shares), and the
// first piece's share; 0 pieces: nothing to join.
__device__ __forceinline__ void leave(int *rec, int row0, int rows, int pieces, int share) {
    *reinterpret_cast<int4 *>(rec) = make_int4(row0, rows, pieces, share);
}

// The same for sequences first, first + step, ...; and, where `rec` has a record for each context, those of sequences without
// tokens: nothing to join.
template <int N, int TOK, bool ONE>
__device__ __forceinline__ void zero_blind(const Args &a, int first, int step, int me, int threads, int *rec) {
    for (int s = first; s < a.S; s += step) {
        Walk<N, TOK, ONE> w;
        w.open(a, s);
        zero_blind(a, w, me, threads);
        if (rec && me == 0 && w.k0 >= w.R) leave(rec + 4 * s, 0, 0, 0, 0);
    }
}

// The block tables, read later one entry after another, on their way into L2; line after line over the CTAs, so that
// each SM has the tables' pages at hand.
__device__ __forceinline__ void prefetch_tables(const Args &a, int64_t line) {
    if ((int64_t)a.S * a.maxb <= 1 << 17 && line * 32 < (int64_t)a.S * a.maxb)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.tables + line * 32));
}

// Whether every context of a call gets a share of its own, uncut, and nothing is left to join by a second kernel: there
// are shares enough, and the longest context there may be has few tiles (of `tok` tokens: 64, also where the kernel's are 48,
// or 128 in pairs of CTAs) -- 4, and up to 10 the more of the shares are
// in use (lengths differ: the limit is for contexts that are half of it on average).  Uncut against cut, in us from graphs, 32
// heads: 4 sequences of 64 / 128 / 256 tokens 7.8 / 8.6 / 11.2 against 9.7 / 11.0 / 11.2, and (uncut by hand) 384 / 512 tokens
// 12.6 / 15.3 against 11.2 / 11.1; 64 sequences of 64 / 256 / 384: 7.9 / 12.0 / 14.3 against 10.1 / 15.3 / 18.2, by hand 512 /
// 1024: 17.5 / 27.6 against 19.0 / 25.0; in pairs (128 heads), 64 sequences of 256 / 512 / 768: 11.7 / 17.2 / 21.3 against 20.7 /
// 25.3 / 30.0.  The longest context is what the call's max_seq_len and the block table's width allow.
// Returns the row tiles to count a sequence for, or 0.
inline int whole_contexts(const Args &a, int n, int tok, int shares) {
    const int64_t tiles = (int64_t)a.rows / n + (a.rows % n != 0), most = (int64_t)a.maxb * a.B;
    const int64_t len = a.max_len < most ? a.max_len : most, contexts = a.S * tiles;
    if (contexts > shares) return 0;
    return len <= (4 + 6 * contexts / shares) * tok ? (int)tiles : 0;
}

// Whether a call's cache rows are the first to leave L2: each is read by one row tile, and the pool, one layer's, is a
// quarter of L2 or more, so that no row is found there at the next step.  Block tables, queries, partial results and the
// kernels' code then stay: 64 contexts of 64 to 2048 tokens, 32 heads, 26.2 -> 24.9 us, 128 heads 33.9 -> 32.7; 8 of 16000,
// 64 heads, 45.0 -> 42.2.  Where it is not done: a pool of 18 MB read again and again, 18.8 us against 20.0; 8 x 512 queries
// of 4096, whose rows are read by 128 row tiles, 674 against 894 (all from graphs).
inline bool read_once(const Args &a, int n) {
    return a.rows <= n && (int64_t)a.NB * a.B * (a.V + kRope) * 2 >= 32 << 20;
}

// A tensor map takes the driver half a microsecond to encode; a call has three to six, of the same shapes in every step of
// a serving loop.  The last few of a thread are kept by their shapes, and given this call's address.
struct MapShape {
    int dims, swizzle;
    uint64_t size[3], stride[2];
    uint32_t box[3];
};
inline bool make_map(CUtensorMap *map, void *base, const MapShape &sh) {
    struct Kept {
        MapShape shape;
        CUtensorMap map;
    };
    constexpr unsigned kKept = 16;
    static thread_local Kept kept[kKept];
    static thread_local unsigned used = 0;
    static const PFN_cuTensorMapReplaceAddress_v12000 replace = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapReplaceAddress", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapReplaceAddress_v12000>(p) : nullptr;
    }();
    if (replace)
        for (unsigned i = 0; i < kKept && i < used; ++i) {
            const MapShape &k = kept[i].shape;
            if (k.dims == sh.dims && k.swizzle == sh.swizzle && k.size[0] == sh.size[0] && k.size[1] == sh.size[1] && k.size[2] == sh.size[2] &&
                k.stride[0] == sh.stride[0] && k.stride[1] == sh.stride[1] && k.box[0] == sh.box[0] && k.box[1] == sh.box[1] &&
                k.box[2] == sh.box[2]) {
                *map = kept[i].map;
                return replace(map, base) == CUDA_SUCCESS;
            }
        }
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t size[3] = {sh.size[0], sh.size[1], sh.size[2]}, stride[2] = {sh.stride[0], sh.stride[1]};
    const cuuint32_t step[3] = {1u, 1u, 1u};
    if (enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)sh.dims, base, size, stride, sh.box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            (CUtensorMapSwizzle)sh.swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return false;
    Kept &k = kept[used++ % kKept];
    if (used >= 2 * kKept) used -= kKept;
    k.shape = sh;
    k.map = *map;
    return true;
}

// Rows of V + 64 entries as [chunk of 64 entries][row][64]: a box of `box` rows and `deep` chunks.
inline bool make_rows_map(CUtensorMap *map, const void *base, int64_t rows, int V, int box, int deep) {
    return make_map(map, const_cast<void *>(base),
                    MapShape{3, CU_TENSOR_MAP_SWIZZLE_128B, {64u, (uint64_t)rows, (uint64_t)(V / 64 + 1)}, {(uint64_t)(V + kRope) * 2, 128u},
                             {64u, (uint32_t)box, (uint32_t)deep}});
}

}  // namespace latent
}  // namespace pkv
