// Latent attention on the 5th-generation tensor cores (bf16).
//
// A row tile is up to N (16, 32 or 64) consecutive query rows of one sequence, a
// row being one head of one query; a decode step's heads, or the heads of a few
// drafted tokens, are one.  It is attended against tiles of 48 or 64 tokens, transposed:
//     S^T = C Q^T   [64 tokens x N rows]        (C: the tile's cache rows, 9 or 5 chunks of 64 entries)
//     O^T += L^T P^T [V entries x N rows]       (L: the latent part of C, P = exp2(S scale - ref))
// so the tile itself is the wide operand of both products, read once into shared
// memory for both, a context's row count costs no padding to 128, and O^T (V / 128
// blocks of N columns) and two S^T fit tensor memory for every N up to 64 -- O of 128
// rows alone would fill it.
//
// The cache rows of 8 tokens are one TMA box [chunk][8 rows][128 bytes]: any block
// size from 8 on, six or eight boxes a tile, and both products see 128-byte swizzled
// operands (C by rows, L^T by columns) whose 8-token groups are one stride apart.
//
// Softmax: four warps, or two sets of four; a thread holds two tokens of every fourth pair of columns.
// Maxima over tokens would be shuffles over lanes, so the reference of a row moves
// only when a score passes it by 2^kSlack: usually in the first tile alone.  Sums of
// weights stay in the threads, per token, until the end of the piece.  Weights are
// rounded to bf16 (by 2^-8 of each at most; the sums they are divided by are of the
// rounded weights, in float32).
//
// All contexts' tiles are laid end to end and cut into equal shares, one a CTA.  A
// context cut by share boundaries leaves partial results that a second kernel joins.
//
// What bounds it: DRAM while tiles stream (what 32000 tokens more a context cost, 8 contexts: 6.7 TB/s at 16 and 32 rows,
// 6.3 at 64, of 6.7), before that a chain of loads (lengths, block table, first tile: 3.2 us until it is asked for), after
// it the join (1.2 us between the kernels, 4 in it), and shares that are equal in tiles but end up to 8 us apart.  64 contexts
// of 64 to 2048 tokens, 32 heads: 24.9 us for 73 MB (all times here from CUDA graphs of many calls); 8 of 16000, 64 heads:
// 41.2 us for 149 MB.  Joined in this kernel, by CTAs that wait for one another's pieces (two stages, as
// below), one context of 16000 took 20.0 us, not 22.7, but these 26.7 and 43.7, not 26.5 and 42.5, and 1 to 2 us more from a
// host's stream of calls: such a launch is a cooperative one.
// A tile of 64 takes 36 + 16 products, 1452 cycles at 16 rows, 1920 at 64 (operand bytes out of
// shared memory); 3200 is its share of DRAM.
#include <cmath>

#include "latent_tc.cuh"

namespace pkv {
namespace latent {

namespace {

__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// 16 entries x N rows of O^T (one warp's ld_16x256b: lane / 4 and 8 on the entries, 2 (lane mod 4)
// and the next of every 8 the rows), each row times its factor, to bf16 rows `out` of V entries:
// transposed through N * 32 bytes of shared memory, in 16-byte stores.
template <int V, int N>
__device__ __forceinline__ void emit(const float (&o)[N / 2], const float (&inv)[N / 8][2], uint32_t stage, int lane, __nv_bfloat16 *out,
                                     int rows) {
    const int h = (lane >> 3) & 1;
#pragma unroll
    for (int j = 0; j < N / 8; j += 2) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int jj = j + (e >> 1), at = 4 * jj + 2 * (e & 1);
            w[e] = pack_bf16x2(o[at] * inv[jj][0], o[at + 1] * inv[jj][1]);
        }
        const int c = 8 * (j + (lane >> 4)) + (lane & 7);
        stmatrix_x4_trans(stage + (uint32_t)(c * 32 + ((h ^ ((c >> 2) & 1)) << 4)), w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
        const int c = (lane + 32 * i) >> 1, hh = lane & 1;
        const float4 v = lds128(stage + (uint32_t)(c * 32 + ((hh ^ ((c >> 2) & 1)) << 4)));
        if (c < rows) *reinterpret_cast<float4 *>(out + (int64_t)c * V + 8 * hh) = v;
    }
    __syncwarp();
}

template <int V, int N>
struct L {
    static constexpr int kChunks = V / 64 + 1;
    // Tokens of a tile: 64, or 48 where three stages of those fit and two of 64: a stage is loaded anew when its tile's last
    // product is done, and with two nothing is under way for half of that time.  64 contexts of 64 to 2048, 32 heads, 26.5 ->
    // 24.8 us, 140, 16 heads, 38.9 -> 35.9, one of 16000 22.6 -> 18.9; some with few tiles to a share got slower: 4 of
    // 64, 32 heads, 7.1 -> 7.6, 16 of 1024, 16 heads, 11.5 -> 12.4, 20 x 4 queries of 8 heads 18.8 -> 19.4.  Five stages of 32
    // tokens: 26.0, 37.9, 25.4.  (A product's 64 rows then reach into what lies behind the tile, for scores that no one
    // looks at.)
    static constexpr int kTok = V == 512 && N <= 32 ? 48 : 64, kAll = (1 << kTok / 8) - 1;
    static constexpr int kGroup = kChunks * 1024;  // bytes of 8 tokens
    static constexpr int kTile = kTok / 8 * kGroup;
    static constexpr int kPart0 = V / 64 - 2;      // chunks of the tile's first part; the second, awaited last, has three
    static constexpr int kQ = kChunks * N * 128;
    static constexpr int kQBufs = N <= 16 || (V == 256 && N == 32) ? 2 : 1;  // the next piece's queries are loaded under this one's, where they fit
    static constexpr int kP = 64 * 128;
    // softmax warps: four for each 32 rows of 64 (a tile of 64 rows keeps four busy for 1000 cycles), else four
    static constexpr int kSets = N >= 32 ? 2 : 1, kCols1 = N / kSets, kSoftmax = 128 * kSets;
    static constexpr int kThreads = 96 + kSoftmax;  // and a producer, and a warp that issues each product
    static constexpr int kMisc = 3 * 1024;
    static constexpr int kMax = 232448;  // shared memory of a CTA
    static constexpr int kStages = (kMax - kMisc - kQBufs * kQ - kP) / kTile < 4 ? (kMax - kMisc - kQBufs * kQ - kP) / kTile : 4;
    static constexpr int ring = 0, q = kStages * kTile, p = q + kQBufs * kQ, misc = p + kP;
    static constexpr int total = misc + kMisc;
    static_assert((8 - kTok / 8) * kGroup <= kQBufs * kQ, "the last stage's product ends in Q");
    static constexpr int kBlocks = V / 128;              // of O^T
    static constexpr uint32_t kS = kBlocks * N;          // first column of S^T
    static constexpr uint32_t kCols = kS + 2 * N <= 128 ? 128 : kS + 2 * N <= 256 ? 256 : 512;
    static_assert(kStages >= 2 && total <= kMax, "shared memory");
    static_assert(kS + 2 * N <= kCols, "tensor memory");
};

struct alignas(8) Misc {
    uint64_t full[2][4], empty[2][4], q_full[2], q_empty[2], s_full[2], s_free[2], p_full, pv_done, o_free, desc_full[kDescs], desc_empty[kDescs], fin[2];
    Piece piece[kDescs];
    float red[4][64];
    int lim[64];         // tokens that a row of the piece sees
    uint32_t nf[2][64];  // by each set's rows: exponents of a token's scores, all of them together
    uint32_t groups[4];  // valid 8-token groups of a stage's tile
    uint32_t tmem;
    int dead;
};
static_assert(sizeof(Misc) <= 3 * 1024, "misc");

struct Ws {
    int *rec;      // [shares][4]: what the context that begins in a share left for the join; or one for each context
    float *o;      // [shares][2][N][V]
    float *ml;     // [shares][2][2][N]: reference (base 2), sum of weights
};
inline size_t ws_bytes(int shares, int n, int v) {
    return (size_t)shares * 16 + (size_t)shares * 2 * n * (v + 2) * 4 + 512;
}
__device__ __forceinline__ Ws ws_of(const Args &a, int shares, int n, int v) {
    Ws w;
    w.o = (float *)a.ws;
    w.ml = w.o + (size_t)shares * 2 * n * v;
    w.rec = (int *)(w.ml + (size_t)shares * 2 * 2 * n);
    return w;
}

template <int V, int N>
__global__ void __launch_bounds__(L<V, N>::kThreads, 1)
latent_mma_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_c0,
                  const __grid_constant__ CUtensorMap tm_c1, const __grid_constant__ Args a, int by_context) {
    using X = L<V, N>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Misc &m = *reinterpret_cast<Misc *>(smem + X::misc);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = gridDim.x, cta = blockIdx.x;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 8; ++i) mbar_init(&m.full[i >> 2][i & 3], 1), mbar_init(&m.empty[i >> 2][i & 3], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&m.q_full[i], 1), mbar_init(&m.q_empty[i], 1);
        mbar_init(&m.s_full[0], 1), mbar_init(&m.s_full[1], 1);
        mbar_init(&m.s_free[0], 4 * X::kSets), mbar_init(&m.s_free[1], 4 * X::kSets);
        mbar_init(&m.p_full, 4 * X::kSets), mbar_init(&m.pv_done, 1), mbar_init(&m.o_free, 4 * X::kSets), mbar_init(&m.fin[0], 1), mbar_init(&m.fin[1], 1);
        for (int i = 0; i < kDescs; ++i) mbar_init(&m.desc_full[i], 1), mbar_init(&m.desc_empty[i], 2 + 4 * X::kSets);
        m.dead = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == 32) {
        prefetch_map(&tm_q), prefetch_map(&tm_c0), prefetch_map(&tm_c1);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&m.tmem)), "r"(X::kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    grid_dependency_wait();
    // the join kernel, which waits for this one before it reads (no other: attention kernels read queries before they wait)
    if (!a.whole) grid_launch_dependents();

    prefetch_tables(a, (int64_t)threadIdx.x * G + cta);
    Share<N, X::kTok, true> sh = locate<N, X::kTok, true>(a, &m.red[0][0], cta, G, X::kThreads);
    const Ws ws = ws_of(a, G, N, V);
    if (threadIdx.x == 0 && !by_context && !a.whole) leave(ws.rec + 4 * cta, 0, 0, 0, 0);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = m.tmem;

    bool dead = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) {  // by whole warps
        if (!dead && !__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) dead = wait_on(bar, parity, &m.dead, a.err);
    };

    if (warp == 0) {
        // ======================= producer =======================
        const uint64_t policy = row_policy(a);
        int tile = 0, np = 0, nq = 0, halves = 0;  // tiles, pieces, queries and parts of tiles issued
        for (;;) {
            const int d = np % kDescs;
            wait(&m.desc_empty[d], (uint32_t)(np / kDescs + 1) & 1u);
            Piece pc;
            const bool more = !dead && sh.take(a, pc);
            if (!more) pc.tiles = 0;
            if (lane == 0) {
                m.piece[d] = pc;
                mbar_arrive(&m.desc_full[d]);
            }
            __syncwarp();
            if (!more) break;
            const int n = pc.tiles;
            const int32_t *table = a.tables + (int64_t)sh.w.s * a.maxb;
            // lane l: the cache row of group l & 7 of tile t + (l >> 3); -1: a bad block; -2: no token
            auto look = [&](int t) {
                const int tok = pc.t0 + (t + (lane >> 3)) * X::kTok + 8 * (lane & 7);
                if (t + (lane >> 3) >= n || tok >= pc.end || (lane & 7) >= X::kTok / 8) return -2;
                const int blk = __ldg(table + (tok >> a.bshift));
                return (unsigned)blk < (unsigned)a.NB ? (blk << a.bshift) + (tok & (a.B - 1)) : -1;
            };
            auto load_q = [&] {
                const int qb = np % X::kQBufs;
                wait(&m.q_empty[qb], (uint32_t)(np / X::kQBufs + 1) & 1u);
                if (dead) return;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&m.q_full[qb], (uint32_t)X::kQ);
                    tma_load_3d(smem_u32(smem + X::q) + (uint32_t)(qb * X::kQ), &tm_q, smem_u32(&m.q_full[qb]), 0, pc.row0, 0);
                }
                ++nq;
                __syncwarp();
            };
            int row = look(0), next = -2;
            if (X::kQBufs == 2 || np == 0) load_q();
            for (int t = 0; t < n && !dead; ++t, ++tile) {
                if ((t & 3) == 0) {
                    if (t) row = next;
                    next = look(t + 4);
                }
                const int st = tile % X::kStages;
                const bool turn = (lane >> 3) == (t & 3) && (lane & 7) < X::kTok / 8;
                // a group without tokens starts past the tensor's end: zeros
                const int y = row >= 0 ? row : a.NB << a.bshift;
                const uint32_t dst = smem_u32(smem + X::ring) + (uint32_t)(st * X::kTile + (lane & 7) * X::kGroup);
                wait(&m.empty[0][st], (uint32_t)(tile / X::kStages + 1) & 1u);
                if (dead) break;
                if (turn && row == -1) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                const uint32_t ok = __ballot_sync(0xffffffffu, row >= 0) >> (8 * (t & 3)) & 0xffu;
                if (lane == 0) {
                    m.groups[st] = ok;
                    mbar_arrive_expect_tx(&m.full[0][st], (uint32_t)(X::kTok * 128 * X::kPart0));
                }
                __syncwarp();
                if (turn) tma_load_3d_hint(dst, &tm_c0, smem_u32(&m.full[0][st]), 0, y, 0, policy);
                ++halves;
                wait(&m.empty[1][st], (uint32_t)(tile / X::kStages + 1) & 1u);
                if (dead) break;
                if (lane == 0) mbar_arrive_expect_tx(&m.full[1][st], (uint32_t)(X::kTile - X::kTok * 128 * X::kPart0));
                __syncwarp();
                if (turn) tma_load_3d_hint(dst + X::kPart0 * 1024, &tm_c1, smem_u32(&m.full[1][st]), 0, y, X::kPart0, policy);
                ++halves;
                if (X::kQBufs == 1 && np > 0 && t == 0) load_q();
                // The tile that this stage takes next, into L2 (64 rows: 8 x 16000 42.5 -> 41.2 us; with three stages no gain,
                // and 36.0 -> 38.9 for 140 contexts of 16 heads).
                if constexpr (X::kStages == 2) {
                    const int ahead = (t & 3) < 2 ? row : next;
                    if ((lane >> 3) == ((t + 2) & 3) && ahead >= 0) prefetch_rows<V>(a, ahead);
                }
            }
            if (lane == 0) {
                if (a.whole) {
                } else if (by_context && pc.out != 2) leave(ws.rec + 4 * pc.seq, pc.row0, pc.rows, pc.out ? sh.reach(cta) : 0, cta);
                else if (pc.out == 1) leave(ws.rec + 4 * cta, pc.row0, pc.rows, sh.reach(cta), cta);
            }
            ++np;
        }
        // no copy outlives the CTA, whoever else gave up
        for (int i = max(0, halves - 2 * X::kStages); i < halves; ++i)
            mbar_wait_bounded(&m.full[i & 1][(i >> 1) % X::kStages], (uint32_t)((i >> 1) / X::kStages) & 1u);
        for (int i = max(0, nq - X::kQBufs); i < nq; ++i) mbar_wait_bounded(&m.q_full[i % X::kQBufs], (uint32_t)(i / X::kQBufs) & 1u);
    } else if (warp == 1) {
        // ======================= issuer of S^T = C Q^T =======================
        constexpr uint32_t id = idesc(64, N, false, false);
        const bool leader = elect_one();
        const uint64_t qd = tc::smem_desc(smem_u32(smem + X::q), 16, 1024);
        const uint64_t cd = tc::smem_desc(smem_u32(smem + X::ring), 16, X::kGroup);
        for (int np = 0, tile = 0;; ++np) {
            const int d = np % kDescs;
            wait(&m.desc_full[d], (uint32_t)(np / kDescs) & 1u);
            const int n = dead ? 0 : m.piece[d].tiles;
            if (n == 0) break;
            const int qb = np % X::kQBufs;
            wait(&m.q_full[qb], (uint32_t)(np / X::kQBufs) & 1u);
            for (int t = 0; t < n; ++t, ++tile) {
                const int st = tile % X::kStages;
                wait(&m.s_free[tile & 1], (uint32_t)((tile >> 1) + 1) & 1u);
                const uint64_t c0 = cd + (uint64_t)(st * (X::kTile >> 4)), q0 = qd + (uint64_t)(qb * (X::kQ >> 4));
                auto part = [&](int lo, int hi) {
#pragma unroll 1
                    for (int c = lo; c < hi; ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc::mma(tmem + X::kS + (uint32_t)((tile & 1) * N), c0 + (uint64_t)((c * 1024 + k * 32) >> 4),
                                    q0 + (uint64_t)((c * N * 128 + k * 32) >> 4), id, c + k > 0 ? 1u : 0u);
                };
                wait(&m.full[0][st], (uint32_t)(tile / X::kStages) & 1u);
                if (dead) break;
                tc::fence_after();
                if (leader) part(0, X::kPart0);
                __syncwarp();
                wait(&m.full[1][st], (uint32_t)(tile / X::kStages) & 1u);
                if (dead) break;
                if (leader) {
                    part(X::kPart0, X::kChunks);
                    tc::commit(&m.s_full[tile & 1]);
                    if (t + 1 == n) tc::commit(&m.q_empty[qb]);
                }
                __syncwarp();
            }
            if (dead) break;
            if (lane == 0) mbar_arrive(&m.desc_empty[d]);
        }
        if (leader) tc::commit(&m.fin[0]);
        __syncwarp();
        mbar_wait_bounded(&m.fin[0], 0);  // every product has ended before the memory goes
    } else if (warp == 2) {
        // ======================= issuer of O^T += L^T P^T =======================
        constexpr uint32_t id = idesc(128, N, true, true);
        const bool leader = elect_one();
        const uint64_t pd = tc::smem_desc(smem_u32(smem + X::p), 1024, 1024);
        const uint64_t ld = tc::smem_desc(smem_u32(smem + X::ring), 1024, X::kGroup);
        for (int np = 0, tile = 0;; ++np) {
            const int d = np % kDescs;
            wait(&m.desc_full[d], (uint32_t)(np / kDescs) & 1u);
            const int n = dead ? 0 : m.piece[d].tiles;
            if (n == 0) break;
            if (np > 0) wait(&m.o_free, (uint32_t)(np - 1) & 1u);
            for (int t = 0; t < n; ++t, ++tile) {
                const int st = tile % X::kStages;
                wait(&m.p_full, (uint32_t)tile & 1u);
                wait(&m.full[0][st], (uint32_t)(tile / X::kStages) & 1u);  // (complete: orders the reads of the tile)
                wait(&m.full[1][st], (uint32_t)(tile / X::kStages) & 1u);
                if (dead) break;
                tc::fence_after();
                if (leader) {
                    const uint64_t l0 = ld + (uint64_t)(st * (X::kTile >> 4));
#pragma unroll 1
                    for (int b = 0; b < X::kBlocks; ++b) {
#pragma unroll
                        for (int k = 0; k < X::kTok / 16; ++k)
                            tc::mma(tmem + (uint32_t)(b * N), l0 + (uint64_t)((b * 2048 + k * 2 * X::kGroup) >> 4),
                                    pd + (uint64_t)((k * 2048) >> 4), id, t == 0 && k == 0 ? 0u : 1u);
                        if (2 * b + 2 == X::kPart0) tc::commit(&m.empty[0][st]);
                    }
                    tc::commit(&m.empty[1][st]);
                    tc::commit(&m.pv_done);
                }
                __syncwarp();
            }
            if (dead) break;
            if (lane == 0) mbar_arrive(&m.desc_empty[d]);
        }
        if (leader) tc::commit(&m.fin[1]);
        __syncwarp();
        mbar_wait_bounded(&m.fin[1], 0);
    } else {
        // ======================= softmax and epilogue =======================
        const int qt = warp & 3;  // quarter of the tensor memory's lanes
        const uint32_t lanes = tmem + ((uint32_t)(qt * 32) << 16);
        constexpr int NL = X::kCols1, J = NL / 8;
        const int set = (warp - 3) >> 2;  // which of the rows
        const float sc = a.scale_log2;
        const uint32_t idle = qt * 16 >= X::kTok ? ~0u : 0u;  // this warp's tokens are none of the tile's
        const int col = set * NL + 2 * (lane & 3), tok0 = qt * 16 + (lane >> 2);  // first column, first token (the other: 8 on)
        // stmatrix: lane gives the address of row (lane & 7) of matrix lane >> 3: tokens 0-7, 8-15 of column block j, then j + 1
        const uint32_t p_s = smem_u32(smem + X::p) + (uint32_t)((qt * 2 + ((lane >> 3) & 1)) * 1024 + (lane & 7) * 128);
        if (sh.blind) zero_blind<N, X::kTok, true>(a, cta, G, threadIdx.x - 96, X::kSoftmax, by_context ? ws.rec : nullptr);
        int tile = 0;
        bool stop = false;  // the softmax warps leave together: they share a barrier
        for (int np = 0;; ++np) {
            const int d = np % kDescs;
            wait(&m.desc_full[d], (uint32_t)(np / kDescs) & 1u);
            if (softmax_any<X::kSoftmax>(dead)) break;
            const Piece pc = m.piece[d];
            if (pc.tiles == 0) break;
            float nref[J][2], l[J][2];  // minus the reference: +inf before the first score
#pragma unroll
            for (int j = 0; j < J; ++j) nref[j][0] = nref[j][1] = INFINITY, l[j][0] = l[j][1] = 0.f;
            if (threadIdx.x - 96 < N) m.lim[threadIdx.x - 96] = min(pc.end, pc.lim0 + by_heads(a, pc.qh0 + (int)threadIdx.x - 96));
            softmax_sync<X::kSoftmax>();
            const int least = m.lim[0];  // tokens that the first row sees
            for (int t = 0; t < pc.tiles; ++t, ++tile) {
                const int st = tile % X::kStages;
                wait(&m.s_full[tile & 1], (uint32_t)(tile >> 1) & 1u);
                wait(&m.full[0][st], (uint32_t)(tile / X::kStages) & 1u);  // (complete: orders the read of groups)
                tc::fence_after();
                uint32_t r[4 * J];
                ld_16x256b(lanes + X::kS + (uint32_t)((tile & 1) * N + set * NL), r);
                tc::wait_ld();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.s_free[tile & 1]);
                const int tb = pc.t0 + t * X::kTok;
                const uint32_t groups = m.groups[st];
                const bool masked = tb + X::kTok > least || groups != X::kAll;
                bool bad[2] = {false, false};
                uint32_t hide[2] = {idle, idle};  // bit 2 j + i: not seen by column 8 j + col + i
                if (masked) {
                    const bool in[2] = {((groups >> (2 * qt)) & 1u) != 0, ((groups >> (2 * qt + 1)) & 1u) != 0};
                    uint32_t nf[2] = {0x7f800000u, 0x7f800000u};
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int c = 8 * j + col + i;
                            const int lim = m.lim[c];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (c < pc.rows) nf[h] &= r[4 * j + 2 * h + i];
                                if (!in[h] || tb + tok0 + 8 * h >= lim) hide[h] |= 1u << (2 * j + i);
                            }
                        }
                    // A row of the cache whose latent part holds an infinity or NaN gives every query a score that is no
                    // number.  It must not reach, through 0 * inf, the rows that do not see it: its latent part is
                    // zeroed here, after its scores were taken, and those that see it get NaN.  (So are rows past
                    // the last token that hold one.)  Scores alone do not tell: finite entries whose products pass
                    // float32's range give every query one too, so the latent part itself is looked at.
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        nf[h] &= __shfl_xor_sync(0xffffffffu, nf[h], 1);
                        nf[h] &= __shfl_xor_sync(0xffffffffu, nf[h], 2);
                    }
                    if constexpr (X::kSets == 2) {
                        if ((lane & 3) == 0) m.nf[set][tok0] = nf[0], m.nf[set][tok0 + 8] = nf[1];
                        softmax_sync<X::kSoftmax>();
                        nf[0] &= m.nf[set ^ 1][tok0], nf[1] &= m.nf[set ^ 1][tok0 + 8];
                    }
                    const bool suspect[2] = {!idle && (nf[0] & 0x7f800000u) == 0x7f800000u, !idle && (nf[1] & 0x7f800000u) == 0x7f800000u};
                    if (__any_sync(0xffffffffu, suspect[0] || suspect[1])) {  // (alike in the two sets' warps of these tokens)
                        wait(&m.full[1][st], (uint32_t)(tile / X::kStages) & 1u);  // (complete: orders the reads of the tile)
                        auto latent = [&](int h, int c, int e) {  // 16 bytes of token h's latent part
                            const int tk = tok0 + 8 * h;
                            return reinterpret_cast<uint4 *>(smem + X::ring + st * X::kTile + (tk >> 3) * X::kGroup + (tk & 7) * 128 + c * 1024 + e * 16);
                        };
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (suspect[h])
                                for (int c = lane & 3; c < V / 64; c += 4)
                                    for (int e = 0; e < 8; ++e) bad[h] |= not_finite(*latent(h, c, e));
                            bad[h] |= __shfl_xor_sync(0xffffffffu, (int)bad[h], 1) != 0;
                            bad[h] |= __shfl_xor_sync(0xffffffffu, (int)bad[h], 2) != 0;
                        }
                        // both sets have looked before one of them zeroes
                        if constexpr (X::kSets == 2) asm volatile("barrier.cta.sync %0, 64;" ::"r"(2 + qt) : "memory");
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (bad[h] && set == 0)
                                for (int c = lane & 3; c < V / 64; c += 4)
                                    for (int e = 0; e < 8; ++e) *latent(h, c, e) = make_uint4(0, 0, 0, 0);
                    }
                }
                // x: log2 of the weights against the references.  Once, if no score passes its row's reference by far; else
                // against 0 where there is none yet, for new references, and a third time.  (A rolled loop: this code is
                // fetched for every tile.)
                float x[4 * J], blank = INFINITY;
#pragma unroll 1
                for (int pass = 0;; ++pass) {
                    float top = -INFINITY;
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float nr = nref[j][i] == INFINITY ? blank : nref[j][i];
                            x[4 * j + i] = fmaf(__uint_as_float(r[4 * j + i]), sc, nr);
                            x[4 * j + 2 + i] = fmaf(__uint_as_float(r[4 * j + 2 + i]), sc, nr);
                        }
                    if (masked || idle)
#pragma unroll
                        for (int e = 0; e < 4 * J; ++e) {
                            const int h = (e >> 1) & 1;
                            x[e] = (hide[h] >> (2 * (e >> 2) + (e & 1))) & 1u ? -INFINITY : bad[h] ? __uint_as_float(0x7fffffffu) : x[e];
                        }
#pragma unroll
                    for (int e = 0; e < 4 * J; e += 2) top = max3_nan(top, x[e], x[e + 1]);
                    if (pass == 2) break;
                    if (pass == 0) {
                        if (tile > 0) wait(&m.pv_done, (uint32_t)(tile - 1) & 1u);  // P is free, and O at rest
                        if (!softmax_any<X::kSoftmax>(!(top <= kSlack) || dead)) break;
                        if (softmax_any<X::kSoftmax>(dead)) {
                            stop = true;
                            break;
                        }
                        blank = 0.f;
                        continue;
                    }
                    // New references for the rows that need one.  The others keep theirs, so no row's result depends on
                    // another's.
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float y = fmaxf(x[4 * j + i], x[4 * j + 2 + i]);
                            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
                            if (lane < 4) m.red[qt][8 * j + col + i] = y;
                        }
                    softmax_sync<X::kSoftmax>();
                    float f[J][2];
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int c = 8 * j + col + i;
                            const float y = fmaxf(fmaxf(m.red[0][c], m.red[1][c]), fmaxf(m.red[2][c], m.red[3][c]));
                            f[j][i] = 1.f;
                            if (nref[j][i] == INFINITY) {
                                if (y > -INFINITY) nref[j][i] = -y;
                            } else if (y > kSlack) {
                                nref[j][i] -= y;
                                f[j][i] = ex2_approx(-y);
                                l[j][i] *= f[j][i];
                            }
                        }
                    softmax_sync<X::kSoftmax>();
                    if (t > 0) {  // O^T has something: scale its columns
                        if (qt == 0 && lane < 4)
#pragma unroll
                            for (int j = 0; j < J; ++j) m.red[0][8 * j + col] = f[j][0], m.red[0][8 * j + col + 1] = f[j][1];
                        softmax_sync<X::kSoftmax>();
                        tc::fence_after();
#pragma unroll 1
                        for (int b = 0; b < X::kBlocks; ++b) {
                            uint32_t o[NL];
                            const uint32_t at = lanes + (uint32_t)(b * N + set * NL);
                            ld_32x32b(at, o);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < NL; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * m.red[0][set * NL + e]);
                            st_32x32b(at, o);
                        }
                        tc::wait_st();
                    }
                }
                if (stop) break;
                uint32_t w2[2 * J];  // [2 j + h]: columns col, col + 1 of block j, token h
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t v = pack_bf16x2(ex2_approx(x[4 * j + 2 * h]), ex2_approx(x[4 * j + 2 * h + 1]));
                        w2[2 * j + h] = v;
                        l[j][0] += bf16x2_lo(v);
                        l[j][1] += bf16x2_hi(v);
                    }
#pragma unroll
                for (int j = 0; j < J; j += 2)
                    stmatrix_x4(p_s + (uint32_t)(((set * J + j + (lane >> 4)) ^ (lane & 7)) << 4), w2[2 * j], w2[2 * j + 1], w2[2 * j + 2],
                                w2[2 * j + 3]);
                fence_proxy_async();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.p_full);
            }
            if (stop) break;
            softmax_sync<X::kSoftmax>();  // red has been read
            // sums of weights over the tokens; then O^T, row by row
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float y = l[j][i];
                    y += __shfl_xor_sync(0xffffffffu, y, 4);
                    y += __shfl_xor_sync(0xffffffffu, y, 8);
                    l[j][i] = y + __shfl_xor_sync(0xffffffffu, y, 16);
                    if (lane < 4) m.red[qt][8 * j + col + i] = l[j][i];
                }
            softmax_sync<X::kSoftmax>();
            float sum[J][2];
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = 8 * j + col + i;
                    sum[j][i] = (m.red[0][c] + m.red[1][c]) + (m.red[2][c] + m.red[3][c]);
                }
            const size_t slot = 2 * (size_t)cta + (pc.out == 1 ? 1 : 0);
            if (pc.out && qt == 0 && lane < 4)
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        ws.ml[slot * 2 * N + 8 * j + col + i] = -nref[j][i];
                        ws.ml[slot * 2 * N + N + 8 * j + col + i] = sum[j][i];
                    }
            wait(&m.pv_done, (uint32_t)(tile - 1) & 1u);
            if (softmax_any<X::kSoftmax>(dead)) break;
            tc::fence_after();
            // O^T, 16 entries at a time; P's memory is free for the transposition
            const uint32_t stage = smem_u32(smem + X::p) + (uint32_t)((set * 4 + qt) * NL * 32);
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) sum[j][i] = sum[j][i] == 0.f ? 0.f : __fdividef(1.f, sum[j][i]);
            auto fetch = [&](int u, uint32_t (&r)[4 * J]) { ld_16x256b(lanes + ((uint32_t)(u & 1) << 20) + (uint32_t)((u >> 1) * N + set * NL), r); };
            auto put = [&](int u, const uint32_t (&r)[4 * J]) {
                const int unit = ((u >> 1) * 4 + qt) * 2 + (u & 1);  // entries 16 unit ..
                if (pc.out) {
                    uint4 *po = reinterpret_cast<uint4 *>(ws.o + slot * N * V) + (size_t)(unit * (N / 8) + set * J) * 32 + lane;
#pragma unroll
                    for (int j = 0; j < J; ++j) po[j * 32] = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                } else {
                    float o[4 * J];
#pragma unroll
                    for (int e = 0; e < 4 * J; ++e) o[e] = __uint_as_float(r[e]);
                    emit<V, NL>(o, sum, stage, lane, (__nv_bfloat16 *)a.out + (int64_t)(pc.row0 + set * NL) * V + 16 * unit, pc.rows - set * NL);
                }
            };
#pragma unroll 1
            for (int u = 0; u < 2 * X::kBlocks; u += 2) {  // (two loads at a time: 0.2 us less)
                uint32_t r0[4 * J], r1[4 * J];
                fetch(u, r0);
                fetch(u + 1, r1);
                tc::wait_ld();
                put(u, r0);
                put(u + 1, r1);
            }
            tc::fence_before();
            softmax_sync<X::kSoftmax>();  // red is read by all before the next piece writes it
            if (lane == 0) {
                mbar_arrive(&m.o_free);
                mbar_arrive(&m.desc_empty[d]);
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(X::kCols) : "memory");
    }
}

// Joins the pieces of cut contexts: CTA (c, y) that of one context (or of the one that begins in share c), SPLIT warps
// 16 entries of 16 rows, in the layout the pieces were stored in.  What it waits for is L2, 1 to 1.5 us for each batch of
// loads.  So the pieces of a context of many (a few long contexts) are divided among four warps (8 contexts of 19 pieces:
// 5 us less), and a batch is two pieces: with four, the registers keep this kernel's CTAs off the SMs until the first
// kernel's have gone (1 to 3 us more).
constexpr int kJoinWarps = 8;

template <int V, int N, int SPLIT>
__global__ void __launch_bounds__(kJoinWarps * 32) latent_mma_join_kernel(const __grid_constant__ Args a, int shares, int by_context) {
    __shared__ __align__(128) unsigned char stage[kJoinWarps / SPLIT][16 * 32];
    __shared__ float part[SPLIT > 1 ? kJoinWarps : 1][16][32];
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Ws ws = ws_of(a, shares, N, V);
    int4 rec = *reinterpret_cast<const int4 *>(ws.rec + 4 * blockIdx.x);
    if (by_context) rec.x = blockIdx.x * a.H, rec.y = a.H;  // (whatever a wait that ran out kept from being left)
    constexpr int kRowUnits = N / 16;
    const int g = warp % SPLIT, work = blockIdx.y * (kJoinWarps / SPLIT) + warp / SPLIT, unit = work / kRowUnits, r0 = work % kRowUnits * 16;
    const int n = rec.z, rows = rec.y - r0, c = rec.w;
    if (n <= 0 || c < 0 || c > shares - n) return;
    const int col = r0 + 2 * (lane & 3);
    float top[4], sum[4] = {}, o[8] = {};  // [2 j + i]: row col + 8 j + i
#pragma unroll
    for (int e = 0; e < 4; ++e) top[e] = -INFINITY;
    for (int k0 = 2 * g; k0 < n && rows > 0; k0 += 2 * SPLIT) {
        float2 m[2][2], l[2][2];
        float4 y[2][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int kk = min(k0 + k, n - 1);
            const size_t slot = (size_t)(kk ? 2 * (c + kk) : 2 * c + 1);
            const float *ml = ws.ml + slot * 2 * N + col;
            const float4 *po = reinterpret_cast<const float4 *>(ws.o + slot * N * V) + (size_t)(unit * (N / 8) + r0 / 8) * 32 + lane;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[k][j] = *reinterpret_cast<const float2 *>(ml + 8 * j);
                l[k][j] = *reinterpret_cast<const float2 *>(ml + N + 8 * j);
                y[k][j] = po[j * 32];
                if (k0 + k >= n) m[k][j] = make_float2(-INFINITY, -INFINITY);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int e = 2 * j + i;
                auto at = [&](const float2 &v) { return i ? v.y : v.x; };
                const float now = fmaxf(top[e], fmaxf(at(m[0][j]), at(m[1][j])));
                const float ref = now == -INFINITY ? 0.f : now, f = exp2f(top[e] - ref);
                top[e] = now;
                sum[e] *= f, o[4 * j + i] *= f, o[4 * j + 2 + i] *= f;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float g2 = exp2f(at(m[k][j]) - ref);
                    if (k0 + k < n) {
                        sum[e] += at(l[k][j]) * g2;
                        o[4 * j + i] += (i ? y[k][j].y : y[k][j].x) * g2;
                        o[4 * j + 2 + i] += (i ? y[k][j].w : y[k][j].z) * g2;
                    }
                }
            }
    }
    if constexpr (SPLIT > 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) part[warp][e][lane] = o[e];
#pragma unroll
        for (int e = 0; e < 4; ++e) part[warp][8 + e][lane] = top[e], part[warp][12 + e][lane] = sum[e];
        __syncthreads();
        if (g) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int at = 4 * (e >> 1) + (e & 1);
            float now = top[e], f[SPLIT];
#pragma unroll
            for (int k = 1; k < SPLIT; ++k) now = fmaxf(now, part[warp + k][8 + e][lane]);
            if (now == -INFINITY) now = 0.f;
#pragma unroll
            for (int k = 0; k < SPLIT; ++k) f[k] = exp2f((k ? part[warp + k][8 + e][lane] : top[e]) - now);
            sum[e] *= f[0], o[at] *= f[0], o[at + 2] *= f[0];
#pragma unroll
            for (int k = 1; k < SPLIT; ++k) {
                sum[e] += part[warp + k][12 + e][lane] * f[k];
                o[at] += part[warp + k][at][lane] * f[k];
                o[at + 2] += part[warp + k][at + 2][lane] * f[k];
            }
        }
    }
    if (rows <= 0) return;
    float inv[2][2];
#pragma unroll
    for (int e = 0; e < 4; ++e) inv[e >> 1][e & 1] = sum[e] == 0.f ? 0.f : 1.f / sum[e];
    emit<V, 16>(o, inv, smem_u32(stage[warp / SPLIT]), lane, (__nv_bfloat16 *)a.out + (int64_t)(rec.x + r0) * V + 16 * unit, rows);
}

// Rows of a row tile: the smallest that holds a sequence's query rows, or 64.
int rows_of(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

template <int V, int N>
pkv_status launch(Args a, cudaStream_t st) {
    static bool done[128];
    const int sms = sm_count();
    if (sms == 0 || !ensure_smem(latent_mma_kernel<V, N>, L<V, N>::total, done)) return PKV_ERR_CUDA;
    using X = L<V, N>;
    CUtensorMap tm_q, tm_c0, tm_c1;
    const int64_t rows = (int64_t)a.NB * a.B;
    if (!make_rows_map(&tm_q, a.q, (int64_t)a.T * a.H, V, N, X::kChunks) || !make_rows_map(&tm_c0, a.cache, rows, V, 8, X::kPart0) ||
        !make_rows_map(&tm_c1, a.cache, rows, V, 8, X::kChunks - X::kPart0))
        return PKV_ERR_CUDA;
    // A decode of no more contexts than shares: the join's CTAs go by contexts, fewer than the shares.
    const int by_context = !a.q_starts && a.S <= sms;
    a.whole = whole_contexts(a, N, 64, sms);
    a.once = read_once(a, N);
    const unsigned grid = a.whole ? (unsigned)(a.S * a.whole) : (unsigned)sms;
    const pkv_status rc = launch_pdl(latent_mma_kernel<V, N>, dim3(grid), dim3(X::kThreads), (size_t)X::total, st, tm_q, tm_c0, tm_c1, a,
                                     by_context);
    if (rc != PKV_OK || a.whole) return rc;
    constexpr unsigned kUnits = V * N / 256;
    const unsigned cuts = by_context ? (unsigned)a.S : (unsigned)sms;
    // (pieces of a context: about shares / contexts)
    if (by_context && a.S * 4 < sms)
        return launch_pdl(latent_mma_join_kernel<V, N, 4>, dim3(cuts, kUnits * 4 / kJoinWarps), dim3(kJoinWarps * 32), 0, st, a, sms, by_context);
    return launch_pdl(latent_mma_join_kernel<V, N, 1>, dim3(cuts, kUnits / kJoinWarps), dim3(kJoinWarps * 32), 0, st, a, sms, by_context);
}

}  // namespace

size_t mma_workspace(int64_t T, int H, int V) {
    const int sms = sm_count();
    return round256(ws_bytes(sms > 0 ? sms : 160, rows_of(T * H), V));
}

pkv_status run_mma(const Args &a, cudaStream_t st) {
    switch (rows_of(a.rows)) {
        case 16: return a.V == 512 ? launch<512, 16>(a, st) : launch<256, 16>(a, st);
        case 32: return a.V == 512 ? launch<512, 32>(a, st) : launch<256, 32>(a, st);
        default: return a.V == 512 ? launch<512, 64>(a, st) : launch<256, 64>(a, st);
    }
}

}  // namespace latent
}  // namespace pkv
