// Latent attention on the 5th-generation tensor cores (bf16), for sequences of more than 64 query
// rows (several queries, or more than 64 heads): pairs of CTAs on one tile.
//
// A row tile is 128 consecutive query rows (a row: one head of one query), 64 a CTA; a tile is 128 tokens.
//     S = Q C^T    [128 rows x 128 tokens]   Q and S by rows over the two CTAs, C by tokens
//     O += P L     [128 rows x V entries]    P and O by rows, L by entries
// with cta_group::2 instructions: each CTA's operands feed both tensor cores, so for a product of 128 x 128
// (or x 256) an SM reads 64 rows of A and half of B from its shared memory -- half of what the transposed
// products of 64 rows read for the same work, which is what bounds those.  O of 64 rows takes 256 columns of
// tensor memory a CTA (V = 512), two S of 64 columns each fit beside it.
//
// Each CTA holds a tile's rows twice, in the two forms the products want: 64 tokens by all entries, and all
// tokens by half of the entries.  Both are read in parts, and a part is loaded anew as soon as the product that read
// it is done: with V = 512 one tile of each form is all that fits beside Q and P.
//
// The leader's (rank 0's) warps issue all products.  What the other CTA has ready it reports to the leader's
// barriers; what the products have done arrives at both CTAs' barriers.
//
// Measured, calls from a host in a row (from CUDA graphs): 8 x 512 queries of 4096, 32 heads, 708 us (679), 79 % (83 %) of the
// measured bf16 rate, a tile 2300 to 2800 cycles where its products are 2176; the transposed kernel took 1272.  4 prompts of
// 3200 to 4000 tokens, 16 heads: 576 us (556).  A decode of 64 contexts of 64 to 2048 tokens, 128 heads: 34.2 us from graphs, 2.6
// times its floor: its tiles come from DRAM, twice (both forms) through the one stage there is, as for 64 x 5 queries (45.7).
//
// Softmax: a thread has one row and a quarter of the tile's tokens (eight warps: with four, whose exponentials alone
// take 512 cycles of each scheduler, a tile took 3300 cycles, not 2200).  References, weights,
// hidden rows, shares and joins as in the transposed kernel.
#include "latent_tc.cuh"

namespace pkv {
namespace latent {

namespace {

constexpr int kRows = 128, kTok = 128;
constexpr int kSoftmax = 256;             // threads of the eight softmax warps
constexpr int kThreads = 128 + kSoftmax;  // two producers, a warp for each product (the other CTA's report loads)

template <int V>
struct L {
    static constexpr int kChunks = V / 64 + 1;
    static constexpr int kPart0 = V / 128;                 // chunks of the first part of the rows by tokens
    static constexpr int kGroupK = kChunks * 1024;         // bytes of 8 tokens, all entries
    static constexpr int kGroupV = V / 128 * 1024;         // 8 tokens, half of the latent entries
    static constexpr int kK = 8 * kGroupK, kV = 16 * kGroupV;
    static constexpr int kQ = kChunks * 64 * 128;
    static constexpr int kP = 64 * kTok * 2;
    static constexpr int q = 0, p = kQ, k = p + kP, v = k + kK, misc = v + kV, total = misc + 2048;
    static constexpr int kBlocks = V / 256;                // products of 256 entries
    static constexpr uint32_t kS = kBlocks * 128;          // first column of S
    static constexpr uint32_t kCols = kS + 128 <= 256 ? 256 : 512;
    static_assert(total <= 232448 && kS + 128 <= kCols, "memory");
};

struct alignas(8) Misc {
    uint64_t k_full[2], k_peer[2], k_empty[2], v_full[2], v_peer[2], v_empty[2], q_full, q_peer, q_empty, s_full[2], s_free[2], p_full, pv_done, o_free;
    uint64_t meta[4], desc_full[kDescs], desc_empty[kDescs], fin[2];
    Piece piece[kDescs];
    float red[4][64];
    uint32_t groups[4];   // valid 8-token groups of a tile
    uint32_t warp_bad[4][2], row_bad[2][2];  // by 32 tokens: scores that are no numbers; latent parts
    uint32_t tmem;
    int dead;
};
static_assert(sizeof(Misc) <= 2048, "misc");

struct Ws {
    int *rec;
    float *o;   // [shares][2][2 CTAs][V / 4][128 threads][4]... one thread's entries, four at a time
    float *ml;  // [shares][2][2 CTAs][2][64]
};
inline size_t ws_bytes(int shares, int v) { return (size_t)shares * 16 + (size_t)shares * 2 * kRows * (v + 2) * 4 + 512; }
__device__ __forceinline__ Ws ws_of(const Args &a, int shares, int v) {
    Ws w;
    w.o = (float *)a.ws;
    w.ml = w.o + (size_t)shares * 2 * kRows * v;
    w.rec = (int *)(w.ml + (size_t)shares * 2 * 2 * kRows);
    return w;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The other CTA's (or the leader's) address of what lies at p here.
__device__ __forceinline__ uint32_t at_rank(const void *p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
// (What these arrivals announce is read by the tensor cores, or has been read from tensor memory: the proxy and
// tcgen05 fences before them order that.  A release at cluster scope would cost a memory barrier, some 1500 cycles.)
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
// Arrives at `bar` of both CTAs when this thread's products so far are done.
__device__ __forceinline__ void commit_both(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
        "h"((unsigned short)3)
        : "memory");
}

// Whether the latent part of token `tok` of a sequence holds an infinity or NaN, as it lies in the cache.  (Out of line, as
// it is seldom asked: inlined, 8 x 512 queries of 4096 took 714 us, not 710.)
template <int V>
__device__ __noinline__ bool latent_not_finite(const Args &a, int seq, int tok) {
    const int blk = __ldg(a.tables + (int64_t)seq * a.maxb + (tok >> a.bshift));
    bool found = false;
    if ((unsigned)blk < (unsigned)a.NB) {
        const int64_t row = ((int64_t)blk << a.bshift) + (tok & (a.B - 1));
        const uint4 *y = reinterpret_cast<const uint4 *>((const unsigned char *)a.cache + row * (V + kRope) * 2);
#pragma unroll 1
        for (int e = 0; e < V / 8; ++e) found |= not_finite(y[e]);
    }
    return found;
}

template <int V>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
latent_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k0, const __grid_constant__ CUtensorMap tm_k1,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ Args a, int by_context) {
    using X = L<V>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Misc &m = *reinterpret_cast<Misc *>(smem + X::misc);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    const uint32_t rank = cluster_rank();
    const bool lead = rank == 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m.k_full[i], 1), mbar_init(&m.k_peer[i], 1), mbar_init(&m.k_empty[i], 1);
            mbar_init(&m.v_full[i], 1), mbar_init(&m.v_peer[i], 1), mbar_init(&m.v_empty[i], 1);
            mbar_init(&m.s_full[i], 1), mbar_init(&m.s_free[i], 16);
            mbar_init(&m.fin[i], 1);
        }
        mbar_init(&m.q_full, 1), mbar_init(&m.q_peer, 1), mbar_init(&m.q_empty, 1);
        mbar_init(&m.p_full, 16), mbar_init(&m.pv_done, 1), mbar_init(&m.o_free, 16);
        for (int i = 0; i < 4; ++i) mbar_init(&m.meta[i], 1);
        for (int i = 0; i < kDescs; ++i) mbar_init(&m.desc_full[i], 1), mbar_init(&m.desc_empty[i], 11);
        m.dead = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == 32) prefetch_map(&tm_q), prefetch_map(&tm_k0), prefetch_map(&tm_k1), prefetch_map(&tm_v), prefetch_map(&tm_o);
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&m.tmem)), "r"(X::kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    cluster_arrive();  // both CTAs' barriers are set up (awaited below)
    grid_dependency_wait();
    // the join kernel, which waits for this one before it reads (no other: attention kernels read queries before they wait)
    if (!a.whole) grid_launch_dependents();
    prefetch_tables(a, (int64_t)threadIdx.x * gridDim.x + blockIdx.x);
    Share<kRows, kTok, false> sh = locate<kRows, kTok, false>(a, &m.red[0][0], pair, pairs, kThreads);
    const Ws ws = ws_of(a, pairs, V);
    if (lead && threadIdx.x == 0 && !by_context && !a.whole) leave(ws.rec + 4 * pair, 0, 0, 0, 0);
    tc::fence_before();
    __syncthreads();
    cluster_wait();
    tc::fence_after();
    const uint32_t tmem = m.tmem;

    bool dead = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) {  // by whole warps
        if (!dead && !__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) dead = wait_on(bar, parity, &m.dead, a.err);
    };

    // lane l: the cache row of group l & 15 of tile t + (l >> 4) of a piece; -1: a bad block; -2: no token
    auto look = [&](const Piece &pc, int t) {
        const int tok = pc.t0 + t * kTok + 8 * lane;
        if (t + (lane >> 4) >= pc.tiles || tok >= pc.end) return -2;
        const int blk = __ldg(a.tables + (int64_t)pc.seq * a.maxb + (tok >> a.bshift));
        return (unsigned)blk < (unsigned)a.NB ? (blk << a.bshift) + (tok & (a.B - 1)) : -1;
    };
    const int none = a.NB << a.bshift;  // where a group without tokens starts: past the tensor's end, zeros

    if (warp == 0) {
        // ======================= producer of pieces, Q and the rows by tokens =======================
        int tile = 0, np = 0, nq = 0, nk = 0;  // tiles, pieces, queries and parts issued
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
            int row = look(pc, 0), next = -2;
            wait(&m.q_empty, (uint32_t)(np + 1) & 1u);
            ++np;
            if (dead) continue;
            if (lane == 0) {
                mbar_arrive_expect_tx(&m.q_full, (uint32_t)X::kQ);
                tma_load_3d(smem_u32(smem + X::q), &tm_q, smem_u32(&m.q_full), 0, pc.row0 + 64 * (int)rank, 0);
            }
            ++nq;
            __syncwarp();
            for (int t = 0; t < pc.tiles && !dead; ++t, ++tile) {
                if ((t & 1) == 0) {
                    if (t) row = next;
                    next = look(pc, t + 2);
                }
                const bool turn = (lane >> 4) == (t & 1);
                const bool mine = turn && ((lane >> 3) & 1) == (int)rank;  // groups of this CTA's 64 tokens
                const uint32_t ok = __ballot_sync(0xffffffffu, row >= 0) >> (16 * (t & 1)) & 0xffffu;
                if (turn && row == -1 && lead) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    wait(&m.k_empty[h], (uint32_t)(tile + 1) & 1u);
                    if (dead) break;
                    if (lane == 0) {
                        if (h == 0) {
                            m.groups[tile & 3] = ok;
                            mbar_arrive(&m.meta[tile & 3]);
                        }
                        mbar_arrive_expect_tx(&m.k_full[h], (uint32_t)(64 * 128 * (h ? X::kChunks - X::kPart0 : X::kPart0)));
                    }
                    __syncwarp();
                    if (mine)
                        tma_load_3d(smem_u32(smem + X::k) + (uint32_t)((lane & 7) * X::kGroupK + h * X::kPart0 * 1024), h ? &tm_k1 : &tm_k0,
                                    smem_u32(&m.k_full[h]), 0, row >= 0 ? row : none, h * X::kPart0);
                    ++nk;
                }
                // The next tile's rows, of whose load nothing is under way yet, into L2, where up to eight row tiles read
                // them: 64 x 5 queries, 32 heads, 48.4 -> 46.2 us, 64 x 4 35.6 -> 34.8, 4 x 8 queries of 128 heads 40.2 ->
                // 39.8.  (More, and they are mostly there: 8 x 64 queries of 32 heads 111 -> 116.  And where rows are the
                // first to leave, it is the load by entries, the later one, that says so: the other, and a decode of 128
                // heads takes 33.9 us, not 32.4.)
                const int ahead = (t & 1) == 0 ? row : next;
                if (a.rows <= 8 * kRows && (lane >> 4) == ((t + 1) & 1) && ((lane >> 3) & 1) == (int)rank && ahead >= 0)
                    prefetch_rows<V>(a, ahead);
            }
            if (lead && lane == 0) {
                if (a.whole) {
                } else if (by_context && pc.out != 2) leave(ws.rec + 4 * pc.seq, pc.row0, pc.rows, pc.out ? sh.reach(pair) : 0, pair);
                else if (pc.out == 1) leave(ws.rec + 4 * pair, pc.row0, pc.rows, sh.reach(pair), pair);
            }
        }
        // no copy outlives the CTA, whoever else gave up
        for (int i = max(0, nk - 2); i < nk; ++i) mbar_wait_bounded(&m.k_full[i & 1], (uint32_t)(i >> 1) & 1u);
        if (nq > 0) mbar_wait_bounded(&m.q_full, (uint32_t)(nq - 1) & 1u);
    } else if (warp == 3) {
        // ======================= producer of the rows by entries =======================
        const uint64_t policy = row_policy(a);
        int tile = 0, nv = 0;
        for (int np = 0;; ++np) {
            const int d = np % kDescs;
            wait(&m.desc_full[d], (uint32_t)(np / kDescs) & 1u);
            if (dead) break;
            const Piece pc = m.piece[d];
            if (pc.tiles == 0) break;
            int row = look(pc, 0), next = -2;
            for (int t = 0; t < pc.tiles && !dead; ++t, ++tile) {
                if ((t & 1) == 0) {
                    if (t) row = next;
                    next = look(pc, t + 2);
                }
                const bool turn = (lane >> 4) == (t & 1);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    wait(&m.v_empty[h], (uint32_t)(tile + 1) & 1u);
                    if (dead) break;
                    if (lane == 0) mbar_arrive_expect_tx(&m.v_full[h], (uint32_t)(X::kV / 2));
                    __syncwarp();
                    if (turn && ((lane >> 3) & 1) == h)
                        tma_load_3d_hint(smem_u32(smem + X::v) + (uint32_t)((lane & 15) * X::kGroupV), &tm_v, smem_u32(&m.v_full[h]), 0,
                                    row >= 0 ? row : none, (int)rank * (V / 128), policy);
                    ++nv;
                }
            }
            if (dead) break;
            if (lane == 0) mbar_arrive(&m.desc_empty[d]);
        }
        for (int i = max(0, nv - 2); i < nv; ++i) mbar_wait_bounded(&m.v_full[i & 1], (uint32_t)(i >> 1) & 1u);
    } else if (warp <= 2 && !lead) {
        // ======================= the other CTA: reports its loads (warp 1: Q, rows by tokens; 2: by entries) =======================
        uint64_t *full = warp == 1 ? m.k_full : m.v_full;
        const uint32_t q_peer = at_rank(&m.q_peer, 0), peer = at_rank(warp == 1 ? m.k_peer : m.v_peer, 0);
        for (int np = 0, tile = 0;; ++np) {
            const int d = np % kDescs;
            wait(&m.desc_full[d], (uint32_t)(np / kDescs) & 1u);
            const int n = dead ? 0 : m.piece[d].tiles;
            if (n == 0) break;
            if (warp == 1) {
                wait(&m.q_full, (uint32_t)np & 1u);
                if (dead) break;
                if (lane == 0) arrive_at(q_peer);
            }
            for (int t = 0; t < n && !dead; ++t, ++tile)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    wait(&full[h], (uint32_t)tile & 1u);
                    if (!dead && lane == 0) arrive_at(peer + 8 * h);
                }
            if (dead) break;
            if (lane == 0) mbar_arrive(&m.desc_empty[d]);
        }
    } else if (warp == 1) {
        // ======================= the leader: issuer of S = Q C^T =======================
        constexpr uint32_t id = idesc(128, kTok, false, false);
        const bool leader = elect_one();
        const uint64_t qd = tc::smem_desc(smem_u32(smem + X::q), 16, 1024);
        const uint64_t kd = tc::smem_desc(smem_u32(smem + X::k), 16, X::kGroupK);
        for (int np = 0, tile = 0;; ++np) {
            const int d = np % kDescs;
            wait(&m.desc_full[d], (uint32_t)(np / kDescs) & 1u);
            const int n = dead ? 0 : m.piece[d].tiles;
            if (n == 0) break;
            wait(&m.q_full, (uint32_t)np & 1u);
            wait(&m.q_peer, (uint32_t)np & 1u);
            for (int t = 0; t < n; ++t, ++tile) {
                const uint32_t s = tmem + X::kS + (uint32_t)((tile & 1) * 64);
                wait(&m.s_free[tile & 1], (uint32_t)((tile >> 1) + 1) & 1u);
                wait(&m.k_full[0], (uint32_t)tile & 1u);
                wait(&m.k_peer[0], (uint32_t)tile & 1u);
                if (dead) break;
                tc::fence_after();
                if (leader) {
#pragma unroll 1  // (rolled: the instruction cache holds what the softmax needs)
                    for (int c = 0; c < X::kPart0; ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma2(s, qd + (uint64_t)((c * 8192 + k * 32) >> 4), kd + (uint64_t)((c * 1024 + k * 32) >> 4), id, c + k > 0 ? 1u : 0u);
                    commit_both(&m.k_empty[0]);
                }
                __syncwarp();
                wait(&m.k_full[1], (uint32_t)tile & 1u);
                wait(&m.k_peer[1], (uint32_t)tile & 1u);
                if (dead) break;
                tc::fence_after();
                if (leader) {
#pragma unroll 1
                    for (int c = X::kPart0; c < X::kChunks; ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma2(s, qd + (uint64_t)((c * 8192 + k * 32) >> 4), kd + (uint64_t)((c * 1024 + k * 32) >> 4), id, 1u);
                    commit_both(&m.k_empty[1]);
                    commit_both(&m.s_full[tile & 1]);
                    if (t + 1 == n) commit_both(&m.q_empty);
                }
                __syncwarp();
            }
            if (dead) break;
            if (lane == 0) mbar_arrive(&m.desc_empty[d]);
        }
        if (leader) commit_both(&m.fin[0]);
        __syncwarp();
    } else if (warp == 2) {
        // ======================= the leader: issuer of O += P L =======================
        constexpr uint32_t id = idesc(128, 256, false, true);
        const bool leader = elect_one();
        const uint64_t pd = tc::smem_desc(smem_u32(smem + X::p), 16, 1024);
        const uint64_t vd = tc::smem_desc(smem_u32(smem + X::v), 1024, X::kGroupV);
        for (int np = 0, tile = 0;; ++np) {
            const int d = np % kDescs;
            wait(&m.desc_full[d], (uint32_t)(np / kDescs) & 1u);
            const int n = dead ? 0 : m.piece[d].tiles;
            if (n == 0) break;
            if (np > 0) wait(&m.o_free, (uint32_t)(np - 1) & 1u);
            for (int t = 0; t < n; ++t, ++tile) {
                wait(&m.p_full, (uint32_t)tile & 1u);
                auto half = [&](int h) {  // 4 steps of 16 tokens
#pragma unroll 1
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int b = 0; b < X::kBlocks; ++b)
                            mma2(tmem + (uint32_t)(b * 128), pd + (uint64_t)((h * 8192 + k * 32) >> 4),
                                 vd + (uint64_t)((b * 2048 + (4 * h + k) * 2 * X::kGroupV) >> 4), id, t == 0 && h + k == 0 ? 0u : 1u);
                };
                wait(&m.v_full[0], (uint32_t)tile & 1u);
                wait(&m.v_peer[0], (uint32_t)tile & 1u);
                if (dead) break;
                tc::fence_after();
                if (leader) {
                    half(0);
                    commit_both(&m.v_empty[0]);
                }
                __syncwarp();
                wait(&m.v_full[1], (uint32_t)tile & 1u);
                wait(&m.v_peer[1], (uint32_t)tile & 1u);
                if (dead) break;
                tc::fence_after();
                if (leader) {
                    half(1);
                    commit_both(&m.v_empty[1]);
                    commit_both(&m.pv_done);
                }
                __syncwarp();
            }
            if (dead) break;
            if (lane == 0) mbar_arrive(&m.desc_empty[d]);
        }
        if (leader) commit_both(&m.fin[1]);
        __syncwarp();
    } else if (warp >= 4) {
        // ======================= softmax and epilogue =======================
        const int qt = warp & 3;  // quarter of the tensor memory's lanes
        const int row = (qt & 1) * 32 + lane, half = qt >> 1;  // of the CTA's rows; of the tile's tokens, and then
        const int q2 = warp >> 2 & 1, me = 2 * half + q2;      // of that half's
        const uint32_t lanes = tmem + ((uint32_t)(qt * 32) << 16);
        const float sc = a.scale_log2;
        unsigned char *p_row = smem + X::p + half * 8192 + row * 128;
        const int p_chunk = 4 * q2;
        const uint32_t p_full = at_rank(&m.p_full, 0), o_free = at_rank(&m.o_free, 0);
        const uint32_t s_free[2] = {at_rank(&m.s_free[0], 0), at_rank(&m.s_free[1], 0)};
        if (sh.blind && lead) zero_blind<kRows, kTok, false>(a, pair, pairs, threadIdx.x - 128, kSoftmax, by_context ? ws.rec : nullptr);
        int tile = 0;
        bool stop = false;  // the four warps leave together: they share a barrier
        for (int np = 0;; ++np) {
            const int d = np % kDescs;
            wait(&m.desc_full[d], (uint32_t)(np / kDescs) & 1u);
            if (softmax_any<kSoftmax>(dead)) break;
            const Piece pc = m.piece[d];
            if (pc.tiles == 0) break;
            float nref = INFINITY;       // minus the reference: +inf before the first score
            uint64_t l2 = f32x2(0.f, 0.f);  // sums of the weights of even and odd tokens
            const int r = 64 * (int)rank + row;
            const int least = pc.lim0 + by_heads(a, pc.qh0);                     // tokens that the first row sees
            const int lim = min(pc.end, pc.lim0 + by_heads(a, pc.qh0 + r));    // that this row sees
            for (int t = 0; t < pc.tiles; ++t, ++tile) {
                wait(&m.meta[tile & 3], (uint32_t)(tile >> 2) & 1u);
                wait(&m.s_full[tile & 1], (uint32_t)(tile >> 1) & 1u);
                tc::fence_after();
                uint32_t s[32];
                ld_32x32b(lanes + X::kS + (uint32_t)((tile & 1) * 64 + 32 * q2), s);
                tc::wait_ld();
                const uint32_t groups = m.groups[tile & 3];
                tc::fence_before();
                __syncwarp();
                if (lane == 0) arrive_at(s_free[tile & 1]);
                const int tb = pc.t0 + t * kTok;
                const bool masked = tb + kTok > least || groups != 0xffffu;
                uint32_t bad = 0u, wipe = 0u;  // rows that hold an infinity or NaN: among this thread's tokens; among those it zeroes
                if (masked) {
                    // A row of the cache whose latent part holds an infinity or NaN gives every query a score that is no
                    // number.  Finite entries whose products pass float32's range may do so too, and there a score of
                    // -infinity is a weight of 0: so the rows themselves decide, looked at only if some score is none.
                    float most = 0.f;
#pragma unroll
                    for (int c = 0; c < 32; c += 2) most = max3_nan(most, fabsf(__uint_as_float(s[c])), fabsf(__uint_as_float(s[c + 1])));
                    if (softmax_any<kSoftmax>(!(most < INFINITY))) {
                        // the tokens that gave all of this CTA's rows one, a word of 32 tokens a warp
                        uint32_t nf = 0u;
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if ((s[c] & 0x7f800000u) == 0x7f800000u) nf |= 1u << c;
                        const uint32_t all = __reduce_and_sync(0xffffffffu, nf);
                        if (lane == 0) m.warp_bad[qt][q2] = all;
                        softmax_sync<kSoftmax>();
                        if (q2 == 0) {  // four warps, tokens 64 half + 32 (qt & 1) .., one a lane; this CTA has half of a row alone
                            const uint32_t suspect = m.warp_bad[2 * half][qt & 1] & m.warp_bad[2 * half + 1][qt & 1];
                            const int at = 64 * half + 32 * (qt & 1) + lane;
                            const bool found = (suspect >> lane) & (groups >> (at >> 3)) & 1u ? latent_not_finite<V>(a, pc.seq, tb + at) : false;
                            wipe = __ballot_sync(0xffffffffu, found);
                            if (lane == 0) m.row_bad[half][qt & 1] = wipe;
                        }
                        softmax_sync<kSoftmax>();
                        bad = m.row_bad[half][q2];
                    }
                }
                // log2 of the weights without the reference
                float x[32];
#pragma unroll
                for (int c = 0; c < 32; c += 2)
                    f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), f32x2(sc, sc), f32x2(0.f, 0.f)), x[c], x[c + 1]);
                if (masked) {
                    const uint32_t g4 = groups >> (8 * half + 4 * q2);
                    const int seen = lim - tb - 64 * half - 32 * q2;  // of this thread's tokens the row sees so many
                    uint32_t hide = seen <= 0 ? 0xffffffffu : seen >= 32 ? 0u : 0xffffffffu << seen;
                    hide |= (g4 & 1u ? 0u : 0xffu) | (g4 & 2u ? 0u : 0xff00u) | (g4 & 4u ? 0u : 0xff0000u) | (g4 & 8u ? 0u : 0xff000000u);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        if ((bad >> c) & 1u) x[c] = __uint_as_float(0x7fffffffu);  // (-infinity too: 0 times an infinity)
                        if ((hide >> c) & 1u) x[c] = -INFINITY;
                    }
                }
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 32; c += 2) top = max3_nan(top, x[c], x[c + 1]);
                const bool over = nref == INFINITY ? !(top == -INFINITY) : !(top + nref <= kSlack);
                if (softmax_any<kSoftmax>(over || dead)) {
                    if (softmax_any<kSoftmax>(dead)) {
                        stop = true;
                        break;
                    }
                    // Some score passed its row's reference by far, or is the row's first: new references for such rows.
                    // The others keep theirs, so no row's result depends on another's.
                    float y = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 32; ++c) y = fmaxf(y, x[c]);
                    if (nref != INFINITY) y += nref;
                    m.red[me][row] = y;
                    softmax_sync<kSoftmax>();
                    y = fmaxf(fmaxf(m.red[0][row], m.red[1][row]), fmaxf(m.red[2][row], m.red[3][row]));
                    softmax_sync<kSoftmax>();
                    float f = 1.f;
                    if (nref == INFINITY) {
                        if (y > -INFINITY) nref = -y;
                    } else if (y > kSlack) {
                        nref -= y;
                        f = ex2_approx(-y);
                        l2 = fma_f32x2(l2, f32x2(f, f), f32x2(0.f, 0.f));
                    }
                    if (t > 0) {
                        wait(&m.pv_done, (uint32_t)(tile - 1) & 1u);  // O at rest
                        tc::fence_after();
                        if (__any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
                            for (int b = q2 * (V / 128); b < (q2 + 1) * (V / 128); ++b) {
                                uint32_t o[32];
                                ld_32x32b(lanes + (uint32_t)(b * 32), o);
                                tc::wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                st_32x32b(lanes + (uint32_t)(b * 32), o);
                            }
                            tc::wait_st();
                        }
                    }
                }
                const float nr = nref == INFINITY ? 0.f : nref;
                uint32_t w[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    float lo, hi;
                    f32x2_split(add_f32x2(f32x2(x[2 * c], x[2 * c + 1]), f32x2(nr, nr)), lo, hi);
                    w[c] = pack_bf16x2(ex2_approx(lo), ex2_approx(hi));
                    l2 = add_f32x2(l2, f32x2(bf16x2_lo(w[c]), bf16x2_hi(w[c])));
                }
                if (tile > 0) wait(&m.pv_done, (uint32_t)(tile - 1) & 1u);  // P is free
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<uint4 *>(p_row + (((p_chunk + c) ^ (row & 7)) << 4)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                if (wipe) {
                    // Such a row must not reach, through 0 * infinity, the queries that do not see it, nor may what lies
                    // behind the last token: this CTA's half of its latent part is zeroed.
                    wait(&m.v_full[0], (uint32_t)tile & 1u);
                    wait(&m.v_full[1], (uint32_t)tile & 1u);
                    const int tk = 64 * half + row;  // (as many tokens as rows)
                    if ((wipe >> lane) & 1u) {
                        unsigned char *g = smem + X::v + (tk >> 3) * X::kGroupV + (tk & 7) * 128;
#pragma unroll 1
                        for (int e = 0; e < V / 128; ++e)
#pragma unroll 1
                            for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4 *>(g + e * 1024 + k * 16) = make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                }
                fence_proxy_async();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) arrive_at(p_full);
            }
            if (stop) break;
            softmax_sync<kSoftmax>();  // red has been read
            float l_even, l_odd;
            f32x2_split(l2, l_even, l_odd);
            m.red[me][row] = l_even + l_odd;
            softmax_sync<kSoftmax>();
            const float sum = (m.red[0][row] + m.red[1][row]) + (m.red[2][row] + m.red[3][row]);
            const size_t slot = (2 * (size_t)pair + (pc.out == 1 ? 1 : 0)) * 2 + rank;
            if (pc.out && me == 0) ws.ml[slot * 128 + row] = -nref, ws.ml[slot * 128 + 64 + row] = sum;
            wait(&m.pv_done, (uint32_t)(tile - 1) & 1u);
            if (softmax_any<kSoftmax>(dead)) break;
            tc::fence_after();
            const float inv = sum == 0.f ? 0.f : __fdividef(1.f, sum);
            // entries of column j of block b: half V / 2 + 128 b + j
            float4 *po = reinterpret_cast<float4 *>(ws.o + slot * 64 * V) + qt * 32 + lane;
            const uint32_t o_at = lanes + (uint32_t)(q2 * (V / 4));
            if (pc.out) {
#pragma unroll 1
                for (int b = 0; b < V / 128; ++b) {
                    uint32_t o[32];
                    ld_32x32b(o_at + (uint32_t)(b * 32), o);
                    tc::wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        po[((q2 * (V / 128) + b) * 8 + e) * 128] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                                               __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                }
            } else {
                // 32 rows of 32 entries at a time through this warp's 2 KB of P's memory (free by now), and out by a
                // bulk copy, or, where not all of the rows are the piece's, by hand: stores straight from the registers
                // would write 32 rows' sectors each, at twice the time.
                unsigned char *stage = smem + X::p + (warp - 4) * 2048;
                const int r0 = r - lane, x0 = half * (V / 2) + q2 * (V / 4);
                uint32_t o[32];
                ld_32x32b(o_at, o);
#pragma unroll 1
                for (int b = 0; b < V / 128; ++b) {
                    tc::wait_ld();
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                    if (b + 1 < V / 128) ld_32x32b(o_at + (uint32_t)((b + 1) * 32), o);
                    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the copy before has read it
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 4; ++e)  // (64-byte swizzle)
                        *reinterpret_cast<uint4 *>(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) =
                            make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                    if (r0 + 32 <= pc.rows) {
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) {
                            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                                             reinterpret_cast<uint64_t>(&tm_o)),
                                         "r"(smem_u32(stage)), "r"(x0 + b * 32), "r"(pc.row0 + r0)
                                         : "memory");
                            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        }
                    } else {
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int rr = 8 * i + (lane >> 2), e = lane & 3;
                            const uint4 y = *reinterpret_cast<const uint4 *>(stage + rr * 64 + ((e ^ ((rr >> 1) & 3)) << 4));
                            if (r0 + rr < pc.rows)
                                *reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.out + ((int64_t)pc.row0 + r0 + rr) * V + x0 + b * 32 + 8 * e) = y;
                        }
                        __syncwarp();
                    }
                }
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
            }
            tc::fence_before();
            softmax_sync<kSoftmax>();  // red is read by all before the next piece writes it
            if (lane == 0) {
                arrive_at(o_free);
                mbar_arrive(&m.desc_empty[d]);
            }
        }
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the output copies that this thread issued
    __syncwarp();
    if (warp == 1) {  // every product has ended before the memory goes
        mbar_wait_bounded(&m.fin[0], 0);
        mbar_wait_bounded(&m.fin[1], 0);
    }
    tc::fence_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();  // nothing arrives at a CTA that is gone
    if (warp == 1) {
        tc::fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(X::kCols) : "memory");
    }
}

// Joins the pieces of cut contexts: CTA (c, y) that of one context (or of the one that begins in share c), 16 entries (of
// each half) of the 64 rows of one CTA, a thread 16 entries of one row, SPLIT threads its pieces (a few long contexts have
// many).
template <int V, int SPLIT>
__global__ void __launch_bounds__(128 * SPLIT) latent_pair_join_kernel(const __grid_constant__ Args a, int shares, int by_context) {
    __shared__ float part[SPLIT > 1 ? SPLIT - 1 : 1][18][128];
    grid_dependency_wait();
    const Ws ws = ws_of(a, shares, V);
    int4 rec = *reinterpret_cast<const int4 *>(ws.rec + 4 * blockIdx.x);
    if (by_context) rec.x = blockIdx.x * a.H, rec.y = a.H;  // (whatever a wait that ran out kept from being left)
    const int rank = blockIdx.y & 1, at = blockIdx.y >> 1, g = threadIdx.x >> 7, me = threadIdx.x & 127;
    const int row = me & 63, half = me >> 6, r = 64 * rank + row;
    const int n = rec.z, c = rec.w;
    if (n <= 0 || c < 0 || c > shares - n || 64 * rank >= rec.y) return;
    float top = -INFINITY, sum = 0.f, o[16] = {};
    for (int k0 = 2 * g; k0 < n; k0 += 2 * SPLIT) {
        float m[2], l[2];
        float4 y[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int kk = min(k0 + k, n - 1);
            const size_t slot = (size_t)(kk ? 2 * (c + kk) : 2 * c + 1) * 2 + rank;
            m[k] = k0 + k < n ? ws.ml[slot * 128 + row] : -INFINITY;
            l[k] = ws.ml[slot * 128 + 64 + row];
            const float4 *po = reinterpret_cast<const float4 *>(ws.o + slot * 64 * V) + at * 4 * 128 + me;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[k][e] = po[e * 128];
        }
        const float now = fmaxf(top, fmaxf(m[0], m[1])), ref = now == -INFINITY ? 0.f : now, f = exp2f(top - ref);
        top = now;
        sum *= f;
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] *= f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (k0 + k < n) {
                const float f2 = exp2f(m[k] - ref);
                sum += l[k] * f2;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[4 * e] += y[k][e].x * f2, o[4 * e + 1] += y[k][e].y * f2, o[4 * e + 2] += y[k][e].z * f2, o[4 * e + 3] += y[k][e].w * f2;
            }
    }
    if constexpr (SPLIT > 1) {
        if (g) {
#pragma unroll
            for (int e = 0; e < 16; ++e) part[g - 1][e][me] = o[e];
            part[g - 1][16][me] = top, part[g - 1][17][me] = sum;
        }
        __syncthreads();
        if (g) return;
        float now = top, f[SPLIT];
#pragma unroll
        for (int k = 1; k < SPLIT; ++k) now = fmaxf(now, part[k - 1][16][me]);
        if (now == -INFINITY) now = 0.f;
#pragma unroll
        for (int k = 0; k < SPLIT; ++k) f[k] = exp2f((k ? part[k - 1][16][me] : top) - now);
        sum *= f[0];
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] *= f[0];
#pragma unroll
        for (int k = 1; k < SPLIT; ++k) {
            sum += part[k - 1][17][me] * f[k];
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] += part[k - 1][e][me] * f[k];
        }
    }
    if (r >= rec.y) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
    __nv_bfloat16 *out = (__nv_bfloat16 *)a.out + ((int64_t)rec.x + r) * V + half * (V / 2) + at * 16;
    *reinterpret_cast<uint4 *>(out) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(out + 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

// The output's rows: boxes of 32 rows of 32 entries.
bool make_out_map(CUtensorMap *map, void *out, int64_t rows, int V) {
    return make_map(map, out, MapShape{2, CU_TENSOR_MAP_SWIZZLE_64B, {(uint64_t)V, (uint64_t)rows, 0u}, {(uint64_t)V * 2, 0u}, {32u, 32u, 0u}});
}

template <int V>
pkv_status launch(Args a, cudaStream_t st) {
    using X = L<V>;
    static bool done[128];
    const int pairs = sm_count() / 2;
    if (pairs == 0 || !ensure_smem(latent_pair_kernel<V>, X::total, done)) return PKV_ERR_CUDA;
    CUtensorMap tm_q, tm_k0, tm_k1, tm_v, tm_o;
    const int64_t rows = (int64_t)a.NB * a.B;
    if (!make_rows_map(&tm_q, a.q, (int64_t)a.T * a.H, V, 64, X::kChunks) || !make_rows_map(&tm_k0, a.cache, rows, V, 8, X::kPart0) ||
        !make_rows_map(&tm_k1, a.cache, rows, V, 8, X::kChunks - X::kPart0) || !make_rows_map(&tm_v, a.cache, rows, V, 8, V / 128) ||
        !make_out_map(&tm_o, a.out, (int64_t)a.T * a.H, V))
        return PKV_ERR_CUDA;
    // A decode of no more contexts than shares: the join's CTAs go by contexts.
    const int by_context = !a.q_starts && a.S <= pairs;
    a.whole = whole_contexts(a, kRows, kTok, pairs);
    a.once = read_once(a, kRows);
    const unsigned ctas = 2 * (a.whole ? (unsigned)(a.S * a.whole) : (unsigned)pairs);
    const pkv_status rc = launch_pdl(latent_pair_kernel<V>, dim3(ctas), dim3(kThreads), (size_t)X::total, st, tm_q, tm_k0, tm_k1,
                                     tm_v, tm_o, a, by_context);
    if (rc != PKV_OK || a.whole) return rc;
    const dim3 grid(by_context ? (unsigned)a.S : (unsigned)pairs, V / 16);
    if (by_context && a.S * 4 < pairs) return launch_pdl(latent_pair_join_kernel<V, 4>, grid, dim3(512), 0, st, a, pairs, by_context);
    return launch_pdl(latent_pair_join_kernel<V, 1>, grid, dim3(128), 0, st, a, pairs, by_context);
}

}  // namespace

size_t pair_workspace(int V) {
    const int sms = sm_count();
    return round256(ws_bytes((sms > 0 ? sms : 160) / 2, V));
}

pkv_status run_pair(const Args &a, cudaStream_t st) { return a.V == 512 ? launch<512>(a, st) : launch<256>(a, st); }

}  // namespace latent
}  // namespace pkv
