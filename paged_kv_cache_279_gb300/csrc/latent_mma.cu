// Latent attention on the 5th-generation tensor cores (bf16).
//
// A row tile is up to N (16, 32 or 64) consecutive query rows of one sequence, a
// row being one head of one query; a decode step's heads, or the heads of a few
// drafted tokens, are one.  It is attended against tiles of 64 tokens, transposed:
//     S^T = C Q^T   [64 tokens x N rows]        (C: the tile's cache rows, 9 or 5 chunks of 64 entries)
//     O^T += L^T P^T [V entries x N rows]       (L: the latent part of C, P = exp2(S scale - ref))
// so the tile itself is the wide operand of both products, read once into shared
// memory for both, a context's row count costs no padding to 128, and O^T (V / 128
// blocks of N columns) and two S^T fit tensor memory for every N up to 64 -- O of 128
// rows alone would fill it.
//
// The cache rows of 8 tokens are one TMA box [chunk][8 rows][128 bytes]: any block
// size from 8 on, eight boxes a tile, and both products see 128-byte swizzled
// operands (C by rows, L^T by columns) whose 8-token groups are one stride apart.
//
// Softmax: four warps, a thread holds two tokens of every fourth pair of columns.
// Maxima over tokens would be shuffles over lanes, so the reference of a row moves
// only when a score passes it by 2^kSlack: usually in the first tile alone.  Sums of
// weights stay in the threads, per token, until the end of the piece.  Weights are
// rounded to bf16 (by 2^-8 of each at most; the sums they are divided by are of the
// rounded weights, in float32).
//
// All contexts' tiles are laid end to end and cut into equal shares, one a CTA.  A
// context cut by share boundaries leaves partial results that a second kernel joins.
#include <cmath>

#include "latent.cuh"
#include "pkv_ptx.cuh"

namespace pkv {
namespace latent {

namespace {

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

constexpr int kTok = 64;       // tokens of a tile
constexpr int kThreads = 224;  // producer warp, a warp that issues each product, four softmax warps
constexpr int kDescs = 4;
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

// Maximum of three that is NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Barrier of the softmax warps, alone and with a vote.
constexpr int kSoftmax = 128;
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kSoftmax) : "memory"); }
__device__ __forceinline__ bool softmax_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "n"(kSoftmax)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

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
    static constexpr int kGroup = kChunks * 1024;  // bytes of 8 tokens
    static constexpr int kTile = kTok / 8 * kGroup;
    static constexpr int kPart0 = V / 128;         // chunks of the tile's first part; the second has the rest
    static constexpr int kQ = kChunks * N * 128;
    static constexpr int kQBufs = N <= 32 ? 2 : 1;  // the next piece's queries are loaded under this one's, where they fit
    static constexpr int kP = kTok * 128;
    static constexpr int kMisc = 4096;
    static constexpr int kMax = 232448;  // shared memory of a CTA
    static constexpr int kStages = (kMax - kMisc + 2048 - kQBufs * kQ - kP) / kTile < 4 ? (kMax - kMisc + 2048 - kQBufs * kQ - kP) / kTile : 4;
    static constexpr int q = 0, p = kQBufs * kQ, ring = p + kP, misc = ring + kStages * kTile;
    static constexpr int total = misc + 2048;
    static constexpr int kBlocks = V / 128;              // of O^T
    static constexpr uint32_t kS = kBlocks * N;          // first column of S^T
    static constexpr uint32_t kCols = kS + 2 * N <= 128 ? 128 : kS + 2 * N <= 256 ? 256 : 512;
    static_assert(kStages >= 2 && total <= kMax, "shared memory");
    static_assert(kS + 2 * N <= kCols, "tensor memory");
};

// One share's part of a context.
struct Piece {
    int tiles;     // 0: no more pieces
    int t0, end;   // first token of the first tile; tokens that some row of the row tile sees
    int row0, rows;
    int lim0;      // tokens that row r sees: lim0 + (qh0 + r) / H
    int qh0;
    int out;       // 0: the whole context; 1: its first tiles; 2: later ones
};

struct alignas(8) Misc {
    uint64_t full[2][4], empty[2][4], q_full[2], q_empty[2], s_full[2], s_free[2], p_full, pv_done, o_free, desc_full[kDescs], desc_empty[kDescs], fin[2];
    Piece piece[kDescs];
    float red[4][64];
    uint32_t groups[4];  // valid 8-token groups of a stage's tile
    uint32_t tmem;
    int dead;
};
static_assert(sizeof(Misc) <= 2048, "misc");

// The walk over contexts (sequence, row tile): row tile k of a sequence is rows
// [k N, k N + N) of its n H query rows.  Its last row's query sees
//     p0 + 1 + floor(min(k N + N - 1, n H - 1) / H)  tokens, p0 = L - n0 the first query's position,
// A context counts kHead tiles more than it has, at its start: what its queries' load and the
// storing of its output take.  Its tiles are, but for the last row tile, floor((k + c) / m) with m = 64 H / N and
// c = floor((N - 1 + H (p0 + 64)) / N): sums over k have a closed form.
template <int N>
struct Walk {
    int s, k, R;           // sequence, row tile, row tiles of the sequence
    int L, q0, nH, p0, k0; // k0: first row tile with a query that sees a token
    bool flagged;
    __device__ __forceinline__ void open(const Args &a, int seq) {
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
    __device__ __forceinline__ int end(const Args &a, int kk) const {  // tokens row tile kk sees
        if (!a.q_starts) return L;
        const int last = min((kk + 1) * N, nH) - 1;
        return min(L, p0 + 1 + last / a.H);
    }
    __device__ __forceinline__ int tiles(const Args &a, int kk) const { return (end(a, kk) + kTok - 1) / kTok; }
    // tiles, heads included, of row tiles k0 .. kk - 1, kk < R
    __device__ __forceinline__ int64_t before(const Args &a, int kk) const {
        if (kk <= k0) return 0;
        const int64_t m = (int64_t)kTok / N * a.H;  // N divides 64
        const int64_t c = (N - 1 + (int64_t)a.H * (p0 + kTok)) >> (N == 16 ? 4 : N == 32 ? 5 : 6);  // floor: p0 may be below -64
        return G(kk + c, m) - G(k0 + c, m) + (int64_t)kHead * (kk - k0);
    }
    static __device__ __forceinline__ int64_t G(int64_t x, int64_t m) {  // sum of floor(j / m), j < x
        const int64_t q = x / m;
        return m * (q * (q - 1) / 2) + q * (x - q * m);
    }
    __device__ __forceinline__ int64_t total(const Args &a) const {
        if (k0 >= R) return 0;
        if (!a.q_starts) return (int64_t)R * (tiles(a, 0) + kHead);  // one query: every row tile sees all
        return before(a, R - 1) + tiles(a, R - 1) + kHead;
    }
};

struct Ws {
    int *rec;      // [shares][4]: first row, rows, pieces of the context that begins in a share and is cut
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

constexpr int kMinShare = 2;  // tiles of a share

template <int V, int N>
__global__ void __launch_bounds__(kThreads, 1)
latent_mma_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_c0,
                  const __grid_constant__ CUtensorMap tm_c1, const __grid_constant__ Args a) {
    using X = L<V, N>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Misc &m = *reinterpret_cast<Misc *>(smem + X::misc);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = gridDim.x, cta = blockIdx.x;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 8; ++i) mbar_init(&m.full[i >> 2][i & 3], 1), mbar_init(&m.empty[i >> 2][i & 3], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&m.q_full[i], 1), mbar_init(&m.q_empty[i], 1);
        mbar_init(&m.s_full[0], 1), mbar_init(&m.s_full[1], 1);
        mbar_init(&m.s_free[0], 4), mbar_init(&m.s_free[1], 4);
        mbar_init(&m.p_full, 4), mbar_init(&m.pv_done, 1), mbar_init(&m.o_free, 4), mbar_init(&m.fin[0], 1), mbar_init(&m.fin[1], 1);
        for (int i = 0; i < kDescs; ++i) mbar_init(&m.desc_full[i], 1), mbar_init(&m.desc_empty[i], 6);
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
    grid_launch_dependents();  // the join kernel; it waits for this one before it reads

    // The block tables, read later one entry after another, on their way into L2.
    if (const int64_t line = (int64_t)cta * kThreads + threadIdx.x; (int64_t)a.S * a.maxb <= 1 << 17 && line * 32 < (int64_t)a.S * a.maxb)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.tables + line * 32));

    // Where this CTA's share begins: each thread sums the tiles of a run of sequences,
    // one of them finds the share's first tile in its run.
    int64_t *scan = reinterpret_cast<int64_t *>(m.red);  // warps' totals; then the first tile's offset, and its row tile
    Walk<N> &begin = *reinterpret_cast<Walk<N> *>(scan + 10);
    const int run = (a.S + kThreads - 1) / kThreads;
    const int sb = min(a.S, (int)threadIdx.x * run), se = min(a.S, sb + run);
    int64_t mine = 0;
    Walk<N> w;
    for (int s = sb; s < se; ++s) {
        w.open(a, s);
        mine += w.total(a);
        if (w.flagged && s % G == cta) flag_error(a.err, PKV_DEVERR_SEQ_LEN);
    }
    int64_t incl = mine;
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int64_t base = 0, total = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) base += scan[i];
        total += scan[i];
    }
    const int64_t excl = base + incl - mine;
    int64_t parts = total >= (int64_t)G * kMinShare ? G : (int)total / kMinShare;
    if (parts < 1) parts = 1;
    const bool idle = total == 0 || cta >= parts;
    int64_t first = 0, last = 0;
    if (!idle && total < (1 << 24)) {  // 32-bit division is a fifth of the time (parts <= 152)
        first = (uint32_t)cta * (uint32_t)total / (uint32_t)parts;
        last = (uint32_t)(cta + 1) * (uint32_t)total / (uint32_t)parts;
    } else if (!idle) {
        first = (int64_t)cta * total / parts;
        last = (int64_t)(cta + 1) * total / parts;
    }
    if (!idle && first >= excl && first < excl + mine) {
        int64_t off = first - excl;
        int s = sb;
        for (;; ++s) {
            w.open(a, s);
            const int64_t t = w.total(a);
            if (off < t) break;
            off -= t;
        }
        int k;
        if (!a.q_starts) {
            k = (int)(off / (w.tiles(a, 0) + kHead));
            off -= (int64_t)k * (w.tiles(a, 0) + kHead);
        } else {
            int lo = w.k0, hi = w.R;  // the last k with before(k) <= off
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (w.before(a, mid) <= off) lo = mid;
                else hi = mid;
            }
            k = lo;
            off -= w.before(a, k);
        }
        w.k = k;
        begin = w;
        scan[8] = off;
    }
    const Ws ws = ws_of(a, G, N, V);
    if (threadIdx.x == 0) ws.rec[4 * cta + 2] = 0;
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = m.tmem;
    const int64_t at_off = scan[8];
    w = begin;
    __syncthreads();

    bool dead = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) {  // by whole warps
        bool ok = dead;
        for (uint32_t i = 0; i < kWaitLimit && !ok; ++i) {
            ok = mbar_try_wait(bar, parity);
            if ((i & 255u) == 255u && *(volatile int *)&m.dead) break;
        }
        if (__any_sync(0xffffffffu, !ok)) {
            dead = true;
            *(volatile int *)&m.dead = 1;
            flag_error(a.err, PKV_DEVERR_TIMEOUT);
        }
    };

    if (idle) {
    } else if (warp == 0) {
        // ======================= producer =======================
        int64_t off = at_off;
        int64_t left = last - first;
        int tile = 0, np = 0, nq = 0, halves = 0;  // tiles, pieces, queries and parts of tiles issued
        for (;;) {
            const int d = np % kDescs;
            wait(&m.desc_empty[d], (uint32_t)(np / kDescs + 1) & 1u);
            if (left == 0 || dead) {
                if (lane == 0) {
                    m.piece[d].tiles = 0;
                    mbar_arrive(&m.desc_full[d]);
                }
                break;
            }
            // of the context's kHead + nt tiles, `take` from `off` on are this share's
            const int nt = w.tiles(a, w.k);
            const int take = (int)min((int64_t)nt + kHead - off, left);
            const int i0 = max(0, (int)off - kHead), n = max(0, (int)off + take - kHead) - i0;
            if (n > 0) {
                Piece pc;
                pc.tiles = n;
                pc.t0 = i0 * kTok;
                pc.end = w.end(a, w.k);
                pc.qh0 = w.k * N;
                pc.row0 = w.q0 * a.H + pc.qh0;
                pc.rows = min(N, w.nH - pc.qh0);
                pc.lim0 = w.p0 + 1;
                pc.out = n == nt ? 0 : i0 == 0 ? 1 : 2;
                if (lane == 0) {
                    m.piece[d] = pc;
                    mbar_arrive(&m.desc_full[d]);
                    if (pc.out == 1) {  // how many shares the rest of the context reaches into
                        const int64_t stop = last + (nt - n);  // the context's end in the row of all tiles
                        ws.rec[4 * cta] = pc.row0;
                        ws.rec[4 * cta + 1] = pc.rows;
                        ws.rec[4 * cta + 2] = (int)(share_owner(stop - 1, total, parts) - cta) + 1;
                    }
                }
                __syncwarp();
                const int32_t *table = a.tables + (int64_t)w.s * a.maxb;
                // lane l: the cache row of group l & 7 of tile t + (l >> 3); -1: a bad block; -2: no token
                auto look = [&](int t) {
                    const int tok = pc.t0 + t * kTok + 8 * lane;
                    if (t + (lane >> 3) >= n || tok >= pc.end) return -2;
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
                if (X::kQBufs == 2) load_q();
                for (int t = 0; t < n && !dead; ++t, ++tile) {
                    if ((t & 3) == 0) {
                        if (t) row = next;
                        next = look(t + 4);
                    }
                    const int st = tile % X::kStages;
                    const bool turn = (lane >> 3) == (t & 3);
                    // a group without tokens starts past the tensor's end: zeros
                    const int y = row >= 0 ? row : a.NB << a.bshift;
                    const uint32_t dst = smem_u32(smem + X::ring) + (uint32_t)(st * X::kTile + (lane & 7) * X::kGroup);
                    wait(&m.empty[0][st], (uint32_t)(tile / X::kStages + 1) & 1u);
                    if (dead) break;
                    if (turn && row == -1) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                    const uint32_t ok = __ballot_sync(0xffffffffu, row >= 0) >> (8 * (t & 3)) & 0xffu;
                    if (lane == 0) {
                        m.groups[st] = ok;
                        mbar_arrive_expect_tx(&m.full[0][st], (uint32_t)(kTok * 128 * X::kPart0));
                    }
                    __syncwarp();
                    if (turn) tma_load_3d(dst, &tm_c0, smem_u32(&m.full[0][st]), 0, y, 0);
                    ++halves;
                    wait(&m.empty[1][st], (uint32_t)(tile / X::kStages + 1) & 1u);
                    if (dead) break;
                    if (lane == 0) mbar_arrive_expect_tx(&m.full[1][st], (uint32_t)(X::kTile - kTok * 128 * X::kPart0));
                    __syncwarp();
                    if (turn) tma_load_3d(dst + X::kPart0 * 1024, &tm_c1, smem_u32(&m.full[1][st]), 0, y, X::kPart0);
                    ++halves;
                    if (X::kQBufs == 1 && t == 0) load_q();
                }
                ++np;
            }
            left -= take;
            off = 0;
            if (left > 0 && ++w.k >= w.R) {
                do {
                    if (w.s + 1 >= a.S) {  // lengths that changed under the call
                        dead = true;
                        break;
                    }
                    w.open(a, w.s + 1);
                } while (w.k0 >= w.R);
            }
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
                auto part = [&](auto lo, auto hi) {
#pragma unroll
                    for (int c = lo(); c < hi(); ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc::mma(tmem + X::kS + (uint32_t)((tile & 1) * N), c0 + (uint64_t)((c * 1024 + k * 32) >> 4),
                                    q0 + (uint64_t)((c * N * 128 + k * 32) >> 4), id, c + k > 0 ? 1u : 0u);
                };
                wait(&m.full[0][st], (uint32_t)(tile / X::kStages) & 1u);
                if (dead) break;
                tc::fence_after();
                if (leader) part([] { return 0; }, [] { return X::kPart0; });
                __syncwarp();
                wait(&m.full[1][st], (uint32_t)(tile / X::kStages) & 1u);
                if (dead) break;
                if (leader) {
                    part([] { return X::kPart0; }, [] { return X::kChunks; });
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
#pragma unroll
                    for (int b = 0; b < X::kBlocks; ++b) {
#pragma unroll
                        for (int k = 0; k < kTok / 16; ++k)
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
        constexpr int J = N / 8;
        const float sc = a.scale_log2;
        const int col = 2 * (lane & 3), tok0 = qt * 16 + (lane >> 2);  // first column, first token (the other: 8 on)
        // stmatrix: lane gives the address of row (lane & 7) of matrix lane >> 3: tokens 0-7, 8-15 of column block j, then j + 1
        const uint32_t p_s = smem_u32(smem + X::p) + (uint32_t)((qt * 2 + ((lane >> 3) & 1)) * 1024 + (lane & 7) * 128);
        int tile = 0;
        bool stop = false;  // the four warps leave together: they share a barrier
        for (int np = 0;; ++np) {
            const int d = np % kDescs;
            wait(&m.desc_full[d], (uint32_t)(np / kDescs) & 1u);
            if (softmax_any(dead)) break;
            const Piece pc = m.piece[d];
            if (pc.tiles == 0) break;
            float nref[J][2], l[J][2];  // minus the reference: +inf before the first score
#pragma unroll
            for (int j = 0; j < J; ++j) nref[j][0] = nref[j][1] = INFINITY, l[j][0] = l[j][1] = 0.f;
            const int least = pc.lim0 + pc.qh0 / a.H;  // tokens that the first row sees
            for (int t = 0; t < pc.tiles; ++t, ++tile) {
                const int st = tile % X::kStages;
                wait(&m.s_full[tile & 1], (uint32_t)(tile >> 1) & 1u);
                wait(&m.full[0][st], (uint32_t)(tile / X::kStages) & 1u);  // (complete: orders the read of groups)
                tc::fence_after();
                uint32_t r[4 * J];
                ld_16x256b(lanes + X::kS + (uint32_t)((tile & 1) * N), r);
                tc::wait_ld();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.s_free[tile & 1]);
                const int tb = pc.t0 + t * kTok;
                const uint32_t groups = m.groups[st];
                const bool masked = tb + kTok > least || groups != 0xffu;
                bool bad[2] = {false, false};
                uint32_t hide[2] = {0u, 0u};  // bit 2 j + i: not seen by column 8 j + col + i
                if (masked) {
                    const bool in[2] = {((groups >> (2 * qt)) & 1u) != 0, ((groups >> (2 * qt + 1)) & 1u) != 0};
                    uint32_t nf[2] = {0x7f800000u, 0x7f800000u};
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int c = 8 * j + col + i;
                            const int lim = min(pc.end, pc.lim0 + (pc.qh0 + c) / a.H);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (c < pc.rows) nf[h] &= r[4 * j + 2 * h + i];
                                if (!in[h] || tb + tok0 + 8 * h >= lim) hide[h] |= 1u << (2 * j + i);
                            }
                        }
                    // A row of the cache that holds an infinity or NaN gives every query such a score.  It
                    // must not reach, through 0 * inf, the rows that do not see it: its latent part is
                    // zeroed here, after its scores were taken, and those that see it get NaN.  So are rows
                    // past the last token in sight, whatever they hold.
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        nf[h] &= __shfl_xor_sync(0xffffffffu, nf[h], 1);
                        nf[h] &= __shfl_xor_sync(0xffffffffu, nf[h], 2);
                        bad[h] = (nf[h] & 0x7f800000u) == 0x7f800000u;
                        const int tk = tok0 + 8 * h;
                        if (bad[h] || (in[h] && tb + tk >= pc.end)) {
                            unsigned char *g = smem + X::ring + st * X::kTile + (tk >> 3) * X::kGroup + (tk & 7) * 128;
                            for (int c = lane & 3; c < V / 64; c += 4)
                                for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4 *>(g + c * 1024 + e * 16) = make_uint4(0, 0, 0, 0);
                        }
                    }
                }
                float x[4 * J];
                // log2 of the weights against the references (`blank`: against 0 where there is none yet);
                // the largest, or NaN
                auto weigh = [&](float blank) {
                    float top = -INFINITY;
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float nr = nref[j][i] == INFINITY ? blank : nref[j][i];
                            x[4 * j + i] = fmaf(__uint_as_float(r[4 * j + i]), sc, nr);
                            x[4 * j + 2 + i] = fmaf(__uint_as_float(r[4 * j + 2 + i]), sc, nr);
                            if (masked) {
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    x[4 * j + 2 * h + i] = (hide[h] >> (2 * j + i)) & 1u ? -INFINITY
                                                           : bad[h]                      ? __uint_as_float(0x7fffffffu)
                                                                                         : x[4 * j + 2 * h + i];
                            }
                            top = max3_nan(top, x[4 * j + i], x[4 * j + 2 + i]);
                        }
                    return top;
                };
                const float top = weigh(INFINITY);
                if (tile > 0) wait(&m.pv_done, (uint32_t)(tile - 1) & 1u);  // P is free, and O at rest
                if (softmax_any(!(top <= kSlack) || dead)) {
                    if (softmax_any(dead)) {
                        stop = true;
                        break;
                    }
                    // Some score passed its row's reference by far, or is the row's first: new references
                    // for such rows.  The others keep theirs, so no row's result depends on another's.
                    weigh(0.f);
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
                    softmax_sync();
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
                                f[j][i] = exp2f(-y);
                                l[j][i] *= f[j][i];
                            }
                        }
                    softmax_sync();
                    if (t > 0) {  // O^T has something: scale its columns
                        if (qt == 0 && lane < 4)
#pragma unroll
                            for (int j = 0; j < J; ++j) m.red[0][8 * j + col] = f[j][0], m.red[0][8 * j + col + 1] = f[j][1];
                        softmax_sync();
                        tc::fence_after();
                        constexpr int W = N < 32 ? 16 : 32;
#pragma unroll 1
                        for (int b = 0; b < X::kBlocks * N / W; ++b) {
                            uint32_t o[W];
                            ld_32x32b(lanes + (uint32_t)(b * W), o);
                            tc::wait_ld();
                            const int c0 = b * W % N;
#pragma unroll
                            for (int e = 0; e < W; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * m.red[0][c0 + e]);
                            st_32x32b(lanes + (uint32_t)(b * W), o);
                        }
                        tc::wait_st();
                    }
                    weigh(0.f);
                }
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
                    stmatrix_x4(p_s + (uint32_t)(((j + (lane >> 4)) ^ (lane & 7)) << 4), w2[2 * j], w2[2 * j + 1], w2[2 * j + 2],
                                w2[2 * j + 3]);
                fence_proxy_async();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.p_full);
            }
            if (stop) break;
            softmax_sync();  // red has been read
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
            softmax_sync();
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
            if (softmax_any(dead)) break;
            tc::fence_after();
            // O^T, 16 entries at a time; P's memory is free for the transposition
            const uint32_t stage = smem_u32(smem + X::p) + (uint32_t)(qt * N * 32);
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) sum[j][i] = sum[j][i] == 0.f ? 0.f : 1.f / sum[j][i];
            auto fetch = [&](int u, uint32_t (&r)[4 * J]) { ld_16x256b(lanes + ((uint32_t)(u & 1) << 20) + (uint32_t)((u >> 1) * N), r); };
            auto put = [&](int u, const uint32_t (&r)[4 * J]) {
                const int unit = ((u >> 1) * 4 + qt) * 2 + (u & 1);  // entries 16 unit ..
                if (pc.out) {
                    uint4 *po = reinterpret_cast<uint4 *>(ws.o + slot * N * V) + (size_t)unit * J * 32 + lane;
#pragma unroll
                    for (int j = 0; j < J; ++j) po[j * 32] = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                } else {
                    float o[4 * J];
#pragma unroll
                    for (int e = 0; e < 4 * J; ++e) o[e] = __uint_as_float(r[e]);
                    emit<V, N>(o, sum, stage, lane, (__nv_bfloat16 *)a.out + (int64_t)pc.row0 * V + 16 * unit, pc.rows);
                }
            };
            uint32_t r0[4 * J], r1[4 * J];  // one is loaded while the other is stored
            fetch(0, r0);
#pragma unroll 1
            for (int u = 0; u < 2 * X::kBlocks; u += 2) {
                tc::wait_ld();
                fetch(u + 1, r1);
                put(u, r0);
                tc::wait_ld();
                if (u + 2 < 2 * X::kBlocks) fetch(u + 2, r0);
                put(u + 1, r1);
            }
            tc::fence_before();
            softmax_sync();  // red is read by all before the next piece writes it
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

// Joins the pieces of cut contexts: CTA (c, y) the one that begins in share c, a warp 16 entries of 16
// rows, in the layout the pieces were stored in.  Small units of work, and the loads of several pieces in
// flight: a long context has one piece a share.
constexpr int kJoinWarps = 8;

template <int V, int N>
__global__ void __launch_bounds__(kJoinWarps * 32) latent_mma_join_kernel(const __grid_constant__ Args a, int shares) {
    __shared__ __align__(128) unsigned char sh[kJoinWarps * 16 * 32];
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // queries that see nothing, but for those in a row tile with others
    for (int s = blockIdx.y * gridDim.x + blockIdx.x; s < a.S; s += gridDim.x * gridDim.y) {
        Walk<N> w;
        w.open(a, s);
        const int64_t vecs = min((int64_t)w.k0 * N, (int64_t)w.nH) * (V / 8);
        uint4 *o = reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.out + (int64_t)w.q0 * a.H * V);
        for (int64_t i = threadIdx.x; i < vecs; i += kJoinWarps * 32) o[i] = make_uint4(0, 0, 0, 0);
    }
    const Ws ws = ws_of(a, shares, N, V);
    const int c = blockIdx.x, n = ws.rec[4 * c + 2];
    if (n == 0) return;
    constexpr int kRowUnits = N / 16;
    const int work = blockIdx.y * kJoinWarps + warp, unit = work / kRowUnits, r0 = work % kRowUnits * 16;
    const int row0 = ws.rec[4 * c] + r0, rows = ws.rec[4 * c + 1] - r0;
    if (rows <= 0) return;
    const int col = r0 + 2 * (lane & 3);
    auto ml_of = [&](int k, int j) { return ws.ml + (size_t)(k ? 2 * (c + k) : 2 * c + 1) * 2 * N + col + 8 * j; };
    float ref[2][2], sum[2][2] = {}, o[8] = {};
#pragma unroll
    for (int j = 0; j < 2; ++j) ref[j][0] = ref[j][1] = -INFINITY;
#pragma unroll 4
    for (int k = 0; k < n; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 m = *reinterpret_cast<const float2 *>(ml_of(k, j));
            ref[j][0] = fmaxf(ref[j][0], m.x), ref[j][1] = fmaxf(ref[j][1], m.y);
        }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) ref[j][i] = ref[j][i] == -INFINITY ? 0.f : ref[j][i];
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
        const float4 *po = reinterpret_cast<const float4 *>(ws.o + (size_t)(k ? 2 * (c + k) : 2 * c + 1) * N * V) +
                           (size_t)(unit * (N / 8) + r0 / 8) * 32 + lane;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 m = *reinterpret_cast<const float2 *>(ml_of(k, j)), l = *reinterpret_cast<const float2 *>(ml_of(k, j) + N);
            const float4 y = po[j * 32];
            const float f0 = exp2f(m.x - ref[j][0]), f1 = exp2f(m.y - ref[j][1]);
            sum[j][0] += l.x * f0, sum[j][1] += l.y * f1;
            o[4 * j] += y.x * f0, o[4 * j + 1] += y.y * f1, o[4 * j + 2] += y.z * f0, o[4 * j + 3] += y.w * f1;
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) sum[j][i] = sum[j][i] == 0.f ? 0.f : 1.f / sum[j][i];
    emit<V, 16>(o, sum, smem_u32(sh) + (uint32_t)(warp * 16 * 32), lane, (__nv_bfloat16 *)a.out + (int64_t)row0 * V + 16 * unit, rows);
}

// Rows of V + 64 entries as [chunk of 64 entries][row][64]: a box of `box` rows and `deep` chunks.
bool make_map(CUtensorMap *map, const void *base, int64_t rows, int V, int box, int deep) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const int chunks = V / 64 + 1;
    cuuint64_t dims[3] = {64u, (cuuint64_t)rows, (cuuint64_t)chunks};
    cuuint64_t strides[2] = {(cuuint64_t)(V + kRope) * 2, 128u};
    cuuint32_t boxd[3] = {64u, (cuuint32_t)box, (cuuint32_t)deep};
    cuuint32_t estr[3] = {1u, 1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, boxd, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a row tile: the smallest that holds a sequence's query rows, or 64.
int rows_of(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

template <int V, int N>
pkv_status launch(const Args &a, cudaStream_t st) {
    static bool done[128];
    const int sms = sm_count();
    if (sms == 0 || !ensure_smem(latent_mma_kernel<V, N>, L<V, N>::total, done)) return PKV_ERR_CUDA;
    using X = L<V, N>;
    CUtensorMap tm_q, tm_c0, tm_c1;
    const int64_t rows = (int64_t)a.NB * a.B;
    if (!make_map(&tm_q, a.q, (int64_t)a.T * a.H, V, N, X::kChunks) || !make_map(&tm_c0, a.cache, rows, V, 8, X::kPart0) ||
        !make_map(&tm_c1, a.cache, rows, V, 8, X::kChunks - X::kPart0))
        return PKV_ERR_CUDA;
    const pkv_status rc = launch_pdl(latent_mma_kernel<V, N>, dim3((unsigned)sms), dim3(kThreads), (size_t)X::total, st, tm_q, tm_c0, tm_c1, a);
    if (rc != PKV_OK) return rc;
    return launch_pdl(latent_mma_join_kernel<V, N>, dim3((unsigned)sms, (unsigned)(V * N / 256 / kJoinWarps)), dim3(kJoinWarps * 32), 0, st, a, sms);
}

}  // namespace

size_t mma_workspace(int64_t T, int H, int V) {
    const int sms = sm_count();
    return round256(ws_bytes(sms > 0 ? sms : 160, rows_of(T * H), V));
}

pkv_status run_mma(const Args &a, cudaStream_t st) {
    const int64_t rows = (int64_t)(a.q_starts ? a.max_q : 1) * a.H;
    switch (rows_of(rows)) {
        case 16: return a.V == 512 ? launch<512, 16>(a, st) : launch<256, 16>(a, st);
        case 32: return a.V == 512 ? launch<512, 32>(a, st) : launch<256, 32>(a, st);
        default: return a.V == 512 ? launch<512, 64>(a, st) : launch<256, 64>(a, st);
    }
}

}  // namespace latent
}  // namespace pkv
