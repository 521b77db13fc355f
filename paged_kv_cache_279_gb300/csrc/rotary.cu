// Rotation of queries and keys by their positions, alone (rotary_embed) and on
// the way into a paged cache (kv_cache_write_rotary, latent_cache_write).
//
// Pair i of the R / 2 rotated pairs of a row at position p turns by the angle
// p f_i, scaled by the amplitude a:
//     c = a cos(p f_i), s = a sin(p f_i);  y1 = x1 c - x2 s;  y2 = x2 c + x1 s
// in float32, rounded once to the rows' type.
//
// Angles.  In float32 the product p f_i of a far position is off by up to
// 2^-25 of itself, 0.03 radians at a million.  Here it is held in turns as a
// 64-bit binary fraction: f_i / 2 pi = G 2^-64 once, then p G modulo 2^64 is the
// angle modulo one turn, off by p times G's error (its last place, and f_i 2^-72 of
// the constant's 64 bits: p (2^-64 + f_i 2^-72) turns at most), in one
// integer multiplication, with no 64-bit floating point and no table of
// positions.  Its signed value converts to float32 half turns with a relative
// error of 2^-24, and sincospif needs no range reduction there.
//
// One launch moves up to three kinds of rows: Q (rotated, stored by token), K
// (rotated, stored by slot), V (copied, stored by slot).  A thread moves 16
// entries: 8 pairs (two runs of 8 where pairs are R / 2 apart) or 16 entries
// that are only copied, as 16-byte vectors.  What bounds it: DRAM traffic for
// long inputs, for short ones the launch and one chain of dependent loads
// (position, angle).  So each CTA computes the sines and cosines of its tokens
// once, one pair a thread, into shared memory, for all heads, while the loads of
// the threads' first entries are in flight.  Measured, from CUDA graphs: 64 tokens of 32 to 48 heads 2 us; 16384 tokens of 32
// heads of 128 bf16 46.4 us (5.8 TB/s, 87 % of a plain copy), 16001 of 32 + 8 + 8 heads into a cache 64.5 us (6.1 TB/s).  A second unit in
// flight a thread (70 instead of 40 registers) takes 6 to 18 % longer, 32 registers by spilling 7 % longer.
#include <cmath>

#include "pkv_internal.cuh"
#include "pkv_ptx.cuh"

namespace pkv {

namespace {

constexpr int kRotThreads = 256;
constexpr int kMaxPairs = 128;  // R <= 256
constexpr int kMaxTok = 8;      // tokens of one CTA

struct RotSeg {
    const unsigned char *src;
    unsigned char *dst;
    int64_t src_t, src_h, dst_t, dst_h;  // bytes from token to token, head to head (dst_t, dst_h: rows stored by token)
    int64_t row;                         // bytes of a cache row (rows stored by slot); 0: stored by token
    int heads;
    uint32_t units, units_magic;  // units of 16 entries in one head's row
    uint32_t end;                 // units of this and the earlier kinds of rows in one token
    int rot0, rot1;               // first and last + 1 rotated unit; rot0 == rot1: copied
};

struct RotArgs {
    RotSeg seg[3];
    const int64_t *slots;
    const int32_t *positions;
    const double *freqs;
    unsigned int *err;
    int64_t num_slots;
    int T, tok, pairs, block;
    uint32_t pairs_magic, total, total_magic;  // total: units of one token
    float amplitude;
};

// n / d for n < 2^16 and 1 <= d <= 2^16, magic = ceil(2^32 / d)
__device__ __forceinline__ uint32_t div16(uint32_t n, uint32_t d, uint32_t magic) {
    return d == 1 ? n : __umulhi(n, magic);
}

// f / 2 pi modulo 1 in 64 binary places, truncated: f = m 2^(e - 52) with a
// 53-bit m, and 2^66 / 2 pi = 11743562013128004905.985, so
// f / 2 pi 2^64 = (m 11743562013128004906) 2^(e - 54), too large by 2^-69.4 of itself.  Zero, subnormal, infinite and NaN
// frequencies give 0.
__device__ __forceinline__ uint64_t turns64(double f) {
    const uint64_t b = (uint64_t)__double_as_longlong(f);
    const int ex = (int)((b >> 52) & 0x7ff);
    if (ex == 0 || ex == 0x7ff) return 0;
    const uint64_t m = (b & 0xfffffffffffffull) | (1ull << 52);
    const uint64_t k = 11743562013128004906ull;
    const uint64_t lo = m * k, hi = __umul64hi(m, k);
    const int sh = 54 - (ex - 1023);  // right shift of hi:lo
    uint64_t g;
    if (sh >= 128) g = 0;
    else if (sh >= 64) g = hi >> (sh - 64);
    else if (sh > 0) g = (hi << (64 - sh)) | (lo >> sh);
    else if (sh > -64) g = lo << -sh;
    else g = 0;
    return b >> 63 ? 0ull - g : g;
}

__device__ __forceinline__ float2 cos_sin(int32_t p, double f, float amplitude) {
    const uint64_t a = (uint64_t)(int64_t)p * turns64(f);
    const float half_turns = __ll2float_rn((long long)a) * 0x1p-63f;
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(amplitude * c, amplitude * s);
}

template <int BYTES>  // of an entry
struct Unit {
    uint4 v[BYTES];  // 16 entries: the first half the first entries of 8 pairs (or 16 in order)
};

template <int BYTES, bool INTER>
__device__ __forceinline__ void turn(Unit<BYTES> &u, const float2 *cs) {
    uint32_t *w = reinterpret_cast<uint32_t *>(u.v);
    if constexpr (BYTES == 2) {
        if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = bf16x2_lo(w[i]), b = bf16x2_hi(w[i]);
                w[i] = pack_bf16x2(a * cs[i].x - b * cs[i].y, b * cs[i].x + a * cs[i].y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a0 = bf16x2_lo(w[i]), a1 = bf16x2_hi(w[i]), b0 = bf16x2_lo(w[4 + i]), b1 = bf16x2_hi(w[4 + i]);
                const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
                w[i] = pack_bf16x2(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
                w[4 + i] = pack_bf16x2(b0 * c0.x + a0 * c0.y, b1 * c1.x + a1 * c1.y);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t &wa = w[INTER ? 2 * i : i], &wb = w[INTER ? 2 * i + 1 : 8 + i];
            const float a = __uint_as_float(wa), b = __uint_as_float(wb);
            wa = __float_as_uint(a * cs[i].x - b * cs[i].y);
            wb = __float_as_uint(b * cs[i].x + a * cs[i].y);
        }
    }
}

// Where a unit of work lies: token, source and destination of its two halves.
struct Place {
    const unsigned char *src;
    unsigned char *dst;
    int second;  // bytes from the first 8 entries to the second 8
    int pair;    // first pair, or -1: copied
    int tok;     // token in the CTA
};

template <int BYTES, bool INTER>
__device__ __forceinline__ bool place(const RotArgs &a, int t0, uint32_t w, Place &pl) {
    const uint32_t tk = div16(w, a.total, a.total_magic);
    const int64_t t = t0 + (int)tk;
    if (t >= a.T) return false;
    uint32_t u = w - tk * a.total;
    const int g = u >= a.seg[1].end ? 2 : u >= a.seg[0].end ? 1 : 0;
    const RotSeg &s = a.seg[g];
    u -= g == 0 ? 0u : a.seg[g - 1].end;
    const uint32_t h = div16(u, s.units, s.units_magic);
    const int j = (int)(u - h * s.units);
    int at = 16 * j;
    pl.second = 8 * BYTES;
    pl.pair = -1;
    pl.tok = (int)tk;
    if (j >= s.rot0 && j < s.rot1) {
        pl.pair = 8 * (j - s.rot0);
        if (!INTER) {
            at = 16 * s.rot0 + pl.pair;
            pl.second = a.pairs * BYTES;
        }
    }
    pl.src = s.src + t * s.src_t + h * s.src_h + at * BYTES;
    if (s.row == 0) {
        pl.dst = s.dst + t * s.dst_t + h * s.dst_h + at * BYTES;
        return true;
    }
    const int64_t slot = a.slots[t];
    if (slot < 0) return false;
    if (slot >= a.num_slots) {
        if (j == 0 && h == 0) flag_error(a.err, PKV_DEVERR_SLOT);
        return false;
    }
    const int64_t blk = slot / a.block;  // block sizes are powers of two, but this is once a unit
    pl.dst = s.dst + ((blk * s.heads + h) * a.block + (slot - blk * a.block)) * s.row + at * BYTES;
    return true;
}

template <int BYTES, bool INTER>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotArgs a) {
    __shared__ float2 cs[kMaxTok * kMaxPairs];
    grid_dependency_wait();
    const int t0 = blockIdx.x * a.tok;
    const uint32_t n = a.total * (uint32_t)a.tok, step = gridDim.y * kRotThreads;
    uint32_t w = blockIdx.y * kRotThreads + threadIdx.x;
    constexpr int kHalf = BYTES / 2;  // 16-byte vectors of 8 entries
    Place pl;
    Unit<BYTES> u;
    bool live = w < n && place<BYTES, INTER>(a, t0, w, pl);
    auto load = [&] {
#pragma unroll
        for (int i = 0; i < kHalf * 2; ++i)
            u.v[i] = *reinterpret_cast<const uint4 *>(pl.src + (i < kHalf ? 0 : pl.second) + 16 * (i % kHalf));
    };
    if (live) load();
    for (int i = threadIdx.x; i < a.tok * a.pairs; i += kRotThreads) {
        const int tk = (int)div16((uint32_t)i, (uint32_t)a.pairs, a.pairs_magic);
        if (t0 + tk < a.T) cs[i] = cos_sin(a.positions[t0 + tk], a.freqs[i - tk * a.pairs], a.amplitude);
    }
    __syncthreads();
    while (true) {
        if (live) {
            if (pl.pair >= 0) turn<BYTES, INTER>(u, cs + pl.tok * a.pairs + pl.pair);
#pragma unroll
            for (int i = 0; i < kHalf * 2; ++i)
                *reinterpret_cast<uint4 *>(pl.dst + (i < kHalf ? 0 : pl.second) + 16 * (i % kHalf)) = u.v[i];
        }
        w += step;
        if (w >= n) break;
        live = place<BYTES, INTER>(a, t0, w, pl);
        if (live) load();
    }
}

uint32_t magic32(uint32_t d) { return (uint32_t)((0x100000000ull + d - 1) / d); }

// Fills one kind of rows; `units` of 16 entries in a row of `dim`, rotated from
// entry off to off + rot.
void set_seg(RotArgs &a, int g, const void *src, void *dst, int64_t src_t, int64_t src_h, int64_t dst_t, int64_t dst_h,
             int64_t row, int heads, int dim, int off, int rot) {
    RotSeg &s = a.seg[g];
    s.src = (const unsigned char *)src;
    s.dst = (unsigned char *)dst;
    s.src_t = src_t, s.src_h = src_h, s.dst_t = dst_t, s.dst_h = dst_h, s.row = row;
    s.heads = heads;
    s.units = (uint32_t)(dim / 16);
    s.units_magic = magic32(s.units);
    s.rot0 = off / 16;
    s.rot1 = (off + rot) / 16;
    s.end = (g ? a.seg[g - 1].end : 0) + (uint32_t)heads * s.units;
}

pkv_status launch_rotary(RotArgs &a, int dtype, int interleaved, void *stream) {
    a.total = a.seg[2].end;
    a.total_magic = magic32(a.total);
    a.pairs_magic = magic32((uint32_t)a.pairs);
    a.err = device_error_word();
    // Few tokens: one a CTA, its rows spread over CTAs of one unit a thread
    // (64 tokens of 48 heads: 128 CTAs).  Many: as many tokens as give each
    // thread one pair's sine and cosine, so that those are computed once for
    // all heads.
    const int sms = sm_count();
    if (sms == 0) return PKV_ERR_CUDA;
    int most = kRotThreads / a.pairs;
    most = most < 1 ? 1 : most > kMaxTok ? kMaxTok : most;
    // ... and of those counts the one that leaves the fewest threads idle in the last round over the units
    int tok = 1;
    uint32_t idle = 0xffffffffu;  // threads without a unit, of 2^16 rounds' threads
    for (int t = 1; t <= most && (t == 1 || ((int64_t)a.T / t >= 8 * sms && (int64_t)t * a.total < 65536)); ++t) {
        const uint32_t n = a.total * (uint32_t)t, rounds = (n + kRotThreads - 1) / kRotThreads;
        const uint32_t waste = (uint32_t)(((uint64_t)(rounds * kRotThreads - n) << 16) / (rounds * kRotThreads));
        if (waste <= idle) tok = t, idle = waste;
    }
    a.tok = tok;
    const int64_t groups = ((int64_t)a.T + tok - 1) / tok;
    const uint32_t per = (a.total * (uint32_t)tok + kRotThreads - 1) / kRotThreads;
    const unsigned gy = groups < 8 * sms ? per : 1;
    auto kern = dtype == PKV_F32 ? (interleaved ? rotary_kernel<4, true> : rotary_kernel<4, false>)
                                 : (interleaved ? rotary_kernel<2, true> : rotary_kernel<2, false>);
    return launch_pdl(kern, dim3((unsigned)groups, gy), dim3(kRotThreads), 0, (cudaStream_t)stream, a);
}

// Checks shared by the three calls.
pkv_status check_rotation(int num_tokens, int dim, int rotary_dim, int offset, float amplitude, int interleaved, int dtype) {
    if (num_tokens < 0 || dim < 1 || rotary_dim < 1 || offset < 0 || offset > dim || rotary_dim > dim - offset)
        return PKV_ERR_INVALID;
    if (!std::isfinite(amplitude) || (interleaved != 0 && interleaved != 1)) return PKV_ERR_INVALID;
    if (dtype != PKV_F32 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (dim % 16 || rotary_dim % 16 || offset % 16 || rotary_dim > 2 * kMaxPairs) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

constexpr int kMaxUnits = 65535;  // of one token's rows

// Strides in entries: whole 16-byte vectors.
bool strides_ok(const int64_t *s, int n, int64_t elt) {
    for (int i = 0; i < n; ++i)
        if (s[i] > (int64_t)1 << 56 || s[i] < -((int64_t)1 << 56) || (s[i] * elt) & 15) return false;
    return true;
}

// Whether rows of `dim` entries, token and head strides s, lie apart: no i < tokens and j < heads but (0, 0) with
// |i s[0] +- j s[1]| < dim.
bool rows_apart(const int64_t *s, int tokens, int heads, int dim) {
    uint64_t st = (uint64_t)(s[0] < 0 ? -s[0] : s[0]), sh = (uint64_t)(s[1] < 0 ? -s[1] : s[1]), n = (uint64_t)tokens, d = (uint64_t)dim;
    if (heads < 2) return tokens < 2 || st >= d;
    if (sh < d) return false;
    if (tokens < 2) return true;
    if (st < d) return false;
    // one kind of steps within the other's, as in all usual layouts
    if (st >= sh ? (st - d) / sh >= (uint64_t)(heads - 1) : (sh - d) / st >= n - 1) return true;
    for (int j = 1; j < heads; ++j) {
        const unsigned __int128 x = (unsigned __int128)sh * (unsigned)j, i = x / st;
        const uint64_t r = (uint64_t)(x % st);
        if ((i < n && r < d) || (i + 1 < n && st - r < d)) return false;
    }
    return true;
}

// Rows written (s[0], s[1]) and read (s[2], s[3]): written rows lie apart, and are the rows read where out is x.
bool rows_ok(const void *out, const void *x, const int64_t *s, int tokens, int heads, int dim) {
    if (out == x && ((tokens > 1 && s[0] != s[2]) || (heads > 1 && s[1] != s[3]))) return false;
    return rows_apart(s, tokens, heads, dim);
}

}  // namespace

}  // namespace pkv

using namespace pkv;

PKV_API pkv_status rotary_frequencies(double *out, int rotary_dim, double base, double factor, double original_len,
                                      double low_turns, double high_turns) {
    if (!out || rotary_dim < 2 || rotary_dim % 2) return PKV_ERR_INVALID;
    if (!std::isfinite(base) || !(base > 0.0) || !std::isfinite(factor) || !(factor > 0.0)) return PKV_ERR_INVALID;
    if (!std::isfinite(original_len) || original_len < 0.0) return PKV_ERR_INVALID;
    if (original_len > 0.0 && !(std::isfinite(low_turns) && std::isfinite(high_turns) && low_turns < high_turns))
        return PKV_ERR_INVALID;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rotary_dim);
        double w = 0.0;  // the part of the frequency that stays as it is
        if (original_len > 0.0) {
            const double turns = original_len * f / 6.283185307179586476925;
            w = (turns - low_turns) / (high_turns - low_turns);
            w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
        }
        out[i] = f * (w + (1.0 - w) / factor);
        if (!std::isfinite(out[i])) return PKV_ERR_INVALID;  // (the calls would take it for 0)
    }
    return PKV_OK;
}

PKV_API pkv_status rotary_embed(void *out, const void *x, const int32_t *positions, const double *frequencies, int num_tokens,
                                int num_heads, int head_dim, int rotary_dim, int offset, const int64_t *strides,
                                float amplitude, int interleaved, int dtype, void *stream) {
    if (num_heads < 1) return PKV_ERR_INVALID;
    const pkv_status rc = check_rotation(num_tokens, head_dim, rotary_dim, offset, amplitude, interleaved, dtype);
    if (rc != PKV_OK) return rc;
    if ((int64_t)num_heads * (head_dim / 16) > kMaxUnits) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (!out || !x || !positions || !frequencies || !aligned16(out) || !aligned16(x)) return PKV_ERR_INVALID;
    const int64_t elt = dtype == PKV_F32 ? 4 : 2;
    const int64_t dense[4] = {(int64_t)num_heads * head_dim, head_dim, (int64_t)num_heads * head_dim, head_dim};
    const int64_t *s = strides ? strides : dense;
    if (!strides_ok(s, 4, elt) || !rows_ok(out, x, s, num_tokens, num_heads, head_dim)) return PKV_ERR_INVALID;
    RotArgs a{};
    a.positions = positions;
    a.freqs = frequencies;
    a.T = num_tokens;
    a.pairs = rotary_dim / 2;
    a.block = 1;
    a.amplitude = amplitude;
    set_seg(a, 0, x, out, s[2] * elt, s[3] * elt, s[0] * elt, s[1] * elt, 0, num_heads, head_dim, offset, rotary_dim);
    set_seg(a, 1, x, out, 0, 0, 0, 0, 0, 0, 16, 0, 0);
    set_seg(a, 2, x, out, 0, 0, 0, 0, 0, 0, 16, 0, 0);
    return launch_rotary(a, dtype, interleaved, stream);
}

PKV_API pkv_status kv_cache_write_rotary(void *q_out, const void *q, const void *k_new, const void *v_new, void *k_cache,
                                         void *v_cache, const int64_t *slot_mapping, const int32_t *positions,
                                         const double *frequencies, int num_tokens, int num_heads, int num_kv_heads,
                                         int head_dim, int rotary_dim, int offset, int block_size, int num_blocks,
                                         const int64_t *strides, float amplitude, int interleaved, int dtype, void *stream) {
    if (num_heads < 0 || num_kv_heads < 1 || block_size < 1 || num_blocks < 1) return PKV_ERR_INVALID;
    const pkv_status rc = check_rotation(num_tokens, head_dim, rotary_dim, offset, amplitude, interleaved, dtype);
    if (rc != PKV_OK) return rc;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PKV_ERR_UNSUPPORTED;
    if (((int64_t)num_heads + 2 * (int64_t)num_kv_heads) * (head_dim / 16) > kMaxUnits) return PKV_ERR_UNSUPPORTED;
    if ((num_heads > 0) != (q != nullptr) || (q != nullptr) != (q_out != nullptr)) return PKV_ERR_INVALID;
    if (num_tokens == 0) return PKV_OK;
    if (!k_new || !v_new || !k_cache || !v_cache || !slot_mapping || !positions || !frequencies) return PKV_ERR_INVALID;
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache))
        return PKV_ERR_INVALID;
    const int64_t elt = dtype == PKV_F32 ? 4 : 2, D = head_dim, qd = num_heads * D, kd = num_kv_heads * D;
    const int64_t dense[8] = {qd, D, qd, D, kd, D, kd, D};
    const int64_t *s = strides ? strides : dense;
    if (num_heads && (!strides_ok(s, 4, elt) || !rows_ok(q_out, q, s, num_tokens, num_heads, head_dim))) return PKV_ERR_INVALID;
    if (!strides_ok(s + 4, 4, elt)) return PKV_ERR_INVALID;
    RotArgs a{};
    a.slots = slot_mapping;
    a.positions = positions;
    a.freqs = frequencies;
    a.num_slots = (int64_t)num_blocks * block_size;
    a.T = num_tokens;
    a.pairs = rotary_dim / 2;
    a.block = block_size;
    a.amplitude = amplitude;
    set_seg(a, 0, q, q_out, s[2] * elt, s[3] * elt, s[0] * elt, s[1] * elt, 0, num_heads, head_dim, offset, rotary_dim);
    set_seg(a, 1, k_new, k_cache, s[4] * elt, s[5] * elt, 0, 0, D * elt, num_kv_heads, head_dim, offset, rotary_dim);
    set_seg(a, 2, v_new, v_cache, s[6] * elt, s[7] * elt, 0, 0, D * elt, num_kv_heads, head_dim, 0, 0);
    return launch_rotary(a, dtype, interleaved, stream);
}

PKV_API pkv_status latent_cache_write(void *q_out, const void *q_rope, const void *latent, const void *k_rope, void *cache,
                                      const int64_t *slot_mapping, const int32_t *positions, const double *frequencies,
                                      int num_tokens, int num_heads, int latent_dim, int block_size, int num_blocks,
                                      const int64_t *strides, float amplitude, int interleaved, int dtype, void *stream) {
    constexpr int kRope = PKV_LATENT_ROPE_DIM;
    if (num_heads < 0 || latent_dim < 1 || block_size < 1 || num_blocks < 1) return PKV_ERR_INVALID;
    const pkv_status rc = check_rotation(num_tokens, kRope, kRope, 0, amplitude, interleaved, dtype);
    if (rc != PKV_OK) return rc;
    if (latent_dim != 256 && latent_dim != 512) return PKV_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64) return PKV_ERR_UNSUPPORTED;
    if ((int64_t)num_heads * (kRope / 16) + (latent_dim + kRope) / 16 > kMaxUnits) return PKV_ERR_UNSUPPORTED;
    if ((num_heads > 0) != (q_rope != nullptr) || (q_rope != nullptr) != (q_out != nullptr)) return PKV_ERR_INVALID;
    if (num_tokens == 0) return PKV_OK;
    if (!latent || !k_rope || !cache || !slot_mapping || !positions || !frequencies) return PKV_ERR_INVALID;
    if (!aligned16(q_rope) || !aligned16(q_out) || !aligned16(latent) || !aligned16(k_rope) || !aligned16(cache)) return PKV_ERR_INVALID;
    const int64_t elt = dtype == PKV_F32 ? 4 : 2, row = latent_dim + kRope, qd = (int64_t)num_heads * kRope;
    const int64_t dense[6] = {qd, kRope, qd, kRope, latent_dim, kRope};
    const int64_t *s = strides ? strides : dense;
    if (num_heads && (!strides_ok(s, 4, elt) || !rows_ok(q_out, q_rope, s, num_tokens, num_heads, kRope))) return PKV_ERR_INVALID;
    if (!strides_ok(s + 4, 2, elt)) return PKV_ERR_INVALID;
    RotArgs a{};
    a.slots = slot_mapping;
    a.positions = positions;
    a.freqs = frequencies;
    a.num_slots = (int64_t)num_blocks * block_size;
    a.T = num_tokens;
    a.pairs = kRope / 2;
    a.block = block_size;
    a.amplitude = amplitude;
    set_seg(a, 0, q_rope, q_out, s[2] * elt, s[3] * elt, s[0] * elt, s[1] * elt, 0, num_heads, kRope, 0, kRope);
    set_seg(a, 1, k_rope, (unsigned char *)cache + latent_dim * elt, s[5] * elt, 0, 0, 0, row * elt, 1, kRope, 0, kRope);
    set_seg(a, 2, latent, cache, s[4] * elt, 0, 0, 0, row * elt, 1, latent_dim, 0, 0);
    return launch_rotary(a, dtype, interleaved, stream);
}
