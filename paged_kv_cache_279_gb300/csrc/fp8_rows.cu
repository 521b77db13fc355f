// Row-scaled FP8 (E4M3) cache: kv_cache_write_fp8_rows quantises new K/V rows
// as it stores them, kv_cache_read_fp8_rows gathers the values of stored rows
// back.  Source: "KV cache & PagedAttention -- vi sao chatbot AI ton bo nho"
// (aiwiki.vn), the paragraph on quantisation and offloading; the page fixes no
// format (see pkv.h for the one taken here).
//
// A row x (one token's K or V of one KV head) is held as head_dim codes and
// one byte e + 127:
//     e = the smallest integer with max |x_i| <= 448 * 2^e, held in [-100, 120]
//     code_i = e4m3(x_i * 2^-e)            value_i = e4m3(code_i) * 2^e
// A power of two costs no accuracy in a floating format (every value keeps its
// 3 fraction bits; at most one binade of the 18 that E4M3 spans is unused) and
// makes both products exact: x_i * 2^-e is rounded once, to the code, and a
// value has 4 significant bits, so it is a bf16 number.  No division anywhere.
//
// Both kernels move each byte once and are bound by HBM for many tokens and by
// the launch for few.  A lane takes 16 elements of a row, 32 bytes of bf16 in one
// access, where the plain rows lie on 32-byte boundaries, else 8: 65536 tokens of
// 8 KV heads of 128 are read in 63.5 us (6.4 TB/s, 94 % of a plain copy; 73 us with
// 8), 16384 written in 20.6 (4.9 TB/s; 22.6 with 8).
#include <type_traits>

#include "pkv_internal.cuh"
#include "scored.cuh"

namespace pkv {

// 16-byte and 32-byte accesses of consecutive words.
template <int W>
__device__ __forceinline__ void load_words(const void *p, uint32_t (&w)[W]) {
    static_assert(W == 2 || W == 4 || W == 8, "");
    if constexpr (W == 2) {
        const uint2 v = *static_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    } else if constexpr (W == 4) {
        const uint4 v = *static_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    }
}
template <int W>
__device__ __forceinline__ void store_words(void *p, const uint32_t (&w)[W]) {
    static_assert(W == 2 || W == 4 || W == 8, "");
    if constexpr (W == 2) {
        *static_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (W == 4) {
        *static_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                     "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    }
}

// E (8 or 16) consecutive elements of a row, as float.
template <int E>
__device__ __forceinline__ void load_row(const float *p, float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < E; i += E / 2) {
        uint32_t w[E / 2];
        load_words(p + i, w);
#pragma unroll
        for (int k = 0; k < E / 2; ++k) x[i + k] = __uint_as_float(w[k]);
    }
}
template <int E>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *p, float (&x)[E]) {
    uint32_t w[E / 2];
    load_words(p, w);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        x[2 * i] = bf16x2_lo(w[i]);
        x[2 * i + 1] = bf16x2_hi(w[i]);
    }
}
template <int E>
__device__ __forceinline__ void store_row(float *p, const float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < E; i += E / 2) {
        uint32_t w[E / 2];
#pragma unroll
        for (int k = 0; k < E / 2; ++k) w[k] = __float_as_uint(x[i + k]);
        store_words(p + i, w);
    }
}
template <int E>
__device__ __forceinline__ void store_row(__nv_bfloat16 *p, const float (&x)[E]) {
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    store_words(p, w);
}

// The scale byte of a row whose largest finite magnitude is `amax`: with amax
// = 1.m * 2^(b - 127) and 448 = 1.75 * 2^8, e = b - 135, plus one when 1.m is
// above 1.75.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int s = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)min(kMaxScaleByte, max(kMinScaleByte, s));
}

// One group of head_dim / E lanes per (token, KV head), K and V together: each
// lane holds E elements of both rows, the group's maximum comes from
// log2(head_dim / E) shuffles, and every lane stores E codes (a 64-byte or
// 128-byte row per group).
template <typename T, int D, int E>
__global__ void __launch_bounds__(256)
kv_cache_write_fp8_rows_kernel(const T *__restrict__ k_new, const T *__restrict__ v_new,
                               unsigned char *__restrict__ k_cache, unsigned char *__restrict__ v_cache,
                               unsigned char *__restrict__ k_scales, unsigned char *__restrict__ v_scales,
                               const int64_t *__restrict__ slot_mapping, uint32_t num_rows, int num_kv_heads, int bshift,
                               int64_t num_slots, unsigned int *err) {
    // a dependent attention kernel may start its launch; it waits for this grid before reading the cache
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kLanes = D / E;
    const uint32_t row = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;  // (num_rows < 2^31)
    const int c = threadIdx.x % kLanes;
    const bool live = row < num_rows;
    const uint32_t t = live ? row / (uint32_t)num_kv_heads : 0u;
    const int h = (int)(row - t * num_kv_heads);
    const int64_t slot = live ? slot_mapping[t] : -1;
    if (slot >= num_slots && c == 0 && h == 0) flag_error(err, PKV_DEVERR_SLOT);
    const bool store = slot >= 0 && slot < num_slots;
    float x[2][E];
    if (store) {
        load_row(k_new + (int64_t)row * D + E * c, x[0]);
        load_row(v_new + (int64_t)row * D + E * c, x[1]);
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) x[0][j] = x[1][j] = 0.f;
    }
    const int64_t blk = slot >> bshift, off = slot - (blk << bshift);
    const int64_t dst = (((blk * num_kv_heads + h) << bshift) + off);  // cache row
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const float m = fabsf(x[w][j]);
            amax = m < INFINITY ? fmaxf(amax, m) : amax;  // infinities and NaN do not set the scale
        }
#pragma unroll
        for (int sh = kLanes / 2; sh > 0; sh >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, sh));
        if (!store) continue;
        const uint32_t b = scale_byte(amax);
        const float inv = __uint_as_float((254u - b) << 23);  // 2^-e, a normal number
        uint32_t code[E / 4];
#pragma unroll
        for (int j = 0; j < E / 4; ++j)
            code[j] = e4m3x2(x[w][4 * j] * inv, x[w][4 * j + 1] * inv) |
                      (e4m3x2(x[w][4 * j + 2] * inv, x[w][4 * j + 3] * inv) << 16);
        store_words((w ? v_cache : k_cache) + dst * D + E * c, code);
        if (c == 0) (w ? v_scales : k_scales)[dst] = (unsigned char)b;
    }
}

// One lane per E codes of a (token, KV head) row, K and V together.
template <typename T, int D, int E>
__global__ void __launch_bounds__(256)
kv_cache_read_fp8_rows_kernel(T *__restrict__ k_out, T *__restrict__ v_out, const unsigned char *__restrict__ k_cache,
                              const unsigned char *__restrict__ v_cache, const unsigned char *__restrict__ k_scales,
                              const unsigned char *__restrict__ v_scales, const int64_t *__restrict__ slot_mapping,
                              uint32_t num_rows, int num_kv_heads, int bshift, int64_t num_slots, unsigned int *err) {
    constexpr int kLanes = D / E;
    const uint32_t row = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;  // (num_rows < 2^31)
    const int c = threadIdx.x % kLanes;
    if (row >= num_rows) return;
    const uint32_t t = row / (uint32_t)num_kv_heads;
    const int h = (int)(row - t * num_kv_heads);
    const int64_t slot = slot_mapping[t];
    if (slot < 0) return;  // padding: the output row is left as it was
    if (slot >= num_slots) {
        if (c == 0 && h == 0) flag_error(err, PKV_DEVERR_SLOT);
        return;
    }
    const int64_t blk = slot >> bshift, off = slot - (blk << bshift);
    const int64_t src = (((blk * num_kv_heads + h) << bshift) + off);
    uint32_t code[2][E / 4];
    load_words(k_cache + src * D + E * c, code[0]);
    load_words(v_cache + src * D + E * c, code[1]);
    const float f[2] = {row_scale(k_scales[src]), row_scale(v_scales[src])};
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float x[E];
#pragma unroll
        for (int j = 0; j < E / 4; ++j) e4m3x4_to_float(code[w][j], x + 4 * j);
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] *= f[w];
        store_row((w ? v_out : k_out) + (int64_t)row * D + E * c, x);
    }
}

// Argument checks shared by the two calls; *blocks = 0 when there is nothing to do.
static pkv_status check_rows(const void *a, const void *b, const void *k_cache, const void *v_cache, const void *k_scales,
                             const void *v_scales, const int64_t *slots, int num_tokens, int num_kv_heads, int head_dim,
                             int block_size, int num_blocks, int dtype, int64_t *blocks, bool *wide) {
    *blocks = 0;
    if (num_tokens < 0 || num_kv_heads < 1 || head_dim < 1 || block_size < 1 || num_blocks < 1) return PKV_ERR_INVALID;
    if (dtype != PKV_F32 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (block_size != 16 && block_size != 32) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (!a || !b || !k_cache || !v_cache || !k_scales || !v_scales || !slots) return PKV_ERR_INVALID;
    if (!aligned16(a) || !aligned16(b) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scales) ||
        !aligned16(v_scales))
        return PKV_ERR_INVALID;
    const int64_t rows = (int64_t)num_tokens * num_kv_heads;
    if (rows > INT32_MAX) return PKV_ERR_UNSUPPORTED;  // (K and V rows of more would not fit the device)
    *wide = ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 31u) == 0;
    const int per_cta = 256 / (head_dim / (*wide ? 16 : 8));
    *blocks = (rows + per_cta - 1) / per_cta;
    return PKV_OK;
}

}  // namespace pkv

using namespace pkv;

PKV_API pkv_status kv_cache_write_fp8_rows(const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                                           void *k_scales, void *v_scales, const int64_t *slot_mapping, int num_tokens,
                                           int num_kv_heads, int head_dim, int block_size, int num_blocks, int dtype,
                                           void *stream) {
    int64_t blocks;
    bool wide;
    const pkv_status rc = check_rows(k_new, v_new, k_cache, v_cache, k_scales, v_scales, slot_mapping, num_tokens,
                                     num_kv_heads, head_dim, block_size, num_blocks, dtype, &blocks, &wide);
    if (rc != PKV_OK || blocks == 0) return rc;
    auto go = [&](auto kern, auto *k, auto *v) {
        kern<<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(
            k, v, (unsigned char *)k_cache, (unsigned char *)v_cache, (unsigned char *)k_scales, (unsigned char *)v_scales,
            slot_mapping, (uint32_t)(num_tokens * num_kv_heads), num_kv_heads, block_size == 16 ? 4 : 5,
            (int64_t)num_blocks * block_size, device_error_word());
        return launch_status();
    };
    auto pick = [&](auto t, auto e) {
        using T = decltype(t);
        constexpr int E = decltype(e)::value;
        auto *k = (const T *)k_new;
        auto *v = (const T *)v_new;
        return head_dim == 128 ? go(kv_cache_write_fp8_rows_kernel<T, 128, E>, k, v) : go(kv_cache_write_fp8_rows_kernel<T, 64, E>, k, v);
    };
    auto size = [&](auto t) {
        return wide ? pick(t, std::integral_constant<int, 16>{}) : pick(t, std::integral_constant<int, 8>{});
    };
    return dtype == PKV_F32 ? size(float{}) : size(__nv_bfloat16{});
}

PKV_API pkv_status kv_cache_read_fp8_rows(void *k_out, void *v_out, const void *k_cache, const void *v_cache,
                                          const void *k_scales, const void *v_scales, const int64_t *slot_mapping,
                                          int num_tokens, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                          int dtype, void *stream) {
    int64_t blocks;
    bool wide;
    const pkv_status rc = check_rows(k_out, v_out, k_cache, v_cache, k_scales, v_scales, slot_mapping, num_tokens,
                                     num_kv_heads, head_dim, block_size, num_blocks, dtype, &blocks, &wide);
    if (rc != PKV_OK || blocks == 0) return rc;
    auto go = [&](auto kern, auto *k, auto *v) {
        kern<<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(
            k, v, (const unsigned char *)k_cache, (const unsigned char *)v_cache, (const unsigned char *)k_scales,
            (const unsigned char *)v_scales, slot_mapping, (uint32_t)(num_tokens * num_kv_heads), num_kv_heads,
            block_size == 16 ? 4 : 5, (int64_t)num_blocks * block_size, device_error_word());
        return launch_status();
    };
    auto pick = [&](auto t, auto e) {
        using T = decltype(t);
        constexpr int E = decltype(e)::value;
        auto *k = (T *)k_out;
        auto *v = (T *)v_out;
        return head_dim == 128 ? go(kv_cache_read_fp8_rows_kernel<T, 128, E>, k, v) : go(kv_cache_read_fp8_rows_kernel<T, 64, E>, k, v);
    };
    auto size = [&](auto t) {
        return wide ? pick(t, std::integral_constant<int, 16>{}) : pick(t, std::integral_constant<int, 8>{});
    };
    return dtype == PKV_F32 ? size(float{}) : size(__nv_bfloat16{});
}
