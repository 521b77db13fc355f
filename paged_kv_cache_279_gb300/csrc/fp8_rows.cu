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
// the launch for few.
#include "pkv_internal.cuh"
#include "scored.cuh"

namespace pkv {

// Eight consecutive elements of a row, as float.
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// The scale byte of a row whose largest finite magnitude is `amax`: with amax
// = 1.m * 2^(b - 127) and 448 = 1.75 * 2^8, e = b - 135, plus one when 1.m is
// above 1.75.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int s = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)min(kMaxScaleByte, max(kMinScaleByte, s));
}

// One group of head_dim / 8 lanes per (token, KV head), K and V together: each
// lane holds 8 elements of both rows, the group's maximum comes from
// log2(head_dim / 8) shuffles, and every lane stores 8 codes (a 64-byte or
// 128-byte row per group).
template <typename T, int D>
__global__ void __launch_bounds__(256)
kv_cache_write_fp8_rows_kernel(const T *__restrict__ k_new, const T *__restrict__ v_new,
                               unsigned char *__restrict__ k_cache, unsigned char *__restrict__ v_cache,
                               unsigned char *__restrict__ k_scales, unsigned char *__restrict__ v_scales,
                               const int64_t *__restrict__ slot_mapping, int64_t num_rows, int num_kv_heads, int bshift,
                               int64_t num_slots, unsigned int *err) {
    // a dependent attention kernel may start its launch; it waits for this grid before reading the cache
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kLanes = D / 8;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t row = i / kLanes;
    const int c = (int)(i % kLanes);
    const bool live = row < num_rows;
    const int64_t t = live ? row / num_kv_heads : 0;
    const int h = (int)(row - t * num_kv_heads);
    const int64_t slot = live ? slot_mapping[t] : -1;
    if (slot >= num_slots && c == 0 && h == 0) flag_error(err, PKV_DEVERR_SLOT);
    const bool store = slot >= 0 && slot < num_slots;
    float x[2][8];
    if (store) {
        load8(k_new + row * D + 8 * c, x[0]);
        load8(v_new + row * D + 8 * c, x[1]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[0][j] = x[1][j] = 0.f;
    }
    const int64_t blk = slot >> bshift, off = slot - (blk << bshift);
    const int64_t dst = (((blk * num_kv_heads + h) << bshift) + off);  // cache row
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float m = fabsf(x[w][j]);
            amax = m < INFINITY ? fmaxf(amax, m) : amax;  // infinities and NaN do not set the scale
        }
#pragma unroll
        for (int sh = kLanes / 2; sh > 0; sh >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, sh));
        if (!store) continue;
        const uint32_t b = scale_byte(amax);
        const float inv = __uint_as_float((254u - b) << 23);  // 2^-e, a normal number
        uint32_t code[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            code[j] = e4m3x2(x[w][4 * j] * inv, x[w][4 * j + 1] * inv) |
                      (e4m3x2(x[w][4 * j + 2] * inv, x[w][4 * j + 3] * inv) << 16);
        *reinterpret_cast<uint2 *>((w ? v_cache : k_cache) + dst * D + 8 * c) = make_uint2(code[0], code[1]);
        if (c == 0) (w ? v_scales : k_scales)[dst] = (unsigned char)b;
    }
}

__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                               pack_bf16x2(x[6], x[7]));
}

// One lane per 8 codes of a (token, KV head) row, K and V together.
template <typename T, int D>
__global__ void __launch_bounds__(256)
kv_cache_read_fp8_rows_kernel(T *__restrict__ k_out, T *__restrict__ v_out, const unsigned char *__restrict__ k_cache,
                              const unsigned char *__restrict__ v_cache, const unsigned char *__restrict__ k_scales,
                              const unsigned char *__restrict__ v_scales, const int64_t *__restrict__ slot_mapping,
                              int64_t num_rows, int num_kv_heads, int bshift, int64_t num_slots, unsigned int *err) {
    constexpr int kLanes = D / 8;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t row = i / kLanes;
    const int c = (int)(i % kLanes);
    if (row >= num_rows) return;
    const int64_t t = row / num_kv_heads;
    const int h = (int)(row - t * num_kv_heads);
    const int64_t slot = slot_mapping[t];
    if (slot < 0) return;  // padding: the output row is left as it was
    if (slot >= num_slots) {
        if (c == 0 && h == 0) flag_error(err, PKV_DEVERR_SLOT);
        return;
    }
    const int64_t blk = slot >> bshift, off = slot - (blk << bshift);
    const int64_t src = (((blk * num_kv_heads + h) << bshift) + off);
    const uint2 code[2] = {*reinterpret_cast<const uint2 *>(k_cache + src * D + 8 * c),
                           *reinterpret_cast<const uint2 *>(v_cache + src * D + 8 * c)};
    const float f[2] = {row_scale(k_scales[src]), row_scale(v_scales[src])};
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float x[8];
        e4m3x4_to_float(code[w].x, x);
        e4m3x4_to_float(code[w].y, x + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= f[w];
        store8((w ? v_out : k_out) + row * D + 8 * c, x);
    }
}

// Argument checks shared by the two calls; *blocks = 0 when there is nothing to do.
static pkv_status check_rows(const void *a, const void *b, const void *k_cache, const void *v_cache, const void *k_scales,
                             const void *v_scales, const int64_t *slots, int num_tokens, int num_kv_heads, int head_dim,
                             int block_size, int num_blocks, int dtype, int64_t *blocks) {
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
    *blocks = ((int64_t)num_tokens * num_kv_heads * (head_dim / 8) + 255) / 256;
    return *blocks > INT32_MAX ? PKV_ERR_UNSUPPORTED : PKV_OK;
}

}  // namespace pkv

using namespace pkv;

PKV_API pkv_status kv_cache_write_fp8_rows(const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                                           void *k_scales, void *v_scales, const int64_t *slot_mapping, int num_tokens,
                                           int num_kv_heads, int head_dim, int block_size, int num_blocks, int dtype,
                                           void *stream) {
    int64_t blocks;
    const pkv_status rc = check_rows(k_new, v_new, k_cache, v_cache, k_scales, v_scales, slot_mapping, num_tokens,
                                     num_kv_heads, head_dim, block_size, num_blocks, dtype, &blocks);
    if (rc != PKV_OK || blocks == 0) return rc;
    auto go = [&](auto kern, auto *k, auto *v) {
        kern<<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(
            k, v, (unsigned char *)k_cache, (unsigned char *)v_cache, (unsigned char *)k_scales, (unsigned char *)v_scales,
            slot_mapping, (int64_t)num_tokens * num_kv_heads, num_kv_heads, block_size == 16 ? 4 : 5,
            (int64_t)num_blocks * block_size, device_error_word());
        return launch_status();
    };
    if (dtype == PKV_F32)
        return head_dim == 128 ? go(kv_cache_write_fp8_rows_kernel<float, 128>, (const float *)k_new, (const float *)v_new)
                               : go(kv_cache_write_fp8_rows_kernel<float, 64>, (const float *)k_new, (const float *)v_new);
    using bf16 = __nv_bfloat16;
    return head_dim == 128 ? go(kv_cache_write_fp8_rows_kernel<bf16, 128>, (const bf16 *)k_new, (const bf16 *)v_new)
                           : go(kv_cache_write_fp8_rows_kernel<bf16, 64>, (const bf16 *)k_new, (const bf16 *)v_new);
}

PKV_API pkv_status kv_cache_read_fp8_rows(void *k_out, void *v_out, const void *k_cache, const void *v_cache,
                                          const void *k_scales, const void *v_scales, const int64_t *slot_mapping,
                                          int num_tokens, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                          int dtype, void *stream) {
    int64_t blocks;
    const pkv_status rc = check_rows(k_out, v_out, k_cache, v_cache, k_scales, v_scales, slot_mapping, num_tokens,
                                     num_kv_heads, head_dim, block_size, num_blocks, dtype, &blocks);
    if (rc != PKV_OK || blocks == 0) return rc;
    auto go = [&](auto kern, auto *k, auto *v) {
        kern<<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(
            k, v, (const unsigned char *)k_cache, (const unsigned char *)v_cache, (const unsigned char *)k_scales,
            (const unsigned char *)v_scales, slot_mapping, (int64_t)num_tokens * num_kv_heads, num_kv_heads,
            block_size == 16 ? 4 : 5, (int64_t)num_blocks * block_size, device_error_word());
        return launch_status();
    };
    if (dtype == PKV_F32)
        return head_dim == 128 ? go(kv_cache_read_fp8_rows_kernel<float, 128>, (float *)k_out, (float *)v_out)
                               : go(kv_cache_read_fp8_rows_kernel<float, 64>, (float *)k_out, (float *)v_out);
    using bf16 = __nv_bfloat16;
    return head_dim == 128 ? go(kv_cache_read_fp8_rows_kernel<bf16, 128>, (bf16 *)k_out, (bf16 *)v_out)
                           : go(kv_cache_read_fp8_rows_kernel<bf16, 64>, (bf16 *)k_out, (bf16 *)v_out);
}
