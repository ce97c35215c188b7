// Library-internal helpers shared by the attention-side kernels: argument checks,
// 16-byte pieces of bf16 / fp32, cross-lane steps.
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "bitnet_w2a8.h"

namespace bitnet_attn {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));

inline bool at(const void *p, uintptr_t align) { return p && ((uintptr_t)p & (align - 1)) == 0; }

inline bool head_dim_ok(int d) { return d == 64 || d == 128; }
inline bool page_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128; }

inline bool heads_ok(int q_heads, int kv_heads) {
    return q_heads >= 1 && q_heads <= 1024 && kv_heads >= 1 && q_heads % kv_heads == 0;
}

inline bitnet_status_t check_cache(const bitnet_kv_cache_t *c) {
    if (!c || !at(c->k, 16) || !at(c->v, 16) || !at(c->k_scale, 4) || !at(c->v_scale, 4) || !at(c->table, 4))
        return BITNET_ERR_INVALID_ARG;
    if (!head_dim_ok(c->head_dim) || !page_ok(c->page) || c->pages < 1 || c->pages > INT32_MAX || c->kv_heads < 1 ||
        c->batch < 1 || c->batch > 65535 || c->slots < 1 || (int64_t)c->slots * c->page > (1 << 30))
        return BITNET_ERR_UNSUPPORTED_SHAPE;
    return BITNET_OK;
}

inline bitnet_status_t launched() { return hipGetLastError() == hipSuccess ? BITNET_OK : BITNET_ERR_HIP; }

// Two fp32 to two bf16 in one word, round to nearest even.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const v2f f = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, v2bf));
}

// 8 consecutive elements from / to 16-byte aligned memory, as fp32.
__device__ __forceinline__ void load8(const uint16_t *p, float f[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float f[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t *p, const float f[8]) {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}
__device__ __forceinline__ void store8(float *p, const float f[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Maximum and sum with the lane 32 (16) places away, by an in-register swap.
__device__ __forceinline__ float max_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_rows16(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float add_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float add_rows16(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

}  // namespace bitnet_attn
