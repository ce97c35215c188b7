// W2A8 products with an epilogue (bias, activation, gate, residual), over all tokens or by expert.
//
//     z[m][n] = s_a[m] * sum_b S[n][b] * A[m][n][b] + bias[n],   y = act(z) (+ residual),  gated: act(z_gate) * z_up
//
// on the int8 matrix cores, as the products without an epilogue: lane (g, j) of a wave supplies row j of 16 weight rows
// and token j of 16 tokens at 16 columns 16 g + 64 s, and receives rows 4g .. 4g + 3 of token j, so that bias, activation
// and residual are a lane's own and the gate and the up projection of an output meet in one lane.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "attention.h"
#include "bitnet_w2a8.h"
#include "layout.h"

using namespace bitnet_attn;
using namespace bitnet_layout;

namespace {

struct FusedArgs {
    const uint8_t *packed;
    const float *scales, *s_a, *bias;
    const int8_t *q;
    const void *residual;
    void *y;
    const int32_t *starts, *rows;  // by expert, else NULL
    int act, rdt, ydt;
    int tokens, slots, experts, N, K;
};

__device__ __forceinline__ v4i decode16(uint32_t w) {  // 16 weights as 64 t in int8
    v4i r;
    r[0] = (int)((w << 6) & 0xC0C0C0C0u);
    r[1] = (int)((w << 4) & 0xC0C0C0C0u);
    r[2] = (int)((w << 2) & 0xC0C0C0C0u);
    r[3] = (int)(w & 0xC0C0C0C0u);
    return r;
}
__device__ __forceinline__ v4i mfma_i8(v4i a, v4i b, v4i c) { return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0); }

// A NaN stays one.
__device__ __forceinline__ float activate(int act, float z) {
    switch (act) {
        case BITNET_ACT_RELU: return z < 0.0f ? 0.0f : z;
        case BITNET_ACT_RELU2: return z < 0.0f ? 0.0f : z * z;
        case BITNET_ACT_SILU: return z / (1.0f + __expf(-z));
        case BITNET_ACT_GELU: {
            const float u = 1.5957691216057308f * (z + 0.044715f * z * z * z);  // 2 sqrt(2 / pi) ...
            return z / (1.0f + __expf(-u));
        }
        default: return z;
    }
}

// Four neighbouring outputs of slot `at` (its token's factor f): z from block sums of 64 t, the epilogue, one store.
template <bool GATED>
__device__ __forceinline__ void finish(const FusedArgs &p, int expert, int64_t at, int n, float f, const float z0[4], const float z1[4]) {
    const int width = GATED ? p.N >> 1 : p.N;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float z = z0[e] * f;
        if (p.bias) z += p.bias[(int64_t)expert * p.N + n + e];
        z = activate(p.act, z);
        if (GATED) {
            float u = z1[e] * f;
            if (p.bias) u += p.bias[(int64_t)expert * p.N + width + n + e];
            z *= u;
        }
        v[e] = z;
    }
    const int64_t idx = at * width + n;
    if (p.residual) {
        if (p.rdt == BITNET_DT_BF16) {
            const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.residual) + idx);
            v[0] += __uint_as_float(w.x << 16);
            v[1] += __uint_as_float(w.x & 0xFFFF0000u);
            v[2] += __uint_as_float(w.y << 16);
            v[3] += __uint_as_float(w.y & 0xFFFF0000u);
        } else {
            const float4 w = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.residual) + idx);
            v[0] += w.x;
            v[1] += w.y;
            v[2] += w.z;
            v[3] += w.w;
        }
    }
    if (p.ydt == BITNET_DT_BF16)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.y) + idx) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
    else
        *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + idx) = make_float4(v[0], v[1], v[2], v[3]);
}

// The expert and first slot of token tile `tile` of `rows` slots each; tiles go through the experts in turn.  Read by every wave for
// itself.  False: there is no such tile.
struct Tile {
    int expert, first, end;  // slots first .. end - 1
};
__device__ __forceinline__ bool find_tile(const FusedArgs &p, int tile, int rows, Tile *out) {
    if (!p.starts) {
        *out = {0, tile * rows, min(p.slots, (tile + 1) * rows)};
        return out->first < p.slots;
    }
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 64) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < p.experts) {
            lo = min(max(p.starts[e], 0), p.slots);
            hi = min(max(p.starts[e + 1], lo), p.slots);
        }
        const int n = (hi - lo + rows - 1) / rows;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int below = __shfl_up(sum, o);
            if (lane >= o) sum += below;
        }
        const int first = before + sum - n;
        const uint64_t who = __ballot(tile >= first && tile < before + sum);
        if (who) {
            const int at = __ffsll((unsigned long long)who) - 1;
            out->expert = e0 + at;
            out->first = __builtin_amdgcn_readlane(lo + (tile - first) * rows, at);
            out->end = min(__builtin_amdgcn_readlane(hi, at), out->first + rows);
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

// One wave: 16 slots x 16 rows (two tiles of 16 rows when gated), all of K.
template <bool GATED>
__global__ __launch_bounds__(256) void fused_kernel(FusedArgs p) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, j = lane & 15;
    const int width = GATED ? p.N >> 1 : p.N, blocks = p.K >> 7, tiles = p.N >> 4;
    const int tile = blockIdx.x * 4 + wave;
    Tile t;
    if (!find_tile(p, blockIdx.y, 16, &t)) return;
    if (tile >= width >> 4) return;
    const int slot = t.first + j;
    int token = -1;
    if (slot < t.end) {
        token = p.rows ? p.rows[slot] : slot;
        if (token >= p.tokens) token = -1;
    }
    const int8_t *q = p.q + (int64_t)max(token, 0) * p.K + 16 * g;
    float z[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
    for (int b = 0; b < blocks; ++b) {
        v4i a[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) a[s] = token >= 0 ? *reinterpret_cast<const v4i *>(q + 128 * b + 64 * s) : v4i{0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            const int64_t brick = ((int64_t)t.expert * tiles + tile + h * (width >> 4)) * blocks + b;
            const uint2 w = *reinterpret_cast<const uint2 *>(p.packed + brick * kBrickBytes + lane * 8);
            const float4 sc = *reinterpret_cast<const float4 *>(p.scales + brick * kTileN + 4 * g);
            v4i c = mfma_i8(decode16(w.x), a[0], v4i{0, 0, 0, 0});
            c = mfma_i8(decode16(w.y), a[1], c);
            z[h][0] = fmaf(sc.x, (float)c[0], z[h][0]);
            z[h][1] = fmaf(sc.y, (float)c[1], z[h][1]);
            z[h][2] = fmaf(sc.z, (float)c[2], z[h][2]);
            z[h][3] = fmaf(sc.w, (float)c[3], z[h][3]);
        }
    }
    if (token < 0) return;
    finish<GATED>(p, t.expert, slot, tile * 16 + 4 * g, p.s_a[token] * 0.015625f, z[0], z[1]);
}

bitnet_status_t run(const FusedArgs &p, int gated, hipStream_t stream) {
    const int width = gated ? p.N >> 1 : p.N;
    const int some = p.experts < p.slots ? p.experts : p.slots;  // experts that can have rows
    const int64_t token_tiles = p.starts ? ((int64_t)p.slots + 15ll * some) / 16 : ((int64_t)p.slots + 15) / 16;
    const int64_t row_groups = (width / 16 + 3) / 4;
    if (token_tiles > 65535) return BITNET_ERR_UNSUPPORTED_SHAPE;
    const dim3 grid((unsigned)row_groups, (unsigned)token_tiles);
    if (gated) hipLaunchKernelGGL(fused_kernel<true>, grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(fused_kernel<false>, grid, dim3(256), 0, stream, p);
    return launched();
}

bool float_type(int dt) { return dt == BITNET_DT_BF16 || dt == BITNET_DT_F32; }

bitnet_status_t check(const FusedArgs &p, int gated) {
    if (!at(p.packed, 16) || !at(p.scales, 16) || !at(p.q, 16) || !at(p.s_a, 4) || (p.bias && !at(p.bias, 16)) ||
        (p.residual && (!at(p.residual, 16) || !float_type(p.rdt))) || !at(p.y, 16) || !float_type(p.ydt) ||
        p.act < BITNET_ACT_NONE || p.act > BITNET_ACT_GELU || (p.residual == p.y && p.rdt != p.ydt))
        return BITNET_ERR_INVALID_ARG;
    if (bitnet_check_shape(p.N, p.K) != BITNET_OK || (gated && p.N % 32)) return BITNET_ERR_UNSUPPORTED_SHAPE;
    return BITNET_OK;
}

}  // namespace

extern "C" {

bitnet_status_t bitnet_w2a8_linear(const uint8_t *packed, const float *scales, const int8_t *q, const float *s_a,
                                   const float *bias, int act, int gated, const void *residual, int rdt, void *y,
                                   int ydt, int M, int N, int K, hipStream_t stream) {
    const FusedArgs p{packed, scales, s_a, bias, q, residual, y, nullptr, nullptr, act, rdt, ydt, M, M, 1, N, K};
    const bitnet_status_t st = check(p, gated);
    if (st != BITNET_OK) return st;
    if (M < 1) return BITNET_ERR_UNSUPPORTED_SHAPE;
    return run(p, gated, stream);
}

bitnet_status_t bitnet_w2a8_grouped(const uint8_t *packed, const float *scales, const int8_t *q, const float *s_a,
                                    int tokens, const int32_t *starts, const int32_t *rows, int experts, int slots,
                                    const float *bias, int act, int gated, void *y, int ydt, int N, int K,
                                    hipStream_t stream) {
    const FusedArgs p{packed, scales, s_a, bias, q, nullptr, y, starts, rows, act, 0, ydt, tokens, slots, experts, N, K};
    const bitnet_status_t st = check(p, gated);
    if (st != BITNET_OK) return st;
    if (!at(starts, 4) || (rows && !at(rows, 4))) return BITNET_ERR_INVALID_ARG;
    if (experts < 1 || experts > 1024 || slots < 1 || slots > (1 << 30) || tokens < 1 || tokens > (1 << 30) ||
        (!rows && tokens < slots))
        return BITNET_ERR_UNSUPPORTED_SHAPE;
    return run(p, gated, stream);
}

}  // extern "C"
