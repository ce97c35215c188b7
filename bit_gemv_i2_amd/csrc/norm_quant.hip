// Residual addition, root-mean-square norm and int8 quantisation of the stream between two products, one pass.
//
//     v = x + d;  x_out = v in x's type;  r = 1 / sqrt(mean x_out^2 + eps);  h = (x_out r) w;  q = rint(h 127 / max|h|)
//
// A row stays in registers between its reads and its writes, so x, the rows of add and the weight are read once and x_out, q
// written once.  The mean of the squares is summed in 64 bits (squares of fp32 values are exact there): its rounding to fp32, and
// with it every code, does then not depend on how a row is cut over lanes.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "attention.h"
#include "bitnet_w2a8.h"

using namespace bitnet_attn;

#pragma clang fp contract(off)

namespace {

constexpr int kMaxWaves = 16;
constexpr int kMaxK = 65536;  // 16 waves of 8 chunks of 8 values a lane
constexpr int kMaxParts = 64;

struct NormArgs {
    const void *x, *add;
    const int32_t *slots;
    const float *gates, *weight;
    void *x_out, *h_out;
    int8_t *q;
    float *s_a;
    int64_t add_rows;
    int parts, K;
    float eps;
};

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Values as they will be read back from memory of type T.
__device__ __forceinline__ void round8(const uint16_t *, float f[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint32_t w = bf16_pair(f[i], f[i + 1]);
        f[i] = __uint_as_float(w << 16);
        f[i + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void round8(const float *, float[8]) {}

// One workgroup per row; a lane holds C chunks of 8 values.
template <typename T, typename A, int C>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs p, int hdt) {
    __shared__ double s_sum[kMaxWaves];
    __shared__ uint32_t s_max[kMaxWaves];
    const int64_t m = blockIdx.x;
    const int tid = threadIdx.x, n = p.K >> 3, threads = blockDim.x, waves = threads >> 6;
    const T *x = static_cast<const T *>(p.x) + m * p.K;
    float f[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int v = tid + c * threads;
        if (v < n) load8(x + 8 * v, f[c]);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) f[c][i] = 0.0f;
    }
    if (p.add) {
        const A *add = static_cast<const A *>(p.add);
        if (p.slots) {
            float d[C][8];
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) d[c][i] = 0.0f;
            for (int j = 0; j < p.parts; ++j) {
                const int slot = p.slots[m * p.parts + j];
                if (slot < 0 || slot >= p.add_rows) continue;
                const float gate = p.gates[m * p.parts + j];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int v = tid + c * threads;
                    float a[8];
                    if (v < n) {
                        load8(add + (int64_t)slot * p.K + 8 * v, a);
#pragma unroll
                        for (int i = 0; i < 8; ++i) d[c][i] += gate * a[i];
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) f[c][i] += d[c][i];
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int v = tid + c * threads;
                float a[8];
                if (v < n) {
                    load8(add + m * p.K + 8 * v, a);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[c][i] += a[i];
                }
            }
        }
        T *out = static_cast<T *>(p.x_out) + m * p.K;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int v = tid + c * threads;
            if (v < n) store8(out + 8 * v, f[c]);
            round8(x, f[c]);
        }
    }

    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fma((double)f[c][i], (double)f[c][i], sum);
#pragma unroll
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    if ((tid & 63) == 0) s_sum[tid >> 6] = sum;
    __syncthreads();
    sum = 0.0;
    for (int i = 0; i < waves; ++i) sum += s_sum[i];
    const float r = (float)(1.0 / sqrt(sum / (double)p.K + (double)p.eps));

    uint32_t most = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int v = tid + c * threads;
        if (v >= n) continue;
        float w[8];
        if (p.weight) load8(p.weight + 8 * v, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[c][i] *= r;
            if (p.weight) f[c][i] *= w[i];
            most = max(most, magnitude(f[c][i]));
        }
        if (p.h_out) {
            if (hdt == BITNET_DT_BF16) store8(static_cast<uint16_t *>(p.h_out) + m * p.K + 8 * v, f[c]);
            else store8(static_cast<float *>(p.h_out) + m * p.K + 8 * v, f[c]);
        }
    }
    if (!p.q) return;
#pragma unroll
    for (int o = 32; o; o >>= 1) most = max(most, (uint32_t)__shfl_xor((int)most, o));
    if ((tid & 63) == 0) s_max[tid >> 6] = most;
    __syncthreads();
    for (int i = 0; i < waves; ++i) most = max(most, s_max[i]);
    const bool bad = most >= 0x7F800000u;  // an infinity or a NaN somewhere in the row
    const float top = fmaxf(__uint_as_float(most), 1e-5f);
    const float inv = __fdiv_rn(127.0f, top);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int v = tid + c * threads;
        if (v >= n) continue;
        uint32_t w[2] = {0, 0};
        if (!bad)
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i >> 2] |= ((uint32_t)(int)__builtin_rintf(f[c][i] * inv) & 0xFFu) << (8 * (i & 3));
        *reinterpret_cast<uint2 *>(p.q + m * p.K + 8 * v) = make_uint2(w[0], w[1]);
    }
    if (tid == 0) p.s_a[m] = bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(top, 127.0f);
}

template <typename T, typename A>
void launch_norm(const NormArgs &p, int M, int hdt, hipStream_t stream) {
    const int n = p.K >> 3;
    const int c = n <= 512 ? 1 : n <= 1024 ? 2 : n <= 2048 ? 4 : 8;
    const dim3 grid(M), block((n + 64 * c - 1) / (64 * c) * 64);
    if (c == 1) hipLaunchKernelGGL((norm_kernel<T, A, 1>), grid, block, 0, stream, p, hdt);
    else if (c == 2) hipLaunchKernelGGL((norm_kernel<T, A, 2>), grid, block, 0, stream, p, hdt);
    else if (c == 4) hipLaunchKernelGGL((norm_kernel<T, A, 4>), grid, block, 0, stream, p, hdt);
    else hipLaunchKernelGGL((norm_kernel<T, A, 8>), grid, block, 0, stream, p, hdt);
}

inline bool float_type(int dt) { return dt == BITNET_DT_BF16 || dt == BITNET_DT_F32; }

}  // namespace

extern "C" bitnet_status_t bitnet_add_norm(const void *x, int xdt, const void *add, int adt, int64_t add_rows,
                                           const int32_t *slots, const float *gates, int parts, const float *weight,
                                           float eps, int M, int K, void *x_out, int8_t *q, float *s_a, void *h_out,
                                           int hdt, hipStream_t stream) {
    if (!at(x, 16) || !float_type(xdt) || (add && (!at(add, 16) || !float_type(adt) || !at(x_out, 16))) ||
        (!add && (slots || x_out)) || (weight && !at(weight, 16)) || (slots && (!at(slots, 4) || !at(gates, 4))) ||
        (!slots && (gates || parts)) || (!q && !h_out) || (q && (!at(q, 16) || !at(s_a, 4))) || (!q && s_a) ||
        (h_out && (!at(h_out, 16) || !float_type(hdt))) || !(eps > 0.0f) || !std::isfinite(eps))
        return BITNET_ERR_INVALID_ARG;
    if (M < 1 || M > 65535 * 1024 || K < 16 || K % 16 || K > kMaxK ||
        (slots && (parts < 1 || parts > kMaxParts || add_rows < 1)))
        return BITNET_ERR_UNSUPPORTED_SHAPE;
    NormArgs p;
    p.x = x; p.add = add; p.slots = slots; p.gates = gates; p.weight = weight; p.x_out = x_out; p.h_out = h_out;
    p.q = q; p.s_a = s_a; p.add_rows = add_rows; p.parts = parts; p.K = K; p.eps = eps;
    const bool x16 = xdt == BITNET_DT_BF16, a16 = add && adt == BITNET_DT_BF16;
    if (x16 && a16) launch_norm<uint16_t, uint16_t>(p, M, hdt, stream);
    else if (x16) launch_norm<uint16_t, float>(p, M, hdt, stream);
    else if (a16) launch_norm<float, uint16_t>(p, M, hdt, stream);
    else launch_norm<float, float>(p, M, hdt, stream);
    return launched();
}
