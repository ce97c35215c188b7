// Residual addition, root-mean-square norm and int8 quantisation of the stream between two products, one pass.
//
//     v = x + d;  x_out = v in x's type;  r = 1 / sqrt(mean x_out^2 + eps);  h = (x_out r) w;  q = rint(h 127 / max|h|)
//
// A row stays in registers between its reads and its writes, so x, the rows of add and the weight are read once and x_out, q
// written once.  The mean of the squares is summed in 64 bits (squares of fp32 values are exact there).  How a row is cut over lanes
// moves the last bits of that sum, some 2^-50 of it, which reaches the factor r in fp32 only where it lies that near to a rounding
// border: about one row in 2^26.
//
// Measured against a large copy's 5.07 TB/s.  16383 x 2560 bf16 with an addition: 294 MB, 53 to 55 us, 5.3 to 5.5 TB/s (it reads more than
// it writes), bound by bytes.  512 rows of 6 parts each: 27.6 MB, 7.7 us in a graph (5.4 at a copy's rate), bound by the chain of a
// row: slots, then parts four at a time, two reductions, codes; waves wait in 70% of their time.  One row 2.9 us: a launch and that chain.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "attention.h"
#include "bitnet_w2a8.h"

using namespace bitnet_attn;

#pragma clang fp contract(off)

namespace {

constexpr int kMaxWaves = 16;
constexpr int kMaxK = 65536;
constexpr int kMaxParts = 64;
// Rows from which on a wave takes a row (2560 wide, bf16: 1024 rows 6.9 us either way, 4096 rows 16.3 against 19.4, 16383 rows 55.7
// against 65.7; 512 rows 6.0 against 5.0).  With parts a workgroup a row stays ahead (512 rows of 6 parts 7.7 against 17.9 us).
constexpr int kWaveRows = 1024;

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

// Sum and maximum over a wave, the same in every lane: within 16 lanes by DPP, then by swaps of rows and of halves (a shuffle through
// LDS at each step costs a row of one token 0.5 us).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32 | dpp<CTRL>((uint32_t)u));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp<kXor1>(v);
    v += dpp<kXor2>(v);
    v += dpp<kHalfMirror>(v);
    v += dpp<kMirror>(v);
    const auto both = [](auto lo, auto hi) {
        return __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | (uint32_t)lo[0]) + __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | (uint32_t)lo[1]);
    };
    uint64_t u = __builtin_bit_cast(uint64_t, v);
    v = both(__builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false),
             __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false));
    u = __builtin_bit_cast(uint64_t, v);
    return both(__builtin_amdgcn_permlane32_swap((uint32_t)u, (uint32_t)u, false, false),
                __builtin_amdgcn_permlane32_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, dpp<kXor1>(v));
    v = max(v, dpp<kXor2>(v));
    v = max(v, dpp<kHalfMirror>(v));
    v = max(v, dpp<kMirror>(v));
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max((uint32_t)a[0], (uint32_t)a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max((uint32_t)b[0], (uint32_t)b[1]);
}

// The codes of a row whose largest magnitude (as bits) is known.
struct Scale {
    bool bad;  // an infinity or a NaN somewhere in the row
    float top, inv;
    __device__ __forceinline__ explicit Scale(uint32_t most)
        : bad(most >= 0x7F800000u), top(fmaxf(__uint_as_float(most), 1e-5f)), inv(__fdiv_rn(127.0f, top)) {}
    __device__ __forceinline__ uint2 codes(const float f[8]) const {
        uint32_t q[2] = {0, 0};
        if (!bad)
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i >> 2] |= ((uint32_t)(int)__builtin_rintf(f[i] * inv) & 0xFFu) << (8 * (i & 3));
        return make_uint2(q[0], q[1]);
    }
    __device__ __forceinline__ float factor() const { return bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(top, 127.0f); }
};

// A lane holds C chunks of 8 values.  WAVE: a wave a row, four rows a workgroup, nothing to wait for; else a workgroup a row, so that
// few rows are cut over many lanes.
template <typename T, typename A, int C, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_kernel(NormArgs p, int rows, int hdt) {
    __shared__ double s_sum[WAVE ? 1 : kMaxWaves];
    __shared__ uint32_t s_max[WAVE ? 1 : kMaxWaves];
    const int tid = WAVE ? threadIdx.x & 63 : threadIdx.x, n = p.K >> 3, threads = WAVE ? 64 : blockDim.x, waves = threads >> 6;
    const int64_t m = WAVE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    if (WAVE && m >= rows) return;
    const T *x = static_cast<const T *>(p.x) + m * p.K;
    // chunks behind the row's end repeat its last one; they count for nothing (where x_out is x, another wave may have stored that one)
    int at[C];
#pragma unroll
    for (int c = 0; c < C; ++c) at[c] = 8 * min(tid + c * threads, n - 1);
    auto there = [&](int c) { return tid + c * threads < n; };
    float f[C][8], w[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) load8(x + at[c], f[c]);
    if (p.add) {
        const A *add = static_cast<const A *>(p.add);
        if (p.slots) {
            float d[C][8];
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) d[c][i] = 0.0f;
            // lane j has part j; kAtOnce parts' rows are asked for together
            constexpr int kAtOnce = C == 1 ? 4 : C == 2 ? 2 : 1;
            const int lane = threadIdx.x & 63, part = min(lane, p.parts - 1);
            const int slot = p.slots[m * p.parts + part];
            const float gate = p.gates[m * p.parts + part];
            for (int j0 = 0; j0 < p.parts; j0 += kAtOnce) {
                float a[kAtOnce][C][8];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const int row = __builtin_amdgcn_readlane(slot, min(j0 + k, p.parts - 1));
#pragma unroll
                    for (int c = 0; c < C; ++c) load8(add + (row < 0 || row >= p.add_rows ? 0 : (int64_t)row * p.K) + at[c], a[k][c]);
                }
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const int row = __builtin_amdgcn_readlane(slot, min(j0 + k, p.parts - 1));
                    if (j0 + k >= p.parts || row < 0 || row >= p.add_rows) continue;
                    const float g = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(gate), j0 + k));
#pragma unroll
                    for (int c = 0; c < C; ++c)
#pragma unroll
                        for (int i = 0; i < 8; ++i) d[c][i] += g * a[k][c][i];
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) f[c][i] += d[c][i];
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float a[8];
                load8(add + m * p.K + at[c], a);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[c][i] += a[i];
            }
        }
        T *out = static_cast<T *>(p.x_out) + m * p.K;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (there(c)) store8(out + at[c], f[c]);
            round8(x, f[c]);
        }
    }
    if (p.weight)
#pragma unroll
        for (int c = 0; c < C; ++c) load8(p.weight + at[c], w[c]);

    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        double part = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) part = fma((double)f[c][i], (double)f[c][i], part);
        sum += there(c) ? part : 0.0;
    }
    sum = wave_sum(sum);
    if (!WAVE) {
        if ((tid & 63) == 0) s_sum[tid >> 6] = sum;
        __syncthreads();
        sum = 0.0;
        for (int i = 0; i < waves; ++i) sum += s_sum[i];
    }
    const float r = (float)(1.0 / sqrt(sum / (double)p.K + (double)p.eps));

    uint32_t most = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[c][i] *= r;
            if (p.weight) f[c][i] *= w[c][i];
            most = there(c) ? max(most, magnitude(f[c][i])) : most;
        }
        if (p.h_out && there(c)) {
            if (hdt == BITNET_DT_BF16) store8(static_cast<uint16_t *>(p.h_out) + m * p.K + at[c], f[c]);
            else store8(static_cast<float *>(p.h_out) + m * p.K + at[c], f[c]);
        }
    }
    if (!p.q) return;
    most = wave_max(most);
    if (!WAVE) {
        if ((tid & 63) == 0) s_max[tid >> 6] = most;
        __syncthreads();
        for (int i = 0; i < waves; ++i) most = max(most, s_max[i]);
    }
    const Scale s(most);
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (there(c)) *reinterpret_cast<uint2 *>(p.q + m * p.K + at[c]) = s.codes(f[c]);
    if (tid == 0) p.s_a[m] = s.factor();
}

// Rows that do not fit the registers: three passes over them, the second and third over x_out (each lane reads what it wrote itself).
template <typename T, typename A>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormArgs p, int hdt) {
    __shared__ double s_sum[kMaxWaves];
    __shared__ uint32_t s_max[kMaxWaves];
    const int tid = threadIdx.x, n = p.K >> 3;
    const int64_t m = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + m * p.K;
    const A *add = static_cast<const A *>(p.add);
    T *out = static_cast<T *>(p.x_out) + m * p.K;
    double sum = 0.0;
    for (int v = tid; v < n; v += 1024) {
        float f[8], a[8];
        load8(x + 8 * v, f);
        if (p.slots) {
            float d[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            for (int j = 0; j < p.parts; ++j) {
                const int slot = p.slots[m * p.parts + j];
                if (slot < 0 || slot >= p.add_rows) continue;
                const float gate = p.gates[m * p.parts + j];
                load8(add + (int64_t)slot * p.K + 8 * v, a);
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] += gate * a[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] += d[i];
        } else if (p.add) {
            load8(add + m * p.K + 8 * v, a);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] += a[i];
        }
        if (p.add) {
            store8(out + 8 * v, f);
            round8(x, f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fma((double)f[i], (double)f[i], sum);
    }
    sum = wave_sum(sum);
    if ((tid & 63) == 0) s_sum[tid >> 6] = sum;
    __syncthreads();
    sum = 0.0;
    for (int i = 0; i < kMaxWaves; ++i) sum += s_sum[i];
    const float r = (float)(1.0 / sqrt(sum / (double)p.K + (double)p.eps));
    const T *from = p.add ? out : x;
    auto normed = [&](int v, float f[8]) {
        load8(from + 8 * v, f);
        float w[8];
        if (p.weight) load8(p.weight + 8 * v, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] *= r;
            if (p.weight) f[i] *= w[i];
        }
    };
    // in the last pass over the row, as h_out may be x
    auto store_h = [&](int v, const float f[8]) {
        if (!p.h_out) return;
        if (hdt == BITNET_DT_BF16) store8(static_cast<uint16_t *>(p.h_out) + m * p.K + 8 * v, f);
        else store8(static_cast<float *>(p.h_out) + m * p.K + 8 * v, f);
    };
    uint32_t most = 0;
    for (int v = tid; v < n; v += 1024) {
        float f[8];
        normed(v, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) most = max(most, magnitude(f[i]));
        if (!p.q) store_h(v, f);
    }
    if (!p.q) return;
    most = wave_max(most);
    if ((tid & 63) == 0) s_max[tid >> 6] = most;
    __syncthreads();
    for (int i = 0; i < kMaxWaves; ++i) most = max(most, s_max[i]);
    const Scale s(most);
    for (int v = tid; v < n; v += 1024) {
        float f[8];
        normed(v, f);
        store_h(v, f);
        *reinterpret_cast<uint2 *>(p.q + m * p.K + 8 * v) = s.codes(f);
    }
    if (tid == 0) p.s_a[m] = s.factor();
}

template <typename T, typename A>
void launch_norm(const NormArgs &p, int M, int hdt, hipStream_t stream) {
    const int n = p.K >> 3;
    if (M >= kWaveRows && n <= 512 && !p.slots) {
        const dim3 grid((M + 3) / 4), block(256);
#define BITNET_NORM(C) hipLaunchKernelGGL((norm_kernel<T, A, C, true>), grid, block, 0, stream, p, M, hdt)
        switch ((n + 63) / 64) {
            case 1: BITNET_NORM(1); return;
            case 2: BITNET_NORM(2); return;
            case 3: BITNET_NORM(3); return;
            case 4: BITNET_NORM(4); return;
            case 5: BITNET_NORM(5); return;
            case 6: BITNET_NORM(6); return;
            default: BITNET_NORM(8); return;
        }
#undef BITNET_NORM
    }
    const int c = n <= 512 ? 1 : n <= 1024 ? 2 : n <= 4096 ? 4 : 0;
    if (c == 0) {
        hipLaunchKernelGGL((norm_long_kernel<T, A>), dim3(M), dim3(1024), 0, stream, p, hdt);
        return;
    }
    const dim3 grid(M), block((n + 64 * c - 1) / (64 * c) * 64);
    if (c == 1) hipLaunchKernelGGL((norm_kernel<T, A, 1, false>), grid, block, 0, stream, p, M, hdt);
    else if (c == 2) hipLaunchKernelGGL((norm_kernel<T, A, 2, false>), grid, block, 0, stream, p, M, hdt);
    else hipLaunchKernelGGL((norm_kernel<T, A, 4, false>), grid, block, 0, stream, p, M, hdt);
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
    // a launch's work items in 32 bits: 64 a row, or up to 1024 (launch_norm)
    if (M < 1 || M > 65535 * 1024 || (M >= 1 << 22 && K > (slots ? 512 : 4096)) || K < 16 || K % 16 || K > kMaxK ||
        (slots && (parts < 1 || parts > kMaxParts || add_rows < 1)))
        return BITNET_ERR_UNSUPPORTED_SHAPE;
    if (h_out && (h_out == x_out || (h_out == x && hdt != xdt))) return BITNET_ERR_INVALID_ARG;
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
