// Attention over whole prompts, packed one behind the other, bf16 on the matrix cores.
//
// out_t = sum_u p_u v_u / sum_u p_u, p_u = exp(scale * q_t.k_u - m): one pass over the keys with the
// running maximum m and sum of the row, so that no score leaves the registers.
//
// Both products are taken transposed: S^T = K Q^T and O^T = V^T P^T, with
// v_mfma_f32_32x32x16_bf16.  A lane then holds one query row (lane % 32) and 16 of its scores for
// 32 keys, the rows 8j + 4 (lane / 32) + r of the result: the softmax needs one exchange between the two
// half-waves and no other, and a lane's scores, rounded to bf16, are its own operand of the second
// product, if that product takes its 16 keys in the order 8x + 4 (lane / 32) + r.  V^T is read from LDS by
// the transposing 16-bit read, which gives a lane 4 keys of one channel: that same order.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "attention.h"
#include "bitnet_w2a8.h"

using namespace bitnet_attn;

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kWaves = 4;
constexpr int kRowsWave = 32;                 // query rows of a wave
constexpr int kRows = kWaves * kRowsWave;     // and of a workgroup
constexpr int kKeys = 64;                     // keys of a tile
constexpr int64_t kMaxTokens = 1 << 24;

struct PromptArgs {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t *starts;
    int64_t tokens;
    int max_len, q_heads, kv_heads, causal;
    float scale2;  // scale * log2(e)
    uint16_t *out;
};

// Byte offset of the 16-byte piece `ch` of row `row` in a tile.  Rows are a multiple of the LDS
// banks apart, so the pieces of a row are permuted by its number: for K a read takes one piece
// of each of 32 rows; for V, 32 bytes (a pair of pieces) of each of 4 rows.
template <int D>
__device__ __forceinline__ int k_at(int row, int ch) {
    return row * (2 * D) + ((ch ^ (row & (D / 8 - 1))) << 4);
}
template <int D>
__device__ __forceinline__ int v_at(int row, int ch) {
    return row * (2 * D) + ((ch ^ ((row & (D / 16 - 1)) << 1)) << 4);
}

template <int D>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_prompt_kernel(PromptArgs p) {
    constexpr int kTileBytes = kKeys * D * 2;
    constexpr int kPieces = kKeys * D / 8 / (64 * kWaves);  // 16-byte pieces of K (and of V) that a thread stages
    constexpr int kKSteps = D / 16;
    constexpr int kDTiles = D / 32;
    __shared__ __align__(16) uint8_t s_k[2][kTileBytes];
    __shared__ __align__(16) uint8_t s_v[2][kTileBytes];

    const int b = blockIdx.z, head = blockIdx.y;
    const int64_t n0 = p.starts[b], n1 = p.starts[b + 1];
    if (n0 < 0 || n1 > p.tokens || n1 <= n0) return;
    const int n = (int)(n1 - n0 < p.max_len ? n1 - n0 : p.max_len);
    const int q0 = (int)(gridDim.x - 1 - blockIdx.x) * kRows;  // the longest rows first
    if (q0 >= n) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = lane & 31, half = lane >> 5;
    const int hk = head / (p.q_heads / p.kv_heads);
    const uint16_t *kg = p.k + n0 * p.k_stride + (int64_t)hk * D;
    const uint16_t *vg = p.v + n0 * p.v_stride + (int64_t)hk * D;

    const int w0 = q0 + wave * kRowsWave;  // this wave's first row
    const int row = w0 + col;              // this lane's query row
    v8bf qf[kKSteps];
    {
        const int r = row < n ? row : n - 1;
        const uint16_t *qg = p.q + (n0 + r) * p.q_stride + (int64_t)head * D + 8 * half;
#pragma unroll
        for (int s = 0; s < kKSteps; ++s) qf[s] = *reinterpret_cast<const v8bf *>(qg + 16 * s);
    }
    const int seen = p.causal && q0 + kRows < n ? q0 + kRows : n;  // keys that any row of the workgroup sees
    const int tiles = (seen + kKeys - 1) / kKeys;

    v16f o[kDTiles];
#pragma unroll
    for (int i = 0; i < kDTiles; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
    float m = -INFINITY, l = 0.0f;

    v4u ks[kPieces], vs[kPieces];
    const auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int id = tid + i * 64 * kWaves, r = t * kKeys + id / (D / 8), ch = id % (D / 8);
            if (r < n) {
                ks[i] = *reinterpret_cast<const v4u *>(kg + r * p.k_stride + ch * 8);
                vs[i] = *reinterpret_cast<const v4u *>(vg + r * p.v_stride + ch * 8);
            } else {  // keys past the end: their weights are 0, so their values must be finite
                ks[i] = v4u{0, 0, 0, 0};
                vs[i] = v4u{0, 0, 0, 0};
            }
        }
    };
    const auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int id = tid + i * 64 * kWaves, r = id / (D / 8), ch = id % (D / 8);
            *reinterpret_cast<v4u *>(s_k[buf] + k_at<D>(r, ch)) = ks[i];
            *reinterpret_cast<v4u *>(s_v[buf] + v_at<D>(r, ch)) = vs[i];
        }
    };

    fetch(0);
    stage(0);
    __syncthreads();
    const int wave_seen = w0 >= n ? 0 : p.causal && w0 + kRowsWave < n ? w0 + kRowsWave : n;
    for (int t = 0; t < tiles; ++t) {
        const int buf = t & 1;
        if (t + 1 < tiles) fetch(t + 1);
        const int u0 = t * kKeys;
        if (u0 < wave_seen) {
            v16f s[2];
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
#pragma unroll
                for (int r = 0; r < 16; ++r) s[tt][r] = 0.0f;
#pragma unroll
                for (int st = 0; st < kKSteps; ++st) {
                    const v8bf a = *reinterpret_cast<const v8bf *>(s_k[buf] + k_at<D>(32 * tt + col, 2 * st + half));
                    s[tt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, qf[st], s[tt], 0, 0, 0);
                }
            }
            // a key is seen if it is in the sequence and, when causal, not behind the row
            const int last = p.causal && row < n - 1 ? row : n - 1;
            if (u0 + kKeys - 1 > (p.causal && w0 < n - 1 ? w0 : n - 1)) {
#pragma unroll
                for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (u0 + 32 * tt + 8 * (r / 4) + 4 * half + r % 4 > last) s[tt][r] = -INFINITY;
            }
            float mt = s[0][0];
#pragma unroll
            for (int r = 1; r < 32; ++r) mt = fmaxf(mt, s[r / 16][r % 16]);
            mt = max_halves(mt) * p.scale2;
            const float mn = fmaxf(m, mt);  // finite: a row sees key 0 in its first tile
            const float alpha = __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            uint32_t pw[16];
            float sum = 0.0f;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float a = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r / 8][2 * r % 16], p.scale2, -mn));
                const float c = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r / 8][2 * r % 16 + 1], p.scale2, -mn));
                sum += a + c;
                pw[r] = bf16_pair(a, c);
            }
            l = __builtin_fmaf(l, alpha, sum);
#pragma unroll
            for (int i = 0; i < kDTiles; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[i][r] *= alpha;
            const int j = lane & 15;
#pragma unroll
            for (int st = 0; st < 4; ++st) {
                const v4u w = {pw[4 * st], pw[4 * st + 1], pw[4 * st + 2], pw[4 * st + 3]};
                const v8bf pf = __builtin_bit_cast(v8bf, w);
#pragma unroll
                for (int i = 0; i < kDTiles; ++i) {
                    v4s f[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int r = 16 * st + 8 * x + 4 * half + (j >> 2);
                        const int ch = 4 * i + 2 * ((lane >> 4) & 1) + ((j & 3) >> 1);
                        f[x] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(s_v[buf] + v_at<D>(r, ch) + 8 * (j & 1)));
                    }
                    const v8bf vf = __builtin_bit_cast(v8bf, __builtin_shufflevector(f[0], f[1], 0, 1, 2, 3, 4, 5, 6, 7));
                    o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf, o[i], 0, 0, 0);
                }
            }
        }
        if (t + 1 < tiles) stage(buf ^ 1);
        __syncthreads();
    }

    l = add_halves(l);
    if (row >= n) return;
    const float inv = 1.0f / l;
    uint16_t *og = p.out + ((n0 + row) * p.q_heads + head) * D + 4 * half;
#pragma unroll
    for (int i = 0; i < kDTiles; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint2 *>(og + 32 * i + 8 * j) =
                make_uint2(bf16_pair(o[i][4 * j] * inv, o[i][4 * j + 1] * inv),
                           bf16_pair(o[i][4 * j + 2] * inv, o[i][4 * j + 3] * inv));
}

}  // namespace

extern "C" bitnet_status_t bitnet_attn_prompt(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                              const void *v, int64_t v_stride, const int32_t *starts, int batch,
                                              int64_t tokens, int max_len, int q_heads, int kv_heads, int head_dim,
                                              int causal, float scale, void *out, hipStream_t stream) {
    if (!at(q, 16) || !at(k, 16) || !at(v, 16) || !at(out, 16) || !at(starts, 4) || !(scale > 0.0f) ||
        !std::isfinite(scale))
        return BITNET_ERR_INVALID_ARG;
    if (!heads_ok(q_heads, kv_heads) || !head_dim_ok(head_dim) || batch < 1 || batch > 65535 || tokens < 1 ||
        tokens > kMaxTokens || max_len < 1 || q_stride < (int64_t)q_heads * head_dim ||
        k_stride < (int64_t)kv_heads * head_dim || v_stride < (int64_t)kv_heads * head_dim || q_stride % 8 || k_stride % 8 ||
        v_stride % 8)
        return BITNET_ERR_UNSUPPORTED_SHAPE;
    PromptArgs p;
    p.q = static_cast<const uint16_t *>(q); p.k = static_cast<const uint16_t *>(k); p.v = static_cast<const uint16_t *>(v);
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.starts = starts; p.tokens = tokens;
    p.max_len = max_len < tokens ? max_len : (int)tokens;
    p.q_heads = q_heads; p.kv_heads = kv_heads; p.causal = causal ? 1 : 0;
    p.scale2 = scale * 1.44269504088896340736f;
    p.out = static_cast<uint16_t *>(out);
    const dim3 grid((unsigned)((p.max_len + kRows - 1) / kRows), (unsigned)q_heads, (unsigned)batch);
    if (head_dim == 64)
        hipLaunchKernelGGL((attn_prompt_kernel<64>), grid, dim3(64 * kWaves), 0, stream, p);
    else
        hipLaunchKernelGGL((attn_prompt_kernel<128>), grid, dim3(64 * kWaves), 0, stream, p);
    return launched();
}
