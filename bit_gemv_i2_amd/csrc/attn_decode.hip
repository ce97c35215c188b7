// Attention of one token per sequence over the paged int8 cache.
//
// out = sum_j p_j v_j / sum_j p_j, p_j = exp(scale * q.k_j), over the cached tokens j: two
// products with the cache, which is read once, so the time is that of the cache's bytes.
//
// Matrix-core formulation.  v_mfma_i32_16x16x64_i8 takes the codes as they lie in memory, with
// no conversion: a tile of 64 tokens is S^T = K Q^T (16 tokens x 64 channels by 64 channels x
// 16 query rows) and O^T = V^T P^T (16 channels x 64 tokens by 64 tokens x 16 query rows).  The other
// operand has to be int8 too, so a query row and a tile's softmax weights are written as a
// few int8 digits to the base 256 under one scale, one product per digit; sums of digits are exact
// in int32 (64 * 127 * 128 < 2^21, 128 * 128 * 128 = 2^21).
//
// Lane l = 16g + c of a result holds rows 4g .. 4g+3 of column c.  The rows of the four score
// tiles are taken from the tokens 16 (i / 4) + 4 tt + i % 4, so that lane (g, c) receives the scores of
// the 16 consecutive tokens 16g .. 16g+15 for query row c: exactly the 16 bytes of the second
// product's operand that this lane has to supply, and tokens of one page (a page is a multiple of 16).
// Nothing moves between lanes but the maxima of a row.
//
// A query row whose tile has maximum mt takes e_j = exp(s_j - mt) <= 1, digits of e_j under
// the tile's own maximum, and joins the running sums with exp(mt - m): a tile far below the
// row's maximum keeps its full digits, so a long flat tail beside one large weight is not lost.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "attention.h"
#include "bitnet_w2a8.h"

using namespace bitnet_attn;

namespace {

constexpr int kWaves = 4;       // waves of a workgroup, which take its tiles in turn
constexpr int kTile = 64;       // tokens of a tile: one int8 product's depth
constexpr int kCols = 16;       // query rows of a product
constexpr int kWantGroups = 512;  // workgroups that a launch is split into where the contexts allow

struct DecodeArgs {
    const void *q;
    int64_t q_stride;
    const int8_t *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *table, *lengths;
    int64_t pages;
    int kv_heads, q_heads, group, page, page_shift, slots, max_len;
    int chunk;    // tiles of one workgroup
    int splits;   // workgroups along the longest context
    float scale2; // scale * log2(e)
    void *out;
    float *part;  // [batch][q_heads][splits][D] sums, then [batch][q_heads][splits][2] (maximum, weight)
};

__device__ __forceinline__ v4i mfma_i8(v4i a, v4i b, v4i c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// Byte i of each of four words, as one word.
template <int I>
__device__ __forceinline__ uint32_t gather_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t sel = 0x0C0C0000u | (uint32_t)((4 + I) << 8) | (uint32_t)I;
    const uint32_t lo = __builtin_amdgcn_perm(b, a, sel);
    const uint32_t hi = __builtin_amdgcn_perm(d, c, sel);
    return lo | (hi << 16);
}

template <int N>
__device__ __forceinline__ void digits4(const uint32_t u[4], int word, v4i out[N]) {
    // u: biased values (128 added to every digit but the top one): byte i is digit i plus its bias
    out[0][word] = (int)(gather_bytes<0>(u[0], u[1], u[2], u[3]) ^ (N > 1 ? 0x80808080u : 0u));
    if constexpr (N > 1) out[1][word] = (int)(gather_bytes<1>(u[0], u[1], u[2], u[3]) ^ (N > 2 ? 0x80808080u : 0u));
    if constexpr (N > 2) out[2][word] = (int)(gather_bytes<2>(u[0], u[1], u[2], u[3]) ^ (N > 3 ? 0x80808080u : 0u));
    if constexpr (N > 3) out[3][word] = (int)gather_bytes<3>(u[0], u[1], u[2], u[3]);
}

// Digit sums (digit 0 lowest) as one fp32 value.
template <int N>
__device__ __forceinline__ float join(const int d[N]) {
    if constexpr (N == 2) return (float)((d[1] << 8) + d[0]);
    if constexpr (N == 3) return __builtin_fmaf((float)((d[2] << 8) + d[1]), 256.0f, (float)d[0]);
    return __builtin_fmaf((float)((d[3] << 8) + d[2]), 65536.0f, (float)((d[1] << 8) + d[0]));
}

template <typename T>
__device__ __forceinline__ void store_one(T *p, float v) {
    if constexpr (sizeof(T) == 2)
        *p = (T)bf16_pair(v, 0.0f);
    else
        *p = v;
}

// QD digits of q (3 for bf16, 4 for fp32), PD digits of the weights (2 for a bf16 output, 3 for fp32).
template <int D, typename QT, typename OT>
__global__ __launch_bounds__(64 * kWaves) void attn_decode_kernel(DecodeArgs p) {
    constexpr int QD = sizeof(QT) == 2 ? 3 : 4;
    constexpr int PD = sizeof(OT) == 2 ? 2 : 3;
    constexpr int kSteps = D / 64;
    constexpr int kDTiles = D / 16;
    constexpr int kRow = D + 4;
    // largest weight of a tile in units of the lowest digit, and the bias of the lower digits
    constexpr float kUnit = PD == 2 ? 127.0f * 256.0f : 127.0f * 65536.0f;
    constexpr float kMagic = 8388608.0f + (PD == 2 ? 128.0f : 32896.0f);

    __shared__ float s_o[kWaves][kCols][kRow];
    __shared__ float s_m[kWaves][kCols], s_l[kWaves][kCols];

    const int b = blockIdx.z, split = blockIdx.x;
    const int chunks = (p.group + kCols - 1) / kCols;
    const int h = blockIdx.y / chunks, first = blockIdx.y % chunks * kCols;
    const int cols = p.group - first < kCols ? p.group - first : kCols;
    const int head0 = h * p.group + first;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c = lane & 15, g = lane >> 4;

    int len = p.lengths[b];
    len = len < p.max_len ? len : p.max_len;
    const int64_t room = (int64_t)p.slots * p.page;
    if (len > room) len = (int)room;
    const int tiles = len > 0 ? (len + kTile - 1) / kTile : 0;
    const int t0 = split * p.chunk;
    const int t1 = t0 + p.chunk < tiles ? t0 + p.chunk : tiles;
    if (split > 0 && t0 >= tiles) return;

    // the query rows' digits: lane (g, c) holds channels 64s + 16g .. +15 of row c
    v4i qd[kSteps][QD];
    float qunit;  // value of a unit of the lowest digit, with the softmax scale
    {
        float f[kSteps][16];
        float most = 0.0f;
        const bool there = c < cols;
        const QT *q = static_cast<const QT *>(p.q) + b * p.q_stride + (int64_t)(head0 + (there ? c : 0)) * D + 16 * g;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            load8(q + 64 * s, f[s]);
            load8(q + 64 * s + 8, f[s] + 8);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                f[s][e] = there ? f[s][e] : 0.0f;
                most = fmaxf(most, fabsf(f[s][e]));
            }
        }
        most = max_halves(max_rows16(most));
        int ex;
        (void)frexpf(most, &ex);  // most < 2^ex, so |value| <= 2^(8 QD - 2)
        const int up = 8 * QD - 2 - ex;
        qunit = ldexpf(p.scale2, -up);
        constexpr uint32_t bias = QD == 3 ? 0x8080u : 0x808080u;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) u[e] = (uint32_t)(int)__builtin_rintf(ldexpf(f[s][4 * w + e], up)) + bias;
                digits4<QD>(u, w, qd[s]);
            }
    }

    float o[kDTiles][4];
#pragma unroll
    for (int i = 0; i < kDTiles; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[i][r] = 0.0f;
    float m = -INFINITY, l = 0.0f;  // l: this lane's share

    const int64_t head_bytes = (int64_t)p.page * D;
    const int32_t *table = p.table + (int64_t)b * p.slots;
    const int last_slot = (len - 1) >> p.page_shift;

    for (int t = t0 + wave; t < t1; t += kWaves) {
        // keys: this lane's rows belong to the tile's 16 tokens number c / 4, its values to number g
        const int kt = t * kTile + 16 * (c >> 2), vt = t * kTile + 16 * g;
        int kslot = kt >> p.page_shift, vslot = vt >> p.page_shift;
        kslot = kslot < last_slot ? kslot : last_slot;  // pieces past the end read the last page and are masked
        vslot = vslot < last_slot ? vslot : last_slot;
        int kp = table[kslot], vp = table[vslot];
        const bool kvalid = (uint32_t)kp < (uint64_t)p.pages, vvalid = (uint32_t)vp < (uint64_t)p.pages;
        kp = kvalid ? kp : 0;
        vp = vvalid ? vp : 0;
        const int8_t *kb = p.k + ((int64_t)kp * p.kv_heads + h) * head_bytes +
                           ((kt & (p.page - 1)) + (c & 3)) * D + 16 * g;
        const int64_t vhead = (int64_t)vp * p.kv_heads + h;
        const int8_t *vb = p.v + vhead * head_bytes + c * p.page + (vt & (p.page - 1));
        const float sk = p.k_scale[vhead] * qunit, sv = p.v_scale[vhead];

        v4i kf[4][kSteps], vf[kDTiles];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int s = 0; s < kSteps; ++s) kf[tt][s] = *reinterpret_cast<const v4i *>(kb + 4 * tt * D + 64 * s);
#pragma unroll
        for (int i = 0; i < kDTiles; ++i) vf[i] = *reinterpret_cast<const v4i *>(vb + 16 * i * p.page);

        float s[16];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
            v4i acc[QD];
#pragma unroll
            for (int d = 0; d < QD; ++d) {
                acc[d] = v4i{0, 0, 0, 0};
#pragma unroll
                for (int st = 0; st < kSteps; ++st) acc[d] = mfma_i8(kf[tt][st], qd[st][d], acc[d]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                int d[QD];
#pragma unroll
                for (int i = 0; i < QD; ++i) d[i] = acc[i][r];
                s[4 * tt + r] = join<QD>(d) * sk;
            }
        }
        const int seen = vvalid ? len - vt : 0;  // of this lane's 16 tokens (may exceed 16 or be negative)
        if (seen < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = i < seen ? s[i] : -INFINITY;
        }
        float mt = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mt = fmaxf(mt, s[i]);
        mt = max_halves(max_rows16(mt));
        const float ref = mt == -INFINITY ? 0.0f : mt;  // a tile of which nothing is seen: all weights 0
        // scales of the four 16-token groups, under the largest
        const float svs = seen > 0 ? sv : 0.0f;
        const float svmax = max_halves(max_rows16(svs));
        const float ratio = svmax > 0.0f ? svs / svmax * kUnit : 0.0f;

        float sum = 0.0f;
        v4i pd[PD];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t u[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float e = __builtin_amdgcn_exp2f(s[4 * w + r] - ref);
                sum += e;
                // one fused product and sum rounds to a whole number in the low bits of the mantissa
                u[r] = __float_as_uint(__builtin_fmaf(e, ratio, kMagic));
            }
            digits4<PD>(u, w, pd);
        }

        const float mn = fmaxf(m, mt);
        const float mref = mn == -INFINITY ? 0.0f : mn;
        const float beta = __builtin_amdgcn_exp2f(mt - mref);
        if (__any(mn > m)) {
            const float alpha = __builtin_amdgcn_exp2f(m - mref);
            l *= alpha;
#pragma unroll
            for (int i = 0; i < kDTiles; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[i][r] *= alpha;
        }
        m = mn;
        l = __builtin_fmaf(sum, beta, l);
        const float w = beta * svmax * (1.0f / kUnit);
#pragma unroll
        for (int i = 0; i < kDTiles; ++i) {
            v4i acc[PD];
#pragma unroll
            for (int d = 0; d < PD; ++d) acc[d] = mfma_i8(vf[i], pd[d], v4i{0, 0, 0, 0});
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                int d[PD];
#pragma unroll
                for (int x = 0; x < PD; ++x) d[x] = acc[x][r];
                o[i][r] = __builtin_fmaf(join<PD>(d), w, o[i][r]);
            }
        }
    }

    // join the waves
    l = add_halves(add_rows16(l));
    if (g == 0) {
        s_m[wave][c] = m;
        s_l[wave][c] = l;
    }
#pragma unroll
    for (int i = 0; i < kDTiles; ++i)
        *reinterpret_cast<v4f *>(&s_o[wave][c][16 * i + 4 * g]) = v4f{o[i][0], o[i][1], o[i][2], o[i][3]};
    __syncthreads();
    for (int i = tid; i < cols * D; i += 64 * kWaves) {
        const int col = i / D, d = i % D;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, s_m[w][col]);
        float ll = 0.0f, oo = 0.0f;
        if (mm != -INFINITY) {
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float a = __builtin_amdgcn_exp2f(s_m[w][col] - mm);
                ll = __builtin_fmaf(a, s_l[w][col], ll);
                oo = __builtin_fmaf(a, s_o[w][col][d], oo);
            }
        }
        const int64_t row = (int64_t)b * p.q_heads + head0 + col;
        if (p.splits == 1) {
            store_one(static_cast<OT *>(p.out) + row * D + d, ll > 0.0f ? oo / ll : 0.0f);
        } else {
            p.part[(row * p.splits + split) * D + d] = oo;
            if (d == 0) {
                float *stat = p.part + (int64_t)gridDim.z * p.q_heads * p.splits * D + (row * p.splits + split) * 2;
                stat[0] = mm;
                stat[1] = ll;
            }
        }
    }
}

// Joins the splits of one query row.
template <int D, typename OT>
__global__ __launch_bounds__(D) void attn_join_kernel(DecodeArgs p) {
    const int b = blockIdx.y, d = threadIdx.x;
    const int64_t row = (int64_t)b * p.q_heads + blockIdx.x;
    int len = p.lengths[b];
    len = len < p.max_len ? len : p.max_len;
    const int64_t room = (int64_t)p.slots * p.page;
    if (len > room) len = (int)room;
    const int tiles = len > 0 ? (len + kTile - 1) / kTile : 0;
    const int n = tiles > p.chunk ? (tiles + p.chunk - 1) / p.chunk : 1;  // the split 0 is always written
    const float *stat = p.part + (int64_t)gridDim.y * p.q_heads * p.splits * D + row * p.splits * 2;
    const float *part = p.part + row * p.splits * D + d;
    float mm = -INFINITY;
    for (int i = 0; i < n; ++i) mm = fmaxf(mm, stat[2 * i]);
    float ll = 0.0f, oo = 0.0f;
    if (mm != -INFINITY)
        for (int i = 0; i < n; ++i) {
            const float a = __builtin_amdgcn_exp2f(stat[2 * i] - mm);
            ll = __builtin_fmaf(a, stat[2 * i + 1], ll);
            oo = __builtin_fmaf(a, part[(int64_t)i * D], oo);
        }
    store_one(static_cast<OT *>(p.out) + row * D + d, ll > 0.0f ? oo / ll : 0.0f);
}

// Tiles of one workgroup: enough workgroups to fill the chip, at least one tile for each wave.
int chunk_of(int batch, int kv_heads, int group, int tiles) {
    const int64_t rows = (int64_t)batch * kv_heads * ((group + kCols - 1) / kCols);
    int64_t splits = (kWantGroups + rows - 1) / rows;
    int64_t chunk = (tiles + splits - 1) / splits;
    return chunk < kWaves ? kWaves : (int)chunk;
}

template <int D, typename QT, typename OT>
void launch_decode(const DecodeArgs &p, int batch, hipStream_t stream) {
    const int chunks = (p.group + kCols - 1) / kCols;
    hipLaunchKernelGGL((attn_decode_kernel<D, QT, OT>), dim3(p.splits, p.kv_heads * chunks, batch), dim3(64 * kWaves), 0,
                       stream, p);
    if (p.splits > 1)
        hipLaunchKernelGGL((attn_join_kernel<D, OT>), dim3(p.q_heads, batch), dim3(D), 0, stream, p);
}

template <int D>
void launch_types(const DecodeArgs &p, int qdt, int odt, int batch, hipStream_t stream) {
    if (qdt == BITNET_DT_BF16)
        odt == BITNET_DT_BF16 ? launch_decode<D, uint16_t, uint16_t>(p, batch, stream)
                              : launch_decode<D, uint16_t, float>(p, batch, stream);
    else
        odt == BITNET_DT_BF16 ? launch_decode<D, float, uint16_t>(p, batch, stream)
                              : launch_decode<D, float, float>(p, batch, stream);
}

bool decode_shape_ok(int batch, int q_heads, int kv_heads, int head_dim, int max_len) {
    return batch >= 1 && batch <= 65535 && heads_ok(q_heads, kv_heads) && head_dim_ok(head_dim) && max_len >= 1 &&
           max_len <= INT32_MAX - kTile;
}

int splits_of(int batch, int q_heads, int kv_heads, int max_len, int *chunk) {
    const int tiles = (max_len + kTile - 1) / kTile;
    *chunk = chunk_of(batch, kv_heads, q_heads / kv_heads, tiles);
    return (tiles + *chunk - 1) / *chunk;
}

}  // namespace

extern "C" {

size_t bitnet_attn_decode_workspace_bytes(int batch, int q_heads, int kv_heads, int head_dim, int max_len) {
    if (!decode_shape_ok(batch, q_heads, kv_heads, head_dim, max_len)) return 0;
    int chunk;
    const int splits = splits_of(batch, q_heads, kv_heads, max_len, &chunk);
    return splits == 1 ? 0 : (size_t)batch * q_heads * splits * (head_dim + 2) * sizeof(float);
}

bitnet_status_t bitnet_attn_decode(const void *q, int qdt, int64_t q_stride, const bitnet_kv_cache_t *cache,
                                   const int32_t *lengths, int max_len, int q_heads, float scale, void *out, int odt,
                                   void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const bitnet_status_t st = check_cache(cache);
    if (st != BITNET_OK) return st;
    if (!at(q, 16) || !at(lengths, 4) || !at(out, 16) || (qdt != BITNET_DT_BF16 && qdt != BITNET_DT_F32) ||
        (odt != BITNET_DT_BF16 && odt != BITNET_DT_F32) || !(scale > 0.0f) || !std::isfinite(scale))
        return BITNET_ERR_INVALID_ARG;
    const int D = cache->head_dim;
    if (!decode_shape_ok(cache->batch, q_heads, cache->kv_heads, D, max_len) || q_stride < (int64_t)q_heads * D ||
        q_stride % 8)
        return BITNET_ERR_UNSUPPORTED_SHAPE;
    DecodeArgs p;
    p.splits = splits_of(cache->batch, q_heads, cache->kv_heads, max_len, &p.chunk);
    const size_t need = bitnet_attn_decode_workspace_bytes(cache->batch, q_heads, cache->kv_heads, D, max_len);
    if (need && (!at(workspace, 256) || workspace_bytes < need)) return BITNET_ERR_INVALID_ARG;
    p.q = q; p.q_stride = q_stride;
    p.k = cache->k; p.v = cache->v; p.k_scale = cache->k_scale; p.v_scale = cache->v_scale;
    p.table = cache->table; p.lengths = lengths; p.pages = cache->pages;
    p.kv_heads = cache->kv_heads; p.q_heads = q_heads; p.group = q_heads / cache->kv_heads;
    p.page = cache->page; p.page_shift = __builtin_ctz((unsigned)cache->page); p.slots = cache->slots; p.max_len = max_len;
    p.scale2 = scale * 1.44269504088896340736f;
    p.out = out; p.part = static_cast<float *>(workspace);
    D == 64 ? launch_types<64>(p, qdt, odt, cache->batch, stream) : launch_types<128>(p, qdt, odt, cache->batch, stream);
    return launched();
}

}  // extern "C"
