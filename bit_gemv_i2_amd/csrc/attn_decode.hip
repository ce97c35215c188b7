// Attention of one token per sequence over the paged int8 cache.
//
// out = sum_j p_j v_j / sum_j p_j, p_j = exp(scale * q.k_j), over the cached tokens j: two
// products with the cache, which is read once, so the time is that of the cache's bytes.
//
// Matrix-core formulation.  v_mfma_i32_16x16x64_i8 takes the codes as they lie in memory, with
// no conversion: a tile of 64 tokens is S^T = K Q^T (16 tokens x 64 channels by 64 channels x
// 16 columns) and O^T = V^T P^T (16 channels x 64 tokens by 64 tokens x 16 columns).  The other operand has
// to be int8 too, so a query row and a tile's softmax weights are written as int8 digits to the
// base 256 under one scale: q 30 bits below the row's largest value in 4 digits, weights, each with the scale of its values
// on it, 23 bits below the largest such product of their tile in 3.  Sums of digits are exact in int32 (64 * 127 * 128 < 2^21, 128 * 128 * 128 = 2^21).
// Up to 4 query heads share a key head: the 16 columns are 4 heads x 4 digits, one product does for all digits, and
// the digits of a score meet in two adds inside a quad of lanes, those of the output once, at the end.
// More heads (WIDE): the 16 columns are heads, and every digit is a product of its own.
//
// Lane l = 16g + c of a result holds rows 4g .. 4g+3 of column c.  The rows of the four score
// tiles are taken from the tokens 16 (i / 4) + 4 tt + i % 4, so that lane (g, c) receives the scores of
// the 16 consecutive tokens 16g .. 16g+15: exactly the 16 bytes of the second
// product's operand that this lane has to supply, and tokens of one page (a page is a multiple of 16).
//
// A query row whose tile has maximum mt takes e_j = exp(s_j - mt) <= 1, digits of e_j * (scale of j's values) under
// the tile's largest, and joins the running sums with exp(mt - m): a tile far below the
// row's maximum keeps its full digits, so a long flat tail beside one large weight is not lost; nor are the small values of
// a page that has the weight, beside the large ones of a page that has none.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "attention.h"
#include "bitnet_w2a8.h"

// The four lanes of a quad take their digits from their own copies of a weight, which must agree to the last bit: no
// product may be fused into one lane's sum and not into the other's.
#pragma clang fp contract(off)

using namespace bitnet_attn;

namespace {

// What bounds it: the cache's bytes.  64 x 8192 tokens, 32 / 8 heads of 128: 1.08 GB in 171 us, 6.3 TB/s, 98% of a bare read;
// one sequence of 131071 tokens, 20 / 5 heads: 168 MB in 35 us (4.8 TB/s) and 4 us to join 98 splits; 16 sequences
// of up to 4000: 42 MB in 14 us and 4 to join, the chain of a wave's three tiles: 2 us to the first keys
// (lengths, pages, keys), then 2 to 3 a tile.  A tile takes some 360 VALU operations of a wave, 1450 cycles; a SIMD's share of
// the bandwidth brings one in 5800.
constexpr int kWaves = 4;       // waves of a workgroup, which take its tiles in turn
constexpr int kTile = 64;       // tokens of a tile: one int8 product's depth
// Workgroups that a launch is split into where the contexts allow: 2 for each of 256 CUs, as many as the registers let
// reside.  (131071 tokens, 20 / 5 heads of 128, with the join: 33.5 us in a graph, 768 34.7, 1024 38.5.)
constexpr int kWantGroups = 512;
// Caches of more bytes than the memory-side cache holds, going by the bound on the lengths, are read past it (non-temporal loads): 1.07 GB in
// 172 us instead of 182, 98% of a bare read's rate; 42 MB, which that cache keeps from call to call, in 18.4 us, but 21.2
// so.  Not for pages of 128: a tile takes half of each 128-byte line of values, and the line has to stay for the
// other half (1.07 GB: 190 us, but 224 so).
constexpr int64_t kStreamBytes = 256ll << 20;

struct DecodeArgs {
    const void *q;
    int64_t q_stride;
    const int8_t *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *table, *lengths;
    int64_t pages;
    int kv_heads, q_heads, group, page, page_shift, slots, max_len;
    int q_bf16, out_bf16;
    int chunk;    // tiles of one workgroup
    int splits;   // workgroups along the longest context
    float scale2; // scale * log2(e)
    void *out;
    float *part;  // [batch][q_heads][splits][D] sums, then [batch][q_heads][splits][2] (maximum, weight)
};

__device__ __forceinline__ v4i mfma_i8(v4i a, v4i b, v4i c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// One byte of each of four words, as one word.  sel: the byte's number in its second, 4 more in its
// second lowest byte, or 0x0C in both for zeros.
__device__ __forceinline__ uint32_t gather_bytes(const uint32_t u[4], uint32_t sel) {
    return __builtin_amdgcn_perm(u[1], u[0], sel) | __builtin_amdgcn_perm(u[3], u[2], sel) << 16;
}

// v + the value that DPP control CTRL brings.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
// The sum over a quad of lanes, the same bits in each.
__device__ __forceinline__ float quad_sum(float v) { return dpp_add<0x4E>(dpp_add<0xB1>(v)); }

// The largest of the four lanes that hold a query row.
__device__ __forceinline__ uint32_t max_row(uint32_t v) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    const uint32_t u = r[0] > r[1] ? r[0] : r[1];
    const auto t = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return t[0] > t[1] ? t[0] : t[1];
}

constexpr uint32_t digit_sel(int i) { return 0x0C0C0000u | (uint32_t)(4 + i) << 8 | (uint32_t)i; }

// Digit sums, digit 0 lowest, as one fp32 value.
__device__ __forceinline__ float join4(int d0, int d1, int d2, int d3) {
    return __builtin_fmaf((float)((d3 << 8) + d2), 65536.0f, (float)((d1 << 8) + d0));
}
__device__ __forceinline__ float join3(int d0, int d1, int d2) {
    return __builtin_fmaf((float)((d2 << 8) + d1), 256.0f, (float)d0);
}

__device__ __forceinline__ void store_out(const DecodeArgs &p, int64_t i, float v) {
    if (p.out_bf16)
        static_cast<uint16_t *>(p.out)[i] = (uint16_t)bf16_pair(v, 0.0f);
    else
        static_cast<float *>(p.out)[i] = v;
}

template <bool STREAM>
__device__ __forceinline__ v4i load16(const int8_t *p) {
    if constexpr (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const v4i *>(p));
    return *reinterpret_cast<const v4i *>(p);
}

template <int D, bool WIDE, bool STREAM>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_decode_kernel(DecodeArgs p) {
    constexpr int kSteps = D / 64;
    constexpr int kDTiles = D / 16;
    constexpr int kHeads = WIDE ? 16 : 4;
    constexpr int kQ = WIDE ? 4 : 1;  // products of the scores
    constexpr int kP = WIDE ? 3 : 1;  // and of the sums
    constexpr int kRow = D + 4;
    constexpr float kUnit = 127.0f * 65536.0f;             // a tile's largest product of weight and scale in units of the lowest digit
    constexpr float kMagic = 8388608.0f + 128.0f * 257.0f;  // 2^23 and a bias of 128 on the two lower digits

    __shared__ __align__(16) float s_o[kWaves][kHeads][kRow];
    __shared__ float s_m[kWaves][kHeads], s_l[kWaves][kHeads];

    const int b = blockIdx.z, split = blockIdx.x;
    const int chunks = (p.group + kHeads - 1) / kHeads;
    const int h = blockIdx.y / chunks, first = blockIdx.y % chunks * kHeads;
    const int heads = p.group - first < kHeads ? p.group - first : kHeads;
    const int head0 = h * p.group + first;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c = lane & 15, g = lane >> 4, dg = c & 3;

    int len = p.lengths[b];
    len = len < p.max_len ? len : p.max_len;
    const int64_t room = (int64_t)p.slots * p.page;
    if (len > room) len = (int)room;
    const int tiles = len > 0 ? (len + kTile - 1) / kTile : 0;
    const int t0 = split * p.chunk;
    const int t1 = t0 + p.chunk < tiles ? t0 + p.chunk : tiles;
    if (split > 0 && t0 >= tiles) return;

    const int64_t head_bytes = (int64_t)p.page * D;
    const int32_t *table = p.table + (int64_t)b * p.slots;
    const int last_slot = (len - 1) >> p.page_shift;

    // Keys: this lane's rows belong to the tile's 16 tokens number c / 4; its values and scores to number g.
    // Loads return in the order in which they were issued, so everything is asked for ahead of what is waited on
    // first: the page numbers two tiles ahead, the next tile's scales and keys as soon as this one's keys are
    // used up, this tile's values before its scores are computed.
    struct Pages { int k, v; };
    const auto pages_of = [&](int t) {
        int kslot = (t * kTile + 16 * (c >> 2)) >> p.page_shift, vslot = (t * kTile + 16 * g) >> p.page_shift;
        kslot = kslot < last_slot ? kslot : last_slot;  // pieces past the end read the last page and are masked
        vslot = vslot < last_slot ? vslot : last_slot;
        return Pages{table[kslot], table[vslot]};
    };
    const auto exists = [&](int page) { return (uint32_t)page < (uint64_t)p.pages; };
    const auto head_of = [&](int page) { return (int64_t)(exists(page) ? page : 0) * p.kv_heads + h; };
    v4i kf[4][kSteps];
    float sk, sv;
    const auto load_keys = [&](int t, Pages pg) {
        sk = p.k_scale[head_of(pg.v)];
        sv = p.v_scale[head_of(pg.v)];
        const int8_t *kb = p.k + head_of(pg.k) * head_bytes +
                           (((t * kTile + 16 * (c >> 2)) & (p.page - 1)) + (c & 3)) * D + 16 * g;
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int s = 0; s < kSteps; ++s) kf[tt][s] = load16<STREAM>(kb + 4 * tt * D + 64 * s);
    };
    Pages now{0, 0}, next{0, 0};
    const bool work = t0 + wave < t1;
    if (work) {
        now = pages_of(t0 + wave);
        next = pages_of(t0 + wave + kWaves);
    }

    // Query digits: lane (g, c) holds digit dg (WIDE: digit i in qd[i]) of channels 64s + 16g .. +15 of its column's head.
    const int head = WIDE ? c : c >> 2;
    v4i qd[kQ][kSteps];
    float qunit;  // what a unit of the lane's (WIDE: of the lowest) digit is worth in a score, in powers of two
    const uint32_t qsel = digit_sel(dg), qflip = dg < 3 ? 0x80808080u : 0u;
    const float weight = WIDE ? 1.0f : __uint_as_float((uint32_t)(127 + 8 * dg) << 23);  // 256^dg
    {
        float f[kSteps][16];
        uint32_t top = 0;  // magnitude bits: an infinity or a NaN is larger than any number
        const bool there = head < heads;
        const int64_t at = b * p.q_stride + (int64_t)(head0 + (there ? head : 0)) * D + 16 * g;
        const auto load_row = [&](const auto *q) {
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                load8(q + 64 * s, f[s]);
                load8(q + 64 * s + 8, f[s] + 8);
            }
        };
        if (p.q_bf16)
            load_row(static_cast<const uint16_t *>(p.q) + at);
        else
            load_row(static_cast<const float *>(p.q) + at);
        if (work) load_keys(t0 + wave, now);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                f[s][e] = there ? f[s][e] : 0.0f;
                const uint32_t u = __float_as_uint(f[s][e]) & 0x7FFFFFFFu;
                top = top > u ? top : u;
            }
        top = max_row(top);
        const float most = __uint_as_float(top);
        int ex;
        (void)frexpf(most, &ex);  // most < 2^ex, so |value| <= 2^30 and its top digit is within +-64
        // a row with an infinity or a NaN has no digits: its scores and its output become NaN
        qunit = top < 0x7F800000u ? ldexpf(p.scale2 * weight, ex - 30) : __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    u[e] = (uint32_t)(int)__builtin_rintf(ldexpf(f[s][4 * w + e], 30 - ex)) + 0x808080u;
                if constexpr (WIDE) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        qd[i][s][w] = (int)(gather_bytes(u, digit_sel(i)) ^ (i < 3 ? 0x80808080u : 0u));
                } else {
                    qd[0][s][w] = (int)(gather_bytes(u, qsel) ^ qflip);
                }
            }
    }
    const uint32_t psel = dg < 3 ? qsel : 0x0C0C0C0Cu, pflip = dg < 2 ? 0x80808080u : 0u;

    float o[kDTiles][4];
    float m = -INFINITY, l = 0.0f;  // l: the share of this lane's tokens
#pragma unroll
    for (int i = 0; i < kDTiles; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[i][r] = 0.0f;

    for (int t = t0 + wave; t < t1; t += kWaves) {
        const int vt = t * kTile + 16 * g;
        const bool vvalid = exists(now.v);
        const int8_t *vb = p.v + head_of(now.v) * head_bytes + c * p.page + (vt & (p.page - 1));
        // A page with a scale that is not finite makes the rows that see it NaN.  Left to the products it need not: an infinity is stored as
        // a code, whose score may come out as -infinity and weigh nothing, and a maximum drops a NaN.
        const float sk_t = __builtin_isfinite(sk) && __builtin_isfinite(sv) ? sk * qunit : __uint_as_float(0x7FC00000u), sv_t = sv;
        v4i vf[kDTiles];
#pragma unroll
        for (int i = 0; i < kDTiles; ++i) vf[i] = load16<STREAM>(vb + 16 * i * p.page);
        const Pages after = pages_of(t + 2 * kWaves);
        __builtin_amdgcn_sched_barrier(0);  // or the compiler moves these loads behind the scores, to spare registers

        float s[16];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
            v4i acc[kQ];
#pragma unroll
            for (int i = 0; i < kQ; ++i) {
                acc[i] = v4i{0, 0, 0, 0};
#pragma unroll
                for (int st = 0; st < kSteps; ++st) acc[i] = mfma_i8(kf[tt][st], qd[i][st], acc[i]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if constexpr (WIDE)
                    s[4 * tt + r] = join4(acc[0][r], acc[1][r], acc[2][r], acc[3][r]) * sk_t;
                else
                    s[4 * tt + r] = __int_as_float(acc[0][r]);  // until the next loads are on their way
            }
        }
        // without a branch, so that the waits below count the loads; behind the last tile that tile once more, from L2
        load_keys(t + kWaves < t1 ? t + kWaves : t, t + kWaves < t1 ? next : now);
        __builtin_amdgcn_sched_barrier(0);
        now = next;
        next = after;

        if constexpr (!WIDE) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = quad_sum((float)__float_as_int(s[i]) * sk_t);
        }
        const int seen = vvalid ? len - vt : 0;  // of this lane's 16 tokens (may exceed 16 or be negative)
        const float svs = seen > 0 ? sv_t : 0.0f;
        if (seen < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = i < seen ? s[i] : -INFINITY;
        }
        float own = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) own = fmaxf(own, s[i]);
        const float mt = max_halves(max_rows16(own));
        const float ref = mt == -INFINITY ? 0.0f : mt;  // a tile of which nothing is seen: all weights 0
        // a unit of the lowest digit: the tile's largest product of a weight and a scale is kUnit of them (the bound keeps its inverse finite)
        const float unit = fmaxf(max_halves(max_rows16(__builtin_amdgcn_exp2f(own - ref) * svs)) * (1.0f / kUnit), 0x1p-126f);
        const float units = 1.0f / unit;

        float sum = 0.0f;
        v4i pd[kP];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t u[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float e = __builtin_amdgcn_exp2f(s[4 * w + r] - ref);
                sum += e;
                // one fused product and sum rounds to a whole number in the low bits of the mantissa
                u[r] = __float_as_uint(__builtin_fmaf(e * svs, units, kMagic));
            }
            if constexpr (WIDE) {
#pragma unroll
                for (int i = 0; i < 3; ++i) pd[i][w] = (int)(gather_bytes(u, digit_sel(i)) ^ (i < 2 ? 0x80808080u : 0u));
            } else {
                pd[0][w] = (int)(gather_bytes(u, psel) ^ pflip);
            }
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
        const float w = beta * unit * weight;
#pragma unroll
        for (int i = 0; i < kDTiles; ++i) {
            v4i acc[kP];
#pragma unroll
            for (int d = 0; d < kP; ++d) acc[d] = mfma_i8(vf[i], pd[d], v4i{0, 0, 0, 0});
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float x;
                if constexpr (WIDE)
                    x = join3(acc[0][r], acc[1][r], acc[2][r]);
                else
                    x = (float)acc[0][r];
                o[i][r] = __builtin_fmaf(x, w, o[i][r]);
            }
        }
    }

    // join the digits, then the waves
    l = add_halves(add_rows16(l));
    if (g == 0 && (WIDE || dg == 0)) {
        s_m[wave][head] = m;
        s_l[wave][head] = l;
    }
#pragma unroll
    for (int i = 0; i < kDTiles; ++i) {
        v4f x;
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = WIDE ? o[i][r] : quad_sum(o[i][r]);
        if (WIDE || (i & 3) == dg) *reinterpret_cast<v4f *>(&s_o[wave][head][16 * i + 4 * g]) = x;
    }
    __syncthreads();
    for (int i = tid; i < heads * D; i += 64 * kWaves) {
        const int col = i / D, d = i % D;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, s_m[w][col]);
        const float ref = mm == -INFINITY ? 0.0f : mm;
        float ll = 0.0f, oo = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float a = __builtin_amdgcn_exp2f(s_m[w][col] - ref);
            ll = __builtin_fmaf(a, s_l[w][col], ll);
            oo = __builtin_fmaf(a, s_o[w][col][d], oo);
        }
        const int64_t row = (int64_t)b * p.q_heads + head0 + col;
        if (p.splits == 1) {
            store_out(p, row * D + d, ll != 0.0f ? oo / ll : 0.0f);
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

// Joins the splits of one query row: 8 runs of splits side by side, 4 channels a lane.
constexpr int kJoinRuns = 8;
template <int D>
__global__ __launch_bounds__(kJoinRuns *D / 4) void attn_join_kernel(DecodeArgs p) {
    __shared__ __align__(16) float s_o[kJoinRuns][D];
    __shared__ float s_l[kJoinRuns];
    const int b = blockIdx.y, tid = threadIdx.x;
    const int run = tid / (D / 4), d = tid % (D / 4) * 4;
    const int64_t row = (int64_t)b * p.q_heads + blockIdx.x;
    int len = p.lengths[b];
    len = len < p.max_len ? len : p.max_len;
    const int64_t room = (int64_t)p.slots * p.page;
    if (len > room) len = (int)room;
    const int tiles = len > 0 ? (len + kTile - 1) / kTile : 0;
    const int n = tiles > p.chunk ? (tiles + p.chunk - 1) / p.chunk : 1;  // the split 0 is always written
    const float2 *stat = reinterpret_cast<const float2 *>(p.part + (int64_t)gridDim.y * p.q_heads * p.splits * D) +
                         row * p.splits;
    const float *part = p.part + row * p.splits * D + d;
    float mm = -INFINITY;  // every wave for itself
    for (int i = tid & 63; i < n; i += 64) mm = fmaxf(mm, stat[i].x);
#pragma unroll
    for (int o = 32; o; o >>= 1) mm = fmaxf(mm, __shfl_xor(mm, o));
    const float ref = mm == -INFINITY ? 0.0f : mm;
    float ll = 0.0f;
    v4f oo = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = run; i < n; i += kJoinRuns) {
        const float2 st = stat[i];
        const v4f x = *reinterpret_cast<const v4f *>(part + (int64_t)i * D);
        const float a = __builtin_amdgcn_exp2f(st.x - ref);
        ll = __builtin_fmaf(a, st.y, ll);
#pragma unroll
        for (int e = 0; e < 4; ++e) oo[e] = __builtin_fmaf(a, x[e], oo[e]);
    }
    *reinterpret_cast<v4f *>(&s_o[run][d]) = oo;
    if (d == 0) s_l[run] = ll;
    __syncthreads();
    for (int i = tid; i < D; i += kJoinRuns * D / 4) {
        float sum = 0.0f, w = 0.0f;
#pragma unroll
        for (int r = 0; r < kJoinRuns; ++r) {
            sum += s_o[r][i];
            w += s_l[r];
        }
        store_out(p, row * D + i, w != 0.0f ? sum / w : 0.0f);
    }
}

// Query heads of one workgroup: the columns of a product, with the digits beside each other or (WIDE) one after the other.
// Groups of 4 are a little faster narrow (16 sequences of up to 4000 tokens, 20 / 5 heads of 128, in a graph: 16.7 us with the join, wide 17.8); larger
// ones would read their keys and values once for every 4 heads (64 x 8192 tokens, 8 key heads of 128: a group of 8 takes 188 us
// wide and 369 narrow, of 16 193 and 743).
int heads_of(int group) { return group <= 4 ? 4 : 16; }

// Contexts of so few tiles are not cut: a tile more for each wave costs 1.25 us, the join 2.8 and, where the host launches it, a
// call's other 5.  One sequence, 20 / 5 heads of 128: 768 tokens whole 7.7 us (8.1 cut) in a graph, 10.5 (15.5) called;
// 1024 tokens 9.0 (8.0) and 10.5 (15.5); 1536 tokens 11.6 (8.1) and 11.6 (15.3).  The limit is the one for calls: between 769 and 1024 tokens a graph
// would be up to 1 us faster cut, a call 5 us slower.
constexpr int kWhole = 4 * kWaves;

// Tiles of one workgroup.  The longest contexts are cut so that all workgroups are resident at once
// (one more than that would double the time), but no finer than a tile for each wave.
int chunk_of(int batch, int kv_heads, int group, int tiles) {
    if (tiles <= kWhole) return kWhole;
    const int heads = heads_of(group);
    const int64_t rows = (int64_t)batch * kv_heads * ((group + heads - 1) / heads);
    const int64_t splits = rows < kWantGroups ? kWantGroups / rows : 1;
    const int64_t chunk = (tiles + splits - 1) / splits;
    return chunk < kWaves ? kWaves : (int)chunk;
}

template <int D, bool WIDE>
void launch_decode(const DecodeArgs &p, dim3 grid, hipStream_t stream) {
    const int64_t bytes = 2ll * grid.z * p.kv_heads * p.max_len * D;
    if (p.page <= 64 && bytes > kStreamBytes)
        hipLaunchKernelGGL((attn_decode_kernel<D, WIDE, true>), grid, dim3(64 * kWaves), 0, stream, p);
    else
        hipLaunchKernelGGL((attn_decode_kernel<D, WIDE, false>), grid, dim3(64 * kWaves), 0, stream, p);
}

template <int D>
void launch(const DecodeArgs &p, int batch, hipStream_t stream) {
    const int heads = heads_of(p.group);
    const dim3 grid(p.splits, p.kv_heads * ((p.group + heads - 1) / heads), batch);
    heads == 4 ? launch_decode<D, false>(p, grid, stream) : launch_decode<D, true>(p, grid, stream);
    if (p.splits > 1)
        hipLaunchKernelGGL((attn_join_kernel<D>), dim3(p.q_heads, batch), dim3(kJoinRuns * D / 4), 0, stream, p);
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
    p.q_bf16 = qdt == BITNET_DT_BF16;
    p.out_bf16 = odt == BITNET_DT_BF16;
    D == 64 ? launch<64>(p, cache->batch, stream) : launch<128>(p, cache->batch, stream);
    return launched();
}

}  // extern "C"
