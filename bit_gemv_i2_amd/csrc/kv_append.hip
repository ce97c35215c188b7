// Rotary positions and the append to the paged int8 cache, in one launch.
//
// A workgroup owns one page of one sequence for one key head (its keys or its values), or
// the same tokens for a few query heads.  Owning a whole page and head makes its scale a reduction
// inside one workgroup: the new values stay in registers between the maximum and the
// codes, so the projection is read once.
//
// What bounds it: the bytes for long prompts (19713 tokens in 8 sequences, 32 / 8 heads of 128, bf16, the turned keys written
// out as well: 489 MB in 107 us, 4.6 TB/s, 96% of a large copy's rate); for one token a chain of four loads, each behind the
// one before (the sequence's bounds, its page, the projection and the scale, the reduction), 4.4 us of which an empty
// launch takes about half.
//
// The arithmetic is specified operation by operation (include/bitnet_w2a8.h), so this
// file must not contract products and sums into fused ones.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "attention.h"
#include "bitnet_w2a8.h"

#pragma clang fp contract(off)

using namespace bitnet_attn;

namespace {

constexpr int64_t kMaxTokens = 1 << 24;  // keeps the launch's thread count inside 32 bits
// Query heads of one workgroup: they share the table row's loads, but a workgroup for each of few heads spreads over more
// CUs.  In a graph, 512 tokens, 20 / 20 heads of 128: 1 head 6.2 us, 2 6.1, 4 7.3, 8 10.3; 19713 tokens, 32 / 8 heads: 115, 107, 110, 111.
constexpr int kQHeads = 2;

struct AppendArgs {
    const void *qkv;
    int64_t row_stride;
    const float *rope;
    int rot, interleaved;
    const int32_t *starts, *before, *table;
    int64_t tokens;
    int max_new, q_heads, kv_heads, slots;
    int64_t pages;
    int8_t *k, *v;
    float *k_scale, *v_scale;
    void *q_out, *k_out;
};

// Channels of one item: two runs of 8, which hold both halves of every pair that they touch.
struct Item {
    int a, b;    // first channel of either run
    bool turned;
};

__device__ __forceinline__ Item item_of(int it, int rot, int interleaved) {
    const bool turned = it < rot / 16;
    if (turned && !interleaved) return {8 * it, 8 * it + rot / 2, true};
    return {16 * it, 16 * it + 8, turned};
}

__device__ __forceinline__ void turn(float a[8], float b[8], const float c[8], const float s[8], int interleaved) {
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x0 = a[2 * e], x1 = a[2 * e + 1];
            a[2 * e] = x0 * c[e] - x1 * s[e];
            a[2 * e + 1] = x1 * c[e] + x0 * s[e];
            const float y0 = b[2 * e], y1 = b[2 * e + 1];
            b[2 * e] = y0 * c[4 + e] - y1 * s[4 + e];
            b[2 * e + 1] = y1 * c[4 + e] + y0 * s[4 + e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x0 = a[e], x1 = b[e];
            a[e] = x0 * c[e] - x1 * s[e];
            b[e] = x1 * c[e] + x0 * s[e];
        }
    }
}

// Largest magnitudes are compared as the bits of the numbers without their sign, in whose order a NaN is above everything: the float
// maximum would drop it, and with it every trace of it in the page.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ int code_of(float x, float inv) {
    return (int)fminf(fmaxf(__builtin_rintf(x * inv), -127.0f), 127.0f);
}

// 4 codes of older tokens, brought to a scale that grew.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r |= ((uint32_t)(int)__builtin_rintf((float)(int8_t)(w >> (8 * i)) * ratio) & 0xFFu) << (8 * i);
    return r;
}

template <typename T, int D, int PAGE>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs p) {
    constexpr int kItems = D / 16;
    constexpr int kThreads = PAGE * kItems < 256 ? PAGE * kItems : 256;
    constexpr int kRows = kThreads / kItems;  // tokens of one pass
    constexpr int kPass = PAGE / kRows;
    constexpr int kVRow = PAGE + 16;
    __shared__ uint32_t s_max[4];
    __shared__ __align__(16) int8_t s_v[D * kVRow];

    const int b = blockIdx.z, unit = blockIdx.y, tid = threadIdx.x;
    const int64_t n0 = p.starts[b], n1 = p.starts[b + 1];
    const int64_t bef = p.before[b];
    // the device-side integers are not trusted with an address
    if (n0 < 0 || n1 > p.tokens || n1 <= n0 || bef < 0) return;
    const int64_t n = n1 - n0 < p.max_new ? n1 - n0 : p.max_new;
    const int64_t slot = bef / PAGE + blockIdx.x;
    const int64_t base = slot * PAGE;
    if (base >= bef + n) return;
    const int r0 = bef > base ? (int)(bef - base) : 0;                         // first new row of the page
    const int r1 = bef + n - base < PAGE ? (int)(bef + n - base) : PAGE;       // and the one behind the last
    const int64_t t0 = n0 + base - bef;                                        // token of row 0 (may not exist)
    const bool held = slot < p.slots;                                          // the table can name this page
    const int it = tid % kItems, row = tid / kItems;
    const T *qkv = static_cast<const T *>(p.qkv);

    if (unit >= 2 * p.kv_heads) {  // queries
        const int h0 = (unit - 2 * p.kv_heads) * kQHeads;
        const Item ch = item_of(it, p.rot, p.interleaved);
        for (int r = r0 + row; r < r1; r += kRows) {
            float c[8], s[8];
            if (ch.turned && held) {
                const float *cs = p.rope + (base + r) * p.rot + 8 * it;
                load8(cs, c);
                load8(cs + p.rot / 2, s);
            }
            const T *x = qkv + (t0 + r) * p.row_stride;
            T *y = static_cast<T *>(p.q_out) + (t0 + r) * p.q_heads * D;
#pragma unroll
            for (int i = 0; i < kQHeads; ++i) {
                const int h = h0 + i;
                if (h >= p.q_heads) break;
                float a[8], bb[8];
                load8(x + h * D + ch.a, a);
                load8(x + h * D + ch.b, bb);
                if (ch.turned && held) turn(a, bb, c, s, p.interleaved);
                if (!held) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) a[e] = bb[e] = 0.0f;
                }
                store8(y + h * D + ch.a, a);
                store8(y + h * D + ch.b, bb);
            }
        }
        return;
    }

    const bool is_k = unit < p.kv_heads;
    const int h = is_k ? unit : unit - p.kv_heads;
    const Item ch = item_of(it, is_k ? p.rot : 0, p.interleaved);
    int pid = held ? p.table[(int64_t)b * p.slots + slot] : -1;
    if ((uint32_t)pid >= (uint64_t)p.pages) pid = -1;
    float *scale = is_k ? p.k_scale : p.v_scale;
    if (pid >= 0) scale += (int64_t)pid * p.kv_heads + h;
    const float old = pid >= 0 && r0 > 0 ? *scale : 0.0f;

    float a[kPass][8], bb[kPass][8];
    uint32_t most = 0;
    const T *x = qkv + (p.q_heads + (is_k ? 0 : p.kv_heads) + h) * D;
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
        const int r = row + i * kRows;
        if (r >= r0 && r < r1) {
            load8(x + (t0 + r) * p.row_stride + ch.a, a[i]);
            load8(x + (t0 + r) * p.row_stride + ch.b, bb[i]);
            if (ch.turned && held) {
                float c[8], s[8];
                const float *cs = p.rope + (base + r) * p.rot + 8 * it;
                load8(cs, c);
                load8(cs + p.rot / 2, s);
                turn(a[i], bb[i], c, s, p.interleaved);
            }
            if (!held) {
#pragma unroll
                for (int e = 0; e < 8; ++e) a[i][e] = bb[i][e] = 0.0f;
            }
            if (is_k && p.k_out) {
                T *y = static_cast<T *>(p.k_out) + ((t0 + r) * p.kv_heads + h) * D;
                store8(y + ch.a, a[i]);
                store8(y + ch.b, bb[i]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) most = umax(most, umax(magnitude(a[i][e]), magnitude(bb[i][e])));
        }
    }
    if (pid < 0) return;  // no page: nothing is stored (uniform over the workgroup)

    // the page's scale
#pragma unroll
    for (int o = 32; o; o >>= 1) most = umax(most, __shfl_xor(most, o));
    if ((tid & 63) == 0) s_max[tid >> 6] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) most = umax(most, s_max[i]);
    const float want = __uint_as_float(umax(most, __float_as_uint(1e-5f))) / 127.0f;
    const float now = __uint_as_float(umax(magnitude(old), magnitude(want)));  // NaN stays NaN until the page begins anew
    const float inv = 1.0f / now;
    if (tid == 0) *scale = now;

    const int64_t head = ((int64_t)pid * p.kv_heads + h) * (PAGE * D);
    const bool grew = r0 > 0 && now > old;
    const float ratio = old / now;
    if (is_k) {
        int8_t *kc = p.k + head;
        if (grew)  // rare: one token in some twenty raises a page's scale (64 sequences, a token each, 20 / 5 heads: all grow 8.2 us, none 4.9)
            for (int i = tid; i < r0 * (D / 16); i += kThreads) {
                uint4 w = reinterpret_cast<uint4 *>(kc)[i];
                w = make_uint4(rescale4(w.x, ratio), rescale4(w.y, ratio), rescale4(w.z, ratio), rescale4(w.w, ratio));
                reinterpret_cast<uint4 *>(kc)[i] = w;
            }
#pragma unroll
        for (int i = 0; i < kPass; ++i) {
            const int r = row + i * kRows;
            if (r >= r0 && r < r1) {
                uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    w[e / 4] |= ((uint32_t)code_of(a[i][e], inv) & 0xFFu) << (8 * (e % 4));
                    w[2 + e / 4] |= ((uint32_t)code_of(bb[i][e], inv) & 0xFFu) << (8 * (e % 4));
                }
                *reinterpret_cast<uint2 *>(kc + r * D + ch.a) = make_uint2(w[0], w[1]);
                *reinterpret_cast<uint2 *>(kc + r * D + ch.b) = make_uint2(w[2], w[3]);
            }
        }
        return;
    }

    // values lie with the positions fastest: through LDS, then 16 positions a store
    int8_t *vc = p.v + head;
    if (grew)
        for (int i = tid; i < D * (PAGE / 16); i += kThreads) {
            const int c0 = i % (PAGE / 16) * 16;
            int8_t *at = vc + (i / (PAGE / 16)) * PAGE + c0;
            if (c0 + 16 <= r0) {
                uint4 w = *reinterpret_cast<uint4 *>(at);
                w = make_uint4(rescale4(w.x, ratio), rescale4(w.y, ratio), rescale4(w.z, ratio), rescale4(w.w, ratio));
                *reinterpret_cast<uint4 *>(at) = w;
            } else {
                for (int e = 0; c0 + e < r0; ++e) at[e] = (int8_t)__builtin_rintf((float)at[e] * ratio);
            }
        }
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
        const int r = row + i * kRows;
        if (r >= r0 && r < r1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s_v[(ch.a + e) * kVRow + r] = (int8_t)code_of(a[i][e], inv);
                s_v[(ch.b + e) * kVRow + r] = (int8_t)code_of(bb[i][e], inv);
            }
        }
    }
    __syncthreads();
    const int c_lo = r0 / 16, c_n = (r1 + 15) / 16 - c_lo;  // the 16-position pieces with new rows
    for (int i = tid; i < D * c_n; i += kThreads) {
        const int d = i / c_n, c0 = (c_lo + i % c_n) * 16;
        const int8_t *from = s_v + d * kVRow + c0;
        int8_t *to = vc + d * PAGE + c0;
        if (c0 >= r0 && c0 + 16 <= r1) {
            *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from);
        } else {
            const int e0 = r0 > c0 ? r0 - c0 : 0, e1 = r1 - c0 < 16 ? r1 - c0 : 16;
            for (int e = e0; e < e1; ++e) to[e] = from[e];
        }
    }
}

template <typename T, int D, int PAGE>
void launch_append(const AppendArgs &p, dim3 grid, hipStream_t stream) {
    constexpr int threads = PAGE * (D / 16) < 256 ? PAGE * (D / 16) : 256;
    hipLaunchKernelGGL((append_kernel<T, D, PAGE>), grid, dim3(threads), 0, stream, p);
}

template <typename T, int D>
void launch_page(const AppendArgs &p, int page, dim3 grid, hipStream_t stream) {
    switch (page) {
        case 16: return launch_append<T, D, 16>(p, grid, stream);
        case 32: return launch_append<T, D, 32>(p, grid, stream);
        case 64: return launch_append<T, D, 64>(p, grid, stream);
        default: return launch_append<T, D, 128>(p, grid, stream);
    }
}

}  // namespace

extern "C" bitnet_status_t bitnet_rope_append_kv(const void *qkv, int dt, int64_t row_stride, const float *rope,
                                                 int64_t rope_rows, int rot, int interleaved, const int32_t *starts,
                                                 const int32_t *before, int64_t tokens, int max_new, int q_heads,
                                                 const bitnet_kv_cache_t *cache, void *q_out, void *k_out,
                                                 hipStream_t stream) {
    const bitnet_status_t st = check_cache(cache);
    if (st != BITNET_OK) return st;
    if (!at(qkv, 16) || !at(q_out, 16) || (k_out && !at(k_out, 16)) || !at(starts, 4) || !at(before, 4) ||
        (rot != 0 && !at(rope, 16)) || (dt != BITNET_DT_BF16 && dt != BITNET_DT_F32))
        return BITNET_ERR_INVALID_ARG;
    const int D = cache->head_dim, hk = cache->kv_heads;
    if (!heads_ok(q_heads, hk) || rot < 0 || rot > D || rot % 16 ||
        (rot != 0 && rope_rows < (int64_t)cache->slots * cache->page) || tokens < 1 || tokens > kMaxTokens || max_new < 1 ||
        row_stride < (int64_t)(q_heads + 2 * hk) * D || row_stride % 8)
        return BITNET_ERR_UNSUPPORTED_SHAPE;
    AppendArgs p;
    p.qkv = qkv; p.row_stride = row_stride; p.rope = rope; p.rot = rot; p.interleaved = interleaved ? 1 : 0;
    p.starts = starts; p.before = before; p.table = cache->table; p.tokens = tokens; p.max_new = max_new;
    p.q_heads = q_heads; p.kv_heads = hk; p.slots = cache->slots; p.pages = cache->pages;
    p.k = cache->k; p.v = cache->v; p.k_scale = cache->k_scale; p.v_scale = cache->v_scale;
    p.q_out = q_out; p.k_out = k_out;
    // a run of n tokens touches at most (n + page - 2) / page + 1 pages
    const int64_t most = max_new < tokens ? max_new : tokens;
    const dim3 grid((unsigned)((most + cache->page - 2) / cache->page + 1),
                    (unsigned)(2 * hk + (q_heads + kQHeads - 1) / kQHeads), (unsigned)cache->batch);
    const int page = cache->page;
    if (dt == BITNET_DT_BF16)
        D == 64 ? launch_page<uint16_t, 64>(p, page, grid, stream) : launch_page<uint16_t, 128>(p, page, grid, stream);
    else
        D == 64 ? launch_page<float, 64>(p, page, grid, stream) : launch_page<float, 128>(p, page, grid, stream);
    return launched();
}
