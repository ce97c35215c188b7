// Attention over whole prompts, packed one behind the other, bf16 on the matrix cores.
//
// out_t = sum_u p_u v_u / sum_u p_u, p_u = exp(scale * q_t.k_u - m): one pass over the keys with the
// running reference m and sum of the row, so that no score leaves the registers.
//
// Both products are taken transposed: S^T = K Q^T and O^T = V^T P^T, with
// v_mfma_f32_32x32x16_bf16.  A lane then holds one query row (lane % 32) and 16 of its scores for
// 32 keys, the rows 8j + 4 (lane / 32) + r of the result: the softmax needs one exchange between the two
// half-waves and no other, and a lane's weights, rounded to bf16, are its own operand of the second
// product, if that product takes its 16 keys in the order 8x + 4 (lane / 32) + r.  V^T is read from LDS by
// the transposing 16-bit read, which gives a lane 4 keys of one channel: that same order.
//
// The weights are rounded to 8 bits because the values are bf16 and the matrix cores take two operands of one type; a second bf16 for what the
// rounding drops would be half as many products again.  Their sum is of the unrounded ones.  Relative error of the bf16 outputs 0.0017 to 0.0022; of
// rounding the exact ones 0.0015 to 0.0017.
//
// A wave has 32 rows and runs one software pipeline over steps of 32 keys: beside the 16 products (128 channels) that make
// the scores of step j + 1 and add step j - 1 to the sums, it turns the scores of step j into weights, one a
// product.  K and V come by direct loads into a ring of four steps, two to three steps ahead.
//
// What bounds it (8192 tokens, 20 / 5 heads of 128, causal: 326 us, 1.05 PFLOP/s, 83% of a bf16 product of 8192 x 8192 x 8192 by the library,
// 77% of one of 16384; 9 prompts of up to 2047 tokens, 32 / 8 heads of 64: 94 us, 0.69 PFLOP/s).  The matrix cores are busy
// for 65% of the cycles at 128 channels, at a clock that falls from 2.4 to about 1.9 GHz under the load.  A step of one wave
// alone takes some 1400 cycles, 512 of them products: the issue of its 220 instructions, the direct loads (a quarter), the
// step's end with its reference and barrier.  Two waves a SIMD hide half of that.  A wave's last product stands behind its loop: inside, as a branch
// of each of the four stages, it cost the loop 45 registers of 250 at 128 channels and 4% of the time.  Measured and not kept: 64 rows a wave
// (half the LDS reads, but one wave a SIMD: 420 us against 350 at the time), 8 waves sharing a ring (369), operands read 5
// products ahead (352), the reference checked beside the next step's first products (364), steps of 64 keys at 64 channels (109
// against 106); wave priorities and all first loads ahead of the queries (no change).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "attention.h"
#include "bitnet_w2a8.h"

using namespace bitnet_attn;

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef unsigned short v2u16 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) v8bf lds_v8bf;
typedef __attribute__((address_space(3))) v4u lds_v4u;
typedef __attribute__((address_space(3))) float lds_float;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr int kWaves = 4;
constexpr int kRowsWave = 32;                 // query rows of a wave
constexpr int kKeys = 32;                     // keys of a step
constexpr int kStages = 4;                    // steps of K and of V in LDS
constexpr float kSlack = 8.0f;                // log2 of the largest weight before a row's reference moves
// The lowest reference.  Weights are exp2 of a score less the rounded reference, so all of a row are off by the same 2^(half a unit in its
// last place): nothing for the row, as long as that is a number.
constexpr float kLowest = -0x1p30f;
// A launch of at most so many workgroups shares the keys of each between two halves of its waves, which doubles the workgroups: up
// to where these no longer run at once.  20 heads of 128, one prompt: 512 tokens 12.1 us instead of 15.3, 1536 (240 workgroups)
// 29.1 instead of 30.6, but 2048 (320) 46.6 instead of 41.3; 32 heads of 64: 512 tokens 9.4 instead of 12.6, 1536 (384) 24.4
// instead of 25.9, 2048 (512) 33.9 instead of 33.4, 3000 (768) 56.8 instead of 52.1.  Two steps are too few to share, three are not
// (20 heads of 128: 33 to 64 tokens 7.8 us instead of 6.7, 65 to 96 8.0 instead of 8.3, 128 8.7 instead of 9.7; 32 heads of 64: 64 tokens 5.9
// instead of 5.6, 96 5.9 instead of 6.7, 128 6.6 instead of 7.8).
template <int D>
constexpr int kFewGroups = D == 64 ? 512 : 256;
constexpr int kShareFrom = 2 * kKeys + 1;
constexpr int64_t kMaxTokens = 1 << 22;
constexpr int64_t kMaxTiles = 1u << 30;  // a workgroup's number stays inside 32 bits and the launch's dimensions inside 16
constexpr int64_t kMaxStride = 1 << 23;  // a lane's offset inside a step stays inside 32 bits

struct PromptArgs {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t *starts;
    int64_t tokens;
    int max_len, q_heads, kv_heads, causal;
    uint32_t units;   // batch * kv_heads
    uint32_t blocks;  // blocks of rows in max_len
    float scale2;  // scale * log2(e)
    uint16_t *out;
};

// Place of the 16-byte piece `ch` of row `row` in a tile (and, being its own inverse, the piece at a place).
// Rows are a multiple of the LDS banks apart, so the pieces of a row are permuted by its number: for K a read
// takes one piece of each of 16 rows at a time; for V, 64 bytes of each of 4 rows.
template <int D>
__device__ __forceinline__ int k_piece(int row, int ch) {
    return ch ^ (D == 128 ? row & 15 : (row >> 1) & 7);  // (at 64 channels two rows share the 256 bytes of the banks)
}
template <int D>
__device__ __forceinline__ int v_piece(int row, int ch) {
    return ch ^ (D == 128 ? (row & 3) << 2 : (row & 2) << 1);
}

// N direct loads, 16 bytes a lane: load i from base + offset[i] + 1024 i to lds + 1024 i + 16 * lane (the load's own offset counts on
// both sides).  M0 carries the LDS address; the compiler's is put back.
template <int N>
__device__ __forceinline__ void dma(const void *base, const uint32_t (&offset)[N], uint32_t lds) {
    static_assert(N == 1 || N == 2 || N == 4);
    uint32_t saved;
    if constexpr (N == 1)
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                     "global_load_lds_dwordx4 %2, %3\n\t"
                     "s_mov_b32 m0, %0"
                     : "=&s"(saved)
                     : "s"(lds), "v"(offset[0]), "s"(base)
                     : "memory");
    else if constexpr (N == 2)
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                     "global_load_lds_dwordx4 %2, %4\n\t"
                     "global_load_lds_dwordx4 %3, %4 offset:0x400\n\t"
                     "s_mov_b32 m0, %0"
                     : "=&s"(saved)
                     : "s"(lds), "v"(offset[0]), "v"(offset[1]), "s"(base)
                     : "memory");
    else
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                     "global_load_lds_dwordx4 %2, %6\n\t"
                     "global_load_lds_dwordx4 %3, %6 offset:0x400\n\t"
                     "global_load_lds_dwordx4 %4, %6 offset:0x800\n\t"
                     "global_load_lds_dwordx4 %5, %6 offset:0xc00\n\t"
                     "s_mov_b32 m0, %0"
                     : "=&s"(saved)
                     : "s"(lds), "v"(offset[0]), "v"(offset[1]), "v"(offset[2]), "v"(offset[3]), "s"(base)
                     : "memory");
}

// Waits until at most N of this wave's direct loads are pending, then meets the workgroup.  At the top of step j, K up to step
// j + 2 and V up to step j - 1 have to be there; after them only V of step j and the two of step j - 1's issue may be pending.  The
// issue that follows takes the stages of K j and V j - 2, whose reads were consumed by products of step j - 1.
template <int N>
__device__ __forceinline__ void wait_loads_barrier() {
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The loop's parts are lambdas called with constants for each of its four stages: left to itself the compiler makes them functions.
#define INLINE __attribute__((always_inline))

// PARTS: the waves of a workgroup share its keys in 1 or 2 parts, every PARTS-th step each.
template <int D, int PARTS>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_prompt_kernel(PromptArgs p) {
    constexpr int kRowWaves = kWaves / PARTS;       // waves side by side in the rows
    constexpr int kRows = kRowWaves * kRowsWave;    // query rows of a workgroup
    constexpr int kRowBytes = 2 * D;
    constexpr int kTileBytes = kKeys * kRowBytes;
    constexpr int kK = D / 16;              // products of a step's scores
    constexpr int kD = D / 32;              // channel tiles of the second product, two products each
    constexpr int kSlots = kK + 2 * kD;
    constexpr int kScores = 16 / kSlots;    // weights computed beside a product
    constexpr int kLoads = kTileBytes / 1024 / kRowWaves;  // direct loads of a wave for a step of K (or V)
    // Stages of K [PARTS][kStages][kTileBytes] and then of V.  Sized at the launch: at the 128 KiB of two parts of 128 channels the
    // compiler would plan for one wave a SIMD and put the scores into accumulator registers, from which every one has to be moved.
    extern __shared__ __align__(1024) uint8_t stages[];
    constexpr int kPartBytes = kStages * kTileBytes;
    const uint32_t lds = (uint32_t)(uintptr_t)(lds_u8 *)stages;

    // Workgroups go to the eight dies in turn, each with an L2 of its own.  x is 8 g + die for head g of a group, so that the heads that
    // share keys share an L2, and where batch * kv_heads is a multiple of 8 all row blocks of a sequence do.  Against heads in
    // turn, 9 prompts of 2047 tokens: 32 / 8 heads of 64 channels 205 us instead of 227 (L2 misses to a quarter), 20 / 5 of 128 217
    // instead of 250; one prompt of 8192 the same.
    const uint32_t tile = (blockIdx.z * gridDim.y + blockIdx.y) * 8 + blockIdx.x % 8, level = tile / p.units, unit = tile % p.units;
    if (level >= p.blocks) return;
    const int b = unit / p.kv_heads, hk = unit % p.kv_heads, head = hk * (gridDim.x / 8) + blockIdx.x / 8;
    const int64_t n0 = p.starts[b], n1 = p.starts[b + 1];
    if (n0 < 0 || n1 > p.tokens || n1 <= n0) return;
    const int n = (int)(n1 - n0 < p.max_len ? n1 - n0 : p.max_len);
    const int q0 = (int)(p.blocks - 1 - level) * kRows;  // the longest rows of all heads and sequences first
    if (q0 >= n) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const uint16_t *kg = p.k + n0 * p.k_stride + (int64_t)hk * D;
    const uint16_t *vg = p.v + n0 * p.v_stride + (int64_t)hk * D;

    const int part = wave / kRowWaves, side = wave % kRowWaves;
    const int w0 = q0 + side * kRowsWave;  // this wave's first row
    const int row = w0 + col;              // this lane's
    const int seen = p.causal && q0 + kRows < n ? q0 + kRows : n;  // keys that any row of the workgroup sees
    const int last_step = (seen - 1) / kKeys;
    const int wave_seen = w0 >= n ? 0 : p.causal && w0 + kRowsWave < n ? w0 + kRowsWave : n;
    // Steps from here on are a part's own: its step j is step PARTS j + part of the keys.
    const auto own = [&](int all) INLINE { return (all - part + PARTS - 1) / PARTS; };  // its share of the first `all` steps
    const int steps = last_step / PARTS + 1;
    const int wave_steps = own((wave_seen + kKeys - 1) / kKeys);
    const int whole = own((p.causal && w0 + 1 < n ? w0 + 1 : n) / kKeys);  // steps that every row of the wave sees whole

    // ---- direct loads (no staging registers and no LDS stores): a lane's places in LDS are fixed, and with them its rows and pieces
    const int r_first = (side * kLoads * 1024 + lane * 16) / kRowBytes, place = lane * 16 % kRowBytes / 16;
    constexpr int kRowsLoad = 1024 / kRowBytes;  // rows of a load
    uint32_t k_off[kLoads], v_off[kLoads];       // less the 1024 i that load i adds itself: it is that many bytes of rows on, or more
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = r_first + kRowsLoad * i;
        k_off[i] = (uint32_t)(r * (int)p.k_stride + k_piece<D>(r, place) * 8) * 2u - 1024 * i;
        v_off[i] = (uint32_t)(r * (int)p.v_stride + v_piece<D>(r, place) * 8) * 2u - 1024 * i;
    }
    const uint32_t part_k = lds + part * kPartBytes, part_v = part_k + PARTS * kPartBytes;  // this part's stages
    const uint32_t lds_k = part_k + side * kLoads * 1024, lds_v = part_v + side * kLoads * 1024;
    // Step t of K (V) into its stage.  Past the end the last step again, so that every step counts the same loads; rows past
    // the end repeat the last one, with weights of 0.
    const auto issue = [&](int t, const uint16_t *g, int64_t stride, const uint32_t (&offset)[kLoads], uint32_t to) INLINE {
        to += (t & (kStages - 1)) * kTileBytes;
        t = PARTS * t + part < last_step ? PARTS * t + part : last_step;
        g += (int64_t)t * kKeys * stride;
        const int left = n - 1 - t * kKeys;
        if (left >= kKeys - 1) {
            dma(g, offset, to);
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int back = r_first + kRowsLoad * i - left;
                const uint32_t one[1] = {offset[i] + 1024 * i - (back > 0 ? (uint32_t)(back * (int)stride) * 2u : 0)};
                dma(g, one, to + 1024 * i);
            }
        }
    };
    const auto issue_k = [&](int t) INLINE { issue(t, kg, p.k_stride, k_off, lds_k); };
    const auto issue_v = [&](int t) INLINE { issue(t, vg, p.v_stride, v_off, lds_v); };
    // The loop's loads, step j + 4 of K and j + 2 of V, take the next place of running pointers as long as step j + 4 is a whole one.
    const int quick = own(n / kKeys < last_step + 1 ? n / kKeys : last_step + 1) - 4;
    const uint16_t *k_next = kg + (4 * PARTS + part) * kKeys * p.k_stride, *v_next = vg + (2 * PARTS + part) * kKeys * p.v_stride;
    const auto issue_next = [&](int u) INLINE {  // u = j % 4
        dma(k_next, k_off, lds_k + u * kTileBytes);
        dma(v_next, v_off, lds_v + ((u + 2) & 3) * kTileBytes);
        k_next += PARTS * kKeys * p.k_stride;
        v_next += PARTS * kKeys * p.v_stride;
    };

    issue_k(0);
    issue_k(1);
    v8bf qf[kK];
    {
        const int r = row < n ? row : n - 1;
        const uint16_t *qg = p.q + (n0 + r) * p.q_stride + (int64_t)head * D + 8 * half;
#pragma unroll
        for (int s = 0; s < kK; ++s) qf[s] = *reinterpret_cast<const v8bf *>(qg + 16 * s);
        // Here: the compiler does not count the direct loads, and a wait for these in the loop, where it would put it, would be one for
        // all of those at every step.
#pragma unroll
        for (int s = 0; s < kK; ++s) asm volatile("" : "+v"(qf[s]));
    }
    issue_k(2);
    issue_v(0);
    issue_k(3);
    issue_v(1);

    v16f o[kD];
    float m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < kD; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;

    // operand reads from stage `stage`
    uint32_t k_at[kK], v_at[kD];
#pragma unroll
    for (int s = 0; s < kK; ++s) k_at[s] = part_k + col * kRowBytes + (k_piece<D>(col, 2 * s + half) << 4);
    const int v_row = 4 * half + ((lane & 15) >> 2);
#pragma unroll
    for (int i = 0; i < kD; ++i) {
        v_at[i] = part_v + v_row * kRowBytes +
                  (v_piece<D>(v_row, 4 * i + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) << 4) + 8 * (lane & 1);
    }
    const auto read_k = [&](int stage, int s) INLINE {  // channels 16 s .. +15
        return *(const lds_v8bf *)(uintptr_t)(k_at[s] + stage * kTileBytes);
    };
    const auto read_v = [&](int stage, int s, int i) INLINE {  // keys 16 s .. +15, channels 32 i .. +31, transposed
        v4s f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x)  // 8 rows further on the places are the same
            f[x] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_v4s *)(uintptr_t)(v_at[i] + (stage * kTileBytes + (16 * s + 8 * x) * kRowBytes)));
        return __builtin_bit_cast(v8bf, __builtin_shufflevector(f[0], f[1], 0, 1, 2, 3, 4, 5, 6, 7));
    };
    const auto hide = [&](v16f &s, int step) INLINE {  // keys that a row does not see
        const int last = (p.causal && row < n - 1 ? row : n - 1) - kKeys * (PARTS * step + part) - 4 * half;
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (8 * (r / 4) + r % 4 > last) s[r] = -INFINITY;
    };

    constexpr int kAhead = 3;  // operand reads ahead of their product
    v8bf kf[4], vf[4];
    v16f s0, s1;
    uint32_t p0[8], p1[8];

    // One step: the weights of step j from its scores `sc` into `pc`, beside the scores of step j + 1 into `sn` and the
    // second product of step j - 1 with its weights `pp`.  Written in the order in which it is to be issued: VALU work of a
    // wave runs in the shadow of that wave's matrix products.  u = j % 4, a constant.
    const auto body = [&](int j, int u, v16f &sc, v16f &sn, uint32_t (&pc)[8], uint32_t (&pp)[8]) INLINE {
        float e[2] = {0.0f, 0.0f};
        const auto pack = [&](int id) INLINE {  // weights id - 1 and id, a while after they were computed
            pc[id / 2] = bf16_pair(e[0], e[1]);
            l += e[0];
            l += e[1];
            asm volatile("" : "+v"(pc[id / 2]), "+v"(l));  // here, not behind the next branch
        };
        const auto weights = [&](int slot) INLINE {
#pragma unroll
            for (int c = 0; c < kScores; ++c) {
                const int id = slot * kScores + c;
                const float a = __builtin_fmaf(sc[id], p.scale2, -m);
                if (id > 0 && id % 2 == 0) pack(id - 1);
                e[id % 2] = __builtin_amdgcn_exp2f(a);
            }
        };
#pragma unroll
        for (int s = 0; s < kK; ++s) {
            if (s == 0) {
                const v16f z = {0.0f};
                sn = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[0], qf[0], z, 0, 0, 0);
            } else {
                sn = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[s & 3], qf[s], sn, 0, 0, 0);
            }
            if (s + kAhead < kK)
                kf[(s + kAhead) & 3] = read_k((u + 1) & 3, s + kAhead);
            else
                vf[s + kAhead - kK] = read_v((u + 3) & 3, (s + kAhead - kK) / kD, (s + kAhead - kK) % kD);
            weights(s);
            __builtin_amdgcn_sched_barrier(0);
        }
        float mx = -INFINITY;
#pragma unroll
        for (int s = 0; s < 2 * kD; ++s) {
            const v4u w = {pp[4 * (s / kD)], pp[4 * (s / kD) + 1], pp[4 * (s / kD) + 2], pp[4 * (s / kD) + 3]};
            o[s % kD] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[s & 3], __builtin_bit_cast(v8bf, w), o[s % kD], 0, 0, 0);
            const int a = s + kAhead;
            if (a < 2 * kD)
                vf[a & 3] = read_v((u + 3) & 3, a / kD, a % kD);
            else
                kf[a - 2 * kD] = read_k((u + 2) & 3, a - 2 * kD);
            weights(kK + s);
            if (s >= 2) {
#pragma unroll
                for (int id = (s - 2) * 8 / (2 * kD - 2); id < (s - 1) * 8 / (2 * kD - 2); ++id) {
                    mx = fmaxf(fmaxf(mx, sn[2 * id]), sn[2 * id + 1]);
                    asm volatile("" : "+v"(mx));
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        pack(15);
        if (j + 1 >= whole) {  // the last steps of a row: not beside anything
            hide(sn, j + 1);
            mx = sn[0];
#pragma unroll
            for (int r = 1; r < 16; ++r) mx = fmaxf(mx, sn[r]);
        }
        // The reference m follows the largest score only when that leaves it by more than kSlack: weights up to 2^kSlack lose
        // nothing in bf16 or fp32, and the sums are scaled again a few times a row instead of at every step.  It moves by a
        // whole number, so that the scaling is by a power of two and leaves the digits of weights already rounded.
        const float t = max_halves(mx) * p.scale2;
        if (__any(t > m + kSlack)) {
            // (from further below than any weight reaches it moves to the score itself, as the scaling is by 0)
            const float mn = t > m + kSlack ? (t - m < 256.0f ? m + __builtin_ceilf(t - m) : t) : m;
            const float alpha = __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= alpha;
#pragma unroll
            for (int i = 0; i < kD; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[i][r] *= alpha;
#pragma unroll
            for (int i = 0; i < 8; ++i)  // weights of this step, not yet multiplied
                pc[i] = bf16_pair(__uint_as_float(pc[i] << 16) * alpha, __uint_as_float(pc[i] & 0xFFFF0000u) * alpha);
        }
    };

    // ---- step 0's scores
    wait_loads_barrier<4 * kLoads>();
    if (wave_steps > 0) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s0[r] = 0.0f;
#pragma unroll
        for (int s = 0; s < kK; ++s) s0 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_k(0, s), qf[s], s0, 0, 0, 0);
        if (whole == 0) hide(s0, 0);
        float t = s0[0];
#pragma unroll
        for (int r = 1; r < 16; ++r) t = fmaxf(t, s0[r]);
        // Not below kLowest, also where all these scores are minus infinity: their weights are then 0, and the first score above it takes over.
        m = fmaxf(max_halves(t) * p.scale2, kLowest);
#pragma unroll
        for (int i = 0; i < 8; ++i) p1[i] = 0;  // no step before the first
#pragma unroll
        for (int i = 0; i < kAhead; ++i) kf[i] = read_k(1, i);
    }
    // The first step multiplies weights 0 by stage 3 of V, which nothing has been loaded to yet: zeros, as 0 * x need not be 0.
    for (int i = side * 64 + lane; i < kTileBytes / 16; i += 64 * kRowWaves) ((lds_v4u *)(uintptr_t)(part_v + 3 * kTileBytes))[i] = v4u{0, 0, 0, 0};
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");

    // The wave's own steps, j % 4 a constant in each of the four.
    const auto step = [&](int j, int u) INLINE {
        wait_loads_barrier<3 * kLoads>();
        if (j < quick) {
            issue_next(u);
        } else {
            issue_k(j + 4);
            issue_v(j + 2);
        }
        if (u & 1)
            body(j, u, s1, s0, p1, p0);
        else
            body(j, u, s0, s1, p0, p1);
    };
    for (int j = 0; j < wave_steps; j += 4) {
        step(j, 0);
        if (j + 1 < wave_steps) step(j + 1, 1);
        if (j + 2 < wave_steps) step(j + 2, 2);
        if (j + 3 < wave_steps) step(j + 3, 3);
    }
    // What is left: the last step's second product, and the loads that other waves wait for.
    for (int j = wave_steps; j <= steps; ++j) {
        wait_loads_barrier<3 * kLoads>();
        if (j < steps) {
            issue_k(j + 4);
            issue_v(j + 2);
        }
        if (j > wave_steps || j == 0) continue;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = p0[i], b = p1[i];  // (a choice between the arrays themselves would put them into memory)
            w[i] = j & 1 ? a : b;
        }
        v4u f[2 * kD];
        v2u16 most = {0, 0};
#pragma unroll
        for (int x = 0; x < 2 * kD; ++x) {
            f[x] = __builtin_bit_cast(v4u, read_v((j + 3) & 3, x / kD, x % kD));
#pragma unroll
            for (int e = 0; e < 4; ++e) most = __builtin_elementwise_max(most, __builtin_bit_cast(v2u16, f[x][e] & 0x7FFF7FFFu));
        }
        // This step has keys that some of its rows do not see.  Their weight is 0, which hides a finite value only, so values that are not
        // finite are taken as 0 here and added to the rows that see them, a key at a time.  (8192 tokens, 20 / 5 heads
        // of 128: 330 us; with an infinity in the last key 380, with NaN throughout 820.)
        const bool odd = __any(most[0] >= 0x7F80 || most[1] >= 0x7F80);
        if (odd) {
#pragma unroll
            for (int x = 0; x < 2 * kD; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    f[x][e] &= ((f[x][e] & 0x7F80u) == 0x7F80u ? 0u : 0xFFFFu) | ((f[x][e] & 0x7F800000u) == 0x7F800000u ? 0u : 0xFFFF0000u);
        }
#pragma unroll
        for (int x = 0; x < 2 * kD; ++x) {
            const v4u y = {w[4 * (x / kD)], w[4 * (x / kD) + 1], w[4 * (x / kD) + 2], w[4 * (x / kD) + 3]};
            o[x % kD] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, f[x]), __builtin_bit_cast(v8bf, y), o[x % kD], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);  // the reads are done with before the next barrier gives their stage away
        if (!odd) continue;
        const int key0 = kKeys * (PARTS * (j - 1) + part);
#pragma unroll 1
        for (int u = 0; u < kKeys && key0 + u < n; ++u) {
            const uint16_t *vr = vg + (key0 + u) * p.v_stride;
            bool bad = false;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) bad |= (vr[64 * i + lane] & 0x7F80) == 0x7F80;
            if (!__any(bad)) continue;
            uint32_t word = 0;  // the pair of weights that holds key u's; half-wave (u / 4) % 2 has it
#pragma unroll
            for (int i = 0; i < 8; ++i) word = i == 2 * (u >> 3) + ((u >> 1) & 1) ? w[i] : word;
            word = __shfl(word, col + 8 * (u & 4));
            const float weight = __uint_as_float(u & 1 ? word & 0xFFFF0000u : word << 16);
            const bool sees = !p.causal || row >= key0 + u;
#pragma unroll
            for (int i = 0; i < kD; ++i)
#pragma unroll
                for (int r = 0; r < 16; r += 2) {
                    const uint32_t v = *reinterpret_cast<const uint32_t *>(vr + 32 * i + 8 * (r / 4) + 4 * half + r % 4);
                    if (sees && (v & 0x7F80u) == 0x7F80u) o[i][r] = __builtin_fmaf(weight, __uint_as_float(v << 16), o[i][r]);
                    if (sees && (v & 0x7F800000u) == 0x7F800000u) o[i][r + 1] = __builtin_fmaf(weight, __uint_as_float(v & 0xFFFF0000u), o[i][r + 1]);
                }
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the loads past the end still write to LDS

    l = add_halves(l);
    if constexpr (PARTS == 2) {  // join the parts; the stages are free once every wave's loads are done
        static_assert(kRowWaves * (D / 2 + 2) * 256 <= 2 * PARTS * kPartBytes, "a part's sums fit the stages");
        __syncthreads();
        lds_float *sums = (lds_float *)(uintptr_t)lds + side * ((D / 2 + 2) * 64) + lane, *ml = sums + D / 2 * 64;
        if (part == 1) {
#pragma unroll
            for (int i = 0; i < kD; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) sums[(16 * i + r) * 64] = o[i][r];
            ml[0] = m;
            ml[64] = l;
        }
        __syncthreads();
        if (part == 1) return;
        const float m1 = ml[0], mm = fmaxf(m, m1);  // a row sees key 0, in part 0: above minus infinity where row < n
        const float a0 = __builtin_amdgcn_exp2f(m - mm), a1 = __builtin_amdgcn_exp2f(m1 - mm);
        l = l * a0 + ml[64] * a1;
#pragma unroll
        for (int i = 0; i < kD; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[i][r] = o[i][r] * a0 + sums[(16 * i + r) * 64] * a1;
    }
    if (row >= n) return;
    const float inv = 1.0f / l;
    uint16_t *og = p.out + ((n0 + row) * p.q_heads + head) * D + 4 * half;
#pragma unroll
    for (int i = 0; i < kD; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint2 *>(og + 32 * i + 8 * j) =
                make_uint2(bf16_pair(o[i][4 * j] * inv, o[i][4 * j + 1] * inv),
                           bf16_pair(o[i][4 * j + 2] * inv, o[i][4 * j + 3] * inv));
}

int64_t row_blocks(int64_t len) { return (len + kWaves * kRowsWave - 1) / (kWaves * kRowsWave); }

template <int D, int PARTS>
void launch_parts(PromptArgs p, hipStream_t stream) {
    constexpr int rows = kWaves / PARTS * kRowsWave;
    p.blocks = (uint32_t)(p.max_len + rows - 1) / rows;
    const int64_t rounds = ((int64_t)p.units * p.blocks + 7) / 8;
    const uint32_t y = (uint32_t)(rounds < 65535 ? rounds : 65535), z = (uint32_t)((rounds + y - 1) / y);
    hipLaunchKernelGGL((attn_prompt_kernel<D, PARTS>), dim3(8 * (p.q_heads / p.kv_heads), y, z), dim3(64 * kWaves),
                       2 * PARTS * kStages * kKeys * 2 * D, stream, p);
}

template <int D>
void launch_prompt(const PromptArgs &p, hipStream_t stream) {
    const int64_t groups = (int64_t)p.units * (p.q_heads / p.kv_heads) * row_blocks(p.max_len);
    if (groups <= kFewGroups<D> && p.max_len >= kShareFrom)
        launch_parts<D, 2>(p, stream);
    else
        launch_parts<D, 1>(p, stream);
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
        v_stride % 8 || q_stride > kMaxStride || k_stride > kMaxStride || v_stride > kMaxStride)
        return BITNET_ERR_UNSUPPORTED_SHAPE;
    const int longest = max_len < tokens ? max_len : (int)tokens;
    if ((int64_t)batch * kv_heads * row_blocks(longest) > kMaxTiles) return BITNET_ERR_UNSUPPORTED_SHAPE;
    PromptArgs p;
    p.q = static_cast<const uint16_t *>(q); p.k = static_cast<const uint16_t *>(k); p.v = static_cast<const uint16_t *>(v);
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.starts = starts; p.tokens = tokens;
    p.max_len = longest;
    p.q_heads = q_heads; p.kv_heads = kv_heads; p.causal = causal ? 1 : 0;
    p.units = (uint32_t)batch * kv_heads;
    p.blocks = 0;  // launch_parts
    p.scale2 = scale * 1.44269504088896340736f;
    p.out = static_cast<uint16_t *>(out);
    if (head_dim == 64)
        launch_prompt<64>(p, stream);
    else
        launch_prompt<128>(p, stream);
    return launched();
}
