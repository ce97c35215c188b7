// W2A8 products with an epilogue (bias, activation, gate, residual), over all tokens or by expert.
//
//     z[m][n] = s_a[m] * sum_b S[n][b] * A[m][n][b] + bias[n],   y = act(z) (+ residual),  gated: act(z_gate) * z_up
//
// on the int8 matrix cores, as the products without an epilogue: lane (g, j) of a wave supplies row j of 16 weight rows
// and token j of 16 tokens at 16 columns 16 g + 64 s, and receives tokens 4g .. 4g + 3 of row j, so that bias, activation
// and residual are a lane's own and the gate and the up projection of an output meet in one lane.
#include "fused.h"

using namespace bitnet_fused;

namespace {

typedef unsigned v2u __attribute__((ext_vector_type(2)));

__device__ __forceinline__ v4i decode16(uint32_t w) {  // 16 weights as 64 t in int8
    v4i r;
    r[0] = (int)((w << 6) & 0xC0C0C0C0u);
    r[1] = (int)((w << 4) & 0xC0C0C0C0u);
    r[2] = (int)((w << 2) & 0xC0C0C0C0u);
    r[3] = (int)(w & 0xC0C0C0C0u);
    return r;
}
__device__ __forceinline__ v4i mfma_i8(v4i a, v4i b, v4i c) { return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0); }

// ==========================================================================
// Few rows of an expert (or few tokens): the weights are the work, each read once.  A workgroup has 16 outputs of a token
// (gated: 16 gate rows and the 16 up rows of the same outputs) of one expert; its waves split the blocks of K, at most NB each, and every
// lane has requested all its codes and scales (streaming loads: nobody reads them again) before the first product.  A wave
// brings its slice of up to TOK tokens through LDS (a few wide loads instead of many narrow ones; it reads only what it wrote itself,
// so no barrier), multiplies, and the waves' sums are joined in LDS in a fixed order.  Further tokens of the expert, TOK at a
// time, meet the codes still in registers; with more blocks than the waves hold at once (MULTI, above 96) every pass reads them again.
// By expert, workgroup row y has the y-th expert that has any rows, so that no more than there are slots are launched.
//
// Floor: the weights once (9/32 of a byte each, their scales among it: 2560 x 6912 5 MB, 13824 x 2560 10 MB; 0.8 and 1.6 us at a bare
// read's 6.3 TB/s) and a launch.  Measured in a graph, weights from HBM: 1 token x 2560 x 6912 4.1 us, 8 x 13824 x 2560 gated 5.7, 16 tokens 6.4, 1 x
// 131072 x 2560 19.6 (4.8 TB/s).  What bounds it: few tiles, one workgroup's chain (launch, loads, products, join); many tiles, the
// time in which a workgroup has no weights in flight (its start, join and end: half of some 4 us).
// ==========================================================================
constexpr int kMostWaves = 12;  // 170 registers a lane, and 96 blocks before a wave has to take its blocks in turns

struct RowsArgs {
    FusedArgs p;
    int per, waves;  // blocks a wave, waves
};

template <bool GATED, bool GROUPED, int NB, int TOK, bool MULTI>
__global__ __launch_bounds__(64 * kMostWaves) void rows_kernel(RowsArgs a) {
    constexpr int H = GATED ? 2 : 1;
    constexpr int kSlice = NB * 128 + 16;  // bytes of a token's slice in LDS, 16 more than the columns: rows 4 banks apart
    // loads of the slices: P lanes a token (8 NB pieces of 16 bytes, rounded up to a power of two), 64 / P tokens a load
    constexpr int P = NB > 4 ? 64 : NB > 2 ? 32 : NB > 1 ? 16 : 8, kTogether = 64 / P, kLoads = (TOK + kTogether - 1) / kTogether;
    constexpr int kEnds = TOK > 4 ? 4 : 1;  // outputs that a lane may have to finish
    const FusedArgs &p = a.p;
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, g = l >> 4, j = l & 15;
    const int blocks = p.K >> 7, all_tiles = p.N >> 4, width = GATED ? p.N >> 1 : p.N, tile = blockIdx.x;
    Tile t = {0, 0, p.slots};
    if (GROUPED && !find_expert(p, blockIdx.y, &t)) return;
    const int b0 = w * a.per, b1 = min(blocks, b0 + a.per);

    int8_t *mine = reinterpret_cast<int8_t *>(smem) + w * TOK * kSlice;
    float *sums = reinterpret_cast<float *>(smem + a.waves * TOK * kSlice);  // [wave][4 H][64]

    uint2 code[H][NB];
    float scale[H][NB];
    auto load_weights = [&](int c0) {
        const int last = min(NB, b1 - c0) - 1;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int64_t brick = ((int64_t)t.expert * all_tiles + tile + h * (width >> 4)) * blocks + c0;
            const uint8_t *cp = p.packed + brick * kBrickBytes;  // the same for all lanes: a lane's part is a 32-bit offset
            const float *sp = p.scales + brick * kTileN;
#pragma unroll
            for (int i = 0; i < NB; ++i) {  // past the wave's last block: the last again, not used
                const v2u c = __builtin_nontemporal_load(reinterpret_cast<const v2u *>(cp + min(i, last) * (int)kBrickBytes) + l);
                code[h][i] = make_uint2(c.x, c.y);
                scale[h][i] = __builtin_nontemporal_load(sp + min(i, last) * (int)kTileN + j);
            }
        }
    };

    // Lane m < TOK: the token of slot first + m (past the last: the last again).  One load whether there are indices or not, as a load
    // behind a branch makes the compiler wait for everything before it.
    int first = t.first, n, token;
    auto load_tokens = [&]() {
        n = min(TOK, t.end - first);
        const int slot = first + min(l, n - 1);
        const int32_t *from = GROUPED && p.rows ? p.rows : reinterpret_cast<const int32_t *>(p.s_a);
        const int32_t row = GROUPED ? from[p.rows ? slot : 0] : 0;
        token = GROUPED && p.rows ? row : slot;
    };
    auto followed = [&](int row) { return (uint32_t)row < (uint32_t)p.tokens; };  // else read as token 0 and not stored
    v4i x[kLoads];
    auto load_x = [&](int c0) {
        const int o = min(l & (P - 1), min(NB, b1 - c0) * 8 - 1), safe = followed(token) ? token : 0;
        const int8_t *from = p.q + c0 * 128;
#pragma unroll
        for (int r = 0; r < kLoads; ++r) {
            if (P == 64) {  // a base for all lanes and a lane's 32-bit offset
                const int8_t *row = from + (int64_t)__builtin_amdgcn_readlane(safe, r) * p.K;
                x[r] = *reinterpret_cast<const v4i *>(row + (uint32_t)(o * 16));
            } else {
                x[r] = *reinterpret_cast<const v4i *>(from + (int64_t)__shfl(safe, min(r * kTogether + l / P, TOK - 1)) * p.K + o * 16);
            }
        }
    };
    // what the outputs of a pass need at their end: output tid + r * threads is token (..) / 16, row (..) % 16
    const uint8_t *res = static_cast<const uint8_t *>(p.residual ? p.residual : p.scales);
    int owner[kEnds];
    float factor[kEnds];
    uint32_t residual[kEnds];
    auto load_ends = [&]() {
#pragma unroll
        for (int r = 0; r < kEnds; ++r) {
            const int i = tid + r * (int)blockDim.x, m = min(i >> 4, n - 1);
            owner[r] = __shfl(token, min(m, TOK - 1));
            factor[r] = p.s_a[followed(owner[r]) ? owner[r] : 0];
            const int64_t at = (int64_t)(first + m) * width + tile * 16 + (i & 15);
            if (!GROUPED) residual[r] = *reinterpret_cast<const uint32_t *>(res + (!p.residual ? 0 : p.rdt == BITNET_DT_BF16 ? (at & ~1) * 2 : at * 4));
        }
    };
    float z[H][4];
    auto multiply = [&](int c0) {
        const int nb = min(NB, b1 - c0), o = min(l & (P - 1), nb * 8 - 1);
        int8_t *to = mine + (l / P) * kSlice + o * 16;
#pragma unroll
        for (int r = 0; r < kLoads; ++r)
            if (TOK % kTogether == 0 || r * kTogether + l / P < TOK) *reinterpret_cast<v4i *>(to + r * kTogether * kSlice) = x[r];
        const int8_t *op = mine + min(j, n - 1) * kSlice + g * 16;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            if (i < nb) {
                const v4i q0 = *reinterpret_cast<const v4i *>(op + i * 128), q1 = *reinterpret_cast<const v4i *>(op + i * 128 + 64);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    asm("" : "+v"(code[h][i].x), "+v"(code[h][i].y));  // decoded again in each pass, not kept four times as large across them
                    v4i c = mfma_i8(q0, decode16(code[h][i].x), v4i{0, 0, 0, 0});
                    c = mfma_i8(q1, decode16(code[h][i].y), c);
#pragma unroll
                    for (int e = 0; e < (TOK < 4 ? TOK : 4); ++e) z[h][e] = fmaf(scale[h][i], (float)c[e], z[h][e]);
                }
            }
            if (i & 1) __builtin_amdgcn_sched_barrier(0);
        }
    };

    // By expert the codes are asked for while the rows' indices are on their way; else the activations go first, so that they are in
    // LDS when the codes come.
    load_tokens();
    if (!GROUPED && !MULTI) load_x(b0);
    if (!MULTI) load_weights(b0);
    __builtin_amdgcn_sched_barrier(0);
    if (GROUPED && !MULTI) load_x(b0);
    load_ends();
    float bias[H];
#pragma unroll
    for (int h = 0; h < H; ++h) bias[h] = p.bias ? p.bias[(int64_t)t.expert * p.N + h * width + tile * 16 + j] : 0.0f;
    __builtin_amdgcn_sched_barrier(0);
    for (;;) {
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[h][e] = 0.0f;
        if constexpr (MULTI) {
            for (int c0 = b0; c0 < b1; c0 += NB) {
                load_x(c0);
                load_weights(c0);
                multiply(c0);
            }
        } else {
            multiply(b0);
        }
        // lane (g, j): tokens 4g .. 4g + 3 of row j
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int e = 0; e < (TOK < 4 ? TOK : 4); ++e) sums[((w * H + h) * 4 + e) * 64 + l] = z[h][e];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kEnds; ++r) {
            const int i = tid + r * (int)blockDim.x, m = i >> 4;
            if (m >= n || !followed(owner[r])) continue;
            const int at = (m & 3) * 64 + 16 * (m >> 2) + (i & 15);
            float y[H];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                float sum = 0.0f;
                for (int w4 = 0; w4 < a.waves; w4 += 4) {
                    float v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = sums[(min(w4 + k, a.waves - 1) * H + h) * 256 + at];
#pragma unroll
                    for (int k = 0; k < 4; ++k) sum += w4 + k < a.waves ? v[k] : 0.0f;
                }
                y[h] = sum * (factor[r] * 0.015625f) + bias[h];  // the block sums are those of 64 t
            }
            const int64_t to = (int64_t)(first + m) * width + tile * 16 + (i & 15);
            with_act(p.act, [&](auto act) {
                float v = activate<decltype(act)::value>(y[0]);
                if (GATED) v *= y[H - 1];
                if (!GROUPED && p.residual)
                    v += __uint_as_float(p.rdt != BITNET_DT_BF16 ? residual[r] : to & 1 ? residual[r] & 0xFFFF0000u : residual[r] << 16);
                if (p.ydt == BITNET_DT_BF16) static_cast<uint16_t *>(p.y)[to] = (uint16_t)bf16_pair(v, v);
                else static_cast<float *>(p.y)[to] = v;
            });
        }
        first += TOK;
        if (first >= t.end) break;
        __syncthreads();  // the sums of this pass are read
        load_tokens();
        if (!MULTI) load_x(b0);
        load_ends();
    }
}

// ==========================================================================
// Few rows each of many experts: more tiles of 16 rows than waves fit on the chip.  A workgroup of 4 waves brings up to 16 rows of its
// expert to LDS whole; then every wave runs through row tiles of its own, all of K each, a chunk of NB blocks in hand and the next one
// (of the next tile where this one ends) on its way, so that the stream of weights never pauses for a row's index, an activation
// or an epilogue.  An expert with more than 16 rows takes a pass over all its weights for each 16.
// ==========================================================================
struct StreamArgs {
    FusedArgs p;
    int tiles;  // row tiles of a wave
};

constexpr int kStreamTokens = 16;

template <bool GATED, int NB>
__global__ __launch_bounds__(256) void stream_kernel(StreamArgs a) {
    constexpr int H = GATED ? 2 : 1, TOK = kStreamTokens, Z = 4;
    const FusedArgs &p = a.p;
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, g = l >> 4, j = l & 15;
    const int blocks = p.K >> 7, all_tiles = p.N >> 4, width = GATED ? p.N >> 1 : p.N, row_bytes = p.K + 16;
    Tile t;
    if (!find_expert(p, blockIdx.y, &t)) return;
    // this wave's tiles: first + 4 i, i < count
    const int first_tile = (int)blockIdx.x * 4 * a.tiles + w, most = ((width >> 4) - first_tile + 3) >> 2;
    const int count = most < 0 ? 0 : min(most, a.tiles);
    const int chunks = (blocks + NB - 1) / NB, steps = count * chunks;

    struct Chunk {
        uint2 code[H][NB];
        float scale[H][NB];
    };
    auto fetch = [&](Chunk &x, int tile, int c) {  // chunk c of the wave's tile (past the end: its last)
        const int last = min(NB, blocks - c * NB) - 1;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int64_t brick = ((int64_t)t.expert * all_tiles + tile + h * (width >> 4)) * blocks + c * NB;
            const uint8_t *cp = p.packed + brick * kBrickBytes;  // the same for all lanes: a lane's part is a 32-bit offset
            const float *sp = p.scales + brick * kTileN;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const v2u v = __builtin_nontemporal_load(reinterpret_cast<const v2u *>(cp + min(i, last) * (int)kBrickBytes) + l);
                x.code[h][i] = make_uint2(v.x, v.y);
                x.scale[h][i] = __builtin_nontemporal_load(sp + min(i, last) * (int)kTileN + j);
            }
        }
    };

    for (int first = t.first; first < t.end; first += TOK) {
        const int n = min(TOK, t.end - first);
        Chunk x0, x1;
        int tile = first_tile, c = 0;        // of the chunk in hand
        int next_tile = tile, next_c = 0;    // of the chunk to fetch
        auto advance = [&](int &tt, int &cc) {
            if (++cc == chunks) cc = 0, tt += 4;
        };
        int token = first + min(l, n - 1);
        if (p.rows) token = p.rows[token];
        if (steps > 0) fetch(x0, tile, 0);
        __builtin_amdgcn_sched_barrier(0);
        const int safe = (uint32_t)token < (uint32_t)p.tokens ? token : 0;
        for (int m = w; m < n; m += 4) {  // a wave a row, 1 KB a load
            const int8_t *from = p.q + (int64_t)__builtin_amdgcn_readlane(safe, m) * p.K;
            for (int o = l * 16; o < p.K; o += 1024)
                *reinterpret_cast<v4i *>(smem + m * row_bytes + o) = *reinterpret_cast<const v4i *>(from + o);
        }
        int owner[Z];
        float factor[Z];
#pragma unroll
        for (int e = 0; e < Z; ++e) {
            const int m = 4 * g + e, row = __shfl(token, min(m, n - 1));
            const bool there = (uint32_t)row < (uint32_t)p.tokens;
            owner[e] = m < n && there ? row : -1;
            factor[e] = p.s_a[there ? row : 0] * 0.015625f;  // the block sums are those of 64 t
        }
        __syncthreads();

        float z[H][4];
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[h][e] = 0.0f;
        auto finish_tile = [&](int at_tile) {
            float bias[H];
#pragma unroll
            for (int h = 0; h < H; ++h) bias[h] = p.bias ? p.bias[(int64_t)t.expert * p.N + h * width + at_tile * 16 + j] : 0.0f;
            with_act(p.act, [&](auto act) {
#pragma unroll
                for (int e = 0; e < Z; ++e) {
                    float v = activate<decltype(act)::value>(z[0][e] * factor[e] + bias[0]);
                    if (GATED) v *= z[H - 1][e] * factor[e] + bias[H - 1];
                    if (owner[e] < 0) continue;
                    const int64_t to = (int64_t)(first + 4 * g + e) * width + at_tile * 16 + j;
                    if (p.ydt == BITNET_DT_BF16) static_cast<uint16_t *>(p.y)[to] = (uint16_t)bf16_pair(v, v);
                    else static_cast<float *>(p.y)[to] = v;
                }
            });
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[h][e] = 0.0f;
        };
        auto multiply = [&](const Chunk &x) {
            const int nb = min(NB, blocks - c * NB);
            const unsigned char *op = smem + min(j, n - 1) * row_bytes + c * NB * 128 + g * 16;
#pragma unroll
            for (int i = 0; i < NB; ++i)
                if (i < nb) {
                    const v4i q0 = *reinterpret_cast<const v4i *>(op + i * 128), q1 = *reinterpret_cast<const v4i *>(op + i * 128 + 64);
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        v4i s = mfma_i8(q0, decode16(x.code[h][i].x), v4i{0, 0, 0, 0});
                        s = mfma_i8(q1, decode16(x.code[h][i].y), s);
#pragma unroll
                        for (int e = 0; e < Z; ++e) z[h][e] = fmaf(x.scale[h][i], (float)s[e], z[h][e]);
                    }
                }
            if (c == chunks - 1) finish_tile(tile);
            advance(tile, c);
        };
        auto step = [&](const Chunk &x, Chunk &next) {
            advance(next_tile, next_c);
            fetch(next, next_tile, next_c);
            __builtin_amdgcn_sched_barrier(0);
            multiply(x);
        };
        // Every fetch stands in straight code: behind a branch the compiler would wait for it before the chunk in hand.
        for (int i = 1; steps > 0; ++i) {
            if (i == steps) {
                multiply(x0);
                break;
            }
            step(x0, x1);
            if (++i == steps) {
                multiply(x1);
                break;
            }
            step(x1, x0);
        }
        if (first + TOK < t.end) __syncthreads();  // the rows in LDS are read
    }
}

// Waves of a launch (64 experts of 2560 x 1280: 6 rows an expert 17.6 us, with 2048 19.3, with 8192 19.9; 12 rows 24.6, 28.9 and 26.0), and the
// tiles of 16 rows from which on it is used: as many as the chip holds workgroups of it.
constexpr int kStreamWaves = 4096, kStreamFrom = 1024;

template <bool GATED, int NB>
void launch_stream_nb(const StreamArgs &a, dim3 grid, size_t lds, hipStream_t stream) {
    hipLaunchKernelGGL((stream_kernel<GATED, NB>), grid, dim3(256), lds, stream, a);
}

template <bool GATED>
bool launch_stream(const FusedArgs &p, hipStream_t stream) {
    StreamArgs a{p, 1};
    const int tiles = (GATED ? p.N / 2 : p.N) / 16, some = p.experts < p.slots ? p.experts : p.slots;
    const size_t lds = (size_t)kStreamTokens * (p.K + 16);
    if (lds > 65536) return false;
    a.tiles = (int)(((int64_t)tiles * some + kStreamWaves - 1) / kStreamWaves);
    const dim3 grid((unsigned)((tiles + 4 * a.tiles - 1) / (4 * a.tiles)), (unsigned)some);
    // blocks a chunk: the fewest loads of blocks that are not there, then the longest
    const int blocks = p.K >> 7;
    constexpr int kLow = GATED ? 2 : 4, kHigh = kLow + 4;
    int best = kHigh, waste = blocks;
    for (int n = kHigh; n > kLow; --n) {
        const int over = (blocks + n - 1) / n * n - blocks;
        if (over < waste) waste = over, best = n;
    }
    if (best == kLow + 1) launch_stream_nb<GATED, kLow + 1>(a, grid, lds, stream);
    else if (best == kLow + 2) launch_stream_nb<GATED, kLow + 2>(a, grid, lds, stream);
    else if (best == kLow + 3) launch_stream_nb<GATED, kLow + 3>(a, grid, lds, stream);
    else launch_stream_nb<GATED, kLow + 4>(a, grid, lds, stream);
    return true;
}

constexpr int kMostLds = 163840, kCUs = 256;

int blocks_held(int per) { return per <= 2 ? 2 : per <= 4 ? 4 : per <= 8 ? per : 8; }  // of a wave's: the NB below

template <bool GATED, bool GROUPED, int TOK>
void launch_rows_tok(const RowsArgs &a, dim3 grid, hipStream_t stream) {
    const dim3 block(64 * a.waves);
    const size_t lds = (size_t)a.waves * (TOK * (blocks_held(a.per) * 128 + 16) + (GATED ? 2 : 1) * 1024);
#define BITNET_ROWS(NB, MULTI) hipLaunchKernelGGL((rows_kernel<GATED, GROUPED, NB, TOK, MULTI>), grid, block, lds, stream, a)
    switch (a.per) {
        case 1: case 2: BITNET_ROWS(2, false); return;
        case 3: case 4: BITNET_ROWS(4, false); return;
        case 5: BITNET_ROWS(5, false); return;
        case 6: BITNET_ROWS(6, false); return;
        case 7: BITNET_ROWS(7, false); return;
        case 8: BITNET_ROWS(8, false); return;
        default: BITNET_ROWS(8, true);
    }
#undef BITNET_ROWS
}
template <bool GATED, bool GROUPED>
void launch_rows(const RowsArgs &a, int tok, dim3 grid, hipStream_t stream) {
    if (tok == 1) launch_rows_tok<GATED, GROUPED, 1>(a, grid, stream);
    else if (tok == 4) launch_rows_tok<GATED, GROUPED, 4>(a, grid, stream);
    else if (tok == 8) launch_rows_tok<GATED, GROUPED, 8>(a, grid, stream);
    else launch_rows_tok<GATED, GROUPED, 16>(a, grid, stream);
}

void run_rows(const FusedArgs &p, int gated, hipStream_t stream) {
    RowsArgs a{p, 0, 0};
    const int blocks = p.K >> 7, tiles = (gated ? p.N / 2 : p.N) / 16;
    const int some = p.starts ? (p.experts < p.slots ? p.experts : p.slots) : 1;  // experts that can have rows
    const int64_t work = (int64_t)tiles * some;
    const int usual = (p.slots + some - 1) / some;
    // 64 experts of 2560 x 1280: 2 rows an expert 17.6 us against the rows kernel's 16.5, 6 rows 18.4 against 25.1, 12 rows 24.1 against 33.0;
    // 8 of 6912 x 2560: 4 rows 13.4 against 12.8, 8 rows 14.7 against 14.8.
    if (p.starts && usual > 4 && work >= kStreamFrom && (gated ? launch_stream<true>(p, stream) : launch_stream<false>(p, stream))) return;
    // Tokens of a pass: a pass reads them whether they are there or not, but two passes cost more than one of twice as many. 13824 x 2560 gated, in
    // passes of 1, 4, 8 and 16 tokens: 1 token 4.9, 5.2, 5.6, 6.2 us; 4 tokens 9.1, 5.2, 5.7, 6.2; 8 tokens 14.7, 7.0, 5.7, 6.4;
    // 12 tokens 20.3, 8.8, 8.0, 6.4.
    int tok = usual == 1 ? 1 : usual <= 4 ? 4 : usual <= 8 ? 8 : 16;
    auto over = [&](int n) { return (blocks + n - 1) / n; };
    // Waves in fours, so that the SIMDs have as many each, of 4 to 8 blocks: 8 x 13824 x 2560 gated 5.7 us with 4 waves, 6.1 with 3, 5.9 with 5,
    // 7.0 with 10; 8 x 20480 x 3200 7.9 with 4, 9.6 with 5, 9.2 with 7; 16 x 2560 x 6912 5.6 with 8, 7.0 with 4, 6.1 with 11.  Two for
    // short columns: 64 experts of 2560 x 1280 16.0 with 2, 20.8 with 4.
    //     From 64 blocks on the rule fits one token and not several: 1 x 2560 x 13824 6.2 us, with 4 waves in turns 8.6; 1 x 13824 x 11008 gated 12.5
    // and 14.0; but 8 x 13824 x 8192 gated 12.6 and 11.5, 16 x 13824 x 11008 gated 24.3 and 17.8, 16 x 5120 x 13824 27.6 and 15.2, since
    // from 65 on 16 tokens of 9 to 12 waves do not fit in LDS and every product is done in passes of 8.
    a.waves = blocks > 12 ? min((over(8) + 3) / 4 * 4, kMostWaves) : blocks > 3 ? 2 : 1;
    a.per = over(a.waves);
    a.waves = over(a.per);
    // All of LDS for tokens, even where it leaves one workgroup a CU: 16 x 2560 x 6912 5.6 us (141 KB), in passes of 8 tokens 7.0; 16 x 13824 x
    // 8192 gated 14.3 and 21.1.
    while (tok > 4 && a.waves * (tok * (blocks_held(a.per) * 128 + 16) + (gated ? 2 : 1) * 1024) > kMostLds) tok >>= 1;
    const dim3 grid((unsigned)tiles, (unsigned)some);
    if (p.starts) gated ? launch_rows<true, true>(a, tok, grid, stream) : launch_rows<false, true>(a, tok, grid, stream);
    else gated ? launch_rows<true, false>(a, tok, grid, stream) : launch_rows<false, false>(a, tok, grid, stream);
}

// Whether the tiles of w2a8_tiles.hip take it.
//     By expert (rows or stream against tiles): 12 rows, 64 experts of 2560 x 1280 24.1 us against 31.6, 24 rows 39.8 against 34.4; 16 rows, 8 experts
// of 6912 x 2560 22.6 against 20.4, of 2560 x 6912 32.5 against 32.6, 32 rows 30.8 against 26.9 and 46.3 against 33.1.  The host knows
// the mean alone, and these are even plans.  Where one expert has most of the rows its passes of 16 follow one another: 900 rows to 64
// experts of 2560 x 1280 19.4 us, with 100 of them at one expert 63, 225 122, 450 229; 128 rows to 8 of 6912 x 2560 14.4, with 64 at one
// 38, 120 70.
//     Else by passes of 16 tokens and tiles of 16 rows a CU, which is what rows cost, while tiles of this few tokens take the time of one chain over
// K: 2560 x 2560 64 tokens 9.5 us against 17.0, 128 17.0 against 17.5; 13824 x 2560 gated 64 15.7 against 17.0, 80 18.3 against 16.8; 20480 x
// 3200 32 17.9 against 19.4, 40 24.8 against 19.7; 65536 x 2560 32 37.4 against 23.2; 2560 x 6912 128 26.7 against 31.8.  Where neither form suits,
// bitnet_w2a8_gemm, which has no epilogue, is the faster product: 13824 x 2560 from 40 to 128 tokens, narrow matrices to 512.
bool many(int64_t slots, int experts, bool grouped, int N) {
    if (grouped) return slots > 16ll * experts;
    const int64_t passes = (slots + 15) / 16;
    return passes > 1 && passes * max(N / 16, 2 * kCUs) > 14 * kCUs;
}

bitnet_status_t run(const FusedArgs &p, int gated, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (many(p.slots, p.experts, p.starts, p.N)) {
        if (!at(workspace, 16) || workspace_bytes < digits_bytes(p.tokens, p.K)) return BITNET_ERR_INVALID_ARG;
        return launch_tiles(p, gated, workspace, stream);
    }
    run_rows(p, gated, stream);
    return launched();
}

constexpr int kMostRows = 1 << 24;  // tokens and slots
constexpr int kMostK = 1 << 24;     // offsets inside 16 rows of weights in 32 bits
constexpr int64_t kMostWeights = (int64_t)1 << 34;  // of a matrix: scales' offsets in 32 bits, row tiles in a launch's size

bool float_type(int dt) { return dt == BITNET_DT_BF16 || dt == BITNET_DT_F32; }

bitnet_status_t check(const FusedArgs &p, int gated) {
    if (!at(p.packed, 16) || !at(p.scales, 16) || !at(p.q, 16) || !at(p.s_a, 4) || (p.bias && !at(p.bias, 16)) ||
        (p.residual && (!at(p.residual, 16) || !float_type(p.rdt))) || !at(p.y, 16) || !float_type(p.ydt) ||
        p.act < BITNET_ACT_NONE || p.act > BITNET_ACT_GELU || (p.residual == p.y && p.rdt != p.ydt))
        return BITNET_ERR_INVALID_ARG;
    if (bitnet_check_shape(p.N, p.K) != BITNET_OK || (gated && p.N % 32) || p.K > kMostK || (int64_t)p.N * p.K > kMostWeights)
        return BITNET_ERR_UNSUPPORTED_SHAPE;
    return BITNET_OK;
}

}  // namespace

extern "C" {

size_t bitnet_w2a8_linear_workspace_bytes(int M, int N, int K) {
    return M < 1 || bitnet_check_shape(N, K) != BITNET_OK || !many(M, 1, false, N) ? 0 : digits_bytes(M, K);
}

bitnet_status_t bitnet_w2a8_linear(const uint8_t *packed, const float *scales, const int8_t *q, const float *s_a,
                                   const float *bias, int act, int gated, const void *residual, int rdt, void *y,
                                   int ydt, int M, int N, int K, void *workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
    const FusedArgs p{packed, scales, s_a, bias, q, residual, y, nullptr, nullptr, act, rdt, ydt, M, M, 1, N, K};
    const bitnet_status_t st = check(p, gated);
    if (st != BITNET_OK) return st;
    if (M < 1 || M > kMostRows) return BITNET_ERR_UNSUPPORTED_SHAPE;
    return run(p, gated, workspace, workspace_bytes, stream);
}

size_t bitnet_w2a8_grouped_workspace_bytes(int tokens, int slots, int experts, int N, int K) {
    return tokens < 1 || slots < 1 || experts < 1 || bitnet_check_shape(N, K) != BITNET_OK || !many(slots, experts, true, N) ? 0 : digits_bytes(tokens, K);
}

bitnet_status_t bitnet_w2a8_grouped(const uint8_t *packed, const float *scales, const int8_t *q, const float *s_a,
                                    int tokens, const int32_t *starts, const int32_t *rows, int experts, int slots,
                                    const float *bias, int act, int gated, void *y, int ydt, int N, int K,
                                    void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const FusedArgs p{packed, scales, s_a, bias, q, nullptr, y, starts, rows, act, 0, ydt, tokens, slots, experts, N, K};
    const bitnet_status_t st = check(p, gated);
    if (st != BITNET_OK) return st;
    if (!at(starts, 4) || (rows && !at(rows, 4))) return BITNET_ERR_INVALID_ARG;
    if (experts < 1 || experts > 1024 || slots < 1 || slots > kMostRows || tokens < 1 || tokens > kMostRows || (!rows && tokens < slots))
        return BITNET_ERR_UNSUPPORTED_SHAPE;
    return run(p, gated, workspace, workspace_bytes, stream);
}

}  // extern "C"
