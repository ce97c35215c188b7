// Products with epilogues over many rows, on the matrix cores' 6-bit and 4-bit formats.
//
// An int8 activation is two digits, q = 16 h + l with -8 <= h, l <= 8.  The 6-bit format (3 exponent, 2 mantissa bits) holds the upper
// digit as h and the lower one as l / 16, both exactly, so that their sum is q / 16; a ternary weight t is the 4-bit float 2 t, whose two
// upper bits are its 2-bit code.  One 32x32x64 step in mixed formats, without scale operands, multiplies 32 tokens by 32 rows over 64
// columns, and the steps of both digits add up to sums of q t / 8, which the epilogue multiplies by 8.  Eight times a block's sum is a
// whole number below 2^24, so block sums are exact in fp32 and come out the same as int8
// products' (checked bit for bit), at the same rate as int8.  What it saves is everything beside the matrix cores: a block
// sum needs no conversion before its scale (one fused multiply-add an output and block instead of two operations), 16 codes
// become operands in three operations instead of seven, and the 32 x 32 shape leaves a wave room for 4 to 6 vector operations
// under every step where the 16 x 16 shape leaves 2 under each of twice as many.
//
// The digits are made once a call by a small kernel of their own: 1.5 bytes a value, in the order in which the codes of the tile
// layout come out of their words.
//
// Measured, digits and products together: 8192 tokens x 6912 x 2560, gated, 165 to 175 us, 1.66 to 1.76 POP/s (the plain product's
// kernel 192 to 198 us; a large int8 library product runs at 2.55 POP/s); 512 x 13824 x 2560 30 us (30), 256
// tokens 19.5 (21.7).  Four steps a 32 x 32 block, two digits each of two halves, are what int8 takes too.  What bounds it with many tiles is
// that its parts overlap too little, no unit being full: of the cycles in which a CU has work (4095 tokens by expert) the matrix cores
// are busy in 48%, the vector units in 54% (matrix steps' issue among them), LDS's reads and writes in 28% (direct loads not counted, no
// bank conflicts); a wave waits for its turn in 32% of its time and for data or the barrier in 24%.  Each block begins with a barrier and 18 LDS
// reads before its first step.  A step that takes 14.3 ns with 32 workgroups on the card takes 20 to 23 with all 512, which with 4420 steps
// a SIMD is 88 to 102 of the products' 170 us.  With few tiles it is one workgroup's chain of blocks, prologue and
// epilogue (1.4 us).  Raising waves' priorities in turn, touching the weights' lines ahead and parting the
// direct loads among the steps changed nothing.
#include "fused.h"

using namespace bitnet_fused;

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v12i __attribute__((ext_vector_type(12)));

constexpr int kDigitRow = 192;  // bytes of the digits of one token and block: [64-column step][half][upper digits 24][lower 24]

// --------------------------------------------------------------------------------------------- digits
// Four digits of 6 bits from four int8 values: a sign and the code of 0 .. 8 (0, 12, 16, 18, 20, 21, 22, 23, 24) or, for the lower
// digit, of its 16th (0 .. 8: the codes are the numbers themselves, below the smallest normal number and just above it).
__device__ __forceinline__ uint32_t pick(uint32_t index, uint32_t t0, uint32_t t1, uint32_t t2, uint32_t t3) {
    const uint32_t sel = index & 0x07070707u;
    const uint32_t ones = (index >> 3) & 0x01010101u, mask = (ones << 8) - ones;
    const uint32_t a = __builtin_amdgcn_perm(t1, t0, sel), b = __builtin_amdgcn_perm(t3, t2, sel);
    return (a & ~mask) | (b & mask);
}
__device__ __forceinline__ uint32_t squeeze(uint32_t c) {  // 6 bits of every byte, side by side
    const uint32_t u = (c & 0x003F003Fu) | ((c & 0x3F003F00u) >> 2);
    return (u & 0xFFFu) | ((u >> 4) & 0xFFF000u);
}
__device__ __forceinline__ uint32_t lower4(uint32_t q) {
    return squeeze(pick(q, 0x03020100u, 0x07060504u, 0x25262728u, 0x21222324u));
}
__device__ __forceinline__ uint32_t upper4(uint32_t q) {  // (q + 8) >> 4; its sign is that of q, or it is zero
    const uint32_t h = ((q >> 4) & 0x0F0F0F0Fu) + ((q >> 3) & 0x01010101u);
    return squeeze(pick(h, 0x12100C00u, 0x17161514u, 0x15161718u, 0x0C101214u) | ((q >> 2) & 0x20202020u));
}

// One lane: 32 columns of a token.  Column order, in every 16: that of the codes' nibbles in a word, 0 8 1 9 2 10 3 11, 4 12 ...
// The 48 bytes of a lane go through LDS, so that a wave stores whole kilobytes (4001 x 2560 x 2560 as a whole 51.7 us instead of 55.7).
__global__ __launch_bounds__(256) void digits_kernel(const int8_t *__restrict__ q, uint8_t *__restrict__ out, int64_t pieces) {
    __shared__ uint4 s_out[256 * 3];
    const int64_t first = (int64_t)blockIdx.x * 256, i = min(first + threadIdx.x, pieces - 1);
    const uint4 x[2] = {reinterpret_cast<const uint4 *>(q)[2 * i], reinterpret_cast<const uint4 *>(q)[2 * i + 1]};
    uint32_t d[12];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint32_t v[4] = {__builtin_amdgcn_perm(x[half].z, x[half].x, 0x05010400u), __builtin_amdgcn_perm(x[half].z, x[half].x, 0x07030602u),
                               __builtin_amdgcn_perm(x[half].w, x[half].y, 0x05010400u), __builtin_amdgcn_perm(x[half].w, x[half].y, 0x07030602u)};
#pragma unroll
        for (int digit = 0; digit < 2; ++digit) {
            uint32_t g[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) g[k] = digit ? lower4(v[k]) : upper4(v[k]);
            uint32_t *to = d + 6 * digit + 3 * half;
            to[0] = g[0] | (g[1] << 24);
            to[1] = (g[1] >> 8) | (g[2] << 16);
            to[2] = (g[2] >> 16) | (g[3] << 8);
        }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) s_out[3 * threadIdx.x + k] = make_uint4(d[4 * k], d[4 * k + 1], d[4 * k + 2], d[4 * k + 3]);
    __syncthreads();
    uint4 *to = reinterpret_cast<uint4 *>(out) + 3 * first;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int at = 256 * k + threadIdx.x;
        if (first * 3 + at < pieces * 3) to[at] = s_out[at];
    }
}

// --------------------------------------------------------------------------------------------- tiles
// A workgroup of 4 waves: 64 tokens x 256 weight rows (gated: 128 gate rows and the 128 up rows of the same outputs); a wave has all
// tokens and 64 rows, as 2 x 2 products of 32 x 32.  Two workgroups share a CU: while one waits (at its barrier, for LDS, in its
// prologue or epilogue) the other has the matrix cores.  Every block of 128 columns is brought to LDS by direct loads, two
// blocks ahead.  Digits lie there as 12 pieces of 16 bytes a token, piece i of token t at (i + t / 4) mod 12, which spreads 16 tokens'
// reads over all banks.  A wave works on one of its two row tiles at a time: under each of the 8 steps of it, it drains four sums
// of the other (finished) row tile into fp32 with their scale, and makes words of that row tile's weights.
// KS = 2, where the tiles are no more than the CUs: one workgroup of 8 waves a CU, the second four take every other block and
// their sums are added once at the end (512 x 2560 x 6912 35.6 us instead of 39.6, 64 x 13824 x 2560 gated
// 16.7 instead of 17.7).  With more tiles than CUs the two workgroups of a CU are that already.
constexpr int kThreads = 256, kStages = 3, kTokens = 64;
constexpr int kDigitStage = kTokens * kDigitRow, kWeightStage = 16 * 512, kScaleStage = 16 * 16 * 4;
constexpr int kStage = kDigitStage + kWeightStage + kScaleStage;
constexpr int kCUs = 256;
constexpr int kBand = 4;  // token tiles that share the rows' tiles (4001 x 2560 x 2560: 53.6 us, with 8 56.3, 16 56.7; 8192 x 6912 x 2560: 173, 178, 180)

// 16 bytes a lane from base + offset into LDS at lds + 16 * lane, the next kilobyte of LDS for each further load; M0 carries the
// LDS address and is restored.
__device__ __forceinline__ void dma3(const void *base, const uint32_t (&off)[3], uint32_t lds) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %5, %4\n\t"
        "s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %6, %4\n\t"
        "s_mov_b32 m0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %7, %4\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(lds), "s"(lds + 1024), "s"(lds + 2048), "s"(base), "v"(off[0]), "v"(off[1]), "v"(off[2])
        : "memory");
}
__device__ __forceinline__ void dma1(const void *base, uint32_t off, uint32_t lds) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %3, %2\n\ts_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(__builtin_amdgcn_readfirstlane(lds)), "s"(base), "v"(off)
        : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <bool GATED, int KS>
__global__ __launch_bounds__(kThreads * KS, 2) void tiles_kernel(FusedArgs p, const uint8_t *__restrict__ digits, int row_tiles, int token_tiles) {
    constexpr int kCols = GATED ? 128 : 256;        // outputs of a token
    constexpr int kRow = kCols + 4;                 // floats from token to token of the output tile in LDS
    extern __shared__ __align__(1024) unsigned char all_lds[];
    __shared__ float s_sa[kTokens];

    // Workgroups go to the eight dies in turn; each die takes a run of tiles, and in a run kBand token tiles share every
    // tile of rows, so that a die's L2 holds what its workgroups read together.
    const int G = gridDim.x, die = blockIdx.x & 7, each = G >> 3, more = G & 7;
    const int t = die * each + min(die, more) + ((int)blockIdx.x >> 3);
    const int band = t / (kBand * row_tiles), in_band = t - band * kBand * row_tiles;
    const int band_tiles = min(kBand, token_tiles - band * kBand);
    const int tn = in_band / band_tiles;
    Tile tile;
    if (!find_tile(p, band * kBand + in_band % band_tiles, kTokens, &tile)) return;

    const int tid = threadIdx.x, l = tid & 63;
    const int all_w = __builtin_amdgcn_readfirstlane(tid >> 6), w = all_w & 3, part = all_w >> 2;
    unsigned char *lds = all_lds + part * kStages * kStage;  // of this part of K
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
    const int half = l >> 5, col = l & 31;
    const int blocks = p.K >> 7, all_tiles = p.N >> 4;

    // sources of this wave's direct loads
    uint32_t from[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int at = (3 * w + i) * 64 + l;  // 16-byte piece of the stage
        const int row = at / 12, piece = (at % 12 - ((row >> 2) & 3) + 12) % 12;
        const int slot = min(tile.first + row, tile.end - 1);
        int token = p.rows ? p.rows[slot] : slot;
        token = token < 0 || token >= p.tokens ? 0 : token;  // its row is not written
        from[i] = (uint32_t)token * (uint32_t)(blocks * kDigitRow) + piece * 16;  // digits of a call stay below 4 GiB
    }
    // 16-row tile of a stage's slot: the wave's two row tiles of 32 lie in slots 4 w .. 4 w + 3
    auto row_tile = [&](int slot) {
        if (GATED) {
            const int i = min(tn * 8 + (slot >> 2) * 2 + (slot & 1), (all_tiles >> 1) - 1);
            return i + (slot & 2 ? all_tiles >> 1 : 0);
        }
        return min(tn * 16 + slot, all_tiles - 1);
    };
    const int64_t expert_tiles = (int64_t)tile.expert * all_tiles;
    const uint8_t *weights[2];  // of the first of two row tiles each; the second one (the upper half of the lanes) lies behind it or is it
    uint32_t weights_at[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int first = row_tile(4 * w + 2 * i), second = row_tile(4 * w + 2 * i + 1);
        weights[i] = p.packed + (expert_tiles + first) * blocks * kBrickBytes;
        weights_at[i] = (uint32_t)(half * (second - first) * blocks * (int)kBrickBytes + col * 16);
    }
    const float *scales = p.scales + (expert_tiles + row_tile(4 * w)) * blocks * kTileN;
    const uint32_t scales_at = (uint32_t)(row_tile(4 * w + ((l >> 2) & 3)) - row_tile(4 * w)) * (uint32_t)(blocks * (int)kTileN * 4) + (l & 3) * 16;  // N K <= 2^34

    auto issue = [&](int i, int stage) {  // this wave's loads of its i-th block (past the last: the last again)
        const int bb = min(KS * i + part, blocks - 1);
        const uint32_t st = lds0 + (uint32_t)(stage * kStage);
        dma3(digits + (int64_t)bb * kDigitRow, from, st + 3 * w * 1024);
#pragma unroll
        for (int k = 0; k < 2; ++k) dma1(weights[k] + (int64_t)bb * kBrickBytes, weights_at[k], st + kDigitStage + (2 * w + k) * 1024);
        if (l < 16) dma1(scales + (int64_t)bb * kTileN, scales_at, st + kDigitStage + kWeightStage + w * 256);
    };
    constexpr int kLoads = 6;

    float y[2][2][16];
    v16f c[2][2];
    float sc[2] = {0.0f, 0.0f};
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) y[a][b][e] = 0.0f, c[a][b][e] = 0.0f;
    v12i ao[2][2];         // digits of 32 tokens [token tile][step]: upper 6 words, lower 6
    v4i bw[2][2];          // weights [row tile][step]
    uint2 wr[2][2];        // packed words [row tile][16 columns of the half], both steps

    uint32_t piece_at[2][3];  // of this lane's token
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int k = 0; k < 3; ++k) piece_at[s][k] = (uint32_t)(col * 12 + ((2 * s + half) * 3 + k + ((col >> 2) & 3)) % 12) * 16;
    auto read_ao = [&](const unsigned char *base, int s) {
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) {
            const v4i x0 = *reinterpret_cast<const v4i *>(base + piece_at[s][0] + ti * 32 * kDigitRow);
            const v4i x1 = *reinterpret_cast<const v4i *>(base + piece_at[s][1] + ti * 32 * kDigitRow);
            const v4i x2 = *reinterpret_cast<const v4i *>(base + piece_at[s][2] + ti * 32 * kDigitRow);
            ao[ti][s] = __builtin_shufflevector(__builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7), __builtin_shufflevector(x2, x2, 0, 1, 2, 3, -1, -1, -1, -1),
                                                0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11);
        }
    };
    auto read_wr = [&](const unsigned char *base, int tj) {
        const unsigned char *at = base + kDigitStage + (4 * w + 2 * tj + (col >> 4)) * 512 + (32 * half + (l & 15)) * 8;
        wr[tj][0] = *reinterpret_cast<const uint2 *>(at);
        wr[tj][1] = *reinterpret_cast<const uint2 *>(at + 128);
    };
    auto read_sc = [&](const unsigned char *base, int tj) {
        return *reinterpret_cast<const float *>(base + kDigitStage + kWeightStage + ((4 * w + 2 * tj) * 16 + col) * 4);
    };
    auto decode = [&](int tj, int i) {  // word i & 3 of step i >> 2
        const uint32_t x = i >> 2 ? wr[tj][(i >> 1) & 1].y : wr[tj][(i >> 1) & 1].x;
        bw[tj][i >> 2][i & 3] = (int)((i & 1 ? x : x << 2) & 0xCCCCCCCCu);
    };
    auto step = [&](int ti, int tj, int s, int digit) {
        v12i &a = ao[ti][s];
        if (tj == 0 && digit == 0) asm("" : "+v"(a));  // twelve registers in a row: the loads' own, not copies for each digit
        const v4i b = bw[tj][s];
        const v8i a8 = digit ? __builtin_shufflevector(a, a, 6, 7, 8, 9, 10, 11, -1, -1) : __builtin_shufflevector(a, a, 0, 1, 2, 3, 4, 5, -1, -1);
        const v8i b8 = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
        const v16f zero = {};
        // operands: 6-bit (format 3) tokens as rows, 4-bit (format 4) weights as columns; scale operands of 0 are the instruction without any
        c[ti][tj] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, s == 0 && digit == 0 ? zero : c[ti][tj], 3, 4, 0, 0, 0, 0);
    };
    // The 8 steps of row tile tj, and what goes under them: the other row tile's drain, and (tj = 0) its weights.
    auto work = [&](int tj) {
        const int o = 1 - tj;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            step(k & 1, tj, k >> 2, (k >> 1) & 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int dt = k >> 2, de = 4 * (k & 3) + e;
                y[dt][o][de] = fmaf(sc[o], c[dt][o][de], y[dt][o][de]);
            }
            if (tj == 0) decode(1, k);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    issue(0, 0);
    issue(1, 1);
    // The barrier at the top of a block publishes its stage (every wave has waited for its own loads of it) and frees the stage of the
    // block before for the next but one: every read of that stage has been waited for.
    auto block = [&](int i, int stage) {  // stage = i % kStages, a constant where it is called: LDS addresses are then all immediate
        wait_loads_barrier<kLoads>();
        issue(i + 2, (stage + 2) % kStages);
        if (KS > 1 && KS * i + part >= blocks) return;  // the last turn, an odd block in the other part
        const unsigned char *base = lds + stage * kStage;
        read_wr(base, 0);
        read_ao(base, 0);
        read_wr(base, 1);
        sc[0] = read_sc(base, 0);
        const float sc1 = read_sc(base, 1);
        read_ao(base, 1);
#pragma unroll
        for (int k = 0; k < 8; ++k) decode(0, k);
        work(0);
        sc[1] = sc1;
        work(1);
    };
    const int turns = (blocks + KS - 1) / KS;
    for (int i = 0;;) {
        block(i, 0);
        if (++i == turns) break;
        block(i, 1);
        if (++i == turns) break;
        block(i, 2);
        if (++i == turns) break;
    }
#pragma unroll
    for (int ti = 0; ti < 2; ++ti)
#pragma unroll
        for (int e = 0; e < 16; ++e) y[ti][1][e] = fmaf(sc[1], c[ti][1][e], y[ti][1][e]);

    // Epilogue: a lane has rows col of its two row tiles and 16 tokens of each 32; through LDS to whole rows of outputs.
    if (tid < kTokens) {
        const int slot = min(tile.first + tid, tile.end - 1);
        const int token = p.rows ? p.rows[slot] : slot;
        s_sa[tid] = token < 0 || token >= p.tokens ? 0.0f : p.s_a[token];
    }
    wait_loads_barrier<0>();
    if constexpr (KS > 1) {  // the second part's sums join the first's
        float *sums = reinterpret_cast<float *>(all_lds) + (tid & 255);
        if (part) {
#pragma unroll
            for (int i = 0; i < 64; ++i) sums[i * 256] = y[i >> 5][(i >> 4) & 1][i & 15];
        }
        wait_loads_barrier<0>();
        if (!part) {
#pragma unroll
            for (int i = 0; i < 64; ++i) y[i >> 5][(i >> 4) & 1][i & 15] += sums[i * 256];
        }
        wait_loads_barrier<0>();
    }
    float *out = reinterpret_cast<float *>(all_lds);
    const int width = GATED ? p.N >> 1 : p.N;
    float bias[2] = {0.0f, 0.0f};
    if (p.bias) {
#pragma unroll
        for (int tj = 0; tj < 2; ++tj) bias[tj] = p.bias[(int64_t)tile.expert * p.N + row_tile(4 * w + 2 * tj + (col >> 4)) * 16 + (l & 15)];
    }
    if (KS == 1 || !part) with_act(p.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
#pragma unroll
        for (int ti = 0; ti < 2; ++ti)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int row = ti * 32 + 8 * (e >> 2) + 4 * half + (e & 3);
                const float f = s_sa[row] * 8.0f;  // the block sums are those of (q / 16) (2 t)
                const float z0 = y[ti][0][e] * f + bias[0], z1 = y[ti][1][e] * f + bias[1];
                float *at = out + row * kRow;
                if (GATED) {
                    at[w * 32 + col] = activate<ACT>(z0) * z1;
                } else {
                    at[w * 64 + col] = activate<ACT>(z0);
                    at[w * 64 + 32 + col] = activate<ACT>(z1);
                }
            }
    });
    wait_loads_barrier<0>();
    constexpr int kPieces = kCols / 8;
#pragma unroll 4
    for (int i = tid; i < kTokens * kPieces; i += kThreads * KS) {
        const int row = i / kPieces, n = tn * kCols + (i % kPieces) * 8, slot = tile.first + row;
        if (slot >= tile.end || n >= width) continue;
        if (p.rows) {
            const int token = p.rows[slot];
            if (token < 0 || token >= p.tokens) continue;
        }
        float v[8];
        load8(out + row * kRow + (i % kPieces) * 8, v);
        const int64_t at = (int64_t)slot * width + n;
        if (p.residual) {
            float r[8];
            if (p.rdt == BITNET_DT_BF16) load8(static_cast<const uint16_t *>(p.residual) + at, r);
            else load8(static_cast<const float *>(p.residual) + at, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += r[e];
        }
        if (p.ydt == BITNET_DT_BF16) store8(static_cast<uint16_t *>(p.y) + at, v);
        else store8(static_cast<float *>(p.y) + at, v);
    }
}

template <bool GATED>
bitnet_status_t launch(const FusedArgs &p, const uint8_t *digits, hipStream_t stream) {
    const int64_t tiles = token_tiles(p, kTokens);
    const int row_tiles = (p.N + 255) / 256;
    constexpr int out_bytes = kTokens * ((GATED ? 128 : 256) + 4) * 4, stages = kStages * kStage;
    const dim3 grid((unsigned)(tiles * row_tiles));
    if (tiles * row_tiles <= kCUs) hipLaunchKernelGGL((tiles_kernel<GATED, 2>), grid, dim3(2 * kThreads), 2 * stages, stream, p, digits, row_tiles, (int)tiles);
    else hipLaunchKernelGGL((tiles_kernel<GATED, 1>), grid, dim3(kThreads), out_bytes > stages ? out_bytes : stages, stream, p, digits, row_tiles, (int)tiles);
    return launched();
}

}  // namespace

namespace bitnet_fused {

size_t digits_bytes(int tokens, int K) { return (size_t)tokens * (size_t)(K / 128) * kDigitRow; }

bitnet_status_t launch_tiles(const FusedArgs &p, int gated, void *digits, hipStream_t stream) {
    const int64_t pieces = (int64_t)p.tokens * (p.K / 32);
    if ((int64_t)p.tokens * p.K > INT32_MAX) return BITNET_ERR_UNSUPPORTED_SHAPE;  // 1.5 bytes a value: offsets in 32 bits
    if (token_tiles(p, kTokens) * (((int64_t)p.N + 255) / 256) > (1 << 23)) return BITNET_ERR_UNSUPPORTED_SHAPE;  // the launch's work items in 32 bits
    hipLaunchKernelGGL(digits_kernel, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, stream, p.q, static_cast<uint8_t *>(digits), pieces);
    return gated ? launch<true>(p, static_cast<const uint8_t *>(digits), stream) : launch<false>(p, static_cast<const uint8_t *>(digits), stream);
}

}  // namespace bitnet_fused
