// Library-internal parts of the products with epilogues: arguments, activations, decoding, and which token tile of which expert a
// workgroup has.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "attention.h"
#include "bitnet_w2a8.h"
#include "layout.h"

namespace bitnet_fused {

using namespace bitnet_attn;
using namespace bitnet_layout;

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

// A NaN stays one.
template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == BITNET_ACT_RELU) return z < 0.0f ? 0.0f : z;
    if constexpr (ACT == BITNET_ACT_RELU2) return z < 0.0f ? 0.0f : z * z;
    if constexpr (ACT == BITNET_ACT_SILU) return z / (1.0f + __expf(-z));
    if constexpr (ACT == BITNET_ACT_GELU) {
        const float u = 1.5957691216057308f * (z + 0.044715f * z * z * z);  // 2 sqrt(2 / pi) ...
        return z / (1.0f + __expf(-u));
    }
    return z;
}

// f(the activation as a type): one branch around an epilogue.  A branch at each value made the epilogue of a 64 x 256 tile 3.5 us long
// where it now takes 1.4.
template <int ACT>
struct Act {
    static constexpr int value = ACT;
};
template <typename F>
__device__ __forceinline__ void with_act(int act, F &&f) {
    switch (act) {
        case BITNET_ACT_RELU: return f(Act<BITNET_ACT_RELU>());
        case BITNET_ACT_RELU2: return f(Act<BITNET_ACT_RELU2>());
        case BITNET_ACT_SILU: return f(Act<BITNET_ACT_SILU>());
        case BITNET_ACT_GELU: return f(Act<BITNET_ACT_GELU>());
        default: return f(Act<BITNET_ACT_NONE>());
    }
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

// The `rank`-th expert that has any rows, and all its slots.  By ballots and counts of bits: a scan by shuffles made a product of one
// token with 2 of 8 experts 6.3 us long instead of 5.6.
__device__ __forceinline__ bool find_expert(const FusedArgs &p, int rank, Tile *out) {
    const int lane = threadIdx.x & 63;
    for (int e0 = 0; e0 < p.experts; e0 += 64) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < p.experts) {
            lo = min(max(p.starts[e], 0), p.slots);
            hi = min(max(p.starts[e + 1], lo), p.slots);
        }
        const uint64_t some = __ballot(hi > lo);
        const int n = __popcll(some);
        if (rank < n) {
            const uint64_t who = __ballot(hi > lo && __popcll(some & ((1ull << lane) - 1)) == rank);
            const int at = __ffsll((unsigned long long)who) - 1;
            *out = {e0 + at, __builtin_amdgcn_readlane(lo, at), __builtin_amdgcn_readlane(hi, at)};
            return true;
        }
        rank -= n;
    }
    return false;
}

// Token tiles of `rows` slots that a launch has to provide for: an expert with rows ends in a tile that may not be full.
inline int64_t token_tiles(const FusedArgs &p, int rows) {
    if (!p.starts) return ((int64_t)p.slots + rows - 1) / rows;
    const int some = p.experts < p.slots ? p.experts : p.slots;
    return ((int64_t)p.slots + (int64_t)some * (rows - 1)) / rows;
}

// The products of many rows (w2a8_tiles.hip): bytes of the activations' digits, and the launches.
size_t digits_bytes(int tokens, int K);
bitnet_status_t launch_tiles(const FusedArgs &p, int gated, void *digits, hipStream_t stream);

}  // namespace bitnet_fused
