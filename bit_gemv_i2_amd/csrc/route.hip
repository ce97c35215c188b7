// The experts of each token and the plan that sorts tokens by expert, on the device alone.
//
// A group of G lanes holds the logits of a token, a lane VPL neighbouring ones, as whole numbers in the order of the
// floats (0: never chosen).  The k largest are taken one after the other: the largest of the group, the lowest lane that
// holds it, which strikes it out.  Neighbours in a lane and the lowest lane make ties go to the lowest expert.
//
// The floor is one read of the logits, the outputs and a launch (16383 x 128 in bf16, 8 chosen: 6.3 MB, 1 us, and a second launch).
// What bounds it there, 11.3 and 7.2 us, is latency: 64 tokens of 8 lanes leave half of a workgroup's waves without a token, a lane's
// 16 logits are 16 loads of 2 bytes, and a round waits for the one before.  Waves wait in 83% of their time in the choosing kernel and
// in 60% in the placing one; the vector units are busy in 38% and 60%.  With few tokens it is the same chain of k rounds and a plan
// of three dependent steps.
//
// The plan is a counting sort.  64 tokens at a time: every expert has a 64-bit mask of the tokens that chose it, so
// that an assignment's place among them is the count of the lower bits: the same plan whatever the order of the
// atomics that set the bits.  Up to kOneLaunch tokens one workgroup does it all; more tokens take a second launch,
// in which every workgroup adds up what the others counted.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "attention.h"
#include "bitnet_w2a8.h"

using namespace bitnet_attn;

namespace {

constexpr int kThreads = 1024;
constexpr int kMaxExperts = 1024, kMaxChosen = 32;
constexpr int kSub = 64;          // tokens of a mask
// Tokens up to which one workgroup does all (64 experts, 6 of them: 64 tokens 7.0 us, 128 10.4, 256 16.1; in two launches 65 to 512
// tokens take 9.4 us, but a second call's time on the host).
constexpr int kOneLaunch = 128;
constexpr int kEach = 64;         // tokens of a workgroup, at least, of the two-launch form (16383 tokens, 8 of 128: 17.9 us; 128: 21.8)
constexpr int kMostBlocks = 256;  // workgroups of the two-launch form

struct RouteArgs {
    const void *logits;
    int64_t row_stride;
    int tokens, experts, k, over_all, per_block;  // per_block: tokens of a workgroup
    int32_t *chosen, *starts, *rows, *slots, *counts;
    float *gates;
};

struct Plan {
    uint64_t mask[kMaxExperts];
    int base[kMaxExperts], total[kMaxExperts];
    int wave[kThreads / 64];
};

__device__ __forceinline__ float as_float(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float as_float(float v) { return v; }

// Floats in the order of unsigned numbers; minus infinity and NaN are 0, minus zero is zero.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u || u == 0xFF800000u) return 0;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// Maximum and sum over G neighbouring lanes, the same in each: within 16 by DPP, then by swaps of rows and of halves.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
template <int G, typename F>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, F &&join) {
    v = join(v, dpp<kXor1>(v));
    v = join(v, dpp<kXor2>(v));
    v = join(v, dpp<kHalfMirror>(v));
    if constexpr (G > 8) v = join(v, dpp<kMirror>(v));
    if constexpr (G > 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = join((uint32_t)r[0], (uint32_t)r[1]);
    }
    if constexpr (G > 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = join((uint32_t)r[0], (uint32_t)r[1]);
    }
    return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    return group_reduce<G>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
    return __uint_as_float(group_reduce<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) { return __float_as_uint(__uint_as_float(a) + __uint_as_float(b)); }));
}

// Experts and gates of tokens t0 .. t1 - 1 of this workgroup; every choice is counted in total[].  What a round costs is mostly what
// its maximum over the group costs, so a group is as small as the registers allow (64 experts: 8 lanes of 8 and 8 tokens a wave
// instead of 64 lanes and one).
template <int G>
struct Kept {  // the choices of every group's token
    float value[kThreads / G][kMaxChosen + 1];
    int16_t expert[kThreads / G][kMaxChosen + 2];
};

template <typename T, int G, int VPL>
__device__ void choose(const RouteArgs &p, int t0, int t1, int *total, Kept<G> &kept) {
    constexpr int kGroups = kThreads / G;
    const int group = threadIdx.x / G, lane = threadIdx.x & 63, sub = lane & (G - 1), first = lane & ~(G - 1);
    const uint64_t mine = (G == 64 ? ~0ull : (1ull << (G & 63)) - 1) << first;
    for (int base = t0; base + (int)(threadIdx.x & ~63u) / G < t1; base += kGroups) {  // as long as the wave has a token
        const int t = base + group;
        const T *row = static_cast<const T *>(p.logits) + (int64_t)min(t, t1 - 1) * p.row_stride;
        uint32_t left[VPL];
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = sub * VPL + v;
            const float x = as_float(row[min(e, p.experts - 1)]);
            left[v] = e < p.experts ? key_of(x) : 0;
        }
        uint32_t best = left[0];
#pragma unroll
        for (int v = 1; v < VPL; ++v) best = max(best, left[v]);
        uint32_t top = group_max<G>(best);
        const float most = value_of(top);
        float sum = 0.0f;
        if (p.over_all) {
#pragma unroll
            for (int v = 0; v < VPL; ++v) sum += left[v] ? __expf(value_of(left[v]) - most) : 0.0f;
            sum = group_sum<G>(sum);
        }
        // Lane j % G keeps choice j, in LDS.  A loop, not rounds in a row: the instructions of 32 rounds take longer to come than to run.
        int16_t *expert = kept.expert[group];
        float *value = kept.value[group];
#pragma unroll 1
        for (int j = 0; j < p.k; ++j) {
            if (j) {
                best = left[0];
#pragma unroll
                for (int v = 1; v < VPL; ++v) best = max(best, left[v]);
                top = group_max<G>(best);
            }
            const uint64_t who = __ballot(best == top) & mine;  // the lowest lane and its first value that hold it
            const int winner = __ffsll((unsigned long long)who) - 1;
            int at = VPL - 1;
#pragma unroll
            for (int v = VPL - 2; v >= 0; --v) at = left[v] == top ? v : at;
            const int struck = lane == winner ? at : -1;
#pragma unroll
            for (int v = 0; v < VPL; ++v) left[v] = v == struck ? 0 : left[v];
            const int e = __shfl(sub * VPL + at, winner);
            if (sub == (j & (G - 1))) {
                expert[j] = (int16_t)(top ? e : -1);
                value[j] = value_of(top);
            }
        }
        if (!p.over_all) {
            float part = 0.0f;
#pragma unroll 1
            for (int j = sub; j < p.k; j += G) part += expert[j] < 0 ? 0.0f : __expf(value[j] - most);
            sum = group_sum<G>(part);
        }
        if (t >= t1) continue;
#pragma unroll 1
        for (int j = sub; j < p.k; j += G) {
            const int e = expert[j];
            const int64_t to = (int64_t)t * p.k + j;
            p.chosen[to] = e;
            p.gates[to] = e < 0 ? 0.0f : __expf(value[j] - most) / sum;
            if (e >= 0) atomicAdd(&total[e], 1);
        }
    }
}

// starts[] of this workgroup's total[] into base[] and, where asked, into memory.  Returns the number of slots in use.
__device__ int scan(const RouteArgs &p, Plan &s, bool write) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int own = tid < p.experts ? s.total[tid] : 0;
    int sum = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int below = __shfl_up(sum, o);
        if (lane >= o) sum += below;
    }
    if (lane == 63) s.wave[tid >> 6] = sum;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kThreads / 64; ++w) {
        if (w < tid >> 6) before += s.wave[w];
        all += s.wave[w];
    }
    if (tid < p.experts) {
        s.base[tid] += before + sum - own;
        if (write) p.starts[tid] = before + sum - own;
    }
    if (write && tid == 0) p.starts[p.experts] = all;
    return all;
}

// Slots of tokens t0 .. t1 - 1, whose experts lie in chosen[]; base[] and an empty mask[] are set.
__device__ void place(const RouteArgs &p, Plan &s, int t0, int t1) {
    for (int at = t0; at < t1; at += kSub) {
        const int n = min(kSub, t1 - at) * p.k;
        const int64_t from = (int64_t)at * p.k;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int e = p.chosen[from + i];
            if (e >= 0) atomicOr((unsigned long long *)&s.mask[e], 1ull << (i / p.k));
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int e = p.chosen[from + i], t = i / p.k;
            int slot = -1;
            if (e >= 0) {
                slot = s.base[e] + __popcll(s.mask[e] & ((1ull << t) - 1));
                p.rows[slot] = at + t;
            }
            p.slots[from + i] = slot;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < p.experts; e += kThreads) {
            s.base[e] += __popcll(s.mask[e]);
            s.mask[e] = 0;
        }
        __syncthreads();
    }
}

__device__ void clear(const RouteArgs &p, Plan &s) {
    const int e = threadIdx.x;
    s.mask[e] = 0;
    s.base[e] = 0;
    s.total[e] = 0;
}

// One workgroup: everything.  Several (counts given): the choice, and how many of the workgroup's tokens chose each expert.
template <typename T, int G, int VPL>
__global__ __launch_bounds__(kThreads) void choose_kernel(RouteArgs p) {
    __shared__ Plan s;
    __shared__ Kept<G> kept;
    static_assert(kEach % kSub == 0 && kThreads == kMaxExperts, "a thread clears an expert");
    const int t0 = blockIdx.x * p.per_block, t1 = min(p.tokens, t0 + p.per_block);
    clear(p, s);
    __syncthreads();
    choose<T, G, VPL>(p, t0, t1, s.total, kept);
    __syncthreads();  // chosen[] of this workgroup is visible to it
    if (p.counts) {
        for (int e = threadIdx.x; e < p.experts; e += kThreads) p.counts[(int64_t)blockIdx.x * p.experts + e] = s.total[e];
        return;
    }
    const int used = scan(p, s, true);
    __syncthreads();
    place(p, s, t0, t1);
    for (int64_t i = used + threadIdx.x; i < (int64_t)p.tokens * p.k; i += kThreads) p.rows[i] = -1;
}

__global__ __launch_bounds__(kThreads) void place_kernel(RouteArgs p) {
    __shared__ Plan s;
    const int t0 = blockIdx.x * p.per_block, t1 = min(p.tokens, t0 + p.per_block);
    clear(p, s);
    __syncthreads();
    // every workgroup's counts: in all, and of the workgroups before this one
    int wide = 64;
    while (wide < p.experts) wide <<= 1;
    const int e = threadIdx.x & (wide - 1);
    if (e < p.experts) {
        int all = 0, before = 0;
        const int step = kThreads / wide;
        for (int b = threadIdx.x / wide; b < (int)gridDim.x; b += 8 * step) {  // eight loads on their way at a time
            int c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = p.counts[(int64_t)min(b + i * step, (int)gridDim.x - 1) * p.experts + e];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                all += b + i * step < (int)gridDim.x ? c[i] : 0;
                before += b + i * step < (int)blockIdx.x ? c[i] : 0;
            }
        }
        atomicAdd(&s.total[e], all);
        atomicAdd(&s.base[e], before);
    }
    __syncthreads();
    const int used = scan(p, s, blockIdx.x == 0);
    __syncthreads();
    place(p, s, t0, t1);
    for (int64_t i = used + (int64_t)blockIdx.x * kThreads + threadIdx.x; i < (int64_t)p.tokens * p.k;
         i += (int64_t)gridDim.x * kThreads)
        p.rows[i] = -1;
}

int blocks_of(int tokens, int *per_block) {
    if (tokens <= kOneLaunch) {
        *per_block = kOneLaunch;
        return 1;
    }
    const int subs = (tokens + kEach - 1) / kEach, each = (subs + kMostBlocks - 1) / kMostBlocks;
    *per_block = each * kEach;
    return (subs + each - 1) / each;
}

template <typename T>
void launch_choose(const RouteArgs &p, int blocks, hipStream_t stream) {
    const dim3 grid(blocks), block(kThreads);
#define BITNET_CHOOSE(G, VPL) hipLaunchKernelGGL((choose_kernel<T, G, VPL>), grid, block, 0, stream, p)
    if (p.experts <= 8) BITNET_CHOOSE(8, 1);
    else if (p.experts <= 16) BITNET_CHOOSE(8, 2);
    else if (p.experts <= 32) BITNET_CHOOSE(8, 4);
    else if (p.experts <= 64) BITNET_CHOOSE(8, 8);
    else if (p.experts <= 128) BITNET_CHOOSE(8, 16);
    else if (p.experts <= 256) BITNET_CHOOSE(16, 16);
    else if (p.experts <= 512) BITNET_CHOOSE(32, 16);
    else BITNET_CHOOSE(64, 16);
#undef BITNET_CHOOSE
}

bool sizes_ok(int tokens, int experts, int k) {
    return tokens >= 1 && k >= 1 && k <= kMaxChosen && k <= experts && experts <= kMaxExperts &&
           (int64_t)tokens * k <= (1 << 30);
}

}  // namespace

extern "C" {

size_t bitnet_route_workspace_bytes(int tokens, int experts, int k) {
    if (!sizes_ok(tokens, experts, k)) return 0;
    int per_block;
    const int blocks = blocks_of(tokens, &per_block);
    return blocks == 1 ? 0 : ((size_t)blocks * experts * sizeof(int32_t) + 255) & ~(size_t)255;
}

bitnet_status_t bitnet_route(const void *logits, int dt, int64_t row_stride, int tokens, int experts, int k,
                             int over_all, int32_t *chosen, float *gates, int32_t *starts, int32_t *rows,
                             int32_t *slots, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if ((dt != BITNET_DT_BF16 && dt != BITNET_DT_F32) || !at(logits, dt == BITNET_DT_BF16 ? 2 : 4) || !at(chosen, 4) ||
        !at(gates, 4) || !at(starts, 4) || !at(rows, 4) || !at(slots, 4))
        return BITNET_ERR_INVALID_ARG;
    if (!sizes_ok(tokens, experts, k) || row_stride < experts || row_stride > ((int64_t)1 << 31)) return BITNET_ERR_UNSUPPORTED_SHAPE;
    const size_t need = bitnet_route_workspace_bytes(tokens, experts, k);
    if (need && (!at(workspace, 16) || workspace_bytes < need)) return BITNET_ERR_INVALID_ARG;
    RouteArgs p;
    p.logits = logits; p.row_stride = row_stride; p.tokens = tokens; p.experts = experts; p.k = k;
    p.over_all = over_all ? 1 : 0; p.chosen = chosen; p.gates = gates; p.starts = starts; p.rows = rows; p.slots = slots;
    const int blocks = blocks_of(tokens, &p.per_block);
    p.counts = blocks == 1 ? nullptr : static_cast<int32_t *>(workspace);
    if (dt == BITNET_DT_BF16) launch_choose<uint16_t>(p, blocks, stream);
    else launch_choose<float>(p, blocks, stream);
    if (blocks > 1) hipLaunchKernelGGL(place_kernel, dim3(blocks), dim3(kThreads), 0, stream, p);
    return launched();
}

}  // extern "C"
