// Host side of the attention operators: the rotary table and the cache's size authority.
#include <cmath>
#include <cstdint>

#include "bitnet_w2a8.h"

extern "C" {

size_t bitnet_kv_cache_bytes(int64_t pages, int kv_heads, int head_dim, int page) {
    if (pages < 1 || pages > INT32_MAX || kv_heads < 1 || kv_heads > 1024) return 0;
    if (head_dim != 64 && head_dim != 128) return 0;
    if (page != 16 && page != 32 && page != 64 && page != 128) return 0;
    return (size_t)pages * kv_heads * page * head_dim;
}

bitnet_status_t bitnet_rope_table(int64_t positions, int rot, double base, double factor, int64_t trained,
                                  float *table) {
    if (!table || !(base > 1.0) || !(factor >= 1.0) || !std::isfinite(base) || !std::isfinite(factor) || trained < 0)
        return BITNET_ERR_INVALID_ARG;
    if (positions < 1 || positions > INT32_MAX || rot < 16 || rot > 128 || rot % 16) return BITNET_ERR_UNSUPPORTED_SHAPE;
    const double two_pi = 6.283185307179586476925286766559;
    const int half = rot / 2;
    double rate[64];
    for (int j = 0; j < half; ++j) {
        const double r = std::pow(base, -2.0 * j / rot);
        double keep = 0.0;  // share of the rate that is left as trained
        if (trained > 0) {
            const double turns = (double)trained * r / two_pi;
            keep = turns <= 1.0 ? 0.0 : turns >= 32.0 ? 1.0 : (turns - 1.0) / 31.0;
        }
        rate[j] = r * (keep + (1.0 - keep) / factor);
    }
    for (int64_t p = 0; p < positions; ++p)
        for (int j = 0; j < half; ++j) {
            const double a = (double)p * rate[j];
            table[p * rot + j] = (float)std::cos(a);
            table[p * rot + half + j] = (float)std::sin(a);
        }
    return BITNET_OK;
}

}  // extern "C"
