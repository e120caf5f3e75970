// order_device.h -- the order of logits (value descending, index ascending) as
// integer keys, shared by the kernels of the log probabilities and of sampling.
#pragma once

#include "q8_device.h"

namespace q8 {

// Order of the top list: larger value first, then lower index; NaN last.  No
// key of a logit is 0.
__device__ __forceinline__ uint32_t value_key(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);       // -0 -> +0
    const uint32_t key = (u >> 31) ? ~u : (u | 0x80000000u);
    return x != x ? 0u : key;
}

__device__ __forceinline__ uint64_t order_key(float x, uint32_t i)
{
    return ((uint64_t)value_key(x) << 32) | (uint32_t)~i;
}

__device__ __forceinline__ float key_value(uint64_t key)
{
    const uint32_t k = (uint32_t)(key >> 32);
    if (k == 0) return __builtin_nanf("");
    return __builtin_bit_cast(float, (k >> 31) ? (k & 0x7fffffffu) : ~k);
}

__device__ __forceinline__ int key_index(uint64_t key) { return (int)~(uint32_t)key; }

// The n-th largest of 64 keys, one per lane, its low half cut (0: fewer than n
// keys are not 0).
__device__ __forceinline__ uint32_t nth_key(uint32_t key, int n)
{
    uint32_t t = 0;
    for (int b = 31; b >= 16; --b) {
        const uint32_t c = t | (1u << b);
        if (__popcll(__ballot(key >= c)) >= n) t = c;
    }
    return t;
}

// The same of 256 keys, four per lane.
__device__ __forceinline__ uint32_t nth_key(u32x4 key, int n)
{
    uint32_t t = 0;
    for (int b = 31; b >= 16; --b) {
        const uint32_t c = t | (1u << b);
        if (__popcll(__ballot(key.x >= c)) + __popcll(__ballot(key.y >= c)) +
                __popcll(__ballot(key.z >= c)) + __popcll(__ballot(key.w >= c)) >= n)
            t = c;
    }
    return t;
}

}  // namespace q8
