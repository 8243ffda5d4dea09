// The maps h -> P h + H that runs, waves and tiles of the gated linear recurrence are joined by,
// and the words that tiles publish them in.  Internal to the library.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssd {

// P = -1 marks a map that begins a sequence anew: what comes before it does not matter, whatever
// it is (a select, so that Inf and NaN stay in their sequence).
struct Map {
    float P, H;
};
template <bool SEQ> __host__ __device__ inline Map then(Map first, Map second) {
    if (SEQ && second.P < 0.f) return second;
    Map m;
    m.H = fmaf(second.P, first.H, second.H);
    m.P = SEQ && first.P < 0.f ? -1.f : first.P * second.P;
    return m;
}
template <bool SEQ> __host__ __device__ inline float apply(Map m, float h) {
    return SEQ && m.P < 0.f ? m.H : fmaf(m.P, h, m.H);
}

// A map as a word that is never 0 in its low half, which stays 0 until the word is published.  The
// one P that the shift would make 0 there is a NaN, and another NaN takes its place.
__host__ __device__ inline uint64_t word_of(Map m) {
    const uint32_t low = __builtin_bit_cast(uint32_t, m.P) + 1u;
    return (uint64_t)__builtin_bit_cast(uint32_t, m.H) << 32 | (low ? low : 0x7fc00001u);
}
// A word that never came is 0: as a map its P is NaN, as a published state (P is 1 there) it is NaN.
__host__ __device__ inline Map map_of(uint64_t w) {
    return {__builtin_bit_cast(float, (uint32_t)w - 1u), __builtin_bit_cast(float, (uint32_t)(w >> 32))};
}
__host__ __device__ inline float state_of(uint64_t w) {
    const Map m = map_of(w);
    return m.P * m.H;
}

}  // namespace ssd
