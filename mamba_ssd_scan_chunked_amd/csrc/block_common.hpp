// Device and host helpers shared by the operators around the scan: the causal
// convolution, the selective scan and the norms.  Internal to the library.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssd {

// V consecutive elements.  Loads and stores go through memcpy at the element's own
// alignment: gfx950 reads and writes 16 bytes at any address that is a multiple of
// the element size in one instruction, so rows of odd length and slices of wider
// rows take the same path as aligned ones.
template <typename T, int V> struct Pack {
    T v[V];
};
template <int V, typename T> __device__ inline Pack<T, V> load_pack(const T* p) {
    Pack<T, V> r;
    __builtin_memcpy(&r, p, sizeof(r));
    return r;
}
template <int V, typename T> __device__ inline void store_pack(T* p, const Pack<T, V>& r) {
    __builtin_memcpy(p, &r, sizeof(r));
}
// The same, past the caches.
template <int V, typename T> __device__ inline void stream_pack(T* p, const Pack<T, V>& r) {
    typedef uint32_t Words __attribute__((ext_vector_type(sizeof(r) >= 8 ? sizeof(r) / 4 : 2), aligned(sizeof(T))));
    if constexpr (sizeof(r) == sizeof(Words)) {
        Words w;
        __builtin_memcpy(&w, &r, sizeof(w));
        __builtin_nontemporal_store(w, (Words*)p);
    } else {
        store_pack<V>(p, r);
    }
}
template <int V, typename T> __device__ inline void load_f32(const T* p, float* out) {
    const Pack<T, V> r = load_pack<V>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = (float)r.v[i];
}
// One rounding to nearest even when T is bf16 (the operator's only one).  STREAM: past the
// caches, for outputs that are larger than they are (see kStreamBytes).  A template's
// parameter: under a test at run time the compiler joins the two stores into a plain one.
template <int V, bool STREAM = false, typename T> __device__ inline void store_f32(T* p, const float* in) {
    Pack<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = (T)in[i];
    if constexpr (STREAM) stream_pack<V>(p, r);
    else store_pack<V>(p, r);
}

// A call whose largest output is above the eight L2 caches' 32 MB stores non-temporally: the
// next kernel would not find it there anyway, and it no longer pushes out what this one still
// reads (4 x 4096 tokens of 5376 channels convolved: 66 us against 78; gated norm of 16384 rows
// of 5120: 134 against 154, its gradients for 8192 rows: 147 against 172; just above the border,
// 40 MB of stream of 4096 rows of 2560: 20 against 24, and 44 against 49 with the norm after it
// that reads the stream).  Smaller ones stay in L2 for the kernel that reads them.
constexpr int64_t kStreamBytes = int64_t(32) << 20;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// e^v for |v| <= 100 from the hardware exp2.  The product v log2(e) is taken as its rounded
// value and its remainder, so the error does not grow with |v| (about 1e-7 relative).  Above
// 88.72 e^v leaves fp32 and the result is +Inf, without the remainder: Inf times it has
// either sign, or is NaN.
__device__ inline float exp_small(float v) {
    const float hi = v * kLog2e;
    const float lo = fmaf(v, 1.925963033500012e-08f, fmaf(v, kLog2e, -hi));
    const float e = __builtin_amdgcn_exp2f(hi);
    return e < __builtin_inff() ? fmaf(e * lo, kLn2, e) : e;
}

// 1 / (1 + e^-v); v beyond +-100 counts as +-100 (1 and, e^100 being Inf, 0: so the gate of the
// type's lowest value is 0 and not a rest of it).
__device__ inline float sigmoid(float v) {
    return __builtin_amdgcn_rcpf(1.f + exp_small(__builtin_amdgcn_fmed3f(-v, -100.f, 100.f)));
}
__device__ inline float silu(float v) { return v * sigmoid(v); }
// The gate of a result that is rounded to T: bf16 takes the plain exp2, whose argument's
// rounding (2^-24 |v| log2 e) is far below bf16's half step and saves six instructions.
template <typename T> __device__ inline float silu_for(float v) { return silu(v); }
template <> __device__ inline float silu_for<__bf16>(float v) {
    return v * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -kLog2e));
}
// d silu / dv = s (1 + v (1 - s)), s = sigmoid(v)
__device__ inline float silu_slope(float v, float s) { return s * (1.f + v * (1.f - s)); }

// log(1 + e^v) = max(v, 0) + log1p(t), t = e^-|v|.  With u = 1 + t rounded and e = t - (u - 1)
// what the rounding lost, log1p(t) = log(u) + e / u to first order, which keeps the relative
// error of a tiny t (u = 1, e = t).  slope: sigmoid(v) = 1 / u or t / u.  Relative error below
// 2^-24 |v| plus a few roundings, from the argument of the exp2.
__device__ inline float softplus_slope(float v, float* slope) {
    const float t = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e), u = 1.f + t;
    const float r = __builtin_amdgcn_rcpf(u), e = t - (u - 1.f);
    *slope = (v >= 0.f ? 1.f : t) * r;
    return fmaxf(v, 0.f) + fmaf(__builtin_amdgcn_logf(u), kLn2, e * r);
}
__device__ inline float softplus(float v) {
    float slope;
    return softplus_slope(v, &slope);
}

// Sum over teams of LANES neighbouring lanes (4 to 64, a power of two), in every lane: DPP
// moves within a row of 16, then the row and half-wave swaps.
template <int CTRL> __device__ inline float dpp_mov(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <int LANES> __device__ inline float lane_team_sum(float v) {
    v += dpp_mov<0xb1>(v);                             // quad_perm 1,0,3,2
    v += dpp_mov<0x4e>(v);                             // quad_perm 2,3,0,1
    if constexpr (LANES > 4) v += dpp_mov<0x141>(v);   // row_half_mirror
    if constexpr (LANES > 8) v += dpp_mov<0x140>(v);   // row_mirror
    if constexpr (LANES > 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if constexpr (LANES > 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}

// Sequence id of a token, clamped so that a bad id cannot leave the per-sequence arrays.
__device__ inline int64_t clamp_id(int32_t id, int64_t nseqs) {
    return id < 0 ? 0 : (id >= nseqs ? nseqs - 1 : id);
}

// Column sums of part (rows x cols), rows in a fixed order: columns below split go to
// out, those below split2 to out2 and the rest to out3 (null: not wanted).
struct ColumnSums {
    const float* part;
    float *out, *out2, *out3;
    int64_t rows, cols, split, split2;
};
hipError_t launch_column_sums(const ColumnSums& c, hipStream_t s);
hipError_t launch_fill(float* p, int64_t n, hipStream_t s);                          // zeros
hipError_t launch_copy(float* dst, const float* src, int64_t n, hipStream_t s);      // src null: zeros

}  // namespace ssd
