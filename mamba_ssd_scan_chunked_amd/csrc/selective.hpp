// Selective scan: parameters and the device code shared by its forward, backward and
// step kernels.  Internal to the library.
//
//   h_t[d][n] = exp(step_t[d] A[d][n]) h_{t-1}[d][n] + step_t[d] x_t[d] B_t[n]
//   y_t[d]    = sum_n C_t[n] h_t[d][n] + D[d] x_t[d],  times silu(z_t[d]) if gated
//   step      = dt + dt_bias, or softplus of it;  A = -exp(A_log)
//
// The decay differs per channel and state, so there is no C B^T product to put on the
// matrix units: the work is one exp2 and four other vector instructions per (token, channel,
// state).  A lane therefore owns a channel with S of its N states in registers and walks the
// tokens; nothing is recomputed per state that is per channel (the step size, its product
// with x) or per token (B, C).
#pragma once
#include "block_common.hpp"
#include "ssd.h"

#include <type_traits>

namespace ssd {

struct SelParams {
    const void *x, *dt, *B, *C, *z;
    const float *A_log, *skip, *dt_bias, *init;
    const int32_t* seq_idx;
    void* y;
    float* fin;
    float *seg_state, *seg_step;     // per (row, segment but the last): end state (D, N), summed steps (D)
    float *ckpt, *ckpt_step;         // per (row, tile): state before it from the segment's start, summed steps
    // gradients
    const float *dy, *dfin;
    float *dx, *ddt, *dz, *dinit;
    float *part_b, *part_c;          // per channel block of a group: (batch, T, G, N)
    float *part_sums;                // per (row, segment): dA_log (D, N), dD (D), ddt_bias (D)
    float *seg_grad;                 // per (row, segment but the first): gradient reaching its incoming state
    int64_t batch, T, D, G, nseqs, ldx, lddt, ldz, ldb, ldc;
    int64_t seg_len;                 // tokens per segment, a multiple of every tile length
    int nseg;
    int per_group, blocks;           // channels per group, workgroups' channel blocks per group
    int softplus;
};

// How a workgroup shares out its channels and states.  A wave's 64 lanes are M = 64 / CH
// groups of CH channels, each group with S of the states, and W waves hold the rest:
// N = W M S.  CH is 16, 32 or 64, so the 16 lanes of a DPP row always hold the same
// states: B and C are kept one state per lane of the row and reach the multiply-adds as
// row broadcasts, without an instruction or an LDS read per state of their own.
template <int N, int CH_, int S_> struct SelShape {
    static constexpr int CH = CH_, S = S_, M = 64 / CH, W = N / (M * S), THREADS = 64 * W;
    static_assert(W * M * S == N && S <= 16 && CH >= 16, "shape");
};

// What a workgroup works on: CH channels of one group (lanes past the group's last channel
// repeat it and store nothing), one segment of one row.
struct SelPlace {
    int64_t b, d0, g, t0, t1;        // d0: first channel
    int seg, block, chans;           // chans: channels of d0 .. that exist, up to CH
};
template <int CH> __device__ inline SelPlace sel_place(const SelParams& p) {
    SelPlace q;
    const unsigned per_row = (unsigned)(p.G * p.blocks);
    const unsigned cb = blockIdx.x % per_row, rest = blockIdx.x / per_row;
    q.seg = (int)(rest % p.nseg);
    q.b = rest / p.nseg;
    q.g = cb / p.blocks;
    q.block = (int)(cb % p.blocks);
    q.d0 = q.g * p.per_group + q.block * CH;
    q.chans = p.per_group - q.block * CH < CH ? p.per_group - q.block * CH : CH;
    q.t0 = q.seg * p.seg_len;
    q.t1 = q.t0 + p.seg_len < p.T ? q.t0 + p.seg_len : p.T;
    return q;
}

// The value that lane I of every row of 16 lanes holds (a DPP operand of the instruction
// that uses it).
template <int I> __device__ inline float row_lane(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x150 + I, 0xf, 0xf, true));
}
template <int N, typename F, int I = 0> __device__ inline void static_for(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        static_for<N, F, I + 1>(static_cast<F&&>(f));
    }
}

// One value per (token, channel) of a tile of TQ tokens, loaded by the workgroup's threads:
// pair j of a thread is token (tid + THREADS j) / CH, channel (tid + THREADS j) % CH.
// Offsets are bytes from the tile's first token, so that a load is a scalar base and a
// 32-bit offset; in a ragged tile the tokens past the end repeat the last one.
template <typename T, int J, int CH, int THREADS> struct TileLoad {
    unsigned off[J];
    __device__ inline void place(int64_t ld, int chans, int tokens) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int k = threadIdx.x + THREADS * j, c = k % CH, i = k / CH;
            off[j] = (unsigned)(((unsigned)ld * (unsigned)(i < tokens ? i : tokens - 1) + (c < chans ? c : chans - 1)) * sizeof(T));
        }
    }
    __device__ inline void load(const T* base, T (&v)[J]) const {
#pragma unroll
        for (int j = 0; j < J; ++j) v[j] = *(const T*)((const char*)base + off[j]);
    }
};

// Bits i of the tile's tokens t .. t+TQ-1: a sequence starts at (ends after) the token.
struct SeqBits {
    uint64_t starts, ends;
};
template <int TQ> __device__ inline SeqBits seq_bits(const int32_t* ids, int64_t t, int64_t T, int lane) {
    const int64_t i = t + lane;
    const bool in = lane < TQ && i < T;
    const int32_t id = in ? ids[i] : 0;
    const bool first = in && (i == 0 || ids[i - 1] != id);
    const bool last = in && (i == T - 1 || ids[i + 1] != id);
    return SeqBits{__ballot(first), __ballot(last)};
}

// A in log2 units: exp(step A) = exp2(step A2).  Kept finite (A_log above 88 counts as 88:
// any step then decays to nothing), so that the zero steps that pad a tile leave the state
// as it is; a NaN stays one.
__device__ inline float decay_rate(float A_log) {
    const float a = -exp_small(__builtin_amdgcn_fmed3f(A_log, -100.f, 88.f)) * kLog2e;
    return A_log == A_log ? a : A_log;
}
template <int S> __device__ inline void load_decay(const SelParams& p, int64_t d, int64_t N, int n0, float (&A2)[S]) {
    load_f32<S>(p.A_log + d * N + n0, A2);
#pragma unroll
    for (int n = 0; n < S; ++n) A2[n] = decay_rate(A2[n]);
}
__device__ inline float decay(float step, float A2) { return __builtin_amdgcn_exp2f(step * A2); }

// S values of LDS at 4 S bytes' alignment.
template <int S> struct alignas(S < 4 ? 4 * S : 16) States {
    float v[S];
};

template <int S> __device__ inline void load_state(const float* p, float (&h)[S]) {
    if (p) {
        load_f32<S>(p, h);
    } else {
#pragma unroll
        for (int n = 0; n < S; ++n) h[n] = 0.f;
    }
}

// Step sizes from dt + bias, in place.
template <int J> __device__ inline void map_steps(float (&v)[J], int soft) {
    if (soft) {
#pragma unroll
        for (int j = 0; j < J; ++j) v[j] = softplus(v[j]);
    }
}

int64_t sel_ckpt_tile();             // tokens per checkpoint of the backward pass
hipError_t launch_sel_local(const SelParams& p, int dtype, int64_t N, hipStream_t s);
hipError_t launch_sel_combine(const SelParams& p, int64_t N, bool both, hipStream_t s);      // both: backwards too
hipError_t launch_sel_forward(const SelParams& p, int dtype, int64_t N, hipStream_t s);
hipError_t launch_sel_step(const SelParams& p, int dtype, int64_t N, hipStream_t s);
hipError_t launch_sel_locals(const SelParams& p, int dtype, int64_t N, hipStream_t s);
hipError_t launch_sel_reverse(const SelParams& p, int dtype, int64_t N, hipStream_t s);
hipError_t launch_sel_group_sums(const SelParams& p, int64_t N, float* dB, float* dC, hipStream_t s);

#define SSD_SEL_BY_STATE(N, CALL)                                    \
    switch (N) {                                                     \
        case 8: CALL(8); break;                                      \
        case 16: CALL(16); break;                                    \
        case 32: CALL(32); break;                                    \
        case 64: CALL(64); break;                                    \
        default: return hipErrorInvalidValue;                        \
    }

}  // namespace ssd
