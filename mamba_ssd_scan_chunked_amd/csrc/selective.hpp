// Selective scan: parameters and the device code shared by its forward, backward and
// step kernels.  Internal to the library.
//
//   h_t[d][n] = exp(step_t[d] A[d][n]) h_{t-1}[d][n] + step_t[d] x_t[d] B_t[n]
//   y_t[d]    = sum_n C_t[n] h_t[d][n] + D[d] x_t[d],  times silu(z_t[d]) if gated
//   step      = dt + dt_bias, or softplus of it;  A = -exp(A_log)
//
// The decay differs per channel and state, so there is no C B^T product to put on the
// matrix units: the work is one exp2 and four multiply-adds per (token, channel, state),
// and the exp2 takes as many issue cycles as the rest.  A lane therefore owns a channel
// with S of its N states in registers and walks the tokens; nothing is recomputed per
// state that is per channel (the step size, its product with x) or per token (B, C).
#pragma once
#include "block_common.hpp"
#include "ssd.h"

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
    int per_group, blocks;           // channels per group, 64-channel blocks per group
    int softplus;
};

// What a workgroup works on: 64 channels of one group (a lane each; lanes past the group's
// last channel repeat it and store nothing), one segment of one row.
struct SelPlace {
    int64_t b, d, g, t0, t1;
    int seg, block;
    bool mine;                       // the lane's channel exists
};
__device__ inline SelPlace sel_place(const SelParams& p, int lane) {
    SelPlace q;
    const unsigned per_row = (unsigned)(p.G * p.blocks);
    const unsigned cb = blockIdx.x % per_row, rest = blockIdx.x / per_row;
    q.seg = (int)(rest % p.nseg);
    q.b = rest / p.nseg;
    q.g = cb / p.blocks;
    q.block = (int)(cb % p.blocks);
    const int c = q.block * 64 + lane;
    q.mine = c < p.per_group;
    q.d = q.g * p.per_group + (q.mine ? c : p.per_group - 1);
    q.t0 = q.seg * p.seg_len;
    q.t1 = q.t0 + p.seg_len < p.T ? q.t0 + p.seg_len : p.T;
    return q;
}

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

// A in log2 units: exp(step A) = exp2(step A2).  Kept finite, so that the zero steps that
// pad a tile leave the state as it is whatever A_log holds.
__device__ inline float decay_rate(float A_log) { return fmaxf(-expf(A_log) * kLog2e, -3e38f); }
template <int S> __device__ inline void load_decay(const SelParams& p, int64_t d, int64_t N, int n0, float (&A2)[S]) {
    load_f32<S>(p.A_log + d * N + n0, A2);
#pragma unroll
    for (int n = 0; n < S; ++n) A2[n] = decay_rate(A2[n]);
}
__device__ inline float decay(float step, float A2) { return __builtin_amdgcn_exp2f(step * A2); }

template <int S> __device__ inline void load_state(const float* p, float (&h)[S]) {
    if (p) {
        load_f32<S>(p, h);
    } else {
#pragma unroll
        for (int n = 0; n < S; ++n) h[n] = 0.f;
    }
}

// Step size before and after its map.
__device__ inline float step_of(float raw, int soft) { return soft ? softplus(raw) : raw; }

int64_t sel_ckpt_tile();             // tokens per checkpoint of the backward pass
hipError_t launch_sel_local(const SelParams& p, int dtype, int64_t N, bool checkpoints, hipStream_t s);
hipError_t launch_sel_combine(const SelParams& p, int64_t N, bool reverse, hipStream_t s);
hipError_t launch_sel_forward(const SelParams& p, int dtype, int64_t N, hipStream_t s);
hipError_t launch_sel_step(const SelParams& p, int dtype, int64_t N, hipStream_t s);
hipError_t launch_sel_reverse_local(const SelParams& p, int dtype, int64_t N, hipStream_t s);
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
