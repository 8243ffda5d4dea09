// Selective scan, gradients.  With G_t = dL/dh_t = g_t C_t + q_t, where g = dL/d(y before
// the gate) and q_t = exp(step_{t+1} A) G_{t+1} reaches token t's state from later tokens
// (dL/dfinal after the last), and p_t = exp(step_t A) h_{t-1}:
//   dB_t[n] = sum_d G step x,  dC_t[n] = sum_d g h,  d(step x) = sum_n G B,
//   dstep = sum_n G p A + x d(step x),  dA = sum_t G p step,  dx = step d(step x) + D g.
//
// The states are not kept by the forward pass: the local pass leaves one before every
// tile of eight tokens, and the reverse pass runs a tile forwards (keeping p and the decays
// in registers) and then backwards.
//
// Bound by vector instructions (the vector units are at work for 83 % of the reverse pass and
// 79 % of the local pass): per (token, channel, state) 7 on the way out, 7 on the way back and
// 3 for the sums over channels.  Measured on an MI355X, 8 x 2048 tokens of 1536 channels with
// 16 states, gated: bf16 0.58 ms, fp32 0.55, of which the reverse pass 0.40, the local pass 0.14
// and the three small launches 0.03.  Eight states a lane need 128 registers for p and the decays
// alone and spill or run two waves per SIMD (0.8 ms and more); the decays computed again on
// the way back, 0.69.
#include "selective.hpp"

namespace ssd {

constexpr int kTile = 8;

// Sums over the 64 lanes of S values for each of the tile's eight tokens.  At every level a
// lane keeps half of what it holds and hands the other half to its partner, so that a level
// halves the work of the next: a token's values first (swaps of 32 and 16 lanes, for eight
// values also lanes of a row), then, as tokens come, pairs of tokens, pairs of pairs and the
// two halves of the tile.  64 sums of four values cost 102 instructions instead of 768.  In
// the end a lane holds the sum of value sum_index<S>(lane) of token sum_token<S>(lane).
template <int S> __device__ inline int sum_index(int lane) { return S == 4 ? lane >> 4 : (lane >> 3 & 1) + 2 * (lane >> 4); }
template <int S> __device__ inline int sum_token(int lane) {
    return S == 4 ? (lane >> 3 & 1) + (lane >> 1 & 2) + (lane << 1 & 4) : (lane >> 2 & 1) + (lane & 2) + (lane << 2 & 4);
}
template <int S> __device__ inline float value_sums(const float (&v)[S], int lane) {
    static_assert(S == 4 || S == 8, "values");
    float a[S / 2], b[S / 4];
#pragma unroll
    for (int k = 0; k < S / 2; ++k) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[k]), __float_as_uint(v[k + S / 2]), false, false);
        a[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
#pragma unroll
    for (int k = 0; k < S / 4; ++k) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a[k]), __float_as_uint(a[k + S / 4]), false, false);
        b[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if constexpr (S == 8) {
        const bool hi = lane & 8;
        return (hi ? b[1] : b[0]) + dpp_mov<0x140>(hi ? b[0] : b[1]);     // row_mirror
    } else {
        return b[0];
    }
}
// Level L of the tokens: lanes with the bit clear go on with `even`, the others with `odd`.
template <int S, int L> __device__ inline float token_sums(float even, float odd, int lane) {
    constexpr int BIT = S == 4 ? 8 >> L : 4 >> L;
    // the partner: row_mirror, row_half_mirror, quad_perm 3,2,1,0 or 1,0,3,2
    constexpr int CTRL = BIT == 8 ? 0x140 : (BIT == 4 ? 0x141 : (BIT == 2 ? 0x1b : 0xb1));
    const bool up = lane & BIT;
    return (up ? odd : even) + dpp_mov<CTRL>(up ? even : odd);
}
// What is kept between tokens: the last unpaired token, pair and half of the tile.
template <int S> struct TileSums {
    float token, pair, half, all;
    template <int I> __device__ inline void forwards(float r, int lane) {
        if constexpr (I & 1) {
            r = token_sums<S, 0>(token, r, lane);
            if constexpr (I & 2) {
                r = token_sums<S, 1>(pair, r, lane);
                if constexpr (I & 4) all = token_sums<S, 2>(half, r, lane);
                else half = r;
            } else {
                pair = r;
            }
        } else {
            token = r;
        }
    }
    template <int I> __device__ inline void backwards(float r, int lane) {
        if constexpr (!(I & 1)) {
            r = token_sums<S, 0>(r, token, lane);
            if constexpr (!(I & 2)) {
                r = token_sums<S, 1>(r, pair, lane);
                if constexpr (!(I & 4)) all = token_sums<S, 2>(r, half, lane);
                else half = r;
            } else {
                pair = r;
            }
        } else {
            token = r;
        }
    }
    __device__ inline float result() const { return S == 4 ? all + dpp_mov<0xb1>(all) : all; }
};

__device__ inline int64_t last_tile(const SelPlace& q) { return q.t0 + (q.t1 - q.t0 - 1) / kTile * kTile; }

// ---------------------------------------------------------------- local pass
// One segment from a zero state (the row's first: from its initial state), eight states a
// lane.  Kept before every tile, and at the segment's end: the state and the sum of the steps
// so far, whose decay exp(A sum) is what an incoming state would still weigh; infinite when a
// sequence starts inside (whatever its own steps are), so that nothing comes through.
// With REV (rows in segments) also what the segment's own tokens send back to its incoming
// state: the sum over its tokens t of P_t C_t g_t, P_t = exp(step_first A) .. exp(step_t A), plus
// P dfinal where its sequence ends; it stops before the first sequence that starts inside.
// Taken in the same direction as the states, so that each decay is computed once for both:
// 0.58 ms for all gradients of the case above, against 0.63 with a pass for each direction and
// 0.61 with those two in one launch.  Sixteen states a lane spill (0.76).
template <typename T, int N, int S, bool SEQ, bool REV>
__global__ __launch_bounds__((SelShape<N, 64, S>::THREADS), 4) void sel_locals_kernel(SelParams p) {
    constexpr int CH = 64, W = N / S, TH = 64 * W, TQ = kTile, J = TQ / W, E = TQ * N / TH;
    static_assert(W * J == TQ && E * TH == TQ * N, "tile shape");
    __shared__ float2 su[TQ][CH];
    __shared__ float gs[REV ? TQ : 1][CH];
    __shared__ float4 Bs[TQ / 4][N], Cs[REV ? TQ / 4 : 1][N];    // four tokens of a state together
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const SelPlace q = sel_place<CH>(p);
    const bool mine = lane < q.chans;
    const int64_t d = q.d0 + (mine ? lane : q.chans - 1);
    const unsigned col = mine ? lane : q.chans - 1;
    const int n0 = w * S;
    const int32_t* ids = SEQ ? p.seq_idx + q.b * p.T : nullptr;
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f;
    float A2[S], h[S], P[S], back[S], sum = 0.f;
    load_decay<S>(p, d, N, n0, A2);
    const int64_t state = d * N + n0, DN = p.D * N;
    load_state<S>(q.seg == 0 && p.init && !SEQ ? p.init + q.b * DN + state : nullptr, h);
#pragma unroll
    for (int n = 0; n < S; ++n) {
        P[n] = 1.f;
        back[n] = 0.f;
    }
    bool cut = false;                     // a sequence has started inside
    bool open = REV && q.seg > 0;         // none has, and there is a segment to send to
    float* sent = open ? p.seg_grad + (q.b * (p.nseg - 1) + q.seg - 1) * DN + state : nullptr;

    const int64_t tok = q.b * p.T + q.t0, tiles = (p.T + TQ - 1) / TQ;
    const T* x = (const T*)p.x + tok * p.ldx + q.d0;
    const T* dt = (const T*)p.dt + tok * p.lddt + q.d0;
    const T* z = (const T*)(p.z ? p.z : p.x) + tok * p.ldz + q.d0;        // (without a gate: not read)
    const T* B = (const T*)p.B + tok * p.ldb + q.g * N;
    const T* C = (const T*)p.C + tok * p.ldc + q.g * N;
    const float* dy = p.dy + tok * p.D + q.d0;
    T xr[J], dr[J], zr[J], br[E], cr[E];
    float yr[J];
    // a wave's tokens are its own, so their rows are scalar addresses; tokens past the
    // segment's end repeat its last one
    auto load = [&](int64_t left) {
        const int tokens = left < TQ ? (int)left : TQ;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int i = w + W * j < tokens ? w + W * j : tokens - 1;
            xr[j] = (x + i * p.ldx)[col];
            dr[j] = (dt + i * p.lddt)[col];
            if (REV && p.z) zr[j] = (z + i * p.ldz)[col];
            if (REV) yr[j] = (dy + i * p.D)[col];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int k = threadIdx.x + TH * e, i = k / N < tokens ? k / N : tokens - 1;
            br[e] = B[i * p.ldb + k % N];
            if (REV) cr[e] = C[i * p.ldc + k % N];
        }
        x += TQ * p.ldx;
        dt += TQ * p.lddt;
        z += TQ * p.ldz;
        B += TQ * p.ldb;
        C += TQ * p.ldc;
        dy += TQ * p.D;
    };
    load(q.t1 - q.t0);
    for (int64_t t = q.t0; t < q.t1; t += TQ) {
        const int tokens = q.t1 - t < TQ ? (int)(q.t1 - t) : TQ;
        if (mine) {
            const int64_t at = (q.b * tiles + t / TQ) * p.D + d;
            store_f32<S>(p.ckpt + at * N + n0, h);
            if (w == 0) p.ckpt_step[at] = sum;
        }
        float step[J], xk[J], g[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            xk[j] = (float)xr[j];
            step[j] = (float)dr[j] + bias;
            if (REV) g[j] = p.z ? yr[j] * silu((float)zr[j]) : yr[j];
        }
        map_steps(step, p.softplus);
        if (tokens < TQ) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (w + W * j >= tokens) step[j] = xk[j] = g[j] = 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < J; ++j) {
            su[w + W * j][lane] = make_float2(step[j], step[j] * xk[j]);
            if (REV) gs[w + W * j][lane] = g[j];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int k = threadIdx.x + TH * e, i = k / N;
            (&Bs[i / 4][k % N].x)[i % 4] = i < tokens ? (float)br[e] : 0.f;
            if (REV) (&Cs[i / 4][k % N].x)[i % 4] = i < tokens ? (float)cr[e] : 0.f;
        }
        __syncthreads();
        if (t + TQ < q.t1) load(q.t1 - t - TQ);
        SeqBits bits{};
        if (SEQ) bits = seq_bits<TQ>(ids, t, p.T, lane);
#pragma unroll
        for (int i4 = 0; i4 < TQ / 4; ++i4) {
            const float4 B4 = Bs[i4][n0 + lane % S], C4 = REV ? Cs[i4][n0 + lane % S] : B4;
            const float Bv[4] = {B4.x, B4.y, B4.z, B4.w}, Cv[4] = {C4.x, C4.y, C4.z, C4.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = 4 * i4 + k;
                if (SEQ && (bits.starts >> i & 1)) {
                    load_state<S>(p.init ? p.init + clamp_id(ids[t + i], p.nseqs) * DN + state : nullptr, h);
                    cut = true;
                    sum = __builtin_inff();
                    if (open && mine) store_f32<S>(sent, back);
                    open = false;
                }
                const float2 s = su[i][lane];
                const float g = REV ? gs[i][lane] : 0.f;
                sum += SEQ && cut ? 0.f : s.x;
                static_for<S>([&](auto I) {
                    constexpr int n = decltype(I)::value;
                    const float a = decay(s.x, A2[n]);
                    h[n] = fmaf(a, h[n], row_lane<n>(Bv[k]) * s.y);
                    if (REV) {
                        P[n] *= a;
                        back[n] = fmaf(P[n], row_lane<n>(Cv[k]) * g, back[n]);
                    }
                });
                if (SEQ && (bits.ends >> i & 1) && open && p.dfin) {
                    float df[S];
                    load_f32<S>(p.dfin + clamp_id(ids[t + i], p.nseqs) * DN + state, df);
#pragma unroll
                    for (int n = 0; n < S; ++n) back[n] = fmaf(P[n], df[n], back[n]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    if (!mine) return;
    if (q.seg < p.nseg - 1) {
        const int64_t at = (q.b * (p.nseg - 1) + q.seg) * p.D + d;
        store_f32<S>(p.seg_state + at * N + n0, h);
        if (w == 0) p.seg_step[at] = sum;
    }
    if (open) {
        if (!SEQ && q.seg == p.nseg - 1 && p.dfin) {
            float df[S];
            load_f32<S>(p.dfin + q.b * DN + state, df);
#pragma unroll
            for (int n = 0; n < S; ++n) back[n] = fmaf(P[n], df[n], back[n]);
        }
        store_f32<S>(sent, back);
    }
}

// ---------------------------------------------------------------- reverse pass
// One workgroup per 64 channels and segment, N/S waves with S states each (four, or eight for
// N = 64).  With four the tile's p and decays take 64 registers, and N = 16 fits three waves per
// SIMD without scratch (packed bf16: 12 bytes a lane); N = 8 at three waves keeps 72 to 116 bytes a
// lane in scratch memory, N = 32 at four 52 to 104.  (2 x 777 packed tokens of 650 channels with 32
// states, fp32, take 60 us here, the vector units at work for 34 % of it.)  The sums over states of
// a token (for y, d(step x) and dstep) meet in LDS, the sums over channels (for dB and dC)
// within the wave and then, over channel blocks, in part_b and part_c.
template <typename T, int N, int S, bool SEQ>
__global__ __launch_bounds__((SelShape<N, 64, S>::THREADS), (N == 32 ? 4 : (N < 32 ? 3 : 2))) void sel_reverse_kernel(SelParams p) {
    constexpr int CH = 64, W = N / S, TH = 64 * W, TQ = kTile, J = TQ / W;
    static_assert(W * J == TQ && TH >= TQ * N, "tile shape");     // a B and a C value per thread
    __shared__ float2 su[TQ][CH];
    __shared__ float gs[TQ][CH];
    __shared__ float4 Bq[TQ / 4][N];                             // four tokens of a state together
    __shared__ __attribute__((aligned(16))) float Bs[TQ][N], Cs[TQ][N];    // a token's states together
    __shared__ float parts[3][W][TQ][CH];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const SelPlace q = sel_place<CH>(p);
    const bool mine = lane < q.chans;
    const int64_t d = q.d0 + (mine ? lane : q.chans - 1);
    const int n0 = w * S;
    const int32_t* ids = SEQ ? p.seq_idx + q.b * p.T : nullptr;
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f, skip = p.skip ? p.skip[d] : 0.f;
    float A2[S], grad[S], dA[S], sum_skip = 0.f, sum_bias = 0.f;
    load_decay<S>(p, d, N, n0, A2);
    const int64_t state = d * N + n0, DN = p.D * N;
    load_state<S>(q.seg < p.nseg - 1 ? p.seg_grad + (q.b * (p.nseg - 1) + q.seg) * DN + state
                                     : (!SEQ && p.dfin ? p.dfin + q.b * DN + state : nullptr), grad);
#pragma unroll
    for (int n = 0; n < S; ++n) dA[n] = 0.f;
    const float* before = q.seg > 0 ? p.seg_state + (q.b * (p.nseg - 1) + q.seg - 1) * DN + state : nullptr;
    const int64_t tiles = (p.T + TQ - 1) / TQ;

    const int64_t first = last_tile(q), tok = q.b * p.T + first;
    const T* x = (const T*)p.x + tok * p.ldx + q.d0;
    const T* dt = (const T*)p.dt + tok * p.lddt + q.d0;
    const T* z = (const T*)(p.z ? p.z : p.x) + tok * p.ldz + q.d0;        // (without a gate: not read)
    const T* B = (const T*)p.B + tok * p.ldb + q.g * N;
    const T* C = (const T*)p.C + tok * p.ldc + q.g * N;
    int64_t row = tok * p.D + d;                                          // of the tile in dy, dx, ddt, dz
    const float* dy = p.dy + tok * p.D + q.d0;
    const unsigned col = mine ? lane : q.chans - 1;
    // part_b and part_c: (block, batch, T, G, N); the lane's value and token after TileSums
    // (with four values two lanes hold the same one, and the even lane stores it)
    const int hold = sum_token<S>(lane);
    const bool stores = S == 8 || lane % 2 == 0;
    int64_t part = ((((int64_t)q.block * p.batch + q.b) * p.T + first + hold) * p.G + q.g) * N + n0 + sum_index<S>(lane);
    for (int64_t t = first; t >= q.t0; t -= TQ) {
        const int tokens = q.t1 - t < TQ ? (int)(q.t1 - t) : TQ;
        T xr[J], dr[J], zr[J];
        float dyk[J], h[S];
        // a wave's tokens are its own, so their rows are scalar addresses
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int i = w + W * j < tokens ? w + W * j : tokens - 1;
            xr[j] = (x + i * p.ldx)[col];
            dr[j] = (dt + i * p.lddt)[col];
            if (p.z) zr[j] = (z + i * p.ldz)[col];
            dyk[j] = (dy + i * p.D)[col];
        }
        const int bi = threadIdx.x / N, bt = bi < tokens ? bi : tokens - 1;       // (threads past the tile repeat it)
        const T br = B[bt * p.ldb + threadIdx.x % N], cr = C[bt * p.ldc + threadIdx.x % N];
        {
            const int64_t at = (q.b * tiles + t / TQ) * p.D + d;
            load_f32<S>(p.ckpt + at * N + n0, h);
            if (before) {
                const float sum = p.ckpt_step[at];
                float in[S];
                load_f32<S>(before, in);
                if (sum != __builtin_inff()) {
#pragma unroll
                    for (int n = 0; n < S; ++n) h[n] = fmaf(decay(sum, A2[n]), in[n], h[n]);
                }
            }
        }
        float xk[J], zk[J], sz[J], slope[J], step[J], g[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            xk[j] = (float)xr[j];
            step[j] = (float)dr[j] + bias;
            g[j] = dyk[j];
            slope[j] = 1.f;
        }
        if (p.softplus) {
#pragma unroll
            for (int j = 0; j < J; ++j) step[j] = softplus_slope(step[j], &slope[j]);
        }
        if (p.z) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                zk[j] = (float)zr[j];
                sz[j] = sigmoid(zk[j]);
                g[j] *= zk[j] * sz[j];
            }
        }
        if (tokens < TQ) {
            // tokens past the end: a zero step leaves the state and its gradient as they are
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (w + W * j >= tokens) step[j] = xk[j] = g[j] = 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < J; ++j) {
            // lanes without a channel of their own add nothing to dB and dC
            su[w + W * j][lane] = make_float2(step[j], mine ? step[j] * xk[j] : 0.f);
            gs[w + W * j][lane] = mine ? g[j] : 0.f;
        }
        if (TH == TQ * N || bi < TQ) {
            const int n = threadIdx.x % N;
            const float b = bi < tokens ? (float)br : 0.f;
            (&Bq[bi / 4][n].x)[bi % 4] = b;
            Bs[bi][n] = b;
            Cs[bi][n] = bi < tokens ? (float)cr : 0.f;
        }
        __syncthreads();
        SeqBits bits{};
        if (SEQ) bits = seq_bits<TQ>(ids, t, p.T, lane);

        float pr[TQ][S], ar[TQ][S];
        TileSums<S> sums_c, sums_b;
        float4 B4;
        static_for<TQ>([&](auto I8) {
            constexpr int i = decltype(I8)::value;
            if (i % 4 == 0) B4 = Bq[i / 4][n0 + lane % S];
            const float Bv = i % 4 == 0 ? B4.x : (i % 4 == 1 ? B4.y : (i % 4 == 2 ? B4.z : B4.w));
            {
                if (SEQ && (bits.starts >> i & 1))
                    load_state<S>(p.init ? p.init + clamp_id(ids[t + i], p.nseqs) * DN + state : nullptr, h);
                const float2 s = su[i][lane];
                const float g = gs[i][lane];
                const States<S> Cv = *(const States<S>*)&Cs[i][n0];
                float acc = 0.f, v[S];
                static_for<S>([&](auto I) {
                    constexpr int n = decltype(I)::value;
                    ar[i][n] = decay(s.x, A2[n]);
                    pr[i][n] = ar[i][n] * h[n];
                    h[n] = pr[i][n] + row_lane<n>(Bv) * s.y;
                    acc = fmaf(Cv.v[n], h[n], acc);
                    v[n] = g * h[n];
                });
                parts[0][w][i][lane] = acc;
                sums_c.template forwards<i>(value_sums<S>(v, lane), lane);
                __builtin_amdgcn_sched_barrier(0);       // (hoisting later tokens' decays costs the occupancy)
            }
        });
        const float total_c = sums_c.result();
        if (stores && hold < tokens) p.part_c[part] = total_c;
        // the way back reads the tile from LDS again: without this the compiler keeps every
        // step size and decay of the way out in registers (120 spilled)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        static_for<TQ>([&](auto I8) {
            constexpr int i = TQ - 1 - decltype(I8)::value;
            {
                if (SEQ && (bits.ends >> i & 1))
                    load_state<S>(p.dfin ? p.dfin + clamp_id(ids[t + i], p.nseqs) * DN + state : nullptr, grad);
                const float2 s = su[i][lane];
                const float g = gs[i][lane];
                const States<S> Bv = *(const States<S>*)&Bs[i][n0], Cv = *(const States<S>*)&Cs[i][n0];
                float du = 0.f, ds = 0.f, v[S];
                static_for<S>([&](auto I) {
                    constexpr int n = decltype(I)::value;
                    const float G = fmaf(Cv.v[n], g, grad[n]);
                    const float m = G * pr[i][n];
                    v[n] = G * s.y;
                    du = fmaf(Bv.v[n], G, du);
                    ds = fmaf(m, A2[n], ds);
                    dA[n] = fmaf(m, s.x, dA[n]);
                    grad[n] = ar[i][n] * G;
                });
                parts[1][w][i][lane] = du;
                parts[2][w][i][lane] = ds;
                sums_b.template backwards<i>(value_sums<S>(v, lane), lane);
                if (SEQ && (bits.starts >> i & 1) && p.dinit && mine)
                    store_f32<S>(p.dinit + clamp_id(ids[t + i], p.nseqs) * DN + state, grad);
                __builtin_amdgcn_sched_barrier(0);
            }
        });
        const float total_b = sums_b.result();
        if (stores && hold < tokens) p.part_b[part] = total_b;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int i = w + W * j;
            float y = skip * xk[j], du = 0.f, ds = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                y += parts[0][k][i][lane];
                du += parts[1][k][i][lane];
                ds += parts[2][k][i][lane];
            }
            const float draw = fmaf(xk[j], du, ds * kLn2) * slope[j];       // ds was taken with A in log2 units
            if (i >= tokens || !mine) continue;
            sum_skip = fmaf(g[j], xk[j], sum_skip);
            sum_bias += draw;
            const int64_t at = row + i * p.D;
            p.dx[at] = fmaf(step[j], du, skip * g[j]);
            p.ddt[at] = draw;
            if (p.z) p.dz[at] = dyk[j] * y * silu_slope(zk[j], sz[j]);
        }
        x -= TQ * p.ldx;
        dt -= TQ * p.lddt;
        z -= TQ * p.ldz;
        B -= TQ * p.ldb;
        C -= TQ * p.ldc;
        dy -= TQ * p.D;
        row -= TQ * p.D;
        part -= TQ * p.G * N;
    }
    if (!SEQ && q.seg == 0 && p.dinit && mine) store_f32<S>(p.dinit + q.b * DN + state, grad);
    float* sums = p.part_sums + (q.b * p.nseg + q.seg) * (DN + 2 * p.D);
#pragma unroll
    for (int n = 0; n < S; ++n) dA[n] *= A2[n] * kLn2;           // dA_log = dA A
    if (mine) store_f32<S>(sums + state, dA);
    if constexpr (W > 1) {
        __syncthreads();
        parts[0][w][0][lane] = sum_skip;
        parts[1][w][0][lane] = sum_bias;
        __syncthreads();
        if (w == 0) {
#pragma unroll
            for (int k = 1; k < W; ++k) {
                sum_skip += parts[0][k][0][lane];
                sum_bias += parts[1][k][0][lane];
            }
        }
    }
    if (w == 0 && mine) {
        sums[DN + d] = sum_skip;
        sums[DN + p.D + d] = sum_bias;
    }
}

// dB and dC: sums over a group's channel blocks, in block order, four values a thread.
__global__ __launch_bounds__(256) void sel_group_sums_kernel(const float* pb, const float* pc, float* dB, float* dC,
                                                             int64_t n4, int blocks) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n4) return;
    const float* src = blockIdx.y ? pc : pb;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    int k = 0;
    for (; k + 8 <= blocks; k += 8) {
        float v[8][4];
#pragma unroll
        for (int u = 0; u < 8; ++u) load_f32<4>(src + ((k + u) * n4 + i) * 4, v[u]);
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] += v[u][e];
    }
    for (; k < blocks; ++k) {
        float v[4];
        load_f32<4>(src + (k * n4 + i) * 4, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += v[e];
    }
    store_f32<4>((blockIdx.y ? dC : dB) + 4 * i, acc);
}

template <typename T, int N, bool REV> static void locals_n(const SelParams& p, hipStream_t s) {
    constexpr int S = 8;
    const dim3 grid((unsigned)(p.batch * p.nseg * p.G * p.blocks)), block(SelShape<N, 64, S>::THREADS);
    if (p.seq_idx) hipLaunchKernelGGL((sel_locals_kernel<T, N, S, true, REV>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((sel_locals_kernel<T, N, S, false, REV>), grid, block, 0, s, p);
}
template <typename T, int N> static void reverse_n(const SelParams& p, hipStream_t s) {
    constexpr int S = N <= 32 ? 4 : 8;
    const dim3 grid((unsigned)(p.batch * p.nseg * p.G * p.blocks)), block(SelShape<N, 64, S>::THREADS);
    if (p.seq_idx) hipLaunchKernelGGL((sel_reverse_kernel<T, N, S, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((sel_reverse_kernel<T, N, S, false>), grid, block, 0, s, p);
}
int64_t sel_ckpt_tile() { return kTile; }

hipError_t launch_sel_locals(const SelParams& p, int dtype, int64_t N, hipStream_t s) {
#define CALL(n)                                                                                                    \
    p.nseg > 1 ? (dtype == SSD_DTYPE_BF16 ? locals_n<__bf16, n, true>(p, s) : locals_n<float, n, true>(p, s))     \
               : (dtype == SSD_DTYPE_BF16 ? locals_n<__bf16, n, false>(p, s) : locals_n<float, n, false>(p, s))
    SSD_SEL_BY_STATE(N, CALL)
#undef CALL
    return hipGetLastError();
}
hipError_t launch_sel_reverse(const SelParams& p, int dtype, int64_t N, hipStream_t s) {
#define CALL(n) dtype == SSD_DTYPE_BF16 ? reverse_n<__bf16, n>(p, s) : reverse_n<float, n>(p, s)
    SSD_SEL_BY_STATE(N, CALL)
#undef CALL
    return hipGetLastError();
}
hipError_t launch_sel_group_sums(const SelParams& p, int64_t N, float* dB, float* dC, hipStream_t s) {
    const int64_t n4 = p.batch * p.T * p.G * N / 4;
    hipLaunchKernelGGL(sel_group_sums_kernel, dim3((unsigned)((n4 + 255) / 256), 2), dim3(256), 0, s, p.part_b, p.part_c,
                       dB, dC, n4, p.blocks);
    return hipGetLastError();
}

}  // namespace ssd
