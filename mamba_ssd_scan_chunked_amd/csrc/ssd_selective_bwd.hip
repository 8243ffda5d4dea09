// Selective scan, gradients.  With G_t = dL/dh_t = g_t C_t + q_t, where g = dL/d(y before
// the gate) and q_t = exp(step_{t+1} A) G_{t+1} reaches token t's state from later tokens
// (dL/dfinal after the last), and p_t = exp(step_t A) h_{t-1}:
//   dB_t[n] = sum_d G step x,  dC_t[n] = sum_d g h,  d(step x) = sum_n G B,
//   dstep = sum_n G p A + x d(step x),  dA = sum_t G p step,  dx = step d(step x) + D g.
//
// The states are not kept by the forward pass: the local pass leaves one before every
// tile of eight tokens, and the reverse pass runs a tile forwards (keeping p in registers)
// and then backwards, the decay being computed again there, which takes fewer cycles than
// the registers that would hold it cost in occupancy.
#include "selective.hpp"

namespace ssd {

constexpr int kTile = 8;

// Sums over the 64 lanes of S values at once: at every level a lane keeps half of the
// values and hands the other half to its partner (swaps of 32 and 16 lanes, then lanes of
// a row), so S values cost about 2 S instructions instead of 6 S.  Returns, in every lane,
// the sum of value sum_index<S>(lane).
template <int CTRL> __device__ inline float dpp_mov(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <int S> __device__ inline int sum_index(int lane) {
    return S == 16 ? (lane >> 2 & 1) + 2 * (lane >> 3 & 1) + 4 * (lane >> 4) : (lane >> 3 & 1) + 2 * (lane >> 4);
}
template <int S> __device__ inline float lane_sums(const float (&v)[S], int lane) {
    static_assert(S == 8 || S == 16, "values");
    constexpr int H = S / 2, Q = S / 4;
    float a[H], b[Q];
#pragma unroll
    for (int k = 0; k < H; ++k) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[k]), __float_as_uint(v[k + H]), false, false);
        a[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
#pragma unroll
    for (int k = 0; k < Q; ++k) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a[k]), __float_as_uint(a[k + Q]), false, false);
        b[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    const bool hi = lane & 8;
    float c[Q / 2];
#pragma unroll
    for (int k = 0; k < Q / 2; ++k) c[k] = (hi ? b[k + Q / 2] : b[k]) + dpp_mov<0x140>(hi ? b[k] : b[k + Q / 2]);   // row_mirror
    float s;
    if constexpr (S == 16) {
        const bool up = lane & 4;
        s = (up ? c[1] : c[0]) + dpp_mov<0x141>(up ? c[0] : c[1]);                       // row_half_mirror
    } else {
        s = c[0] + dpp_mov<0x141>(c[0]);
    }
    s += dpp_mov<0xb1>(s);      // quad_perm 1,0,3,2
    s += dpp_mov<0x4e>(s);      // quad_perm 2,3,0,1
    return s;
}

__device__ inline int64_t last_tile(const SelPlace& q) { return q.t0 + (q.t1 - q.t0 - 1) / kTile * kTile; }

// ---------------------------------------------------------------- local reverse pass
// For rows in segments: what a segment's own tokens send back through its first token, q
// from zero (the row's last segment: from dfinal).  Kept for segments 1 .. nseg-1.
template <typename T, int N, int S, bool SEQ> __global__ __launch_bounds__(64 * (N / S))
void sel_reverse_local_kernel(SelParams p) {
    constexpr int W = N / S, TQ = kTile, J = TQ / W, E = TQ * N / (64 * W);
    __shared__ float2 sg[TQ][64];
    __shared__ float Cs[TQ][N];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const SelPlace q = sel_place(p, lane);
    if (q.seg == 0) return;
    const int32_t* ids = SEQ ? p.seq_idx + q.b * p.T : nullptr;
    const T* dt = (const T*)p.dt + q.b * p.T * p.lddt + q.d;
    const T* z = p.z ? (const T*)p.z + q.b * p.T * p.ldz + q.d : nullptr;
    const T* C = (const T*)p.C + q.b * p.T * p.ldc + q.g * N;
    const float* dy = p.dy + q.b * p.T * p.D + q.d;
    const float bias = p.dt_bias ? p.dt_bias[q.d] : 0.f;
    float A2[S], grad[S];
    load_decay<S>(p, q.d, N, w * S, A2);
    const int64_t state = q.d * N + w * S, DN = p.D * N;
    load_state<S>(!SEQ && q.seg == p.nseg - 1 && p.dfin ? p.dfin + q.b * DN + state : nullptr, grad);
    for (int64_t t = last_tile(q); t >= q.t0; t -= TQ) {
        float step[J], g[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t i = t + w + W * j;
            step[j] = g[j] = 0.f;
            if (i < q.t1) {
                step[j] = step_of((float)dt[i * p.lddt] + bias, p.softplus);
                g[j] = dy[i * p.D] * (z ? silu((float)z[i * p.ldz]) : 1.f);
            }
        }
        float cv[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int k = threadIdx.x + 64 * W * e;
            cv[e] = t + k / N < q.t1 ? (float)C[(t + k / N) * p.ldc + k % N] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < J; ++j) sg[w + W * j][lane] = make_float2(step[j], g[j]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int k = threadIdx.x + 64 * W * e;
            Cs[k / N][k % N] = cv[e];
        }
        __syncthreads();
        SeqBits bits{};
        if (SEQ) bits = seq_bits<TQ>(ids, t, p.T, lane);
#pragma unroll
        for (int i = TQ - 1; i >= 0; --i) {
            if (SEQ && (bits.ends >> i & 1))
                load_state<S>(p.dfin ? p.dfin + clamp_id(ids[t + i], p.nseqs) * DN + state : nullptr, grad);
            const float2 s = sg[i][lane];
#pragma unroll
            for (int n = 0; n < S; ++n) grad[n] = decay(s.x, A2[n]) * fmaf(s.y, Cs[i][w * S + n], grad[n]);
            // what leaves a sequence's first token goes to its initial state, not to the segment before
            if (SEQ && (bits.starts >> i & 1)) load_state<S>(nullptr, grad);
        }
    }
    if (q.mine) store_f32<S>(p.seg_grad + (q.b * (p.nseg - 1) + q.seg - 1) * DN + state, grad);
}

// ---------------------------------------------------------------- reverse pass
// One workgroup per 64 channels and segment, N/S waves with S <= 16 states each (one wave
// for N <= 16: no partial sums over waves, no barriers).
template <typename T, int N, int S, bool SEQ> __global__ __launch_bounds__(64 * (N / S), 2)
void sel_reverse_kernel(SelParams p) {
    constexpr int W = N / S, TQ = kTile, J = TQ / W, E = TQ * N / (64 * W), HOLD = 64 / S;   // HOLD tokens per store
    __shared__ float2 su[TQ][64];
    __shared__ float gs[TQ][64];
    __shared__ float Bs[TQ][N], Cs[TQ][N];
    __shared__ float parts[3][W][TQ][64];                        // of y, d(step x) and dstep
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const SelPlace q = sel_place(p, lane);
    const int32_t* ids = SEQ ? p.seq_idx + q.b * p.T : nullptr;
    const T* x = (const T*)p.x + q.b * p.T * p.ldx + q.d;
    const T* dt = (const T*)p.dt + q.b * p.T * p.lddt + q.d;
    const T* z = p.z ? (const T*)p.z + q.b * p.T * p.ldz + q.d : nullptr;
    const T* B = (const T*)p.B + q.b * p.T * p.ldb + q.g * N;
    const T* C = (const T*)p.C + q.b * p.T * p.ldc + q.g * N;
    const int64_t row = q.b * p.T * p.D + q.d;
    const float bias = p.dt_bias ? p.dt_bias[q.d] : 0.f, skip = p.skip ? p.skip[q.d] : 0.f;
    float A2[S], grad[S], dA[S], sum_skip = 0.f, sum_bias = 0.f;
    load_decay<S>(p, q.d, N, w * S, A2);
    const int64_t state = q.d * N + w * S, DN = p.D * N;
    load_state<S>(q.seg < p.nseg - 1 ? p.seg_grad + (q.b * (p.nseg - 1) + q.seg) * DN + state
                                     : (!SEQ && p.dfin ? p.dfin + q.b * DN + state : nullptr), grad);
#pragma unroll
    for (int n = 0; n < S; ++n) dA[n] = 0.f;
    const float* before = q.seg > 0 ? p.seg_state + (q.b * (p.nseg - 1) + q.seg - 1) * DN + state : nullptr;
    const int64_t tiles = (p.T + TQ - 1) / TQ;
    // part_b and part_c: (block, batch, T, G, N); the lane's value and token of a store
    const int64_t part0 = (((int64_t)q.block * p.batch + q.b) * p.T * p.G + q.g) * N + w * S + sum_index<S>(lane);
    const int hold = lane % HOLD;
    for (int64_t t = last_tile(q); t >= q.t0; t -= TQ) {
        float xk[J], zk[J], dyk[J], slope[J], bv[E], cv[E], h[S];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t i = t + w + W * j;
            xk[j] = zk[j] = dyk[j] = slope[j] = 0.f;
            if (i < q.t1) {
                xk[j] = (float)x[i * p.ldx];
                slope[j] = (float)dt[i * p.lddt] + bias;
                dyk[j] = p.dy[row + i * p.D];
                if (z) zk[j] = (float)z[i * p.ldz];
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int k = threadIdx.x + 64 * W * e;
            const bool in = t + k / N < q.t1;
            bv[e] = in ? (float)B[(t + k / N) * p.ldb + k % N] : 0.f;
            cv[e] = in ? (float)C[(t + k / N) * p.ldc + k % N] : 0.f;
        }
        {
            const int64_t at = (q.b * tiles + t / TQ) * p.D + q.d;
            load_f32<S>(p.ckpt + at * N + w * S, h);
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
        __syncthreads();
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool in = t + w + W * j < q.t1;
            const float raw = slope[j], step = in ? step_of(raw, p.softplus) : 0.f;
            // lanes without a channel of their own add nothing to dB and dC
            su[w + W * j][lane] = make_float2(step, q.mine ? step * xk[j] : 0.f);
            gs[w + W * j][lane] = q.mine ? dyk[j] * (z ? silu(zk[j]) : 1.f) : 0.f;
            slope[j] = p.softplus ? sigmoid(raw) : 1.f;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int k = threadIdx.x + 64 * W * e;
            Bs[k / N][k % N] = bv[e];
            Cs[k / N][k % N] = cv[e];
        }
        __syncthreads();
        SeqBits bits{};
        if (SEQ) bits = seq_bits<TQ>(ids, t, p.T, lane);

        float pr[TQ][S], held = 0.f;
#pragma unroll
        for (int i = 0; i < TQ; ++i) {
            if (SEQ && (bits.starts >> i & 1))
                load_state<S>(p.init ? p.init + clamp_id(ids[t + i], p.nseqs) * DN + state : nullptr, h);
            const float2 s = su[i][lane];
            const float g = gs[i][lane];
            float acc = 0.f, v[S];
#pragma unroll
            for (int n = 0; n < S; ++n) {
                pr[i][n] = decay(s.x, A2[n]) * h[n];
                h[n] = fmaf(s.y, Bs[i][w * S + n], pr[i][n]);
                acc = fmaf(h[n], Cs[i][w * S + n], acc);
                v[n] = g * h[n];
            }
            parts[0][w][i][lane] = acc;
            const float c = lane_sums<S>(v, lane);
            held = hold == i % HOLD ? c : held;
            if (i % HOLD == HOLD - 1 && t + i - (HOLD - 1) + hold < q.t1)
                p.part_c[part0 + (t + i - (HOLD - 1) + hold) * p.G * N] = held;
        }
#pragma unroll
        for (int i = TQ - 1; i >= 0; --i) {
            if (SEQ && (bits.ends >> i & 1))
                load_state<S>(p.dfin ? p.dfin + clamp_id(ids[t + i], p.nseqs) * DN + state : nullptr, grad);
            const float2 s = su[i][lane];
            const float g = gs[i][lane];
            float du = 0.f, ds = 0.f, v[S];
#pragma unroll
            for (int n = 0; n < S; ++n) {
                const float G = fmaf(g, Cs[i][w * S + n], grad[n]);
                const float m = G * pr[i][n];
                v[n] = G * s.y;
                du = fmaf(G, Bs[i][w * S + n], du);
                ds = fmaf(m, A2[n], ds);
                dA[n] = fmaf(m, s.x, dA[n]);
                grad[n] = decay(s.x, A2[n]) * G;
            }
            parts[1][w][i][lane] = du;
            parts[2][w][i][lane] = ds;
            const float c = lane_sums<S>(v, lane);
            held = hold == i % HOLD ? c : held;
            if (i % HOLD == 0 && t + i + hold < q.t1) p.part_b[part0 + (t + i + hold) * p.G * N] = held;
            if (SEQ && (bits.starts >> i & 1) && p.dinit && q.mine)
                store_f32<S>(p.dinit + clamp_id(ids[t + i], p.nseqs) * DN + state, grad);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int i = w + W * j;
            if (t + i >= q.t1) continue;
            float y = skip * xk[j], du = 0.f, ds = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                y += parts[0][k][i][lane];
                du += parts[1][k][i][lane];
                ds += parts[2][k][i][lane];
            }
            const float step = su[i][lane].x, g = gs[i][lane];
            const float draw = fmaf(xk[j], du, ds * kLn2) * slope[j];       // ds was taken with A in log2 units
            sum_skip = fmaf(g, xk[j], sum_skip);
            sum_bias += draw;
            if (!q.mine) continue;
            const int64_t at = row + (t + i) * p.D;
            p.dx[at] = fmaf(step, du, skip * g);
            p.ddt[at] = draw;
            if (z) {
                const float s = sigmoid(zk[j]);
                p.dz[at] = dyk[j] * y * silu_slope(zk[j], s);
            }
        }
    }
    if (!SEQ && q.seg == 0 && p.dinit && q.mine) store_f32<S>(p.dinit + q.b * DN + state, grad);
    float* sums = p.part_sums + (q.b * p.nseg + q.seg) * (DN + 2 * p.D);
#pragma unroll
    for (int n = 0; n < S; ++n) dA[n] *= A2[n] * kLn2;           // dA_log = dA A
    if (q.mine) store_f32<S>(sums + state, dA);
    if constexpr (W > 1) {
        __syncthreads();
        parts[0][w][0][lane] = sum_skip;
        parts[0][w][1][lane] = sum_bias;
        __syncthreads();
        if (w == 0) {
#pragma unroll
            for (int k = 1; k < W; ++k) {
                sum_skip += parts[0][k][0][lane];
                sum_bias += parts[0][k][1][lane];
            }
        }
    }
    if (w == 0 && q.mine) {
        sums[DN + q.d] = sum_skip;
        sums[DN + p.D + q.d] = sum_bias;
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

template <typename T, int N> static void reverse_n(const SelParams& p, bool local, hipStream_t s) {
    constexpr int S = N <= 16 ? N : 16;
    const dim3 grid((unsigned)(p.batch * p.nseg * p.G * p.blocks)), block(64 * (N / S));
    if (local) {
        if (p.seq_idx) hipLaunchKernelGGL((sel_reverse_local_kernel<T, N, S, true>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((sel_reverse_local_kernel<T, N, S, false>), grid, block, 0, s, p);
    } else {
        if (p.seq_idx) hipLaunchKernelGGL((sel_reverse_kernel<T, N, S, true>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((sel_reverse_kernel<T, N, S, false>), grid, block, 0, s, p);
    }
}
static hipError_t reverse(const SelParams& p, int dtype, int64_t N, bool local, hipStream_t s) {
#define CALL(n) dtype == SSD_DTYPE_BF16 ? reverse_n<__bf16, n>(p, local, s) : reverse_n<float, n>(p, local, s)
    SSD_SEL_BY_STATE(N, CALL)
#undef CALL
    return hipGetLastError();
}
hipError_t launch_sel_reverse_local(const SelParams& p, int dtype, int64_t N, hipStream_t s) {
    return reverse(p, dtype, N, true, s);
}
hipError_t launch_sel_reverse(const SelParams& p, int dtype, int64_t N, hipStream_t s) {
    return reverse(p, dtype, N, false, s);
}
hipError_t launch_sel_group_sums(const SelParams& p, int64_t N, float* dB, float* dC, hipStream_t s) {
    const int64_t n4 = p.batch * p.T * p.G * N / 4;
    hipLaunchKernelGGL(sel_group_sums_kernel, dim3((unsigned)((n4 + 255) / 256), 2), dim3(256), 0, s, p.part_b, p.part_c,
                       dB, dC, n4, p.blocks);
    return hipGetLastError();
}

}  // namespace ssd
