// Selective scan, forward: the scan over whole rows or segments, the local pass and the
// combine of split rows, and the single-token step.
#include "selective.hpp"

namespace ssd {

// ---------------------------------------------------------------- scan
// One workgroup per 64 channels: N/S waves, each with the same 64 channels and S of the
// states, so B and C are the same for every lane of a wave and y needs one sum over
// waves per (token, channel) instead of one over lanes.  Per tile of TQ tokens:
//   - the waves share out the tokens, each computing step and step x once (LDS), and
//     stage B and C as fp32; the next tile's loads are issued then;
//   - every wave walks the tile with its states and leaves its part of y in LDS;
//   - the waves share out the tokens again, sum the parts, add D x, gate and store.
template <typename T, int N, int S, bool SEQ> __global__ __launch_bounds__(64 * (N / S))
void sel_forward_kernel(SelParams p) {
    constexpr int W = N / S, TQ = 16, J = TQ / W, E = TQ * N / (64 * W);
    static_assert(TQ % W == 0 && E * 64 * W == TQ * N, "tile shape");
    __shared__ float2 su[TQ][64];
    __shared__ float Bs[TQ][N], Cs[TQ][N];
    __shared__ float part[W][TQ][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const SelPlace q = sel_place(p, lane);
    const int32_t* ids = SEQ ? p.seq_idx + q.b * p.T : nullptr;
    const T* x = (const T*)p.x + q.b * p.T * p.ldx + q.d;
    const T* dt = (const T*)p.dt + q.b * p.T * p.lddt + q.d;
    const T* z = p.z ? (const T*)p.z + q.b * p.T * p.ldz + q.d : nullptr;
    const T* B = (const T*)p.B + q.b * p.T * p.ldb + q.g * N;
    const T* C = (const T*)p.C + q.b * p.T * p.ldc + q.g * N;
    T* y = (T*)p.y + q.b * p.T * p.D + q.d;
    const float bias = p.dt_bias ? p.dt_bias[q.d] : 0.f, skip = p.skip ? p.skip[q.d] : 0.f;
    float A2[S], h[S];
    load_decay<S>(p, q.d, N, w * S, A2);
    const int64_t state = q.d * N + w * S, DN = p.D * N;
    load_state<S>(q.seg > 0 ? p.seg_state + (q.b * (p.nseg - 1) + q.seg - 1) * DN + state
                            : (p.init && !SEQ ? p.init + q.b * DN + state : nullptr), h);

    T xr[J], dr[J], zr[J], br[E], cr[E];
    auto load = [&](int64_t t) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t i = t + w + W * j;
            if (i < q.t1) {
                xr[j] = x[i * p.ldx];
                dr[j] = dt[i * p.lddt];
                if (z) zr[j] = z[i * p.ldz];
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int k = threadIdx.x + 64 * W * e;
            const int64_t i = t + k / N;
            if (i < q.t1) {
                br[e] = B[i * p.ldb + k % N];
                cr[e] = C[i * p.ldc + k % N];
            }
        }
    };
    load(q.t0);
    for (int64_t t = q.t0; t < q.t1; t += TQ) {
        float xk[J], zk[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            // tokens past the end take a zero step: they leave the state as it is
            const bool in = t + w + W * j < q.t1;
            const float step = in ? step_of((float)dr[j] + bias, p.softplus) : 0.f;
            xk[j] = in ? (float)xr[j] : 0.f;
            zk[j] = in && z ? (float)zr[j] : 0.f;
            su[w + W * j][lane] = make_float2(step, step * xk[j]);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int k = threadIdx.x + 64 * W * e;
            const bool in = t + k / N < q.t1;
            Bs[k / N][k % N] = in ? (float)br[e] : 0.f;
            Cs[k / N][k % N] = in ? (float)cr[e] : 0.f;
        }
        __syncthreads();
        if (t + TQ < q.t1) load(t + TQ);
        SeqBits bits{};
        if (SEQ) bits = seq_bits<TQ>(ids, t, p.T, lane);
#pragma unroll
        for (int i = 0; i < TQ; ++i) {
            if (SEQ && (bits.starts >> i & 1))
                load_state<S>(p.init ? p.init + clamp_id(ids[t + i], p.nseqs) * DN + state : nullptr, h);
            const float2 s = su[i][lane];
            float acc = 0.f;
#pragma unroll
            for (int n = 0; n < S; ++n) {
                h[n] = fmaf(decay(s.x, A2[n]), h[n], s.y * Bs[i][w * S + n]);
                acc = fmaf(h[n], Cs[i][w * S + n], acc);
            }
            part[w][i][lane] = acc;
            if (SEQ && (bits.ends >> i & 1) && p.fin && q.mine)
                store_f32<S>(p.fin + clamp_id(ids[t + i], p.nseqs) * DN + state, h);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int i = w + W * j;
            float out = skip * xk[j];
#pragma unroll
            for (int k = 0; k < W; ++k) out += part[k][i][lane];
            if (z) out *= silu_for<T>(zk[j]);
            if (q.mine && t + i < q.t1) y[(t + i) * p.D] = (T)out;
        }
    }
    if (!SEQ && q.seg == p.nseg - 1 && p.fin && q.mine) store_f32<S>(p.fin + q.b * DN + state, h);
}

// ---------------------------------------------------------------- local pass of split rows
// The scan of one segment without its read-out, from a zero state (the first segment:
// from the row's initial state): the segment's end state and the sum of its steps, whose
// decay exp(A sum) is what an incoming state would still weigh; infinite when a sequence
// starts inside, so that nothing comes through.  For the backward pass (CKPT) the same
// two are also kept before every tile.  A wave on its own, up to 16 states a lane.
template <typename T, int N, int S, bool SEQ, bool CKPT, int TQ> __global__ __launch_bounds__(64 * (N / S))
void sel_local_kernel(SelParams p) {
    constexpr int W = N / S, J = TQ / W, E = TQ * N / (64 * W);
    static_assert(TQ % W == 0 && E * 64 * W == TQ * N, "tile shape");
    __shared__ float2 su[TQ][64];
    __shared__ float Bs[TQ][N];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const SelPlace q = sel_place(p, lane);
    if (!CKPT && q.seg == p.nseg - 1) return;
    const int32_t* ids = SEQ ? p.seq_idx + q.b * p.T : nullptr;
    const T* x = (const T*)p.x + q.b * p.T * p.ldx + q.d;
    const T* dt = (const T*)p.dt + q.b * p.T * p.lddt + q.d;
    const T* B = (const T*)p.B + q.b * p.T * p.ldb + q.g * N;
    const float bias = p.dt_bias ? p.dt_bias[q.d] : 0.f;
    float A2[S], h[S], sum = 0.f;
    load_decay<S>(p, q.d, N, w * S, A2);
    const int64_t state = q.d * N + w * S, DN = p.D * N;
    load_state<S>(q.seg == 0 && p.init && !SEQ ? p.init + q.b * DN + state : nullptr, h);
    T xr[J], dr[J], br[E];
    auto load = [&](int64_t t) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t i = t + w + W * j;
            if (i < q.t1) {
                xr[j] = x[i * p.ldx];
                dr[j] = dt[i * p.lddt];
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int k = threadIdx.x + 64 * W * e;
            if (t + k / N < q.t1) br[e] = B[(t + k / N) * p.ldb + k % N];
        }
    };
    load(q.t0);
    const int64_t tiles = (p.T + TQ - 1) / TQ;
    for (int64_t t = q.t0; t < q.t1; t += TQ) {
        if (CKPT && q.mine) {
            const int64_t at = (q.b * tiles + t / TQ) * p.D + q.d;
            store_f32<S>(p.ckpt + at * N + w * S, h);
            if (w == 0) p.ckpt_step[at] = sum;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool in = t + w + W * j < q.t1;
            const float step = in ? step_of((float)dr[j] + bias, p.softplus) : 0.f;
            su[w + W * j][lane] = make_float2(step, in ? step * (float)xr[j] : 0.f);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int k = threadIdx.x + 64 * W * e;
            Bs[k / N][k % N] = t + k / N < q.t1 ? (float)br[e] : 0.f;
        }
        __syncthreads();
        if (t + TQ < q.t1) load(t + TQ);
        SeqBits bits{};
        if (SEQ) bits = seq_bits<TQ>(ids, t, p.T, lane);
#pragma unroll
        for (int i = 0; i < TQ; ++i) {
            if (SEQ && (bits.starts >> i & 1)) {
                load_state<S>(p.init ? p.init + clamp_id(ids[t + i], p.nseqs) * DN + state : nullptr, h);
                sum = __builtin_inff();
            }
            const float2 s = su[i][lane];
            sum += s.x;
#pragma unroll
            for (int n = 0; n < S; ++n) h[n] = fmaf(decay(s.x, A2[n]), h[n], s.y * Bs[i][w * S + n]);
        }
    }
    if (q.seg < p.nseg - 1 && q.mine) {
        const int64_t at = (q.b * (p.nseg - 1) + q.seg) * p.D + q.d;
        store_f32<S>(p.seg_state + at * N + w * S, h);
        if (w == 0) p.seg_step[at] = sum;
    }
}

// In-place scan over a row's segments, a thread per (row, channel, state).  Forward:
// seg_state[s] becomes the state after segment s; reverse: seg_grad[s] (of segment s+1)
// becomes the gradient reaching that segment's incoming state.
template <bool REVERSE> __global__ __launch_bounds__(256) void sel_combine_kernel(SelParams p, int N) {
    const int64_t DN = p.D * N, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.batch * DN) return;
    const int64_t b = i / DN, e = i % DN;
    const int ns = p.nseg - 1;
    float* st = (REVERSE ? p.seg_grad : p.seg_state) + b * ns * DN + e;
    const float* sum = p.seg_step + b * ns * p.D + e / N;
    const float A2 = decay_rate(p.A_log[e]);
    float carry = 0.f;
    // segment s lets exp(A sum) of what enters it through (forward: s = 1 .., reverse:
    // segment s+1 of seg_grad[s]); eight segments' loads are issued ahead
    for (int k0 = 0; k0 < ns; k0 += 8) {
        float l[8], c[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int s = REVERSE ? ns - 1 - k0 - k : k0 + k;
            if (k0 + k < ns) {
                l[k] = st[s * DN];
                c[k] = REVERSE ? (s + 1 < ns ? sum[(s + 1) * p.D] : 0.f) : sum[s * p.D];
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int s = REVERSE ? ns - 1 - k0 - k : k0 + k;
            if (k0 + k >= ns) break;
            // selected, not multiplied by zero: an Inf or NaN of another sequence stays there
            carry = k0 + k == 0 || c[k] == __builtin_inff() ? l[k] : fmaf(decay(c[k], A2), carry, l[k]);
            st[s * DN] = carry;
        }
    }
}

// ---------------------------------------------------------------- step
// One token: N/4 lanes per channel, four states each; bound by the state's read and
// write at large batches and by the launch at small ones.
template <typename T, int N> __global__ __launch_bounds__(256) void sel_step_kernel(SelParams p) {
    constexpr int L = N / 4, R = 256 / L;                // channels per workgroup
    const int c = threadIdx.x % L;
    const int64_t i = (int64_t)blockIdx.x * R + threadIdx.x / L;
    if (i >= p.batch * p.D) return;
    const int64_t b = i / p.D, d = i % p.D, g = d / p.per_group;
    float h[4], A[4], Bv[4], Cv[4];
    load_f32<4>(p.init + i * N + 4 * c, h);
    load_f32<4>(p.A_log + d * N + 4 * c, A);
    load_f32<4>((const T*)p.B + b * p.ldb + g * N + 4 * c, Bv);
    load_f32<4>((const T*)p.C + b * p.ldc + g * N + 4 * c, Cv);
    const float x = (float)((const T*)p.x)[b * p.ldx + d];
    const float step = step_of((float)((const T*)p.dt)[b * p.lddt + d] + (p.dt_bias ? p.dt_bias[d] : 0.f), p.softplus);
    float acc = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        h[k] = fmaf(decay(step, decay_rate(A[k])), h[k], step * x * Bv[k]);
        acc = fmaf(h[k], Cv[k], acc);
    }
    store_f32<4>(p.fin + i * N + 4 * c, h);
#pragma unroll
    for (int k = 1; k < L; k <<= 1) acc += __shfl_xor(acc, k);
    if (c == 0) {
        acc = fmaf(p.skip ? p.skip[d] : 0.f, x, acc);
        if (p.z) acc *= silu_for<T>((float)((const T*)p.z)[b * p.ldz + d]);
        ((T*)p.y)[i] = (T)acc;
    }
}

// ---------------------------------------------------------------- launches
static unsigned sel_grid(const SelParams& p) { return (unsigned)(p.batch * p.nseg * p.G * p.blocks); }

template <typename T, int N> static void forward_n(const SelParams& p, hipStream_t s) {
    constexpr int S = N <= 16 ? 4 : N / 4;
    if (p.seq_idx) hipLaunchKernelGGL((sel_forward_kernel<T, N, S, true>), dim3(sel_grid(p)), dim3(64 * (N / S)), 0, s, p);
    else hipLaunchKernelGGL((sel_forward_kernel<T, N, S, false>), dim3(sel_grid(p)), dim3(64 * (N / S)), 0, s, p);
}
template <typename T, int N, bool CKPT> static void local_n(const SelParams& p, hipStream_t s) {
    constexpr int S = N <= 16 ? N : 16, TQ = CKPT ? 8 : 16;
    const dim3 grid(sel_grid(p)), block(64 * (N / S));
    if (p.seq_idx) hipLaunchKernelGGL((sel_local_kernel<T, N, S, true, CKPT, TQ>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((sel_local_kernel<T, N, S, false, CKPT, TQ>), grid, block, 0, s, p);
}

int64_t sel_ckpt_tile() { return 8; }

hipError_t launch_sel_forward(const SelParams& p, int dtype, int64_t N, hipStream_t s) {
#define CALL(n) dtype == SSD_DTYPE_BF16 ? forward_n<__bf16, n>(p, s) : forward_n<float, n>(p, s)
    SSD_SEL_BY_STATE(N, CALL)
#undef CALL
    return hipGetLastError();
}
hipError_t launch_sel_local(const SelParams& p, int dtype, int64_t N, bool checkpoints, hipStream_t s) {
#define CALL(n)                                                                                              \
    checkpoints ? (dtype == SSD_DTYPE_BF16 ? local_n<__bf16, n, true>(p, s) : local_n<float, n, true>(p, s)) \
                : (dtype == SSD_DTYPE_BF16 ? local_n<__bf16, n, false>(p, s) : local_n<float, n, false>(p, s))
    SSD_SEL_BY_STATE(N, CALL)
#undef CALL
    return hipGetLastError();
}
hipError_t launch_sel_combine(const SelParams& p, int64_t N, bool reverse, hipStream_t s) {
    const dim3 grid((unsigned)((p.batch * p.D * N + 255) / 256));
    if (reverse) hipLaunchKernelGGL(sel_combine_kernel<true>, grid, dim3(256), 0, s, p, (int)N);
    else hipLaunchKernelGGL(sel_combine_kernel<false>, grid, dim3(256), 0, s, p, (int)N);
    return hipGetLastError();
}
template <typename T, int N> static void step_n(const SelParams& p, hipStream_t s) {
    const int64_t threads = p.batch * p.D * (N / 4);
    hipLaunchKernelGGL((sel_step_kernel<T, N>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, p);
}
hipError_t launch_sel_step(const SelParams& p, int dtype, int64_t N, hipStream_t s) {
#define CALL(n) dtype == SSD_DTYPE_BF16 ? step_n<__bf16, n>(p, s) : step_n<float, n>(p, s)
    SSD_SEL_BY_STATE(N, CALL)
#undef CALL
    return hipGetLastError();
}

}  // namespace ssd
