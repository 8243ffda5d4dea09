// Selective scan, forward: the scan over whole rows or segments, the local pass and the
// combine of split rows, and the single-token step.
#include "selective.hpp"

namespace ssd {

// ---------------------------------------------------------------- scan
// Per tile of TQ tokens:
//   - the threads share out the tile's (token, channel) pairs, each computing step and
//     step x once (LDS), and stage B and C as fp32; the next tile's loads are issued then;
//   - every wave walks the tile with its states and leaves its part of y in LDS;
//   - the threads share out the pairs again, sum the parts, add D x, gate and store.
//
// Bound by vector instructions: per (token, channel) 16 states x 5 (a multiply and an exp2 for
// the decay, a multiply by the row broadcast of B, two fused multiply-adds) and some 50 for
// the step size, the gate and the sums.  A wave's instruction takes a SIMD about 1.84 ns and
// exp2 3.95, which makes 0.23 ms for the states alone at 4 x 4096 tokens, 5120 channels, 16
// states and 0.33 with the rest; measured 0.46 (bf16, gated, softplus; fp32 0.47), with the vector
// units at work for 65 % of the time, as 640 workgroups of 32 channels are 2.5 for each of 256
// compute units.  (The 64 bytes that 32 bf16 channels take of a token are half a cache line, and
// most lines are fetched twice: 1066 MB for 507 of inputs, 2.7 TB/s in all.)  Rows whole in 64-channel
// workgroups of four states a lane take 0.65, in 16-channel waves 0.66, with B and C from LDS
// per state instead of by row broadcasts 0.79; two buffers and one barrier a tile 0.59.
// Rows in segments take 64-channel workgroups of four states a lane (16384 tokens of 1536
// channels: 0.18 ms for the local pass, the combine and the scan, at work for 81 and 87 % of the
// two passes; 32-channel ones 0.22).
template <typename T, int N, int CH, int S, bool SEQ>
__global__ __launch_bounds__((SelShape<N, CH, S>::THREADS)) void sel_forward_kernel(SelParams p) {
    using Sh = SelShape<N, CH, S>;
    constexpr int W = Sh::W, TH = Sh::THREADS, TQ = 32, J = TQ * CH / TH, E = (TQ * N + TH - 1) / TH;
    static_assert(J * TH == TQ * CH, "tile shape");
    __shared__ float2 su[TQ][CH];
    __shared__ float4 Bs[TQ / 4][N];                             // four tokens of a state together
    __shared__ __attribute__((aligned(16))) float Cs[TQ][N];     // a token's states together
    __shared__ float part[W][TQ][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const SelPlace q = sel_place<CH>(p);
    const int ch = lane % CH, n0 = (w * Sh::M + lane / CH) * S;
    const bool mine = ch < q.chans;
    const int64_t d = q.d0 + (mine ? ch : q.chans - 1);
    const int32_t* ids = SEQ ? p.seq_idx + q.b * p.T : nullptr;
    const int64_t tok = q.b * p.T + q.t0;
    const T* x = (const T*)p.x + tok * p.ldx + q.d0;
    const T* dt = (const T*)p.dt + tok * p.lddt + q.d0;
    const T* z = (const T*)(p.z ? p.z : p.x) + tok * p.ldz + q.d0;      // (without a gate: read and not used)
    const T* B = (const T*)p.B + tok * p.ldb + q.g * N;
    const T* C = (const T*)p.C + tok * p.ldc + q.g * N;
    T* y = (T*)p.y + tok * p.D + q.d0;
    // of the thread's own pairs: their channel is the same for every j when CH divides TH
    const int pc = threadIdx.x % CH;
    const int64_t pd = q.d0 + (pc < q.chans ? pc : q.chans - 1);
    const float bias = p.dt_bias ? p.dt_bias[pd] : 0.f, skip = p.skip ? p.skip[pd] : 0.f;
    float A2[S], h[S];
    load_decay<S>(p, d, N, n0, A2);
    const int64_t state = d * N + n0, DN = p.D * N;
    load_state<S>(q.seg > 0 ? p.seg_state + (q.b * (p.nseg - 1) + q.seg - 1) * DN + state
                            : (p.init && !SEQ ? p.init + q.b * DN + state : nullptr), h);

    TileLoad<T, J, CH, TH> lx, ld, lz, ly;
    TileLoad<T, E, N, TH> lb, lc;
    ly.place(p.D, q.chans, TQ);
    T xr[J], dr[J], zr[J], br[E], cr[E];
    auto load = [&](int64_t left) {
        if (left < TQ || left == q.t1 - q.t0) {
            const int tokens = left < TQ ? (int)left : TQ;
            lx.place(p.ldx, q.chans, tokens);
            ld.place(p.lddt, q.chans, tokens);
            lz.place(p.ldz, q.chans, tokens);
            lb.place(p.ldb, N, tokens);
            lc.place(p.ldc, N, tokens);
        }
        lx.load(x, xr);
        ld.load(dt, dr);
        if (p.z) lz.load(z, zr);
        lb.load(B, br);
        lc.load(C, cr);
        x += TQ * p.ldx;
        dt += TQ * p.lddt;
        z += TQ * p.ldz;
        B += TQ * p.ldb;
        C += TQ * p.ldc;
    };
    load(q.t1 - q.t0);
    for (int64_t t = q.t0; t < q.t1; t += TQ, y += TQ * p.D) {
        const int tokens = q.t1 - t < TQ ? (int)(q.t1 - t) : TQ;
        float xk[J], zk[J], step[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            xk[j] = (float)xr[j];
            zk[j] = (float)zr[j];
            step[j] = (float)dr[j] + bias;
        }
        map_steps(step, p.softplus);
        if (tokens < TQ) {
            // tokens past the end take a zero step: they leave the state as it is
#pragma unroll
            for (int j = 0; j < J; ++j)
                if ((threadIdx.x + TH * j) / CH >= tokens) step[j] = xk[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < J; ++j) su[(threadIdx.x + TH * j) / CH][pc] = make_float2(step[j], step[j] * xk[j]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int k = threadIdx.x + TH * e, i = k / N;
            if (E * TH > TQ * N && i >= TQ) continue;
            (&Bs[i / 4][k % N].x)[i % 4] = i < tokens ? (float)br[e] : 0.f;
            Cs[i][k % N] = i < tokens ? (float)cr[e] : 0.f;
        }
        __syncthreads();
        if (t + TQ < q.t1) load(q.t1 - t - TQ);
        SeqBits bits{};
        if (SEQ) bits = seq_bits<TQ>(ids, t, p.T, lane);
#pragma unroll
        for (int i4 = 0; i4 < TQ / 4; ++i4) {
            const float4 B4 = Bs[i4][n0 + lane % S];
            const float Bv[4] = {B4.x, B4.y, B4.z, B4.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = 4 * i4 + k;
                if (SEQ && (bits.starts >> i & 1))
                    load_state<S>(p.init ? p.init + clamp_id(ids[t + i], p.nseqs) * DN + state : nullptr, h);
                const float2 s = su[i][ch];
                const States<S> Cv = *(const States<S>*)&Cs[i][n0];
                float acc = 0.f;
                static_for<S>([&](auto I) {
                    constexpr int n = decltype(I)::value;
                    h[n] = fmaf(decay(s.x, A2[n]), h[n], row_lane<n>(Bv[k]) * s.y);
                    acc = fmaf(Cv.v[n], h[n], acc);
                });
                part[w][i][lane] = acc;
                if (SEQ && (bits.ends >> i & 1) && p.fin && mine)
                    store_f32<S>(p.fin + clamp_id(ids[t + i], p.nseqs) * DN + state, h);
            }
        }
        __syncthreads();
        float out[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            out[j] = skip * xk[j];
#pragma unroll
            for (int v = 0; v < W; ++v)
#pragma unroll
                for (int g = 0; g < Sh::M; ++g) out[j] += part[v][(threadIdx.x + TH * j) / CH][g * CH + pc];
        }
        if (p.z) {
#pragma unroll
            for (int j = 0; j < J; ++j) out[j] *= silu_for<T>(zk[j]);
        }
        if (pc < q.chans) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (tokens == TQ || (threadIdx.x + TH * j) / CH < tokens) *(T*)((char*)y + ly.off[j]) = (T)out[j];
        }
    }
    if (!SEQ && q.seg == p.nseg - 1 && p.fin && mine) store_f32<S>(p.fin + q.b * DN + state, h);
}

// ---------------------------------------------------------------- local pass of split rows
// The scan of one segment without its read-out, from a zero state (the first segment:
// from the row's initial state): the segment's end state and the sum of its steps, whose
// decay exp(A sum) is what an incoming state would still weigh; infinite when a sequence
// starts inside (whatever its own steps are), so that nothing comes through.  A wave on its
// own, up to 16 states a lane.
template <typename T, int N, int CH, int S, bool SEQ>
__global__ __launch_bounds__((SelShape<N, CH, S>::THREADS)) void sel_local_kernel(SelParams p) {
    using Sh = SelShape<N, CH, S>;
    constexpr int TQ = 16, TH = Sh::THREADS, J = TQ * CH / TH, E = (TQ * N + TH - 1) / TH;
    static_assert(J * TH == TQ * CH, "tile shape");
    __shared__ float2 su[TQ][CH];
    __shared__ float4 Bs[TQ / 4][N];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const SelPlace q = sel_place<CH>(p);
    if (q.seg == p.nseg - 1) return;
    const int ch = lane % CH, n0 = (w * Sh::M + lane / CH) * S;
    const bool mine = ch < q.chans;
    const int64_t d = q.d0 + (mine ? ch : q.chans - 1);
    const int32_t* ids = SEQ ? p.seq_idx + q.b * p.T : nullptr;
    const int64_t tok = q.b * p.T + q.t0;
    const T* x = (const T*)p.x + tok * p.ldx + q.d0;
    const T* dt = (const T*)p.dt + tok * p.lddt + q.d0;
    const T* B = (const T*)p.B + tok * p.ldb + q.g * N;
    const int pc = threadIdx.x % CH;
    const float bias = p.dt_bias ? p.dt_bias[q.d0 + (pc < q.chans ? pc : q.chans - 1)] : 0.f;
    float A2[S], h[S], sum = 0.f;
    bool cut = false;                     // a sequence has started inside
    load_decay<S>(p, d, N, n0, A2);
    const int64_t state = d * N + n0, DN = p.D * N;
    load_state<S>(q.seg == 0 && p.init && !SEQ ? p.init + q.b * DN + state : nullptr, h);
    TileLoad<T, J, CH, TH> lx, ld;
    TileLoad<T, E, N, TH> lb;
    T xr[J], dr[J], br[E];
    auto load = [&](int64_t left) {
        if (left < TQ || left == q.t1 - q.t0) {
            const int tokens = left < TQ ? (int)left : TQ;
            lx.place(p.ldx, q.chans, tokens);
            ld.place(p.lddt, q.chans, tokens);
            lb.place(p.ldb, N, tokens);
        }
        lx.load(x, xr);
        ld.load(dt, dr);
        lb.load(B, br);
        x += TQ * p.ldx;
        dt += TQ * p.lddt;
        B += TQ * p.ldb;
    };
    load(q.t1 - q.t0);
    for (int64_t t = q.t0; t < q.t1; t += TQ) {
        const int tokens = q.t1 - t < TQ ? (int)(q.t1 - t) : TQ;
        __syncthreads();
        float step[J], xk[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            xk[j] = (float)xr[j];
            step[j] = (float)dr[j] + bias;
        }
        map_steps(step, p.softplus);
        if (tokens < TQ) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                if ((threadIdx.x + TH * j) / CH >= tokens) step[j] = xk[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < J; ++j) su[(threadIdx.x + TH * j) / CH][pc] = make_float2(step[j], step[j] * xk[j]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int k = threadIdx.x + TH * e, i = k / N;
            if (E * TH > TQ * N && i >= TQ) continue;
            (&Bs[i / 4][k % N].x)[i % 4] = i < tokens ? (float)br[e] : 0.f;
        }
        __syncthreads();
        if (t + TQ < q.t1) load(q.t1 - t - TQ);
        SeqBits bits{};
        if (SEQ) bits = seq_bits<TQ>(ids, t, p.T, lane);
#pragma unroll
        for (int i4 = 0; i4 < TQ / 4; ++i4) {
            const float4 B4 = Bs[i4][n0 + lane % S];
            const float Bv[4] = {B4.x, B4.y, B4.z, B4.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = 4 * i4 + k;
                if (SEQ && (bits.starts >> i & 1)) {
                    load_state<S>(p.init ? p.init + clamp_id(ids[t + i], p.nseqs) * DN + state : nullptr, h);
                    cut = true;
                    sum = __builtin_inff();
                }
                const float2 s = su[i][ch];
                sum += SEQ && cut ? 0.f : s.x;
                static_for<S>([&](auto I) {
                    constexpr int n = decltype(I)::value;
                    h[n] = fmaf(decay(s.x, A2[n]), h[n], row_lane<n>(Bv[k]) * s.y);
                });
            }
        }
    }
    if (mine) {
        const int64_t at = (q.b * (p.nseg - 1) + q.seg) * p.D + d;
        store_f32<S>(p.seg_state + at * N + n0, h);
        if (n0 == 0) p.seg_step[at] = sum;
    }
}

// In-place scan over a row's segments, a thread per (row, channel, state).  Forward:
// seg_state[s] becomes the state after segment s; reverse: seg_grad[s] (of segment s+1)
// becomes the gradient reaching that segment's incoming state.  A chain of nseg - 1 steps
// whose loads do not depend on it: those of 32 segments are in flight together (63 steps of
// 24576 states take 15 us with eight in flight and 13.6 with 32).
constexpr int kCombineAhead = 32;
constexpr int kCombineBlock = 64;      // small workgroups: few threads, spread over all units
template <bool REVERSE> __device__ inline void sel_combine(const SelParams& p, int N) {
    const int64_t DN = p.D * N, i = (int64_t)blockIdx.x * kCombineBlock + threadIdx.x;
    if (i >= p.batch * DN) return;
    const int64_t b = i / DN, e = i % DN;
    const int ns = p.nseg - 1;
    float* st = (REVERSE ? p.seg_grad : p.seg_state) + b * ns * DN + e;
    const float* sum = p.seg_step + b * ns * p.D + e / N;
    const float A2 = decay_rate(p.A_log[e]);
    // segment s lets exp(A sum) of what enters it through (forward: s = 1 .., reverse:
    // segment s+1 of seg_grad[s])
    auto segment = [&](int k) { return REVERSE ? ns - 1 - k : k; };
    float carry = 0.f;
    for (int k0 = 0; k0 < ns; k0 += kCombineAhead) {
        float l[kCombineAhead], c[kCombineAhead];
#pragma unroll
        for (int k = 0; k < kCombineAhead; ++k) {
            const int s = segment(k0 + k);
            if (k0 + k >= ns) break;
            l[k] = st[s * DN];
            c[k] = REVERSE ? (s + 1 < ns ? sum[(s + 1) * p.D] : 0.f) : sum[s * p.D];
        }
#pragma unroll
        for (int k = 0; k < kCombineAhead; ++k) {
            if (k0 + k >= ns) break;
            // selected, not multiplied by zero: an Inf or NaN of another sequence stays there
            carry = k0 + k == 0 || c[k] == __builtin_inff() ? l[k] : fmaf(decay(c[k], A2), carry, l[k]);
            st[segment(k0 + k) * DN] = carry;
        }
    }
}
__global__ __launch_bounds__(kCombineBlock) void sel_combine_kernel(SelParams p, int N) {
    if (blockIdx.y) sel_combine<true>(p, N);
    else sel_combine<false>(p, N);
}

// ---------------------------------------------------------------- step
// One token: N/4 lanes per channel, four states each, for R rows of the batch, so that A is
// read and exponentiated once for them and their loads are in flight together.  Bound by
// the state's read and write at large batches and by the launch at small ones.
template <typename T, int N, int R> __global__ __launch_bounds__(256) void sel_step_kernel(SelParams p) {
    constexpr int L = N / 4, PER = 256 / L;              // channels per workgroup
    const int c = threadIdx.x % L;
    const int64_t d = (int64_t)(blockIdx.x % p.blocks) * PER + threadIdx.x / L;
    const int64_t b0 = (int64_t)(blockIdx.x / p.blocks) * R;
    if (d >= p.D) return;
    const int64_t g = d / p.per_group;
    float h[R][4], A2[4], Bv[R][4], Cv[R][4], x[R], step[R], z[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (b0 + r >= p.batch) continue;
        const int64_t b = b0 + r;
        load_f32<4>(p.init + (b * p.D + d) * N + 4 * c, h[r]);
        step[r] = (float)((const T*)p.dt)[b * p.lddt + d];
        x[r] = (float)((const T*)p.x)[b * p.ldx + d];
        if (p.z) z[r] = (float)((const T*)p.z)[b * p.ldz + d];
        load_f32<4>((const T*)p.B + b * p.ldb + g * N + 4 * c, Bv[r]);
        load_f32<4>((const T*)p.C + b * p.ldc + g * N + 4 * c, Cv[r]);
    }
    load_decay<4>(p, d, N, 4 * c, A2);
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f, skip = p.skip ? p.skip[d] : 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) step[r] += bias;
    map_steps(step, p.softplus);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (b0 + r >= p.batch) continue;
        float acc = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[r][k] = fmaf(decay(step[r], A2[k]), h[r][k], step[r] * x[r] * Bv[r][k]);
            acc = fmaf(h[r][k], Cv[r][k], acc);
        }
        store_f32<4>(p.fin + ((b0 + r) * p.D + d) * N + 4 * c, h[r]);
        if constexpr (L == 2) acc += dpp_mov<0xb1>(acc);
        else acc = lane_team_sum<L>(acc);
        if (c == 0) {
            acc = fmaf(skip, x[r], acc);
            if (p.z) acc *= silu_for<T>(z[r]);
            ((T*)p.y)[(b0 + r) * p.D + d] = (T)acc;
        }
    }
}

// ---------------------------------------------------------------- launches
// `blocks` counts the workgroups' channel blocks, which differ between kernels.
static SelParams blocked(const SelParams& p, int ch) {
    SelParams q = p;
    q.blocks = (p.per_group + ch - 1) / ch;
    return q;
}
static dim3 sel_grid(const SelParams& p) { return dim3((unsigned)(p.batch * p.nseg * p.G * p.blocks)); }

template <typename T, int N, int CH, int S> static void forward_shape(const SelParams& p0, hipStream_t s) {
    const SelParams p = blocked(p0, CH);
    const dim3 block(SelShape<N, CH, S>::THREADS);
    if (p.seq_idx) hipLaunchKernelGGL((sel_forward_kernel<T, N, CH, S, true>), sel_grid(p), block, 0, s, p);
    else hipLaunchKernelGGL((sel_forward_kernel<T, N, CH, S, false>), sel_grid(p), block, 0, s, p);
}
// 64-channel workgroups, N/4 states a lane, spend fewer instructions per state; 32-channel ones,
// N/8 states a lane, give twice the waves where there are fewer than three of the larger for
// each of 256 compute units.  1024 tokens of 5120 channels, bf16, us with 32 and 64 channels:
// N = 16: 4 rows (320 workgroups of 64) 132 and 161, 8 rows 223 and 213, 12 rows 310 and 282,
// 32 rows 748 and 642; N = 64: 4 rows 358 and 419, 8 rows 573 and 623, 12 rows 883 and 806.  One
// border for all N: at 8 rows it gives away 10 us with 16 states and wins 50 with 64.
template <typename T, int N> static void forward_n(const SelParams& p, hipStream_t s) {
    if (p.nseg > 1 || p.batch * p.G * ((p.per_group + 63) / 64) >= 768) forward_shape<T, N, 64, N / 4>(p, s);
    else forward_shape<T, N, 32, N / 8>(p, s);
}
template <typename T, int N> static void local_n(const SelParams& p0, hipStream_t s) {
    constexpr int CH = 64, S = N <= 16 ? N : 16;
    const SelParams p = blocked(p0, CH);
    const dim3 block(SelShape<N, CH, S>::THREADS);
    if (p.seq_idx) hipLaunchKernelGGL((sel_local_kernel<T, N, CH, S, true>), sel_grid(p), block, 0, s, p);
    else hipLaunchKernelGGL((sel_local_kernel<T, N, CH, S, false>), sel_grid(p), block, 0, s, p);
}

hipError_t launch_sel_forward(const SelParams& p, int dtype, int64_t N, hipStream_t s) {
#define CALL(n) dtype == SSD_DTYPE_BF16 ? forward_n<__bf16, n>(p, s) : forward_n<float, n>(p, s)
    SSD_SEL_BY_STATE(N, CALL)
#undef CALL
    return hipGetLastError();
}
hipError_t launch_sel_local(const SelParams& p, int dtype, int64_t N, hipStream_t s) {
#define CALL(n) dtype == SSD_DTYPE_BF16 ? local_n<__bf16, n>(p, s) : local_n<float, n>(p, s)
    SSD_SEL_BY_STATE(N, CALL)
#undef CALL
    return hipGetLastError();
}
hipError_t launch_sel_combine(const SelParams& p, int64_t N, bool both, hipStream_t s) {
    const dim3 grid((unsigned)((p.batch * p.D * N + kCombineBlock - 1) / kCombineBlock), both ? 2 : 1);
    hipLaunchKernelGGL(sel_combine_kernel, grid, dim3(kCombineBlock), 0, s, p, (int)N);
    return hipGetLastError();
}
template <typename T, int N, int R> static void step_rows(SelParams p, hipStream_t s) {
    p.blocks = (int)((p.D + 1024 / N - 1) / (1024 / N));
    const dim3 grid((unsigned)(p.blocks * ((p.batch + R - 1) / R)));
    hipLaunchKernelGGL((sel_step_kernel<T, N, R>), grid, dim3(256), 0, s, p);
}
// Four rows per thread once that still leaves 1 << 18 threads (64 rows of 5120 channels with
// 16 states, bf16: 10.7 us against 12.8 for one row a thread).
template <typename T, int N> static void step_n(const SelParams& p, hipStream_t s) {
    if (p.batch * p.D * (N / 4) >= int64_t(1) << 20) step_rows<T, N, 4>(p, s);
    else step_rows<T, N, 1>(p, s);
}
hipError_t launch_sel_step(const SelParams& p, int dtype, int64_t N, hipStream_t s) {
#define CALL(n) dtype == SSD_DTYPE_BF16 ? step_n<__bf16, n>(p, s) : step_n<float, n>(p, s)
    SSD_SEL_BY_STATE(N, CALL)
#undef CALL
    return hipGetLastError();
}

}  // namespace ssd
