// The short causal convolution of a Mamba layer (depthwise, K = 2..4 taps): whole
// sequences, their gradients, and the single-token step.  C entries of include/ssd.h.
//
//   pre[t][d] = bias[d] + sum_j w[d][K-1-j] in[t-j][d],   y = pre or silu(pre),
//
// in[t-j] being the token j back in the same sequence, or, before the sequence's first
// token, the row of its initial state (K-1 rows, oldest first), or zero.
//
// Memory-bound: each thread owns V neighbouring channels and walks a run of tokens with
// the last K-1 inputs in registers, so x is read once (plus K-1 rows per run) and y written
// once; the next four tokens' loads are in flight while four are worked on.  Measured on an
// MI355X, 4 x 4096 tokens of 5376 channels, K = 4 (a device copy moves 5.0 TB/s): forward bf16
// 71 us for 353 MB (63 when the call before has left part of x in the memory-side cache), fp32
// 135 us for 705 MB, 5.0-5.2 TB/s; backward, packed, with states, bf16 209 us for 887 MB, fp32
// 235 us for 1063 MB, 4.2-4.5 TB/s: its 43 vector instructions per element keep the vector
// units at work for 49 % of that time, and 148 registers leave three waves per SIMD.  A step of
// 4 rows takes 2.8 us on the GPU, 10 us with the launch and the binding.
#include "ssd.h"

#include <algorithm>
#include <cstdio>

#include "block_common.hpp"
#include "block_host.hpp"

namespace ssd {

struct ConvParams {
    const void* x;
    const float *w, *bias, *init;
    const int32_t* seq_idx;
    void* y;
    float* fin;
    const float *dy, *dfin;
    float *dx, *dinit;
    float *part, *part_bias;         // runs' sums of dw and dbias, rows of D (K + 1)
    int64_t T, D, nseqs, ldx;
    unsigned nvec, nblk, nrun, L;    // vectors, workgroups over them, runs per row, tokens per run
    int silu;
    int stream;                      // y or dx stored past the caches
};

// A workgroup is one wave on 64 vectors of V channels and one run of tokens, so that every
// decision about tokens and sequences is a scalar one.  The last vector of a row is moved
// back to end with the row (D >= V): it repeats channels of its neighbour with equal
// results, and no access needs a bound per element.
struct Place {
    int64_t c0, b, t0, t1;
    unsigned run;
    bool active;
};
template <int V> __device__ inline Place place_of(const ConvParams& p) {
    Place q;
    const unsigned cv = blockIdx.x % p.nblk * 64 + threadIdx.x;
    q.run = blockIdx.x / p.nblk;
    q.b = q.run / p.nrun;
    q.t0 = (int64_t)(q.run % p.nrun) * p.L;
    q.t1 = q.t0 + p.L < p.T ? q.t0 + p.L : p.T;
    const int64_t c = (int64_t)cv * V;
    q.c0 = c + V <= p.D ? c : p.D - V;
    q.active = cv < p.nvec;
    return q;
}

// Weights as w[k][v]; in memory the K taps of a channel lie together.
template <int V, int K> __device__ inline void load_weights(const ConvParams& p, int64_t c0, float (&w)[K][V]) {
    float flat[V * K];
    load_f32<V * K>(p.w + c0 * K, flat);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < K; ++k) w[k][v] = flat[v * K + k];
}

// win[i] = row i of the sequence's initial state (zero without one).
template <int V, int K> __device__ inline void load_init(const ConvParams& p, int64_t seq, int64_t c0, float (&win)[K - 1][V]) {
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        if (p.init) {
            load_f32<V>(p.init + (seq * (K - 1) + i) * p.D + c0, win[i]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) win[i][v] = 0.f;
        }
    }
}

// The window before token t0: win[i] = input K-1-i tokens back.  Returns how many of
// those K-1 tokens lie in t0's own sequence (its place in it, up to K-1).
template <typename T, int V, int K, bool SEQ>
__device__ inline int open_window(const ConvParams& p, const Place& q, const int32_t* ids, float (&win)[K - 1][V]) {
    const T* x = (const T*)p.x + q.b * p.T * p.ldx + q.c0;
    int m = 0;
#pragma unroll
    for (int lag = 1; lag < K; ++lag)
        if (q.t0 - lag >= 0 && (!SEQ || ids[q.t0 - lag] == ids[q.t0])) m = lag;
    const int64_t seq = SEQ ? clamp_id(ids[q.t0], p.nseqs) : q.b;
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        const int lag = K - 1 - i;
        if (lag <= m) {
            load_f32<V>(x + (q.t0 - lag) * p.ldx, win[i]);
        } else if (p.init) {
            load_f32<V>(p.init + (seq * (K - 1) + K - 1 + m - lag) * p.D + q.c0, win[i]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) win[i][v] = 0.f;
        }
    }
    return m;
}

template <int V, int K> __device__ inline void push(float (&win)[K - 1][V], const float (&in)[V]) {
#pragma unroll
    for (int i = 0; i + 1 < K - 1; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) win[i][v] = win[i + 1][v];
#pragma unroll
    for (int v = 0; v < V; ++v) win[K - 2][v] = in[v];
}

constexpr int kAhead = 4;      // tokens whose loads are issued together

// Sequence ids of tokens t .. t + kAhead (the row's last one past its end).
__device__ inline void fetch_ids(const ConvParams& p, const int32_t* ids, int64_t t, int32_t (&id)[kAhead + 1]) {
#pragma unroll
    for (int u = 0; u <= kAhead; ++u) id[u] = ids[t + u < p.T ? t + u : p.T - 1];
}

template <typename T, int V, int K, bool SEQ, bool STREAM> __device__ inline void conv_forward(const ConvParams& p) {
    const Place q = place_of<V>(p);
    if (!q.active) return;
    const int32_t* ids = SEQ ? p.seq_idx + q.b * p.T : nullptr;
    float w[K][V], bias[V], win[K - 1][V];
    load_weights<V, K>(p, q.c0, w);
    if (p.bias) {
        load_f32<V>(p.bias + q.c0, bias);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) bias[v] = 0.f;
    }
    open_window<T, V, K, SEQ>(p, q, ids, win);
    const T* x = (const T*)p.x + q.b * p.T * p.ldx + q.c0;
    T* y = (T*)p.y + q.b * p.T * p.D + q.c0;
    // the next tokens' loads are in flight while these are worked on
    Pack<T, V> next[kAhead];
    int32_t next_id[kAhead + 1], before = SEQ ? ids[q.t0] : 0;
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (t + u < q.t1) next[u] = load_pack<V>(x + (t + u) * p.ldx);
        if (SEQ) fetch_ids(p, ids, t, next_id);
    };
    fetch(q.t0);
    for (int64_t t = q.t0; t < q.t1; t += kAhead) {
        Pack<T, V> raw[kAhead];
        int32_t id[kAhead + 1];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) raw[u] = next[u];
#pragma unroll
        for (int u = 0; u <= kAhead; ++u) id[u] = SEQ ? next_id[u] : 0;
        fetch(t + kAhead);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (t + u >= q.t1) break;
            const int64_t tt = t + u;
            if (SEQ && id[u] != (u ? id[u - 1] : before)) load_init<V, K>(p, clamp_id(id[u], p.nseqs), q.c0, win);
            float in[V], out[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                in[v] = (float)raw[u].v[v];
                float acc = fmaf(w[K - 1][v], in[v], bias[v]);
#pragma unroll
                for (int i = 0; i < K - 1; ++i) acc = fmaf(w[i][v], win[i][v], acc);
                out[v] = acc;
            }
            if (p.silu) {
#pragma unroll
                for (int v = 0; v < V; ++v) out[v] = silu_for<T>(out[v]);
            }
            store_f32<V, STREAM>(y + tt * p.D, out);
            push<V, K>(win, in);
            if (p.fin && (tt == p.T - 1 || (SEQ && id[u + 1] != id[u]))) {
                const int64_t seq = SEQ ? clamp_id(id[u], p.nseqs) : q.b;
#pragma unroll
                for (int i = 0; i < K - 1; ++i) store_f32<V>(p.fin + (seq * (K - 1) + i) * p.D + q.c0, win[i]);
            }
        }
        before = id[kAhead - 1];
    }
}

template <typename T, int V, int K, bool SEQ> __global__ __launch_bounds__(64, 4) void conv_forward_kernel(ConvParams p) {
    if (p.stream) conv_forward<T, V, K, SEQ, true>(p);
    else conv_forward<T, V, K, SEQ, false>(p);
}

// Gradients.  With g[t] = dy[t] silu'(pre[t]), input row r receives
// sum_j w[K-1-j] g[r+j] over the tokens r+j of its own sequence, and, being one of the
// sequence's last K-1 inputs, its row of dfinal.  A thread walks its run once, keeping
// the K partial sums of the rows t-K+1 .. t (acc[j]: row t-j); after token t row t-K+1
// is complete.  It reads K-1 tokens past its run to complete its last rows, and leaves
// the rows before its run to the run before.  Rows before a sequence's first token are
// those of its initial state and go to dinit.  dw and dbias are summed per run into
// `part` (K+1 arrays of runs x D), then over runs in a fixed order.
template <typename T, int V, int K, bool SEQ, bool STREAM> __device__ inline void conv_backward(const ConvParams& p) {
    const Place q = place_of<V>(p);
    if (!q.active) return;
    const int32_t* ids = SEQ ? p.seq_idx + q.b * p.T : nullptr;
    float w[K][V], bias[V], win[K - 1][V], acc[K][V], dw[K][V], db[V];
    load_weights<V, K>(p, q.c0, w);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) acc[k][v] = dw[k][v] = 0.f;
    }
    if (p.bias) {
        load_f32<V>(p.bias + q.c0, bias);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) bias[v] = 0.f;
    }
    int place = open_window<T, V, K, SEQ>(p, q, ids, win);       // of the token at hand in its sequence, up to K-1
    int64_t seq = SEQ ? clamp_id(ids[q.t0], p.nseqs) : q.b;
    const T* x = (const T*)p.x + q.b * p.T * p.ldx + q.c0;
    const float* dy = p.dy + q.b * p.T * p.D + q.c0;
    float* dx = p.dx + q.b * p.T * p.D + q.c0;
    const int64_t end = q.t1 + K - 1 < p.T ? q.t1 + K - 1 : p.T;

    // the finished sum of the row j back from token tt
    auto emit = [&](int64_t tt, int j, const float (&val)[V]) {
        const int64_t row = tt - j;
        if (place >= j) {
            if (row >= q.t0 && row < q.t1) store_f32<V, STREAM>(dx + row * p.D, val);
        } else if (p.dinit && tt - place >= q.t0 && tt - place < q.t1) {
            store_f32<V>(p.dinit + (seq * (K - 1) + K - 1 + place - j) * p.D + q.c0, val);
        }
    };

    // the next tokens' loads are in flight while these are worked on
    Pack<T, V> next[kAhead];
    Pack<float, V> next_dy[kAhead];
    int32_t next_id[kAhead + 1], before = SEQ ? ids[q.t0] : 0;
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (t + u < end) {
                next[u] = load_pack<V>(x + (t + u) * p.ldx);
                next_dy[u] = load_pack<V>(dy + (t + u) * p.D);
            }
        if (SEQ) fetch_ids(p, ids, t, next_id);
    };
    fetch(q.t0);
    bool open = true;                     // the run's last sequence goes on past the run
    for (int64_t t = q.t0; t < end && open; t += kAhead) {
        Pack<T, V> raw[kAhead];
        Pack<float, V> dyr[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            raw[u] = next[u];
            dyr[u] = next_dy[u];
        }
        int32_t id[kAhead + 1];
#pragma unroll
        for (int u = 0; u <= kAhead; ++u) id[u] = SEQ ? next_id[u] : 0;
        fetch(t + kAhead);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t tt = t + u;
            if (tt >= end || !open) break;
            if (SEQ && id[u] != (u ? id[u - 1] : before)) {
                seq = clamp_id(id[u], p.nseqs);
                place = 0;
                load_init<V, K>(p, seq, q.c0, win);
            }
            const bool mine = tt < q.t1;
            float in[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                in[v] = (float)raw[u].v[v];
                float g = dyr[u].v[v];
                if (p.silu) {
                    float pre = fmaf(w[K - 1][v], in[v], bias[v]);
#pragma unroll
                    for (int i = 0; i < K - 1; ++i) pre = fmaf(w[i][v], win[i][v], pre);
                    g *= silu_slope(pre, sigmoid(pre));
                }
                acc[0][v] = w[K - 1][v] * g;
#pragma unroll
                for (int j = 1; j < K; ++j) acc[j][v] = fmaf(w[K - 1 - j][v], g, acc[j][v]);
                if (mine) {
                    db[v] += g;
                    dw[K - 1][v] = fmaf(g, in[v], dw[K - 1][v]);
#pragma unroll
                    for (int i = 0; i < K - 1; ++i) dw[i][v] = fmaf(g, win[i][v], dw[i][v]);
                }
            }
            emit(tt, K - 1, acc[K - 1]);
            const bool last = tt == p.T - 1 || (SEQ && id[u + 1] != id[u]);
            if (last) {
#pragma unroll
                for (int j = K - 2; j >= 0; --j) {
                    if (p.dfin) {
                        float df[V];
                        load_f32<V>(p.dfin + (seq * (K - 1) + K - 2 - j) * p.D + q.c0, df);
#pragma unroll
                        for (int v = 0; v < V; ++v) acc[j][v] += df[v];
                    }
                    emit(tt, j, acc[j]);
                }
                // the next sequence's rows start from zero; past the run nothing is left to complete
                open = tt + 1 < q.t1;
#pragma unroll
                for (int j = 0; j < K; ++j)
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[j][v] = 0.f;
            } else {
#pragma unroll
                for (int j = K - 1; j > 0; --j)
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[j][v] = acc[j - 1][v];
            }
            push<V, K>(win, in);
            if (place < K - 1) ++place;
        }
        before = id[kAhead - 1];
    }
    const int64_t row = (int64_t)q.run * p.D * (K + 1);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < K; ++k) p.part[row + (q.c0 + v) * K + k] = dw[k][v];
    if (p.part_bias) store_f32<V>(p.part_bias + row + q.c0, db);
}

template <typename T, int V, int K, bool SEQ> __global__ __launch_bounds__(64, 3) void conv_backward_kernel(ConvParams p) {
    if (p.stream) conv_backward<T, V, K, SEQ, true>(p);
    else conv_backward<T, V, K, SEQ, false>(p);
}

// One token: a thread per (row, channel); state_out may be state (each element is read
// and then written by one thread).  A few microseconds of launch and latency at any
// batch that decoding meets.
template <typename T, int K> __global__ __launch_bounds__(256) void conv_step_kernel(ConvParams p, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t b = i / p.D, d = i % p.D;
    const float* st = p.init + b * (K - 1) * p.D + d;
    float* out = p.fin + b * (K - 1) * p.D + d;
    const float in = (float)((const T*)p.x)[b * p.ldx + d];
    float win[K - 1];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) win[k] = st[k * p.D];
    float acc = fmaf(p.w[d * K + K - 1], in, p.bias ? p.bias[d] : 0.f);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) acc = fmaf(p.w[d * K + k], win[k], acc);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) out[k * p.D] = k + 1 < K - 1 ? win[k + 1] : in;
    ((T*)p.y)[i] = (T)(p.silu ? silu_for<T>(acc) : acc);
}

template <typename T, int V, int K, bool BACK> static void launch_conv(const ConvParams& p, int64_t batch, hipStream_t s) {
    const dim3 grid((unsigned)(p.nblk * p.nrun * batch)), block(64);
    if constexpr (BACK) {
        if (p.seq_idx) hipLaunchKernelGGL((conv_backward_kernel<T, V, K, true>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((conv_backward_kernel<T, V, K, false>), grid, block, 0, s, p);
    } else {
        if (p.seq_idx) hipLaunchKernelGGL((conv_forward_kernel<T, V, K, true>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((conv_forward_kernel<T, V, K, false>), grid, block, 0, s, p);
    }
}
template <typename T, int V, bool BACK>
static hipError_t launch_conv_k(int K, const ConvParams& p, int64_t batch, hipStream_t s) {
    if (K == 2) launch_conv<T, V, 2, BACK>(p, batch, s);
    else if (K == 3) launch_conv<T, V, 3, BACK>(p, batch, s);
    else launch_conv<T, V, 4, BACK>(p, batch, s);
    return hipGetLastError();
}
template <typename T> static hipError_t launch_step(int K, const ConvParams& p, int64_t n, hipStream_t s) {
    const dim3 grid((unsigned)((n + 255) / 256)), block(256);
    if (K == 2) hipLaunchKernelGGL((conv_step_kernel<T, 2>), grid, block, 0, s, p, n);
    else if (K == 3) hipLaunchKernelGGL((conv_step_kernel<T, 3>), grid, block, 0, s, p, n);
    else hipLaunchKernelGGL((conv_step_kernel<T, 4>), grid, block, 0, s, p, n);
    return hipGetLastError();
}

}  // namespace ssd

namespace {

using namespace ssd_host;

constexpr int64_t kMaxDim = int64_t(1) << 31;

// Channels per thread and tokens per run.
struct Shape {
    int V;
    int64_t nvec, nblk, L, nrun;
};
Shape shape_of(const ssd_conv_problem_t* p, bool backward) {
    Shape s;
    // 16 bytes of x per thread forward; four channels backward, which keeps K sums, K
    // weights, K weight gradients and the window of each in registers
    s.V = backward ? 4 : (p->dtype == SSD_DTYPE_BF16 ? 8 : 4);
    if (p->channels < s.V) s.V = 1;
    s.nvec = (p->channels + s.V - 1) / s.V;
    s.nblk = (s.nvec + 63) / 64;
    // Runs: as many waves as the chip holds at once (three per SIMD backward, four forward),
    // or a whole number of times that when runs would get longer than `longest`: a run
    // re-reads K-1 rows, but a last round of few waves costs a whole one (4 x 4096 tokens of
    // 5376 channels backward, packed and not: runs of 64 tokens, 1.75 rounds, 217 and 192 us; of
    // 96, 1.2 rounds, 253 and 206; of 114, this rule's 0.98 rounds, 209 and 192; of 128, 0.9
    // rounds, 212 and 193).
    const int64_t longest = backward ? 128 : 32, resident = (backward ? 3 : 4) * 1024;
    const int64_t columns = std::max<int64_t>(1, p->batch * s.nblk);
    const int64_t least = (p->seqlen + longest - 1) / longest;                      // runs per row
    const double all = double(least) * double(columns) / resident;                  // (validate refuses the largest)
    const int64_t rounds = all < 1e9 ? (int64_t)all + 1 : (int64_t)1e9;
    const int64_t runs = std::max(std::max<int64_t>(1, least), rounds * resident / columns);
    s.L = std::max<int64_t>(4, (p->seqlen + runs - 1) / runs);
    s.nrun = std::max<int64_t>(1, (p->seqlen + s.L - 1) / s.L);
    return s;
}

int validate(const ssd_conv_problem_t* p) {
    if (!p) return SSD_ERR_NULL_POINTER;
    if (p->batch < 0 || p->seqlen < 0 || p->channels <= 0 || p->nseqs < 0 || p->ldx < p->channels)
        return SSD_ERR_BAD_SHAPE;
    if (p->batch >= kMaxDim || p->seqlen >= kMaxDim || p->channels >= kMaxDim || p->nseqs >= kMaxDim ||
        p->ldx >= kMaxDim)
        return SSD_ERR_BAD_SHAPE;
    if (p->dtype != SSD_DTYPE_BF16 && p->dtype != SSD_DTYPE_F32) return SSD_ERR_UNSUPPORTED;
    if (p->width < 2 || p->width > 4 || (p->flags & ~uint32_t(SSD_CONV_SILU)) || p->reserved != 0)
        return SSD_ERR_UNSUPPORTED;
    const double elems = double(p->batch) * double(p->seqlen) * double(p->ldx);
    if (elems > 4e17 || double(p->nseqs) * p->channels * 3 > 4e17) return SSD_ERR_BAD_SHAPE;
    // a launch holds fewer than 2^32 threads
    for (bool backward : {false, true}) {
        const Shape s = shape_of(p, backward);
        if (double(s.nblk) * s.nrun * p->batch * 64 >= 4e9) return SSD_ERR_UNSUPPORTED;
    }
    return SSD_OK;
}

struct ConvSizes {
    int64_t x, y, f, w, state, seq, bias;
};
ConvSizes conv_sizes(const ssd_conv_problem_t* p) {
    ConvSizes s;
    const int64_t bt = p->batch * p->seqlen, e = elem_size(p->dtype);
    s.x = bt > 0 ? ((bt - 1) * p->ldx + p->channels) * e : 0;
    s.y = bt * p->channels * e;
    s.f = bt * p->channels * 4;
    s.w = p->channels * p->width * 4;
    s.bias = p->channels * 4;
    s.state = p->nseqs * (p->width - 1) * p->channels * 4;
    s.seq = bt * 4;
    return s;
}

ssd::ConvParams params_of(const ssd_conv_problem_t* p, const Shape& s) {
    ssd::ConvParams c{};
    c.T = p->seqlen;
    c.D = p->channels;
    c.nseqs = p->nseqs;
    c.ldx = p->ldx;
    c.nvec = (unsigned)s.nvec;
    c.nblk = (unsigned)s.nblk;
    c.nrun = (unsigned)s.nrun;
    c.L = (unsigned)s.L;
    c.silu = (p->flags & SSD_CONV_SILU) ? 1 : 0;
    return c;
}

// A single run writes dw and dbias themselves.
int64_t backward_bytes(const ssd_conv_problem_t* p) {
    const int64_t runs = p->batch * shape_of(p, true).nrun;
    return p->seqlen == 0 || runs <= 1 ? 0 : align256(runs * p->channels * (p->width + 1) * 4);
}

int done(const char* what, const ssd_conv_problem_t* p, hipError_t e) {
    if (log_enabled())
        std::fprintf(stderr, "[ssd] conv %s dtype=%d batch=%lld T=%lld D=%lld K=%d -> %s\n", what, p->dtype,
                     (long long)p->batch, (long long)p->seqlen, (long long)p->channels, p->width, hipGetErrorString(e));
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

}  // namespace

extern "C" {

size_t ssd_conv_backward_workspace_size(const ssd_conv_problem_t* p) {
    return validate(p) == SSD_OK ? (size_t)backward_bytes(p) : 0;
}

int ssd_conv_forward(const ssd_conv_problem_t* p, const void* x, const float* weight, const float* bias,
                     const float* init_state, const int32_t* seq_idx, void* y, float* final_state, void* stream) {
    const int v = validate(p);
    if (v != SSD_OK) return v;
    const bool empty = p->batch == 0 || p->seqlen == 0;
    if (!weight || (!empty && (!x || !y))) return SSD_ERR_NULL_POINTER;
    const int q = check_sequences(p, seq_idx);
    if (q != SSD_OK) return q;
    const uintptr_t e = (uintptr_t)elem_size(p->dtype);
    if (misaligned(x, e) || misaligned(y, e) || misaligned(weight, 4) || misaligned(bias, 4) ||
        misaligned(init_state, 4) || misaligned(seq_idx, 4) || misaligned(final_state, 4))
        return SSD_ERR_ALIGNMENT;
    const ConvSizes z = conv_sizes(p);
    const Buf in[] = {{x, z.x}, {weight, z.w}, {bias, z.bias}, {init_state, z.state}, {seq_idx, z.seq}};
    const Buf out[] = {{y, z.y}, {final_state, z.state}};
    const int a = check_alias(in, 5, out, 2);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (empty) {
        // no token: each row's final state is its initial state
        if (seq_idx || !final_state) return SSD_OK;
        return done("forward", p, ssd::launch_copy(final_state, init_state, z.state / 4, st));
    }
    const Shape s = shape_of(p, false);
    ssd::ConvParams c = params_of(p, s);
    c.x = x;
    c.w = weight;
    c.bias = bias;
    c.init = init_state;
    c.seq_idx = seq_idx;
    c.y = y;
    c.fin = final_state;
    c.stream = z.y > ssd::kStreamBytes;
    hipError_t r;
    if (p->dtype == SSD_DTYPE_BF16)
        r = s.V == 8 ? ssd::launch_conv_k<__bf16, 8, false>(p->width, c, p->batch, st)
                     : ssd::launch_conv_k<__bf16, 1, false>(p->width, c, p->batch, st);
    else
        r = s.V == 4 ? ssd::launch_conv_k<float, 4, false>(p->width, c, p->batch, st)
                     : ssd::launch_conv_k<float, 1, false>(p->width, c, p->batch, st);
    return done("forward", p, r);
}

int ssd_conv_backward(const ssd_conv_problem_t* p, const void* x, const float* weight, const float* bias,
                      const float* init_state, const int32_t* seq_idx, const float* dy, const float* dfinal, float* dx,
                      float* dweight, float* dbias, float* dinit, void* workspace, size_t workspace_bytes,
                      void* stream) {
    const int v = validate(p);
    if (v != SSD_OK) return v;
    const bool empty = p->batch == 0 || p->seqlen == 0;
    if (!weight || !dweight || (!empty && (!x || !dy || !dx))) return SSD_ERR_NULL_POINTER;
    const int q = check_sequences(p, seq_idx);
    if (q != SSD_OK) return q;
    const int64_t wsb = backward_bytes(p);
    if (wsb > 0 && !workspace) return SSD_ERR_WORKSPACE;
    if (misaligned(x, (uintptr_t)elem_size(p->dtype)) || misaligned(weight, 4) || misaligned(bias, 4) ||
        misaligned(init_state, 4) || misaligned(seq_idx, 4) || misaligned(dy, 4) || misaligned(dfinal, 4) ||
        misaligned(dx, 4) || misaligned(dweight, 4) || misaligned(dbias, 4) || misaligned(dinit, 4) ||
        misaligned(workspace, 256))
        return SSD_ERR_ALIGNMENT;
    if ((int64_t)workspace_bytes < wsb) return SSD_ERR_WORKSPACE;
    const ConvSizes z = conv_sizes(p);
    const Buf in[] = {{x, z.x}, {weight, z.w}, {bias, z.bias}, {init_state, z.state}, {seq_idx, z.seq}, {dy, z.f}, {dfinal, z.state}};
    const Buf out[] = {{dx, z.f}, {dweight, z.w}, {dbias, z.bias}, {dinit, z.state}, {workspace, wsb}};
    const int a = check_alias(in, 7, out, 5);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t r = hipSuccess;
    if (empty) {
        // no token: nothing reaches the weights, and each row's final state is its initial state
        r = ssd::launch_fill(dweight, z.w / 4, st);
        if (r == hipSuccess) r = ssd::launch_fill(dbias, z.bias / 4, st);
        if (r == hipSuccess && dinit) r = ssd::launch_copy(dinit, seq_idx ? nullptr : dfinal, z.state / 4, st);
        return done("backward", p, r);
    }
    const Shape s = shape_of(p, true);
    ssd::ConvParams c = params_of(p, s);
    c.x = x;
    c.w = weight;
    c.bias = bias;
    c.init = init_state;
    c.seq_idx = seq_idx;
    c.dy = dy;
    c.dfin = dfinal;
    c.dx = dx;
    c.dinit = dinit;
    c.stream = z.f > ssd::kStreamBytes;
    const bool direct = wsb == 0;
    c.part = direct ? dweight : static_cast<float*>(workspace);
    c.part_bias = direct ? dbias : c.part + p->channels * p->width;
    // ids that do not occur keep a zero gradient
    if (seq_idx && dinit) r = ssd::launch_fill(dinit, z.state / 4, st);
    if (r == hipSuccess) {
        if (p->dtype == SSD_DTYPE_BF16)
            r = s.V == 4 ? ssd::launch_conv_k<__bf16, 4, true>(p->width, c, p->batch, st)
                         : ssd::launch_conv_k<__bf16, 1, true>(p->width, c, p->batch, st);
        else
            r = s.V == 4 ? ssd::launch_conv_k<float, 4, true>(p->width, c, p->batch, st)
                         : ssd::launch_conv_k<float, 1, true>(p->width, c, p->batch, st);
    }
    if (r == hipSuccess && !direct) {
        // one row of part per run: D*K weight gradients, then D bias gradients
        ssd::ColumnSums cs{};
        cs.part = c.part;
        cs.out = dweight;
        cs.out2 = dbias;
        cs.split = p->channels * p->width;
        cs.rows = p->batch * s.nrun;
        cs.cols = cs.split2 = p->channels * (p->width + 1);
        r = ssd::launch_column_sums(cs, st);
    }
    return done("backward", p, r);
}

int ssd_conv_step(const ssd_conv_problem_t* p, const void* x, const float* weight, const float* bias,
                  const float* state, float* state_out, void* y, void* stream) {
    if (!p) return SSD_ERR_NULL_POINTER;
    if (p->seqlen != 1 || p->nseqs != p->batch) return SSD_ERR_BAD_SHAPE;
    const int v = validate(p);
    if (v != SSD_OK) return v;
    if (double(p->batch) * p->channels >= 4e9) return SSD_ERR_UNSUPPORTED;       // a thread per (row, channel)
    if (!weight || (p->batch > 0 && (!x || !state || !state_out || !y))) return SSD_ERR_NULL_POINTER;
    const uintptr_t e = (uintptr_t)elem_size(p->dtype);
    if (misaligned(x, e) || misaligned(y, e) || misaligned(weight, 4) || misaligned(bias, 4) || misaligned(state, 4) ||
        misaligned(state_out, 4))
        return SSD_ERR_ALIGNMENT;
    const ConvSizes z = conv_sizes(p);
    const Buf in[] = {{x, z.x}, {weight, z.w}, {bias, z.bias}, {state == state_out ? nullptr : state, z.state}};
    const Buf out[] = {{y, z.y}, {state_out, z.state}};
    const int a = check_alias(in, 4, out, 2);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    if (p->batch == 0) return SSD_OK;
    Shape s = shape_of(p, false);
    ssd::ConvParams c = params_of(p, s);
    c.x = x;
    c.w = weight;
    c.bias = bias;
    c.init = state;
    c.fin = state_out;
    c.y = y;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t n = p->batch * p->channels;
    return done("step", p, p->dtype == SSD_DTYPE_BF16 ? ssd::launch_step<__bf16>(p->width, c, n, st)
                                                      : ssd::launch_step<float>(p->width, c, n, st));
}

}  // extern "C"
