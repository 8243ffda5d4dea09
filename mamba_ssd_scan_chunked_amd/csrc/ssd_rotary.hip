// Root-mean-square norm of B and C per head with the rotation by position, and its
// gradients.  C entries of include/ssd.h.
//
//   v = u r w,  r = 1 / sqrt(mean(u^2) + eps);   (p, q) -> (p cos - q sin, p sin + q cos).
// Gradients: e = the rotation's transpose of dout;  hat = u r;
//   du = r (e w - hat mean(e w hat)),   dw = sum over tokens and heads of e hat.
//
// Memory-bound: every element is read once and written once.  A team of lanes holds a head of a
// token, each lane two packs of V channels that lie half the rotated (or whole) width apart, so
// that a pair is in one lane and all lanes' packs together are whole lines.  A team walks the
// heads of its token, B's and then C's, with the next head's loads in flight: the token's cosines
// and sines (fp64 angles) are formed once for all of them.  Measured on an MI355X (a device copy
// moves 5.1 TB/s), bf16: 8192 tokens of 8 + 32 heads of 128 27.9 us for 168 MB; 16384 tokens of one
// head each 7.0 us on the GPU for 17 MB (one round of waves: latency), 12.5 with the binding;
// gradients of 16384 tokens of 8 + 8 heads 66 us for 336 MB; one decoded token for four rows 3.0 us
// on the GPU, 12 a call.  Fp32: 16384 tokens of one head each 9.6 us on the GPU for 34 MB, 4096 of 8 +
// 32 heads 32 us for 168 MB, gradients of 8192 tokens of 8 + 8 heads 42 us for 201 MB.  Gradients take
// packs of four channels, so that a store instruction's 16-byte pieces of fp32 lie side by side.
#include "ssd.h"

#include <algorithm>
#include <cstdio>

#include "block_common.hpp"
#include "block_host.hpp"

namespace ssd {

struct RotaryParams {
    const void* u[2];                // B, C
    const float* w[2];
    void* out[2];
    const float* dout[2];
    float* du[2];
    const float* freqs;
    const int32_t* positions;
    float* part[2];                  // workgroups' sums of dw, rows of part_stride
    int64_t part_stride;
    int64_t tokens, seqlen, ld[2];
    int heads[2];
    int N, R;
    int chunk, nchunk;               // heads of an item, items per token
    float eps;
    int interleaved, stream;
};

// cos and sin of position times freq.  The angle, in revolutions, is formed in fp64 (three
// roundings: 2^-20 of a radian at 2^31 of them) and reduced to half a revolution before it is
// rounded to fp32.
__device__ inline void turn_of(int64_t position, float freq, float* c, float* s) {
    const double rev = (double)position * ((double)freq * 0.15915494309189535);
    const float part = (float)(rev - rint(rev));
    *c = __builtin_amdgcn_cosf(part);
    *s = __builtin_amdgcn_sinf(part);
}
__device__ inline int64_t position_of(const RotaryParams& p, int64_t t) {
    if (p.positions) return p.positions[t];
    return (unsigned)t % (unsigned)p.seqlen;               // both at most 2^31
}

// A lane's channels: its M units are e = lane, lane + L, ..., each two packs of V channels.
// Halves: pairs are (pack 0, pack 1) at j and j + R / 2; behind the rotated channels the rest is
// split in two the same way.  INTER: pairs lie within a pack; pack 1 is N / 2 behind.
template <int V, int L, int M, bool INTER> struct Unit {
    int c[M][2];
    bool real[M], turned[M];
    float cs[M][V], sn[M][V];
    __device__ inline void place(const RotaryParams& p, int lane) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int e = lane + m * L, first = p.R / (2 * V);
            real[m] = e < p.N / (2 * V);
            turned[m] = INTER || e < first;
            c[m][0] = INTER || e < first ? e * V : p.R + (e - first) * V;
            c[m][1] = INTER ? p.N / 2 + e * V : (e < first ? p.R / 2 + e * V : p.R + (p.N - p.R) / 2 + (e - first) * V);
            if (!real[m]) c[m][0] = c[m][1] = 0;
        }
    }
    __device__ inline int pair(int m, int i) const {
        return INTER ? (i < V / 2 ? c[m][0] / 2 + i : c[m][1] / 2 + i - V / 2) : c[m][0] + i;
    }
    __device__ inline bool turns(const RotaryParams& p, int m, int i) const {
        return INTER ? 2 * pair(m, i) < p.R : turned[m];
    }
    __device__ inline void turn(const RotaryParams& p, int64_t position) {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                cs[m][i] = sn[m][i] = 0.f;
                if (turns(p, m, i)) turn_of(position, p.freqs[pair(m, i)], &cs[m][i], &sn[m][i]);
            }
    }
    // Pairs of unit m turned, by the angles or (BACK) against them.  The channels behind the rotated
    // ones pass by a select: by a turn of angle 0, an infinite or NaN one would spoil its neighbour.
    template <bool BACK> __device__ inline void rotate(const RotaryParams& p, int m, float (&v)[2][V]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int h = V / 2 > 0 ? V / 2 : 1;
            float& a = INTER ? v[i / h][2 * (i % h)] : v[0][i];
            float& b = INTER ? v[i / h][2 * (i % h) + 1] : v[1][i];
            const float s = BACK ? -sn[m][i] : sn[m][i], x = a, y = b;
            const bool on = turns(p, m, i);
            a = on ? fmaf(x, cs[m][i], -y * s) : x;
            b = on ? fmaf(x, s, y * cs[m][i]) : y;
        }
    }
};

// An item: 64 / L tokens and `chunk` of their heads (B's first).  Waves take items in turn.
template <typename T, int V, int L, int M, bool INTER, bool STREAM> __device__ inline void rotary_forward(const RotaryParams& p) {
    const int lane = threadIdx.x % L;
    Unit<V, L, M, INTER> q;
    q.place(p, lane);
    const int64_t items = (p.tokens + 64 / L - 1) / (64 / L) * p.nchunk;
    for (int64_t item = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); item < items; item += (int64_t)gridDim.x * 4) {
        const int64_t t = item / p.nchunk * (64 / L) + threadIdx.x % 64 / L;
        const int h0 = (int)(item % p.nchunk) * p.chunk, h1 = h0 + p.chunk < p.heads[0] + p.heads[1] ? h0 + p.chunk : p.heads[0] + p.heads[1];
        if (t >= p.tokens) continue;         // whole teams: sums stay within a team
        const int lo[2] = {h0 < p.heads[0] ? h0 : p.heads[0], h0 > p.heads[0] ? h0 - p.heads[0] : 0};
        const int hi[2] = {h1 < p.heads[0] ? h1 : p.heads[0], h1 > p.heads[0] ? h1 - p.heads[0] : 0};
        Pack<T, V> raw[2][M][2];
        auto fetch = [&](int k, int head, Pack<T, V> (&r)[M][2]) {
            const T* u = (const T*)p.u[k] + t * p.ld[k] + (int64_t)head * p.N;
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (M == 1 || q.real[m]) r[m][e] = load_pack<V>(u + q.c[m][e]);
        };
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (lo[k] < hi[k]) fetch(k, lo[k], raw[k]);
        q.turn(p, position_of(p, t));
        const float inv = 1.f / (float)p.N;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (lo[k] >= hi[k]) continue;
            float w[M][2][V];
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e) load_f32<V>(p.w[k] + q.c[m][e], w[m][e]);
#pragma unroll 1
            for (int head = lo[k]; head < hi[k]; ++head) {
                float v[M][2][V], sq = 0.f;
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            v[m][e][i] = q.real[m] ? (float)raw[k][m][e].v[i] : 0.f;
                            sq = fmaf(v[m][e][i], v[m][e][i], sq);
                        }
                if (head + 1 < hi[k]) fetch(k, head + 1, raw[k]);
                const float r = 1.f / sqrtf(fmaf(lane_team_sum<L>(sq), inv, p.eps));
                T* out = (T*)p.out[k] + (t * p.heads[k] + head) * p.N;
#pragma unroll
                for (int m = 0; m < M; ++m) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int i = 0; i < V; ++i) v[m][e][i] *= r * w[m][e][i];
                    q.template rotate<false>(p, m, v[m]);
                    if (q.real[m]) {
                        store_f32<V, STREAM>(out + q.c[m][0], v[m][0]);
                        store_f32<V, STREAM>(out + q.c[m][1], v[m][1]);
                    }
                }
            }
        }
    }
}
template <typename T, int V, int L, int M, bool INTER> __global__ __launch_bounds__(256, M == 1 ? 4 : 1) void rotary_forward_kernel(RotaryParams p) {
    if (p.stream) rotary_forward<T, V, L, M, INTER, true>(p);
    else rotary_forward<T, V, L, M, INTER, false>(p);
}

// Waves walk items, with the sums of dw in registers; a workgroup's go to the workspace.
template <typename T, int V, int L, int M, bool INTER, bool STREAM>
__device__ inline void rotary_backward(const RotaryParams& p, float (&sums)[4][2][1024]) {
    const int lane = threadIdx.x % L, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Unit<V, L, M, INTER> q;
    q.place(p, lane);
    float dw[2][M][2][V];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < V; ++i) dw[k][m][e][i] = 0.f;
    const int64_t items = (p.tokens + 64 / L - 1) / (64 / L) * p.nchunk;
    const float inv = 1.f / (float)p.N;
    for (int64_t item = (int64_t)blockIdx.x * 4 + wave; item < items; item += (int64_t)gridDim.x * 4) {
        const int64_t at = item / p.nchunk * (64 / L) + threadIdx.x % 64 / L;
        const bool here = at < p.tokens;
        const int64_t t = here ? at : p.tokens - 1;        // teams past the end repeat the last token, unwritten
        const int h0 = (int)(item % p.nchunk) * p.chunk, h1 = h0 + p.chunk < p.heads[0] + p.heads[1] ? h0 + p.chunk : p.heads[0] + p.heads[1];
        const int lo[2] = {h0 < p.heads[0] ? h0 : p.heads[0], h0 > p.heads[0] ? h0 - p.heads[0] : 0};
        const int hi[2] = {h1 < p.heads[0] ? h1 : p.heads[0], h1 > p.heads[0] ? h1 - p.heads[0] : 0};
        Pack<T, V> raw[2][M][2];
        Pack<float, V> grad[2][M][2];
        auto fetch = [&](int k, int head, Pack<T, V> (&r)[M][2], Pack<float, V> (&g)[M][2]) {
            const T* u = (const T*)p.u[k] + t * p.ld[k] + (int64_t)head * p.N;
            const float* d = p.dout[k] + (t * p.heads[k] + head) * p.N;
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    r[m][e] = load_pack<V>(u + q.c[m][e]);
                    g[m][e] = load_pack<V>(d + q.c[m][e]);
                }
        };
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (lo[k] < hi[k]) fetch(k, lo[k], raw[k], grad[k]);
        q.turn(p, position_of(p, t));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (lo[k] >= hi[k]) continue;
            float w[M][2][V];
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e) load_f32<V>(p.w[k] + q.c[m][e], w[m][e]);
#pragma unroll 1
            for (int head = lo[k]; head < hi[k]; ++head) {
                float u[M][2][V], e[M][2][V], sq = 0.f, dot = 0.f;
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const bool real = here && q.real[m];
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            u[m][f][i] = real ? (float)raw[k][m][f].v[i] : 0.f;
                            e[m][f][i] = real ? grad[k][m][f].v[i] : 0.f;
                            sq = fmaf(u[m][f][i], u[m][f][i], sq);
                        }
                }
                if (head + 1 < hi[k]) fetch(k, head + 1, raw[k], grad[k]);
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    q.template rotate<true>(p, m, e[m]);
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int i = 0; i < V; ++i) dot = fmaf(e[m][f][i] * w[m][f][i], u[m][f][i], dot);
                }
                sq = lane_team_sum<L>(sq);
                dot = lane_team_sum<L>(dot);
                // a team past the end adds nothing, also with eps = 0
                const float r = here ? 1.f / sqrtf(fmaf(sq, inv, p.eps)) : 0.f;
                dot *= inv * r * r;                               // the mean of e w hat, times r
                float* out = p.du[k] + (t * p.heads[k] + head) * p.N;
#pragma unroll
                for (int m = 0; m < M; ++m) {
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        float du[V];
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            dw[k][m][f][i] = fmaf(e[m][f][i], u[m][f][i] * r, dw[k][m][f][i]);
                            du[i] = r * fmaf(e[m][f][i], w[m][f][i], -u[m][f][i] * dot);
                        }
                        if (here && q.real[m]) store_f32<V, STREAM>(out + q.c[m][f], du);
                    }
                }
            }
        }
    }
    // over the teams of a wave, then over the waves
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
#pragma unroll
                for (int d = L; d < 64; d *= 2)
#pragma unroll
                    for (int i = 0; i < V; ++i) dw[k][m][f][i] += __shfl_xor(dw[k][m][f][i], d);
                if (threadIdx.x % 64 < L && q.real[m]) store_f32<V>(&sums[wave][k][q.c[m][f]], dw[k][m][f]);
            }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.N; c += 256) {
        const int k = c >= p.N, at = k ? c - p.N : c;
        p.part[k][blockIdx.x * p.part_stride + at] = sums[0][k][at] + sums[1][k][at] + (sums[2][k][at] + sums[3][k][at]);
    }
}
template <typename T, int V, int L, int M, bool INTER> __global__ __launch_bounds__(256, M == 1 ? 3 : 1) void rotary_backward_kernel(RotaryParams p) {
    __shared__ float sums[4][2][1024];
    if (p.stream) rotary_backward<T, V, L, M, INTER, true>(p, sums);
    else rotary_backward<T, V, L, M, INTER, false>(p, sums);
}

// Heads that no vectors fit (see vector_of): a wave per (token, head), lane l with pairs l,
// l + 64, ... and the channels behind them, read again where they are needed again.  16384 tokens
// of two heads of 99: 16 us on the GPU, gradients 113 (13 and 32 MB, bf16): latency, one head at a time,
// and sums in memory.
template <typename T, bool BACK> __global__ __launch_bounds__(64) void rotary_any_kernel(RotaryParams p) {
    const int lane = threadIdx.x, all = p.heads[0] + p.heads[1];
    if constexpr (BACK) {
        for (int c = lane; c < p.N; c += 64) p.part[0][blockIdx.x * p.part_stride + c] = p.part[1][blockIdx.x * p.part_stride + c] = 0.f;
        __syncthreads();             // a channel's sum is another lane's from here on
    }
    for (int64_t unit = blockIdx.x; unit < p.tokens * all; unit += gridDim.x) {
        const int64_t t = unit / all;
        int head = (int)(unit % all);
        const int k = head >= p.heads[0];
        if (k) head -= p.heads[0];
        const T* u = (const T*)p.u[k] + t * p.ld[k] + (int64_t)head * p.N;
        const int64_t o = (t * p.heads[k] + head) * p.N;
        const int64_t position = position_of(p, t);
        float* dw = BACK ? p.part[k] + blockIdx.x * p.part_stride : nullptr;
        float sq = 0.f;
        for (int c = lane; c < p.N; c += 64) sq = fmaf((float)u[c], (float)u[c], sq);
        const float r = 1.f / sqrtf(lane_team_sum<64>(sq) / p.N + p.eps);
        const int units = p.R / 2 + (p.N - p.R);          // pairs, then single channels
        float dot = 0.f;
        for (int pass = 0; pass < (BACK ? 2 : 1); ++pass) {
            if (pass) dot = lane_team_sum<64>(dot) / p.N;
            for (int j = lane; j < units; j += 64) {
                const bool pair = j < p.R / 2;
                const int c = !pair ? j + p.R / 2 : (p.interleaved ? 2 * j : j), c2 = p.interleaved ? c + 1 : c + p.R / 2;
                float cs = 1.f, sn = 0.f;
                if (pair) turn_of(position, p.freqs[j], &cs, &sn);
                const float h = (float)u[c] * r, h2 = pair ? (float)u[c2] * r : 0.f;
                const float w = p.w[k][c], w2 = pair ? p.w[k][c2] : 0.f;
                if constexpr (!BACK) {
                    ((T*)p.out[k])[o + c] = (T)(h * w * cs - h2 * w2 * sn);
                    if (pair) ((T*)p.out[k])[o + c2] = (T)(h * w * sn + h2 * w2 * cs);
                } else {
                    const float d = p.dout[k][o + c], d2 = pair ? p.dout[k][o + c2] : 0.f;
                    const float e = d * cs + d2 * sn, e2 = d2 * cs - d * sn;
                    if (!pass) {
                        dot += e * w * h + e2 * w2 * h2;
                        dw[c] += e * h;
                        if (pair) dw[c2] += e2 * h2;
                    } else {
                        p.du[k][o + c] = r * (e * w - h * dot);
                        if (pair) p.du[k][o + c2] = r * (e2 * w2 - h2 * dot);
                    }
                }
            }
        }
    }
}

// Sums of the workgroups' rows of dw: 16 columns by 64 rows at a time, then over the 64.
__global__ __launch_bounds__(1024) void rotary_sums_kernel(const float* part, float* b, float* c, int rows, int N) {
    __shared__ float acc[64][17];
    const int col = blockIdx.x * 16 + (threadIdx.x & 15), row = threadIdx.x >> 4;
    float sum = 0.f;
    if (col < 2 * N) {
#pragma unroll 8
        for (int r = row; r < rows; r += 64) sum += part[(int64_t)r * 2 * N + col];
    }
    acc[row][threadIdx.x & 15] = sum;
    __syncthreads();
    if (threadIdx.x < 16 && col < 2 * N) {
        float total = 0.f;
#pragma unroll
        for (int r = 0; r < 64; ++r) total += acc[r][threadIdx.x];
        (col < N ? b : c - N)[col] = total;
    }
}

// Channels of a pack: as many as 16 bytes of what is stored hold, that divide what has to be
// divided, and that leave a head at least four lanes; 0 if there are none (or a head would need
// more than 128 units).
static int vector_of(int64_t N, int64_t R, bool inter, int most) {
    for (int V = most; V >= (inter ? 2 : 1); V /= 2) {
        const bool fits = inter ? N % (2 * V) == 0 : R % (2 * V) == 0 && (N - R) % (2 * V) == 0;
        if (fits && N >= 8 * V) return N / (2 * V) <= 128 ? V : 0;
    }
    return 0;
}
static int lanes_of(int64_t N, int V) {
    const int64_t units = N / (2 * V);
    for (int L = 4; L <= 32; L *= 2)
        if (units <= L) return L;
    return 64;
}
constexpr int64_t kWalkers = 3 * 1024;       // three waves on each SIMD
// How a call is spread: V (0: a wave per head), lanes per head, heads per item, items, workgroups.
struct RotaryShape {
    int V, L, M;
    int64_t chunk, nchunk, items, groups;
};
static RotaryShape shape_of(int64_t tokens, int64_t heads, int64_t N, int64_t R, bool inter, bool wide, bool back) {
    RotaryShape s{};
    s.V = vector_of(N, R, inter, wide ? 8 : 4);
    if (!s.V) {
        s.items = tokens * heads;
        s.groups = std::min<int64_t>(back ? kWalkers / 4 : 65536, s.items);
        return s;
    }
    s.L = lanes_of(N, s.V);
    s.M = N / (2 * s.V) > 64 ? 2 : 1;
    const int64_t teams = (tokens + 64 / s.L - 1) / (64 / s.L);
    // Heads of a token stay together where that gives 8192 waves.  Backward kWalkers waves stay on
    // the chip and walk: few tokens' heads are spread over them once, many tokens' into 16384 items
    // or more, so that no wave walks much longer than another (16384 tokens of 16 heads of 128, bf16:
    // 4096 items 84 us, 8192 77, 16384 71, 32768 73; 2331 tokens of 9 heads of 80, fp32: 2915 items
    // 12.8, 5247 14.2).  On the GPU around the border, spread over the waves once against 16384 items:
    // 16 heads of 128, bf16, 4000 tokens 22.8 and 24.5 us, 4200 23.1 and 23.7, 8192 43.3 and 41.2, 16384
    // 78.5 and 67.1; 9 heads of 80, fp32, 4200 tokens 14.7 and 16.7, 8192 19.3 and 21.3; two heads of
    // 128, 8000 tokens 13.1 and 13.3, 8400 12.3 and 13.6, 16384 16.2 and 16.8.  So for few heads the
    // border lies low, by 2 us at most.
    const int64_t wanted = !back ? 8192 : (teams > kWalkers / 3 ? 16384 : kWalkers);
    const int64_t n = std::max<int64_t>(1, std::min(heads, wanted / std::max<int64_t>(1, teams)));
    s.chunk = (heads + n - 1) / n;
    s.nchunk = (heads + s.chunk - 1) / s.chunk;
    s.items = teams * s.nchunk;
    s.groups = std::min<int64_t>(back ? kWalkers / 4 : 1 << 20, (s.items + 3) / 4);
    return s;
}

template <typename T, bool BACK, int V, int L, int M> static void launch_one(const RotaryParams& p, dim3 grid, hipStream_t s) {
    if constexpr (V > 1) {                   // a pair of neighbours needs a pack of two
        if (p.interleaved) {
            if constexpr (BACK) hipLaunchKernelGGL((rotary_backward_kernel<T, V, L, M, true>), grid, dim3(256), 0, s, p);
            else hipLaunchKernelGGL((rotary_forward_kernel<T, V, L, M, true>), grid, dim3(256), 0, s, p);
            return;
        }
    }
    if constexpr (BACK) hipLaunchKernelGGL((rotary_backward_kernel<T, V, L, M, false>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((rotary_forward_kernel<T, V, L, M, false>), grid, dim3(256), 0, s, p);
}
template <typename T, bool BACK> static hipError_t launch_rotary(const RotaryParams& p, const RotaryShape& k, hipStream_t s) {
    const dim3 grid((unsigned)k.groups);
    constexpr bool WIDE = sizeof(T) == 2 && !BACK;
#define SSD_ROTARY_CASE(VV, LL, MM) \
    if (k.V == VV && k.L == LL && k.M == MM) launch_one<T, BACK, VV, LL, MM>(p, grid, s);
    if (!k.V) hipLaunchKernelGGL((rotary_any_kernel<T, BACK>), grid, dim3(64), 0, s, p);
    if constexpr (WIDE) {
        SSD_ROTARY_CASE(8, 4, 1) SSD_ROTARY_CASE(8, 8, 1) SSD_ROTARY_CASE(8, 16, 1) SSD_ROTARY_CASE(8, 32, 1) SSD_ROTARY_CASE(8, 64, 1)
    }
    SSD_ROTARY_CASE(4, 4, 1) SSD_ROTARY_CASE(4, 8, 1) SSD_ROTARY_CASE(4, 16, 1) SSD_ROTARY_CASE(4, 32, 1) SSD_ROTARY_CASE(4, 64, 1)
    SSD_ROTARY_CASE(4, 64, 2)
    SSD_ROTARY_CASE(2, 4, 1) SSD_ROTARY_CASE(2, 8, 1) SSD_ROTARY_CASE(2, 16, 1) SSD_ROTARY_CASE(2, 32, 1) SSD_ROTARY_CASE(2, 64, 1)
    SSD_ROTARY_CASE(2, 64, 2)
    SSD_ROTARY_CASE(1, 4, 1) SSD_ROTARY_CASE(1, 8, 1) SSD_ROTARY_CASE(1, 16, 1) SSD_ROTARY_CASE(1, 32, 1) SSD_ROTARY_CASE(1, 64, 1)
    SSD_ROTARY_CASE(1, 64, 2)
#undef SSD_ROTARY_CASE
    return hipGetLastError();
}

}  // namespace ssd

namespace {

using namespace ssd_host;

constexpr int64_t kMaxDim = int64_t(1) << 31;
constexpr int64_t kMaxHead = 1024;

int validate(const ssd_rotary_problem_t* p) {
    if (!p) return SSD_ERR_NULL_POINTER;
    if (p->tokens < 0 || p->seqlen < 1 || p->seqlen > kMaxDim || p->b_heads < 1 || p->c_heads < 1 || p->headdim < 1 ||
        p->rotary_dim < 0 || p->rotary_dim > p->headdim || p->rotary_dim % 2 != 0)
        return SSD_ERR_BAD_SHAPE;
    if (p->tokens >= kMaxDim || p->b_heads >= kMaxDim || p->c_heads >= kMaxDim || p->headdim >= kMaxDim)
        return SSD_ERR_BAD_SHAPE;
    if (p->ldb >= kMaxDim || p->ldc >= kMaxDim || p->ldb < p->b_heads * p->headdim || p->ldc < p->c_heads * p->headdim)
        return SSD_ERR_BAD_SHAPE;
    if (!(p->eps >= 0.f) || p->eps > 1e30f) return SSD_ERR_BAD_SHAPE;
    if (p->dtype != SSD_DTYPE_BF16 && p->dtype != SSD_DTYPE_F32) return SSD_ERR_UNSUPPORTED;
    if ((p->flags & ~uint32_t(SSD_ROTARY_INTERLEAVED)) || p->reserved != 0 || p->headdim > kMaxHead)
        return SSD_ERR_UNSUPPORTED;
    // sizes stay far from int64 overflow, a token's heads from that of int
    if (double(p->tokens) * double(std::max(p->ldb, p->ldc)) > 4e17) return SSD_ERR_BAD_SHAPE;
    if (p->b_heads + p->c_heads >= kMaxDim) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

ssd::RotaryShape shape_of(const ssd_rotary_problem_t* p, bool back) {
    return ssd::shape_of(p->tokens, p->b_heads + p->c_heads, p->headdim, p->rotary_dim,
                         (p->flags & SSD_ROTARY_INTERLEAVED) != 0, p->dtype == SSD_DTYPE_BF16 && !back, back);
}
// A single workgroup writes db_weight and dc_weight itself.
int64_t backward_bytes(const ssd_rotary_problem_t* p) {
    const int64_t rows = shape_of(p, true).groups;
    return p->tokens == 0 || rows == 1 ? 0 : align256(rows * 2 * p->headdim * 4);
}

struct RotSizes {
    int64_t b, c, ob, oc, fb, fc, w, freqs, positions;
};
RotSizes rot_sizes(const ssd_rotary_problem_t* p) {
    RotSizes s;
    const int64_t e = elem_size(p->dtype), nb = p->b_heads * p->headdim, nc = p->c_heads * p->headdim;
    s.b = p->tokens > 0 ? ((p->tokens - 1) * p->ldb + nb) * e : 0;
    s.c = p->tokens > 0 ? ((p->tokens - 1) * p->ldc + nc) * e : 0;
    s.ob = p->tokens * nb * e;
    s.oc = p->tokens * nc * e;
    s.fb = p->tokens * nb * 4;
    s.fc = p->tokens * nc * 4;
    s.w = p->headdim * 4;
    s.freqs = p->rotary_dim * 2;
    s.positions = p->tokens * 4;
    return s;
}

ssd::RotaryParams params_of(const ssd_rotary_problem_t* p, const void* B, const void* C, const float* bw,
                            const float* cw, const float* freqs, const int32_t* positions, const ssd::RotaryShape& s) {
    ssd::RotaryParams r{};
    r.u[0] = B;
    r.u[1] = C;
    r.w[0] = bw;
    r.w[1] = cw;
    r.freqs = freqs;
    r.positions = positions;
    r.tokens = p->tokens;
    r.seqlen = p->seqlen;
    r.ld[0] = p->ldb;
    r.ld[1] = p->ldc;
    r.heads[0] = (int)p->b_heads;
    r.heads[1] = (int)p->c_heads;
    r.N = (int)p->headdim;
    r.R = (int)p->rotary_dim;
    r.eps = p->eps;
    r.chunk = (int)s.chunk;
    r.nchunk = (int)s.nchunk;
    r.interleaved = (p->flags & SSD_ROTARY_INTERLEAVED) ? 1 : 0;
    return r;
}

int done(const char* what, const ssd_rotary_problem_t* p, hipError_t e) {
    if (log_enabled())
        std::fprintf(stderr, "[ssd] rotary norm %s dtype=%d tokens=%lld heads=%lld+%lld N=%lld R=%lld -> %s\n", what,
                     p->dtype, (long long)p->tokens, (long long)p->b_heads, (long long)p->c_heads,
                     (long long)p->headdim, (long long)p->rotary_dim, hipGetErrorString(e));
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

}  // namespace

extern "C" {

int ssd_rotary_norm_forward(const ssd_rotary_problem_t* p, const void* B, const void* C, const float* b_weight,
                            const float* c_weight, const float* freqs, const int32_t* positions, void* B_out,
                            void* C_out, void* stream) {
    const int v = validate(p);
    if (v != SSD_OK) return v;
    if (!b_weight || !c_weight || (p->rotary_dim > 0 && !freqs) || (p->tokens > 0 && (!B || !C || !B_out || !C_out)))
        return SSD_ERR_NULL_POINTER;
    const uintptr_t e = (uintptr_t)elem_size(p->dtype);
    if (misaligned(B, e) || misaligned(C, e) || misaligned(B_out, e) || misaligned(C_out, e) ||
        misaligned(b_weight, 4) || misaligned(c_weight, 4) || misaligned(freqs, 4) || misaligned(positions, 4))
        return SSD_ERR_ALIGNMENT;
    const RotSizes n = rot_sizes(p);
    const Buf in[] = {{B, n.b}, {C, n.c}, {b_weight, n.w}, {c_weight, n.w}, {freqs, n.freqs}, {positions, n.positions}};
    const Buf out[] = {{B_out, n.ob}, {C_out, n.oc}};
    const int a = check_alias(in, 6, out, 2);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    if (p->tokens == 0) return SSD_OK;
    const ssd::RotaryShape s = shape_of(p, false);
    ssd::RotaryParams r = params_of(p, B, C, b_weight, c_weight, freqs, positions, s);
    r.out[0] = B_out;
    r.out[1] = C_out;
    r.stream = std::max(n.ob, n.oc) > ssd::kStreamBytes;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return done("forward", p, p->dtype == SSD_DTYPE_BF16 ? ssd::launch_rotary<__bf16, false>(r, s, st)
                                                         : ssd::launch_rotary<float, false>(r, s, st));
}

size_t ssd_rotary_norm_backward_workspace_size(const ssd_rotary_problem_t* p) {
    return validate(p) == SSD_OK ? (size_t)backward_bytes(p) : 0;
}

int ssd_rotary_norm_backward(const ssd_rotary_problem_t* p, const void* B, const void* C, const float* b_weight,
                             const float* c_weight, const float* freqs, const int32_t* positions, const float* dB_out,
                             const float* dC_out, float* dB, float* dC, float* db_weight, float* dc_weight,
                             void* workspace, size_t workspace_bytes, void* stream) {
    const int v = validate(p);
    if (v != SSD_OK) return v;
    if (!b_weight || !c_weight || !db_weight || !dc_weight || (p->rotary_dim > 0 && !freqs) ||
        (p->tokens > 0 && (!B || !C || !dB_out || !dC_out || !dB || !dC)))
        return SSD_ERR_NULL_POINTER;
    const int64_t wsb = backward_bytes(p);
    if (wsb > 0 && !workspace) return SSD_ERR_WORKSPACE;
    const uintptr_t e = (uintptr_t)elem_size(p->dtype);
    if (misaligned(B, e) || misaligned(C, e) || misaligned(b_weight, 4) || misaligned(c_weight, 4) ||
        misaligned(freqs, 4) || misaligned(positions, 4) || misaligned(dB_out, 4) || misaligned(dC_out, 4) ||
        misaligned(dB, 4) || misaligned(dC, 4) || misaligned(db_weight, 4) || misaligned(dc_weight, 4) ||
        (wsb > 0 && misaligned(workspace, 256)))
        return SSD_ERR_ALIGNMENT;
    if ((int64_t)workspace_bytes < wsb) return SSD_ERR_WORKSPACE;
    const RotSizes n = rot_sizes(p);
    const Buf in[] = {{B, n.b}, {C, n.c}, {b_weight, n.w}, {c_weight, n.w}, {freqs, n.freqs}, {positions, n.positions},
                      {dB_out, n.fb}, {dC_out, n.fc}};
    const Buf out[] = {{dB, n.fb}, {dC, n.fc}, {db_weight, n.w}, {dc_weight, n.w}, {workspace, wsb}};
    const int a = check_alias(in, 8, out, 5);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (p->tokens == 0) {
        hipError_t q = ssd::launch_fill(db_weight, p->headdim, st);
        if (q == hipSuccess) q = ssd::launch_fill(dc_weight, p->headdim, st);
        return done("backward", p, q);
    }
    const ssd::RotaryShape s = shape_of(p, true);
    ssd::RotaryParams r = params_of(p, B, C, b_weight, c_weight, freqs, positions, s);
    r.dout[0] = dB_out;
    r.dout[1] = dC_out;
    r.du[0] = dB;
    r.du[1] = dC;
    r.stream = std::max(n.fb, n.fc) > ssd::kStreamBytes;
    float* ws = static_cast<float*>(workspace);
    r.part[0] = wsb > 0 ? ws : db_weight;
    r.part[1] = wsb > 0 ? ws + p->headdim : dc_weight;
    r.part_stride = 2 * p->headdim;
    hipError_t q = p->dtype == SSD_DTYPE_BF16 ? ssd::launch_rotary<__bf16, true>(r, s, st)
                                              : ssd::launch_rotary<float, true>(r, s, st);
    if (q == hipSuccess && wsb > 0) {
        hipLaunchKernelGGL(ssd::rotary_sums_kernel, dim3((unsigned)((2 * p->headdim + 15) / 16)), dim3(1024), 0, st, ws,
                           db_weight, dc_weight, (int)s.groups, (int)p->headdim);
        q = hipGetLastError();
    }
    return done("backward", p, q);
}

}  // extern "C"
