// The gated linear recurrence: whole sequences, their gradients, and the single-token step.
// C entries of include/ssd.h.
//
//   s = sigmoid(r),  L = A s,  a = e^L,  m = 1 - a,  beta = sqrt(1 - a^2) = sqrt(m (2 - m)),
//   h_t = a h_{t-1} + beta sigmoid(i) x,      y = h  or  h silu(z).
// Gradients, q_{t+1} being what token t + 1 sends back (or dfinal after a sequence's last token):
//   g = dy [silu(z)] + q_{t+1},   q_t = a g,   dx = g beta sigmoid(i),
//   M = g L (a h_{t-1} - sigmoid(i) x a^2 / beta),   dr = M (1 - s),   dA_log = sum of M.
//
// Memory-bound if the work is spread over the card and the inputs are read once.  There is one
// state per channel, so a row's channels alone fill a few waves: rows are cut into tiles of
// tokens, a workgroup each.  A tile's tokens stay in registers, in runs of a few tokens per lane;
// runs, waves and tiles are joined as maps h -> P h + H (P the product of the decays): runs and
// waves through LDS, tiles through memory.  A tile publishes its map as soon as it
// has it and takes those of the tiles before it; every 16th tile publishes its final state
// instead, so that a tile reads 15 maps and one state at most and the waiting grows with a
// sixteenth of the tiles.  Maps are always composed in the same order, whoever comes first:
// results are deterministic.  A map of a channel is one 64-bit word that is its own flag (the
// words are zeroed by a launch before), so nothing has to be fenced.  The tiles of a chain (a row's
// 64 channels) are handed out by its counter: a tile waits only for tiles that workgroups already
// running have taken, so every wait ends (and it is bounded besides).  One counter for all chains
// held the card up: 5120 workgroups took 94 us, 10240 of half the size 141.
//
// Backward, a first pass over the tiles leaves the state before every 16th token (not for a row of
// one tile, whose waves join their runs in LDS); then tiles walk from a row's end, maps being q -> P q + Q of
// what a run sends back.
//
// Measured on an MI355X (a device copy moves 5.1 TB/s), bf16, a call: 4 x 4096 tokens of 2560
// channels 71 us for 336 MB, vector units at work for 76 %; 16384 tokens of 1536 with a gate 60 us
// for 252 MB (60 %); gradients of 4 x 4096 x 2560, packed, 273 us: the first pass 73 (252 MB read),
// the second 195 for 925 MB (79 %), sums and zeros 9; of 8 x 2048 x 1536 with a gate 177 (41 and
// 128 for 705 MB).  So both bounds are near: about 45 vector instructions an element forward (six
// of them transcendental) and 130 backward, a third of them the joins'.  Fewer instructions for
// addresses (a branch for whole tiles) were slower, 77 -> 82 us; tiles of half the tokens 78 -> 91,
// of twice as many 107; a workgroup that takes several tiles with the next one's loads in flight
// 105 (200 registers); loads for the tile that would be next while the counter is asked 89.
// Fp32: 4 x 2048 x 2560 70 us for 336 MB, gradients 175 (252 + 587 MB).
// A row of up to 256 tokens (fp32 and backward 128) is one tile of up to eight waves: one launch,
// no first pass (against two tiles that join through memory: 64 rows of 2560 channels,
// gradients of 128 tokens 124 -> 100 us, 256 tokens forward 79 -> 75).  A longer one costs a
// launch for the zeros and some us for the counter and the maps' way between dies: 2 rows of 650
// channels on the GPU 6.3 us for 128 tokens, 8.8 for 256, 11 for 777; gradients 12 for 128, 23 for
// 256, 27 for 777.
#include "ssd.h"

#include <algorithm>
#include <cstdio>

#include "block_common.hpp"
#include "block_host.hpp"
#include "ssd_recurrence_map.hpp"

namespace ssd {

constexpr int kBlock = 64;           // channels of a workgroup
constexpr int kWaves = 8;            // waves of a workgroup, at most: rows of one tile
constexpr int kTileWaves = 4;        // of one of several tiles
constexpr int kGroup = 16;           // tiles from one published state to the next
constexpr int kRunBack = 16;         // tokens of a wave backward, and between states kept for it
constexpr int kCounter = 32;         // words between two chains' counters: a line each

// What the tiles of one direction publish: words (chains, tiles, 64) and (chains, groups, 64).
struct Chain {
    uint64_t *maps, *states;
    unsigned* counters;              // a chain's next tile, kCounter apart
};

struct RecurrenceParams {
    const void *x, *r, *i, *z;
    const float *A_log, *init;
    const int32_t* seq_idx;
    void* y;
    float* fin;
    const float *dy, *dfin;
    float *dx, *dr, *di, *dz, *dinit;
    float *part;                     // tiles' sums of dA_log, rows of D
    float *kept;                     // state before every kRunBack-th token, (batch, n, D)
    Chain chain;
    int64_t batch, T, D, nseqs, ldx, ldr, ldi, ldz;
    int64_t pieces;                  // kept states per row
    unsigned nblk, ntile;            // blocks of channels, tiles per row
    int stream;
};

// A log2(e), kept finite so that a gate of 0 times it is 0 (NaN stays): e^88 log2(e) is 0.7 of fp32's
// largest, so every product with a gate that is not 0 is right, however nearly closed.
__device__ inline float rate_of(float a_log) { return -kLog2e * expf(a_log > 88.f ? 88.f : a_log); }

// sigmoid(v), and sigmoid(-v) to its own relative precision, from t = e^-|v|.  EXACT: the
// exponent's rounding is made good, as in exp_small (beyond +-100 as at +-100, where t is 0; NaN
// stays).  Else t is off by |v| roundings, which for a bf16 v is 2^-16 of v's own step.
struct Gate {
    float s, n;
};
template <bool EXACT> __device__ inline float exp_minus(float v) {
    if constexpr (!EXACT) return __builtin_amdgcn_exp2f(v * -kLog2e);
    const float hi = v * -kLog2e, lo = fmaf(v, -1.925963033500012e-08f, fmaf(v, -kLog2e, -hi));
    const float t = __builtin_amdgcn_exp2f(hi);
    return fmaf(t * lo, kLn2, t);
}
template <bool EXACT> __device__ inline Gate gates_of(float v) {
    float a = fabsf(v);
    if (EXACT) a = a > 100.f ? 100.f : a;
    const float t = exp_minus<EXACT>(a), big = __builtin_amdgcn_rcpf(1.f + t), small = t * big;
    return v < 0.f ? Gate{small, big} : Gate{big, small};
}
template <bool EXACT> __device__ inline float gate_of(float v) {
    if constexpr (EXACT) return gates_of<true>(v).s;
    return __builtin_amdgcn_rcpf(1.f + exp_minus<false>(v));
}

// A decay a = e^L, L <= 0, from K = L log2(e), as one number k.  Near 1 a long memory is a matter
// of m = 1 - a, and k is -m, its sign bit set also where m is 0: m = -L (1 + L/2 + L^2/6 + ...), a
// polynomial fitted to the definition on [-1/8, 0] by interpolation at Chebyshev points (relative
// error 3.4e-8 with its rounded coefficients), these times ln(2)^k for K.  Below, k is a itself:
// what it multiplies (a state, a gradient on its way back, dr and dA_log) is then right relative to
// itself, where 1 - m is a multiple of 2^-24, and 0 from L = -17.3 on.  near stays a mask of the
// wave: as a factor of 1 or 0 it took registers (spills; 16384 x 1536 with a gate 66 us against 61.5).
struct Decay {
    float k;
    bool near;
};
__device__ inline Decay decay_of(float K) {
    float q = fmaf(0.009151561185717583f, K, 0.05545208230614662f);
    q = fmaf(q, K, 0.24022464454174042f);
    q = fmaf(q, K, 0.6931471824645996f);
    const bool near = K > -0.18f;
    return {near ? K * q : __builtin_amdgcn_exp2f(K), near};
}
__device__ inline Decay decay_from(float k) { return {k, __float_as_int(k) < 0}; }
constexpr Decay kKeepAll{-0.f, true};
__device__ inline float beta_of(Decay a) { return __builtin_amdgcn_sqrtf(fmaf(-a.k, a.k, a.near ? -2.f * a.k : 1.f)); }
// a v + u and a v.  Near 1 as v - m v, so that an error of 1's last place does not add up over a
// long memory.
__device__ inline float advance(float v, Decay a, float u) { return (a.near ? v : 0.f) + fmaf(a.k, v, u); }
__device__ inline float decayed(float v, Decay a) { return fmaf(a.k, v, a.near ? v : 0.f); }

// ------------------------------------------------------------------ what tiles publish
__device__ inline void publish(uint64_t* p, Map m) {
    __hip_atomic_store(p, word_of(m), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Up to N words `step` apart, each as soon as it is there.  The bound (about a second) is never
// reached in a call by itself; it ends the waits of calls that were given one workspace at the
// same time.  A word that did not come is 0.
template <int N> __device__ inline void await(const uint64_t* p, int64_t step, int n, uint64_t (&w)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = 0;
    for (int tries = 0; tries < 1 << 20; ++tries) {
        bool all = true;
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (k < n && !(uint32_t)w[k])
                w[k] = __hip_atomic_load(p + k * step, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int k = 0; k < N; ++k) all = all && (k >= n || (uint32_t)w[k]);
        if (all) break;
        __builtin_amdgcn_s_sleep(2);
    }
}

// Shared memory of a workgroup of up to W waves.
template <int RUNS, int W> struct Joint {
    struct Wave {
        float P[RUNS][kBlock], H[RUNS][kBlock];        // maps of its runs, H then their incoming states
        Map total[kBlock];           // its map
        Map before[kBlock];          // of a part of the tiles before
        float sums[kBlock];
    };
    float carry[kBlock];             // state before the tile
    unsigned ticket, pad[3];
    Wave wave[W];
    static constexpr int bytes(int waves) { return (int)sizeof(Joint) - (W - waves) * (int)sizeof(Wave); }
};

// Where a workgroup and a lane work.  LPT lanes with V channels each hold a token's 64 channels;
// the wave's V lane groups hold a run of tokens each.  The last vector of a row is moved back to
// end with it: it repeats channels of its neighbour with equal results.  Between the runs' maps a
// lane stands for one of the 64 places (own).
struct Tile {
    int64_t b, c0, own;
    unsigned at, chain;              // the tile's place in the order of the walk
    int wave, group, slot;
    bool active, here;               // the lane's channels, its place exist
};
template <int V> __device__ inline Tile tile_of(const RecurrenceParams& p) {
    constexpr int LPT = kBlock / V;
    const unsigned chains = p.nblk * (unsigned)p.batch, lane = threadIdx.x & 63;
    Tile q;
    q.chain = blockIdx.x % chains;
    q.at = 0;
    q.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    q.b = q.chain / p.nblk;
    const int64_t first = (int64_t)(q.chain % p.nblk) * kBlock;
    auto channel = [&](int64_t vec) { return vec + V <= p.D ? vec : p.D - V; };
    q.group = lane / LPT;
    q.slot = (lane % LPT) * V;
    q.active = first + q.slot < p.D;
    q.c0 = q.active ? channel(first + q.slot) : 0;
    q.here = first + lane / V * V < p.D;
    q.own = q.here ? channel(first + lane / V * V) + lane % V : 0;
    return q;
}

// The workgroup's tile of its chain, from the chain's counter.
__device__ inline void take_tile(const RecurrenceParams& p, Tile& q, unsigned* ticket) {
    if (p.ntile == 1) return;
    if (threadIdx.x == 0)
        *ticket = __hip_atomic_fetch_add(p.chain.counters + (int64_t)q.chain * kCounter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    q.at = __builtin_amdgcn_readfirstlane(*ticket);
}

// Joins the runs whose maps the lanes left in their wave's P and H: puts into H the state that reaches
// each run, in the order of the walk.  `first` is what reaches the row's first tile, `keep` is
// called with the number of each run of the wave and the state that reaches it (lanes are places).
template <int RUNS, bool SEQ, bool FORWARD, int W, typename Keep>
__device__ inline void join(const Chain& c, Joint<RUNS, W>& j, const Tile& q, unsigned ntile, int waves, float first, Keep keep) {
    const int lane = threadIdx.x & 63;
    const int w = FORWARD ? q.wave : waves - 1 - q.wave;      // place of the wave in the order of the walk
    auto run = [&](int k) { return FORWARD ? k : RUNS - 1 - k; };
    auto total = [&](int k) { return j.wave[FORWARD ? k : waves - 1 - k].total[lane]; };
    Map m[RUNS], all{1.f, 0.f};
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
        m[k] = {j.wave[q.wave].P[run(k)][lane], j.wave[q.wave].H[run(k)][lane]};
        all = then<SEQ>(all, m[k]);
    }
    float h = first;
    if (waves > 1) {
        j.wave[q.wave].total[lane] = all;
        __syncthreads();
    }
    if (ntile > 1) {
        const unsigned group = q.at / kGroup, from = group * kGroup;
        const bool closes = q.at == from + kGroup - 1;        // the group: publishes its state
        const bool ends = q.at + 1 == ntile;                  // nobody follows
        Map own{1.f, 0.f};
        if (w == 0) {
            for (int k = 0; k < waves; ++k) own = then<SEQ>(own, total(k));
            if (!closes && !ends) publish(c.maps + ((int64_t)q.chain * ntile + q.at) * kBlock + lane, own);
        }
        // the tiles of the group before this one, in `waves` parts
        constexpr int kPart = kGroup / kTileWaves;
        const int n = (int)(q.at - from), per = (n + waves - 1) / waves, lo = w * per, hi = lo + per < n ? lo + per : n;
        Map part{1.f, 0.f};
        for (int k = lo; k < hi; k += kPart) {
            uint64_t word[kPart];
            await(c.maps + ((int64_t)q.chain * ntile + from + k) * kBlock + lane, (int64_t)kBlock, hi - k < kPart ? hi - k : kPart, word);
#pragma unroll
            for (int e = 0; e < kPart; ++e)
                if (k + e < hi) part = then<SEQ>(part, map_of(word[e]));
        }
        j.wave[w].before[lane] = part;
        const unsigned ngroup = (ntile + kGroup - 1) / kGroup;
        if (w == 0 && group > 0) {
            uint64_t word[1];
            await(c.states + ((int64_t)q.chain * ngroup + group - 1) * kBlock + lane, (int64_t)0, 1, word);
            h = state_of(word[0]);
        }
        __syncthreads();
        if (w == 0) {
            for (int k = 0; k < waves; ++k) h = apply<SEQ>(j.wave[k].before[lane], h);
            if (closes && !ends)
                publish(c.states + ((int64_t)q.chain * ngroup + group) * kBlock + lane, Map{1.f, apply<SEQ>(own, h)});
            j.carry[lane] = h;
        }
        __syncthreads();
        h = j.carry[lane];
    }
    for (int k = 0; k < w; ++k) h = apply<SEQ>(total(k), h);
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
        keep(run(k), h);
        j.wave[q.wave].H[run(k)][lane] = h;
        h = apply<SEQ>(m[k], h);
    }
    __builtin_amdgcn_wave_barrier();
}

// Sequence of each token of a run, and which tokens begin or end one; from the ids of the run and
// its neighbours.
template <int R> struct Ids {
    int v[R + 2];
};
template <int R> __device__ inline Ids<R> load_ids(const RecurrenceParams& p, int64_t b, int64_t t0) {
    Ids<R> q;
#pragma unroll
    for (int k = 0; k < R + 2; ++k) {
        const int64_t t = t0 + k - 1;
        q.v[k] = p.seq_idx[b * p.T + (t < 0 ? 0 : (t < p.T ? t : p.T - 1))];
    }
    return q;
}
template <int R> struct Runs {
    int id[R];
    unsigned fresh, last;            // bits
};
template <int R> __device__ inline Runs<R> runs_of(const RecurrenceParams& p, const Ids<R>& ids, int64_t t0) {
    Runs<R> q;
    q.fresh = q.last = 0;
    auto id = [&](int k) {
        const int64_t t = t0 + k - 1;
        return t >= 0 && t < p.T ? (int)clamp_id(ids.v[k], p.nseqs) : -1;
    };
    int prev = id(0);
#pragma unroll
    for (int k = 0; k < R; ++k) {
        q.id[k] = id(k + 1);
        if (q.id[k] != prev) {
            if (q.id[k] >= 0) q.fresh |= 1u << k;
            if (k) q.last |= 1u << (k - 1);
        }
        prev = q.id[k];
    }
    if (prev >= 0 && id(R + 1) != prev) q.last |= 1u << (R - 1);
    return q;
}

// Where a run's R tokens from flat token `row` on lie, of which `rest` exist; the last one stands
// for those that do not.
template <typename T> __device__ inline const T* token_at(const void* base, int64_t ld, int64_t row, int64_t rest, bool full, int k) {
    return (const T*)base + (row + (full || k < rest ? k : rest - 1)) * ld;
}

// Keeps a pack of bf16 as it was loaded: without this the compiler converts it once and holds the
// fp32 values, twice the registers, until their last use.
template <typename T, int V> __device__ inline void stay_packed(Pack<T, V>& p) {
    if constexpr (sizeof(p) % 4 == 0 && sizeof(T) < 4) {
        uint32_t w[sizeof(p) / 4];
        __builtin_memcpy(w, &p, sizeof(p));
#pragma unroll
        for (unsigned k = 0; k < sizeof(p) / 4; ++k) asm volatile("" : "+v"(w[k]));
        __builtin_memcpy(&p, w, sizeof(p));
    }
}

// Whole rows.  TOK tokens per wave; KEEP: no output, but the state before every kRunBack-th token.
// W: waves of a workgroup, at most (one kernel for both numbers was 3 % slower with tiles of four).
template <typename T, int V, int TOK, int W, bool SEQ, bool GATE, bool STREAM, bool KEEP>
__global__ __launch_bounds__(64 * W, sizeof(T) == 4 ? 1 : 4) void recurrence_forward_kernel(RecurrenceParams p) {
    constexpr int R = TOK / V, RS = SEQ ? R : 1;
    constexpr bool EXACT = sizeof(T) == 4;
    __shared__ Joint<V, W> j;
    const int waves = blockDim.x >> 6;
    Tile q = tile_of<V>(p);
    take_tile(p, q, &j.ticket);
    if (q.at >= p.ntile) return;             // only in a workspace that another call writes too
    const int64_t w0 = ((int64_t)q.at * waves + q.wave) * TOK, t0 = w0 + q.group * R, rest = p.T - t0, row = q.b * p.T + t0;
    const bool full = w0 + TOK <= p.T;
    float P[R][V], H[R][V];          // map from the run's start to after each token
    Pack<T, V> x[R], r[R], g[R], z[GATE ? R : 1];
    float A[V], end_p[V], end_h[V];
    Runs<RS> s{};
    load_f32<V>(p.A_log + q.c0, A);
#pragma unroll
    for (int k = 0; k < R; ++k) {
        r[k] = load_pack<V>(token_at<T>(p.r, p.ldr, row, rest, full, k) + q.c0);
        g[k] = load_pack<V>(token_at<T>(p.i, p.ldi, row, rest, full, k) + q.c0);
        x[k] = load_pack<V>(token_at<T>(p.x, p.ldx, row, rest, full, k) + q.c0);
    }
    if (SEQ) s = runs_of<RS>(p, load_ids<RS>(p, q.b, t0), t0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = rate_of(A[v]);
        end_p[v] = 1.f;
        end_h[v] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
        Decay a[V];
        float u[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            a[v] = decay_of(A[v] * gate_of<EXACT>((float)r[k].v[v]));
            u[v] = beta_of(a[v]) * (gate_of<EXACT>((float)g[k].v[v]) * (float)x[k].v[v]);
        }
        if (!full) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (k >= rest) a[v] = kKeepAll, u[v] = 0.f;
        }
        const bool fresh = SEQ && (s.fresh >> k & 1);
        if (SEQ && fresh) {
            float h[V];
            if (p.init) load_f32<V>(p.init + (int64_t)s.id[SEQ ? k : 0] * p.D + q.c0, h);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                end_h[v] = p.init ? h[v] : 0.f;
                end_p[v] = 0.f;
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            end_h[v] = H[k][v] = advance(end_h[v], a[v], u[v]);
            end_p[v] = P[k][v] = decayed(end_p[v], a[v]);
        }
        __builtin_amdgcn_sched_barrier(0);       // token by token: the inputs' registers become free
    }
    if (SEQ && s.fresh) {
#pragma unroll
        for (int v = 0; v < V; ++v) end_p[v] = -1.f;
    }
    store_f32<V>(&j.wave[q.wave].P[q.group][q.slot], end_p);
    store_f32<V>(&j.wave[q.wave].H[q.group][q.slot], end_h);
    // a row of packed sequences begins with a fresh token, others with their initial state
    const float first = !SEQ && p.init ? p.init[q.b * p.D + q.own] : 0.f;
    join<V, SEQ, true>(p.chain, j, q, p.ntile, waves, first, [&](int run, float h) {
        if constexpr (KEEP) {
            const int64_t t = w0 + run * R;
            if (run * R % kRunBack == 0 && t < p.T && q.here) p.kept[(q.b * p.pieces + t / kRunBack) * p.D + q.own] = h;
        }
    });
    if (KEEP || !q.active) return;
    if constexpr (GATE) {            // not before: its registers would cost a wave per SIMD
#pragma unroll
        for (int k = 0; k < R; ++k) z[k] = load_pack<V>(token_at<T>(p.z, p.ldz, row, rest, full, k) + q.c0);
    }
    float h0[V];
    load_f32<V>(&j.wave[q.wave].H[q.group][q.slot], h0);
#pragma unroll
    for (int k = 0; k < R; ++k) {
        if (k >= rest) break;
        const bool fresh = SEQ && (s.fresh >> k & 1);
        float h[V], y[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (fresh) h0[v] = 0.f;                          // P is 0 from here on in the run
            h[v] = fmaf(P[k][v], h0[v], H[k][v]);
            y[v] = GATE ? h[v] * silu_for<T>((float)z[GATE ? k : 0].v[v]) : h[v];
        }
        store_f32<V, STREAM>((T*)p.y + (row + k) * p.D + q.c0, y);
        if (p.fin && (SEQ ? (s.last >> k & 1) : k + 1 == rest))
            store_f32<V>(p.fin + (SEQ ? (int64_t)s.id[SEQ ? k : 0] : q.b) * p.D + q.c0, h);
    }
}

// Gradients of whole rows, tiles from the last to the first.
template <typename T, int V, bool SEQ, bool GATE, bool STREAM>
__global__ __launch_bounds__(64 * kWaves) void recurrence_backward_kernel(RecurrenceParams p) {
    constexpr int TOK = kRunBack, R = TOK / V;
    constexpr bool EXACT = sizeof(T) == 4;
    extern __shared__ __align__(16) float shared[];
    Joint<V, kWaves>& j = *(Joint<V, kWaves>*)shared;          // as much of it as the waves need
    const int waves = blockDim.x >> 6;
    Tile q = tile_of<V>(p);
    take_tile(p, q, &j.ticket);
    if (q.at >= p.ntile) return;             // only in a workspace that another call writes too
    const unsigned tile = p.ntile - 1 - q.at;
    const int64_t piece = (int64_t)tile * waves + q.wave, w0 = piece * TOK, t0 = w0 + q.group * R, rest = p.T - t0;
    const int64_t row = q.b * p.T + t0;
    const bool full = w0 + TOK <= p.T;
    Runs<SEQ ? R : 1> s{};
    Pack<T, V> x[R], r[R], g[R], z[GATE ? R : 1];
    float a[R][V], gy[R][V], A[V];
    float hp[R][V];                  // what each token adds, then the state before it
    // the state before the first token of a sequence
    auto begin = [&](int k, float (&h)[V]) {
        if (p.init) {
            load_f32<V>(p.init + (int64_t)s.id[SEQ ? k : 0] * p.D + q.c0, h);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = 0.f;
        }
    };
    if (SEQ) s = runs_of<SEQ ? R : 1>(p, load_ids<SEQ ? R : 1>(p, q.b, t0), t0);
    float end_p[V], end_h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) end_p[v] = 1.f, end_h[v] = 0.f;
    // the state before the wave's first token (or the row's), of the lane's place
    float h0 = 0.f;
    if (p.kept) {
        if (w0 < p.T) h0 = p.kept[(q.b * p.pieces + piece) * p.D + q.own];
    } else if (!SEQ && p.init) {
        h0 = p.init[q.b * p.D + q.own];
    }
    if (q.active) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            r[k] = load_pack<V>(token_at<T>(p.r, p.ldr, row, rest, full, k) + q.c0);
            g[k] = load_pack<V>(token_at<T>(p.i, p.ldi, row, rest, full, k) + q.c0);
            x[k] = load_pack<V>(token_at<T>(p.x, p.ldx, row, rest, full, k) + q.c0);
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            load_f32<V>(token_at<float>(p.dy, p.D, row, rest, full, k) + q.c0, gy[k]);
            if constexpr (GATE) z[k] = load_pack<V>(token_at<T>(p.z, p.ldz, row, rest, full, k) + q.c0);
        }
        load_f32<V>(p.A_log + q.c0, A);
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = rate_of(A[v]);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (SEQ && (s.fresh >> k & 1)) begin(k, end_h);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                Decay d = decay_of(A[v] * gate_of<EXACT>((float)r[k].v[v]));
                hp[k][v] = beta_of(d) * (gate_of<EXACT>((float)g[k].v[v]) * (float)x[k].v[v]);
                if (!full && k >= rest) d = kKeepAll, hp[k][v] = gy[k][v] = 0.f;
                a[k][v] = d.k;
                end_h[v] = advance(end_h[v], d, hp[k][v]);
                end_p[v] = decayed(end_p[v], d);
            }
            stay_packed(r[k]);
            stay_packed(g[k]);
            stay_packed(x[k]);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (SEQ && s.fresh) {
#pragma unroll
            for (int v = 0; v < V; ++v) end_p[v] = -1.f;
        }
    }
    store_f32<V>(&j.wave[q.wave].P[q.group][q.slot], end_p);
    store_f32<V>(&j.wave[q.wave].H[q.group][q.slot], end_h);
    __builtin_amdgcn_wave_barrier();
    {
        const int lane = threadIdx.x & 63;
        Map run[V];
#pragma unroll
        for (int k = 0; k < V; ++k) run[k] = {j.wave[q.wave].P[k][lane], j.wave[q.wave].H[k][lane]};
        if (!p.kept && waves > 1) {          // a single tile: from the waves before
            Map all{1.f, 0.f};
#pragma unroll
            for (int k = 0; k < V; ++k) all = then<SEQ>(all, run[k]);
            j.wave[q.wave].before[lane] = all;
            __syncthreads();
            for (int k = 0; k < q.wave; ++k) h0 = apply<SEQ>(j.wave[k].before[lane], h0);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            j.wave[q.wave].H[k][lane] = h0;
            h0 = apply<SEQ>(run[k], h0);
        }
    }
    __builtin_amdgcn_wave_barrier();
    if (q.active) {
        float h[V];
        load_f32<V>(&j.wave[q.wave].H[q.group][q.slot], h);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const bool last = SEQ ? (s.last >> k & 1) : k + 1 == rest;
            if (SEQ && (s.fresh >> k & 1)) begin(k, h);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float u = hp[k][v];
                hp[k][v] = h[v];
                h[v] = advance(h[v], decay_from(a[k][v]), u);
            }
            if constexpr (GATE) {
                float dz[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float zv = (float)z[k].v[v], sz = gate_of<EXACT>(zv);
                    dz[v] = gy[k][v] * h[v] * silu_slope(zv, sz);
                    gy[k][v] *= zv * sz;
                }
                if (k < rest) store_f32<V, STREAM>(p.dz + (row + k) * p.D + q.c0, dz);
            }
            if (last && p.dfin) {
                float d[V];
                load_f32<V>(p.dfin + (SEQ ? (int64_t)s.id[SEQ ? k : 0] : q.b) * p.D + q.c0, d);
#pragma unroll
                for (int v = 0; v < V; ++v) gy[k][v] += d[v];
            }
        }
    }
    // backwards through the run, from nothing; the product of its decays is in place
#pragma unroll
    for (int v = 0; v < V; ++v) end_h[v] = 0.f;
    if (q.active) {
#pragma unroll
        for (int k = R - 1; k >= 0; --k) {
            const bool fresh = SEQ && (s.fresh >> k & 1);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float e = gy[k][v] + end_h[v];
                end_h[v] = fresh ? 0.f : decayed(e, decay_from(a[k][v]));
            }
        }
    }
    store_f32<V>(&j.wave[q.wave].H[q.group][q.slot], end_h);
    join<V, SEQ, false>(p.chain, j, q, p.ntile, waves, 0.f, [](int, float) {});
    float dA[V];
#pragma unroll
    for (int v = 0; v < V; ++v) dA[v] = 0.f;
    if (q.active) {
        float e[V];
        load_f32<V>(&j.wave[q.wave].H[q.group][q.slot], e);
#pragma unroll
        for (int k = R - 1; k >= 0; --k) {
            if (k >= rest) continue;
            float dx[V], dr[V], di[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Decay ak = decay_from(a[k][v]);
                const float d = gy[k][v] + e[v], decay = (ak.near ? 1.f : 0.f) + ak.k;
                const Gate sr = gates_of<EXACT>((float)r[k].v[v]), si = gates_of<EXACT>((float)g[k].v[v]);
                // a L first: L alone times a state can leave fp32, and a be 0
                const float aL = decay * (A[v] * sr.s * kLn2), beta = beta_of(ak), in = si.s * (float)x[k].v[v];
                const float ratio = beta > 0.f ? aL * __builtin_amdgcn_rcpf(beta) : 0.f;
                const float M = d * fmaf(aL, hp[k][v], -in * decay * ratio);
                dx[v] = d * beta * si.s;
                di[v] = d * beta * in * si.n;
                dr[v] = M * sr.n;
                dA[v] += M;
                e[v] = decayed(d, ak);
            }
            store_f32<V, STREAM>(p.dx + (row + k) * p.D + q.c0, dx);
            store_f32<V, STREAM>(p.dr + (row + k) * p.D + q.c0, dr);
            store_f32<V, STREAM>(p.di + (row + k) * p.D + q.c0, di);
            const bool fresh = SEQ ? (s.fresh >> k & 1) : t0 + k == 0;
            if (fresh) {
                if (p.dinit) store_f32<V>(p.dinit + (SEQ ? (int64_t)s.id[SEQ ? k : 0] : q.b) * p.D + q.c0, e);
#pragma unroll
                for (int v = 0; v < V; ++v) e[v] = 0.f;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // sums over the runs of each wave, then over the waves
    store_f32<V>(&j.wave[q.wave].P[q.group][q.slot], dA);
    __builtin_amdgcn_wave_barrier();
    const int lane = threadIdx.x & 63;
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) sum += j.wave[q.wave].P[k][lane];
    if (waves > 1) {
        j.wave[q.wave].sums[lane] = sum;
        __syncthreads();
    }
    if (q.wave == 0 && q.here) {
        for (int w = 1; w < waves; ++w) sum += j.wave[w].sums[lane];
        p.part[(q.b * p.ntile + tile) * p.D + q.own] = sum;
    }
}

// One token: a thread per (row, channel).  On the GPU 64 x 2560 with a gate 3.2 us (bf16) and 3.5
// (fp32): a launch; 256 x 5120 7.7 and 8.5 for 24 and 37 MB.
template <typename T> __global__ __launch_bounds__(256) void recurrence_step_kernel(RecurrenceParams p) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= p.batch * p.D) return;
    const int64_t b = n / p.D, c = n % p.D;
    constexpr bool EXACT = sizeof(T) == 4;
    const Decay a = decay_of(rate_of(p.A_log[c]) * gate_of<EXACT>((float)((const T*)p.r)[b * p.ldr + c]));
    const float u = beta_of(a) * (gate_of<EXACT>((float)((const T*)p.i)[b * p.ldi + c]) * (float)((const T*)p.x)[b * p.ldx + c]);
    const float h = advance(p.init[n], a, u);
    p.fin[n] = h;
    ((T*)p.y)[n] = (T)(p.z ? h * silu_for<T>((float)((const T*)p.z)[b * p.ldz + c]) : h);
}

// Zeros for the words that tiles publish, 16 bytes a store, and for a second array.
__global__ __launch_bounds__(256) void recurrence_clear_kernel(uint4* p, int64_t n, float* q, int64_t m) {
    const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t i = first; i < n; i += step) p[i] = uint4{0, 0, 0, 0};
    for (int64_t i = first; i < m; i += step) q[i] = 0.f;
}
static hipError_t launch_clear(void* p, int64_t bytes, float* q, int64_t floats, hipStream_t s) {
    const int64_t n = bytes / 16, g = (std::max(n, floats) + 255) / 256;
    if (g <= 0) return hipSuccess;
    hipLaunchKernelGGL(recurrence_clear_kernel, dim3((unsigned)(g < 2048 ? g : 2048)), dim3(256), 0, s, (uint4*)p, n, q, floats);
    return hipGetLastError();
}

// ------------------------------------------------------------------ launches
enum Pass { kForward, kKeep, kBackward };
template <Pass PASS, typename T, int V, bool SEQ, bool GATE, bool STREAM>
static void launch_one(const RecurrenceParams& p, int waves, hipStream_t s) {
    const dim3 grid(p.nblk * (unsigned)p.batch * p.ntile), block(64 * waves);
    // fp32 has half the vector instructions a byte to spare: shorter runs start sooner (2 x 16 tokens
    // of 650 channels 6.6 -> 4.6 us, 2 x 777 13.3 -> 11.9, 4 x 2048 x 2560 73.9 -> 71.7)
    constexpr int TOK = V == 1 || sizeof(T) == 4 ? 16 : 32;
    if constexpr (PASS == kBackward)
        hipLaunchKernelGGL((recurrence_backward_kernel<T, V, SEQ, GATE, STREAM>), grid, block,
                           (Joint<V, kWaves>::bytes(waves)), s, p);
    else if (waves <= kTileWaves)
        hipLaunchKernelGGL((recurrence_forward_kernel<T, V, TOK, kTileWaves, SEQ, GATE, STREAM, PASS == kKeep>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((recurrence_forward_kernel<T, V, TOK, kWaves, SEQ, GATE, STREAM, PASS == kKeep>), grid, block, 0, s, p);
}
template <Pass PASS, typename T, int V, bool STREAM> static void launch_seq(const RecurrenceParams& p, int waves, hipStream_t s) {
    if constexpr (PASS != kKeep) {
        if (p.z) {
            if (p.seq_idx) launch_one<PASS, T, V, true, true, STREAM>(p, waves, s);
            else launch_one<PASS, T, V, false, true, STREAM>(p, waves, s);
            return;
        }
    }
    if (p.seq_idx) launch_one<PASS, T, V, true, false, STREAM>(p, waves, s);
    else launch_one<PASS, T, V, false, false, STREAM>(p, waves, s);
}
// Rows narrower than a vector take a channel per lane.
template <Pass PASS, typename T, int V> static void launch_width(const RecurrenceParams& p, int waves, hipStream_t s) {
    if (p.D < V) return launch_seq<PASS, T, 1, false>(p, waves, s);
    if constexpr (PASS != kKeep) {
        if (p.stream) return launch_seq<PASS, T, V, true>(p, waves, s);
    }
    launch_seq<PASS, T, V, false>(p, waves, s);
}
// Vectors are 16 bytes of the activations, but backwards of the fp32 gradients: with eight
// channels a lane, whose stores of 16 bytes lie 32 apart, three gradients of 4 x 4096 x 2560 went
// out at 4.0 TB/s, with four at 5.4.
constexpr int vector_of(Pass pass, bool bf16) { return bf16 && pass != kBackward ? 8 : 4; }
template <Pass PASS> static hipError_t launch_pass(bool bf16, const RecurrenceParams& p, int waves, hipStream_t s) {
    if (bf16) launch_width<PASS, __bf16, vector_of(PASS, true)>(p, waves, s);
    else launch_width<PASS, float, vector_of(PASS, false)>(p, waves, s);
    return hipGetLastError();
}

}  // namespace ssd

namespace {

using namespace ssd_host;

constexpr int64_t kMaxDim = int64_t(1) << 31;

// Blocks of channels, waves of a workgroup and tiles per row.
struct Shape {
    int64_t nblk, waves, ntile;
};
Shape shape_of(const ssd_recurrence_problem_t* p, bool back) {
    Shape s;
    s.nblk = (p->channels + ssd::kBlock - 1) / ssd::kBlock;
    const bool narrow = p->channels < ssd::vector_of(ssd::kForward, p->dtype == SSD_DTYPE_BF16);
    const int64_t tokens = back || narrow || p->dtype == SSD_DTYPE_F32 ? ssd::kRunBack : 32;          // of a wave
    const int64_t runs = std::max<int64_t>(1, (p->seqlen + tokens - 1) / tokens);
    s.waves = runs <= ssd::kWaves ? runs : ssd::kTileWaves;
    s.ntile = (runs + s.waves - 1) / s.waves;
    return s;
}

int validate(const ssd_recurrence_problem_t* p) {
    if (!p) return SSD_ERR_NULL_POINTER;
    if (p->batch < 0 || p->seqlen < 0 || p->channels <= 0 || p->nseqs < 0) return SSD_ERR_BAD_SHAPE;
    if (p->batch >= kMaxDim || p->seqlen >= kMaxDim || p->channels >= kMaxDim || p->nseqs >= kMaxDim)
        return SSD_ERR_BAD_SHAPE;
    for (int64_t ld : {p->ldx, p->ldr, p->ldi, p->ldz})
        if (ld < p->channels || ld >= kMaxDim) return SSD_ERR_BAD_SHAPE;
    if (p->dtype != SSD_DTYPE_BF16 && p->dtype != SSD_DTYPE_F32) return SSD_ERR_UNSUPPORTED;
    if (p->flags != 0) return SSD_ERR_UNSUPPORTED;
    const double widest = double(std::max({p->ldx, p->ldr, p->ldi, p->ldz}));
    if (double(p->batch) * double(p->seqlen) * widest > 4e17 || double(p->nseqs) * p->channels > 4e17)
        return SSD_ERR_BAD_SHAPE;
    // a launch holds fewer than 2^32 threads, a tile's chains fewer than 2^31
    for (bool back : {false, true}) {
        const Shape s = shape_of(p, back);
        if (double(p->batch) * s.nblk >= 2e9 || double(p->batch) * s.nblk * s.ntile * 64 * s.waves >= 4e9)
            return SSD_ERR_UNSUPPORTED;
    }
    return SSD_OK;
}

struct RecSizes {
    int64_t x, r, i, z, y, f, d, state, seq;
};
RecSizes rec_sizes(const ssd_recurrence_problem_t* p) {
    RecSizes s;
    const int64_t bt = p->batch * p->seqlen, e = elem_size(p->dtype);
    auto span = [&](int64_t ld) { return bt > 0 ? ((bt - 1) * ld + p->channels) * e : 0; };
    s.x = span(p->ldx);
    s.r = span(p->ldr);
    s.i = span(p->ldi);
    s.z = span(p->ldz);
    s.y = bt * p->channels * e;
    s.f = bt * p->channels * 4;
    s.d = p->channels * 4;
    s.state = p->nseqs * s.d;
    s.seq = bt * 4;
    return s;
}

bool empty(const ssd_recurrence_problem_t* p) { return p->batch == 0 || p->seqlen == 0; }

// What the tiles publish, in bytes from the workspace's start: counters, maps, states.
struct ChainSpace {
    int64_t maps, states, total;
};
ChainSpace chain_space(const ssd_recurrence_problem_t* p, const Shape& s) {
    ChainSpace c{};
    if (empty(p) || s.ntile == 1) return c;
    const int64_t chains = p->batch * s.nblk, groups = (s.ntile + ssd::kGroup - 1) / ssd::kGroup;
    c.maps = align256(chains * ssd::kCounter * 4);
    c.states = c.maps + chains * s.ntile * ssd::kBlock * 8;
    c.total = align256(c.states + chains * groups * ssd::kBlock * 8);
    return c;
}
// Backwards: both directions' chains, the kept states, the tiles' sums.
struct BackwardSpace {
    int64_t back, kept, part, total;
};
int64_t pieces_of(const ssd_recurrence_problem_t* p) { return (p->seqlen + ssd::kRunBack - 1) / ssd::kRunBack; }
BackwardSpace backward_space(const ssd_recurrence_problem_t* p) {
    BackwardSpace w{};
    if (empty(p)) return w;
    const Shape s = shape_of(p, true);
    const int64_t pieces = pieces_of(p);
    const bool keep = s.ntile > 1;                       // a single tile finds its states itself
    w.back = keep ? chain_space(p, shape_of(p, false)).total : 0;
    w.kept = w.back + chain_space(p, s).total;
    w.part = w.kept + (keep ? align256(p->batch * pieces * p->channels * 4) : 0);
    w.total = w.part + (p->batch * s.ntile > 1 ? align256(p->batch * s.ntile * p->channels * 4) : 0);
    return w;
}
int64_t forward_bytes(const ssd_recurrence_problem_t* p) { return chain_space(p, shape_of(p, false)).total; }
int64_t backward_bytes(const ssd_recurrence_problem_t* p) { return backward_space(p).total; }

ssd::Chain chain_at(const ssd_recurrence_problem_t* p, const Shape& s, void* at) {
    const ChainSpace c = chain_space(p, s);
    char* base = static_cast<char*>(at);
    ssd::Chain r{};
    if (c.total) {
        r.counters = reinterpret_cast<unsigned*>(base);
        r.maps = reinterpret_cast<uint64_t*>(base + c.maps);
        r.states = reinterpret_cast<uint64_t*>(base + c.states);
    }
    return r;
}

ssd::RecurrenceParams params_of(const ssd_recurrence_problem_t* p, const void* x, const void* r, const void* i,
                                const float* A_log, const void* z, const float* init, const int32_t* seq_idx) {
    ssd::RecurrenceParams c{};
    c.x = x;
    c.r = r;
    c.i = i;
    c.z = z;
    c.A_log = A_log;
    c.init = init;
    c.seq_idx = seq_idx;
    c.batch = p->batch;
    c.T = p->seqlen;
    c.D = p->channels;
    c.nseqs = p->nseqs;
    c.ldx = p->ldx;
    c.ldr = p->ldr;
    c.ldi = p->ldi;
    c.ldz = p->ldz;
    c.pieces = pieces_of(p);
    return c;
}

int done(const char* what, const ssd_recurrence_problem_t* p, hipError_t e) {
    if (log_enabled())
        std::fprintf(stderr, "[ssd] recurrence %s dtype=%d batch=%lld T=%lld D=%lld -> %s\n", what, p->dtype,
                     (long long)p->batch, (long long)p->seqlen, (long long)p->channels, hipGetErrorString(e));
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

// One pass over the rows; `space` holds its chain, zeroed.
template <ssd::Pass PASS>
hipError_t run_pass(const ssd_recurrence_problem_t* p, ssd::RecurrenceParams c, void* space, hipStream_t st) {
    const Shape s = shape_of(p, PASS == ssd::kBackward);
    c.nblk = (unsigned)s.nblk;
    c.ntile = (unsigned)s.ntile;
    c.chain = chain_at(p, s, space);
    return ssd::launch_pass<PASS>(p->dtype == SSD_DTYPE_BF16, c, (int)s.waves, st);
}

}  // namespace

extern "C" {

size_t ssd_recurrence_workspace_size(const ssd_recurrence_problem_t* p) {
    return validate(p) == SSD_OK ? (size_t)forward_bytes(p) : 0;
}
size_t ssd_recurrence_backward_workspace_size(const ssd_recurrence_problem_t* p) {
    return validate(p) == SSD_OK ? (size_t)backward_bytes(p) : 0;
}

int ssd_recurrence_forward(const ssd_recurrence_problem_t* p, const void* x, const void* r, const void* i,
                           const float* A_log, const void* z, const float* init_state, const int32_t* seq_idx, void* y,
                           float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
    const int v = validate(p);
    if (v != SSD_OK) return v;
    if (!A_log || (!empty(p) && (!x || !r || !i || !y))) return SSD_ERR_NULL_POINTER;
    const int q = check_sequences(p, seq_idx);
    if (q != SSD_OK) return q;
    const int64_t wsb = forward_bytes(p);
    if (wsb > 0 && !workspace) return SSD_ERR_WORKSPACE;
    const uintptr_t e = (uintptr_t)elem_size(p->dtype);
    if (misaligned(x, e) || misaligned(r, e) || misaligned(i, e) || misaligned(z, e) || misaligned(y, e) ||
        misaligned(A_log, 4) || misaligned(init_state, 4) || misaligned(seq_idx, 4) || misaligned(final_state, 4) ||
        (wsb > 0 && misaligned(workspace, 256)))
        return SSD_ERR_ALIGNMENT;
    if ((int64_t)workspace_bytes < wsb) return SSD_ERR_WORKSPACE;
    const RecSizes n = rec_sizes(p);
    const Buf in[] = {{x, n.x}, {r, n.r}, {i, n.i}, {A_log, n.d}, {z, n.z}, {init_state, n.state}, {seq_idx, n.seq}};
    const Buf out[] = {{y, n.y}, {final_state, n.state}, {workspace, wsb}};
    const int a = check_alias(in, 7, out, 3);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (empty(p)) {
        // no token: each row's final state is its initial state
        if (seq_idx || !final_state) return SSD_OK;
        return done("forward", p, ssd::launch_copy(final_state, init_state, n.state / 4, st));
    }
    ssd::RecurrenceParams c = params_of(p, x, r, i, A_log, z, init_state, seq_idx);
    c.y = y;
    c.fin = final_state;
    c.stream = n.y > ssd::kStreamBytes;
    hipError_t h = ssd::launch_clear(workspace, wsb, nullptr, 0, st);
    if (h == hipSuccess) h = run_pass<ssd::kForward>(p, c, workspace, st);
    return done("forward", p, h);
}

int ssd_recurrence_step(const ssd_recurrence_problem_t* p, const void* x, const void* r, const void* i,
                        const float* A_log, const void* z, const float* state, float* state_out, void* y, void* stream) {
    if (!p) return SSD_ERR_NULL_POINTER;
    if (p->seqlen != 1 || p->nseqs != p->batch) return SSD_ERR_BAD_SHAPE;
    const int v = validate(p);
    if (v != SSD_OK) return v;
    if (double(p->batch) * p->channels >= 4e9) return SSD_ERR_UNSUPPORTED;       // a thread per (row, channel)
    if (!A_log || (p->batch > 0 && (!x || !r || !i || !state || !state_out || !y))) return SSD_ERR_NULL_POINTER;
    const uintptr_t e = (uintptr_t)elem_size(p->dtype);
    if (misaligned(x, e) || misaligned(r, e) || misaligned(i, e) || misaligned(z, e) || misaligned(y, e) ||
        misaligned(A_log, 4) || misaligned(state, 4) || misaligned(state_out, 4))
        return SSD_ERR_ALIGNMENT;
    const RecSizes n = rec_sizes(p);
    const Buf in[] = {{x, n.x}, {r, n.r}, {i, n.i}, {A_log, n.d}, {z, n.z}, {state == state_out ? nullptr : state, n.state}};
    const Buf out[] = {{y, n.y}, {state_out, n.state}};
    const int a = check_alias(in, 6, out, 2);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    if (p->batch == 0) return SSD_OK;
    ssd::RecurrenceParams c = params_of(p, x, r, i, A_log, z, state, nullptr);
    c.y = y;
    c.fin = state_out;
    const dim3 grid((unsigned)((p->batch * p->channels + 255) / 256));
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (p->dtype == SSD_DTYPE_BF16) hipLaunchKernelGGL((ssd::recurrence_step_kernel<__bf16>), grid, dim3(256), 0, st, c);
    else hipLaunchKernelGGL((ssd::recurrence_step_kernel<float>), grid, dim3(256), 0, st, c);
    return done("step", p, hipGetLastError());
}

int ssd_recurrence_backward(const ssd_recurrence_problem_t* p, const void* x, const void* r, const void* i,
                            const float* A_log, const void* z, const float* init_state, const int32_t* seq_idx,
                            const float* dy, const float* dfinal, float* dx, float* dr, float* di, float* dA_log,
                            float* dz, float* dinit, void* workspace, size_t workspace_bytes, void* stream) {
    const int v = validate(p);
    if (v != SSD_OK) return v;
    if (!A_log || !dA_log || (!empty(p) && (!x || !r || !i || !dy || !dx || !dr || !di || (z && !dz))))
        return SSD_ERR_NULL_POINTER;
    const int q = check_sequences(p, seq_idx);
    if (q != SSD_OK) return q;
    const int64_t wsb = backward_bytes(p);
    if (wsb > 0 && !workspace) return SSD_ERR_WORKSPACE;
    const uintptr_t e = (uintptr_t)elem_size(p->dtype);
    if (misaligned(x, e) || misaligned(r, e) || misaligned(i, e) || misaligned(z, e) || misaligned(A_log, 4) ||
        misaligned(init_state, 4) || misaligned(seq_idx, 4) || misaligned(dy, 4) || misaligned(dfinal, 4) ||
        misaligned(dx, 4) || misaligned(dr, 4) || misaligned(di, 4) || misaligned(dA_log, 4) || misaligned(dz, 4) ||
        misaligned(dinit, 4) || (wsb > 0 && misaligned(workspace, 256)))
        return SSD_ERR_ALIGNMENT;
    if ((int64_t)workspace_bytes < wsb) return SSD_ERR_WORKSPACE;
    const RecSizes n = rec_sizes(p);
    const Buf in[] = {{x, n.x}, {r, n.r}, {i, n.i}, {A_log, n.d}, {z, n.z}, {init_state, n.state}, {seq_idx, n.seq},
                      {dy, n.f}, {dfinal, n.state}};
    const Buf out[] = {{dx, n.f}, {dr, n.f}, {di, n.f}, {dA_log, n.d}, {z ? dz : nullptr, n.f}, {dinit, n.state}, {workspace, wsb}};
    const int a = check_alias(in, 9, out, 7);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e2 = hipSuccess;
    if (empty(p)) {
        // no token: nothing reaches the decays, and each row's final state is its initial state
        e2 = ssd::launch_fill(dA_log, p->channels, st);
        if (e2 == hipSuccess && dinit) e2 = ssd::launch_copy(dinit, seq_idx ? nullptr : dfinal, n.state / 4, st);
        return done("backward", p, e2);
    }
    ssd::RecurrenceParams c = params_of(p, x, r, i, A_log, z, init_state, seq_idx);
    const BackwardSpace w = backward_space(p);
    char* base = static_cast<char*>(workspace);
    const Shape s = shape_of(p, true);
    const bool direct = p->batch * s.ntile == 1;         // a single tile writes dA_log itself
    // ids that do not occur keep a zero gradient
    e2 = ssd::launch_clear(base, w.kept, dinit, seq_idx && dinit ? n.state / 4 : 0, st);
    if (e2 == hipSuccess && s.ntile > 1) {
        c.kept = reinterpret_cast<float*>(base + w.kept);
        e2 = run_pass<ssd::kKeep>(p, c, base, st);
    }
    if (e2 == hipSuccess) {
        c.dy = dy;
        c.dfin = dfinal;
        c.dx = dx;
        c.dr = dr;
        c.di = di;
        c.dz = dz;
        c.dinit = dinit;
        c.part = direct ? dA_log : reinterpret_cast<float*>(base + w.part);
        c.stream = n.f > ssd::kStreamBytes;
        e2 = run_pass<ssd::kBackward>(p, c, base + w.back, st);
    }
    if (e2 == hipSuccess && !direct) {
        ssd::ColumnSums cs{};
        cs.part = c.part;
        cs.out = dA_log;
        cs.rows = p->batch * s.ntile;
        cs.cols = cs.split = cs.split2 = p->channels;
        e2 = ssd::launch_column_sums(cs, st);
    }
    return done("backward", p, e2);
}

}  // extern "C"
