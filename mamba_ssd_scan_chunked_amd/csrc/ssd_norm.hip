// The norms around a Mamba block and their gradients.  C entries of include/ssd.h.
//
// Gated norm, after the scan (per row and group of consecutive channels):
//   gate first:  u = x silu(z),  out = u r w
//   gate after:  u = x,          out = u r w silu(z)        r = 1 / sqrt(mean(u^2) + eps)
// Residual norm, before a block (whole rows):
//   u = residual + scale x,  out = u r w,  u kept in fp32 as the stream
//
// Memory-bound.  A row (of a group) is held by a team of TEAM lanes, CH packs of four
// channels each, so every input is read once; sums of squares are fp32 butterflies within a
// wave and meet in LDS above it.  It stays in registers forward and, up to 8192 channels, in the
// gradients (but for 68 bytes a lane of the residual norm's at 513 to 768 channels and 44 at
// 4097 to 8192); gradients of wider groups keep 380 to 2270 bytes a lane in scratch memory.
//
// Gradients, with e = dL/d(u r w) and hat = u r:
//   du = r (e w - hat mean(e w hat)),   dw = sum over rows of e hat.
// A team walks several rows of one group (as it does forward), with dw (and the residual's dscale) in
// registers; the teams' sums go to the workspace and are added in a fixed order.
//
// Measured on an MI355X (a device copy moves 5.0 TB/s, calls that read more than they write up
// to 5.7), bf16: gated norm of 16384 rows of 5120 (fp32 x) 131 us, 5.1 TB/s; its gradients for
// 8192 rows in eight groups 146 us, 5.2 TB/s; residual norm's gradients for 16384 rows of 2560
// with a scale 163 us, 5.6 TB/s; four decoded rows of 2560 4.3 us on the GPU, 12 us with the
// launch and the binding.  Gradients by width, 42 million channels in all, gated and residual
// with a scale, TB/s: 768 channels 5.0 and 4.3, 1024 5.0 and 5.1, 2560 5.3 and 5.6, 4096 4.8 and
// 5.0, 5120 4.5 and 4.2, 8192 4.7 and 4.6; of scratch, 12288 1.1 and 1.5, 16384 1.3 and 1.5,
// 32768 0.5 and 0.5.
#include "ssd.h"

#include <algorithm>
#include <cstdio>

#include "block_common.hpp"
#include "block_host.hpp"

namespace ssd {

struct NormParams {
    const void *x, *z;               // z: the gate, or the residual stream (fp32)
    const float *w, *scale;
    void* out;
    float* res;                      // the residual stream after the addition
    const float *dout, *dstream;
    float *dx, *dz;                  // dz: of the gate, or of the residual
    float *part, *part_scale;        // teams' sums of dw and dscale, rows of part_stride
    int64_t part_stride;
    int64_t rows, D, ldx, ldz;
    int size, groups;                // channels per group, groups per row
    int64_t slots;                   // teams per group (backward)
    float eps;
    int stream;                      // outputs stored past the caches
};

constexpr int kV = 4;                // channels per pack

// Lanes of a team: TEAM of them (several teams in a workgroup of 256 when that is less), or,
// TEAM 0, a whole workgroup of as many waves as the row needs.
template <int TEAM> __device__ inline int team_lanes() { return TEAM ? TEAM : (int)blockDim.x; }
template <int TEAM> __device__ inline int team_lane() { return TEAM ? threadIdx.x % (TEAM ? TEAM : 1) : threadIdx.x; }
template <int TEAM> __device__ inline unsigned team_index() {
    return TEAM ? blockIdx.x * (256 / (TEAM ? TEAM : 1)) + threadIdx.x / (TEAM ? TEAM : 1) : blockIdx.x;
}

// Sum over the lanes of a team, in every lane.  The waves of a workgroup-sized team meet in
// `red`; two sums in turn need one buffer each (between two uses of a buffer lies the
// other sum's barrier).
template <int TEAM> __device__ inline float team_sum(float v, float (&red)[16]) {
    v = lane_team_sum<(TEAM == 0 || TEAM > 64 ? 64 : TEAM)>(v);
    if constexpr (TEAM == 0 || TEAM > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        const int w = threadIdx.x & 15;
        v = lane_team_sum<16>(w < (int)blockDim.x / 64 ? red[w] : 0.f);
    }
    return v;
}

// Pack c of the team lane: channels 4 (c lanes + lane) .. +3 of the group, of which
// `n` exist.  Whole packs load in one piece, the last of an odd group one by one.
template <typename T> __device__ inline void load_part(const T* p, int n, float (&v)[kV]) {
    if (n >= kV) {
        load_f32<kV>(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = i < n ? (float)p[i] : 0.f;
    }
}
template <bool STREAM = false, typename T> __device__ inline void store_part(T* p, int n, const float (&v)[kV]) {
    if (n >= kV) {
        store_f32<kV, STREAM>(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (i < n) p[i] = (T)v[i];
    }
}

enum { kGateFirst = 0, kGateAfter = 1, kResidual = 2 };
// One row (of a group) per team: rows in flight hide each other's latency.
template <typename TX, typename TO, int MODE, int TEAM, int CH, bool STREAM>
__device__ inline void norm_forward(const NormParams& p) {
    __shared__ float red[16];
    const int lane = team_lane<TEAM>(), lanes = team_lanes<TEAM>();
    const unsigned unit = team_index<TEAM>();
    if (TEAM && TEAM < 256 && unit >= p.rows * p.groups) return;
    const int64_t row = unit / (unsigned)p.groups, c0 = (int64_t)(unit % (unsigned)p.groups) * p.size;
    float u[CH][kV], gate[CH][kV];
    float sq = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = (c * lanes + lane) * kV, n = p.size - i;
        if (n <= 0) continue;
        load_part((const TX*)p.x + row * p.ldx + c0 + i, n, u[c]);
        if constexpr (MODE == kResidual) {
            if (p.z) load_part((const float*)p.z + row * p.ldz + i, n, gate[c]);
        } else {
            load_part((const TO*)p.z + row * p.ldz + c0 + i, n, gate[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = (c * lanes + lane) * kV, n = p.size - i;
        if (n <= 0) continue;
        if constexpr (MODE == kResidual) {
            if (p.scale) {
                float g[kV];
                load_part(p.scale + i, n, g);
#pragma unroll
                for (int v = 0; v < kV; ++v) u[c][v] *= g[v];
            }
            if (p.z) {
#pragma unroll
                for (int v = 0; v < kV; ++v) u[c][v] += gate[c][v];
            }
            store_part<STREAM>(p.res + row * p.D + i, n, u[c]);
        } else {
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                gate[c][v] = silu_for<TO>(gate[c][v]);
                if (MODE == kGateFirst) u[c][v] *= gate[c][v];
            }
        }
#pragma unroll
        for (int v = 0; v < kV; ++v)
            if (v < n) sq = fmaf(u[c][v], u[c][v], sq);
    }
    const float r = 1.f / sqrtf(team_sum<TEAM>(sq, red) / (float)p.size + p.eps);
    TO* out = (TO*)p.out + row * p.D + c0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = (c * lanes + lane) * kV, n = p.size - i;
        if (n <= 0) continue;
        float w[kV], o[kV];
        load_part(p.w + c0 + i, n, w);
#pragma unroll
        for (int v = 0; v < kV; ++v) o[v] = u[c][v] * r * w[v] * (MODE == kGateAfter ? gate[c][v] : 1.f);
        store_part<STREAM>(out + i, n, o);
    }
}

template <typename TX, typename TO, int MODE, int TEAM, int CH>
__global__ __launch_bounds__(TEAM ? 256 : 1024) void norm_forward_kernel(NormParams p) {
    if (p.stream) norm_forward<TX, TO, MODE, TEAM, CH, true>(p);
    else norm_forward<TX, TO, MODE, TEAM, CH, false>(p);
}

// Waves per SIMD that the backward is built for; teams are launched to fill them, and walk
// the rows.  A pack takes about 45 registers, so four waves (128 registers) hold two of them;
// the teams of more packs, 16 waves of one workgroup, can have no more registers than that.
constexpr int backward_waves(int team, int ch) { return ch <= 1 ? 5 : (ch <= 2 || team == 0 ? 4 : (ch <= 3 ? 3 : 2)); }

template <typename TX, typename TO, int MODE, int TEAM, int CH, bool STREAM>
__device__ inline void norm_backward(const NormParams& p) {
    __shared__ float red[2][16];
    const int lane = team_lane<TEAM>(), lanes = team_lanes<TEAM>();
    const unsigned team = team_index<TEAM>();
    if (TEAM && team >= p.slots * p.groups) return;
    const int64_t slot = team / (unsigned)p.groups, c0 = (int64_t)(team % (unsigned)p.groups) * p.size;
    // w and the scale once: a load of them in the loop would wait for the next row's loads before it
    float w[CH][kV], g[CH][kV], dw[CH][kV], ds[CH][kV];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = (c * lanes + lane) * kV, n = p.size - i;
        if (n > 0) load_part(p.w + c0 + i, n, w[c]);
        if (MODE == kResidual && p.scale && n > 0) load_part(p.scale + i, n, g[c]);
#pragma unroll
        for (int v = 0; v < kV; ++v) dw[c][v] = ds[c][v] = 0.f;
    }
    // u (residual: the saved stream), e = dL/d(u r w); the gate (residual: dL/dstream) in z
    float nu[CH][kV], ne[CH][kV], nz[CH][kV], nx[CH][kV];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = (c * lanes + lane) * kV, n = p.size - i;
            if (n <= 0) continue;
            load_part(p.dout + row * p.D + c0 + i, n, ne[c]);
            if constexpr (MODE == kResidual) {
                load_part(p.res + row * p.D + i, n, nu[c]);
                if (p.dstream) load_part(p.dstream + row * p.D + i, n, nz[c]);
                if (p.scale) load_part((const TX*)p.x + row * p.ldx + i, n, nx[c]);
            } else {
                load_part((const TX*)p.x + row * p.ldx + c0 + i, n, nx[c]);
                load_part((const TO*)p.z + row * p.ldz + c0 + i, n, nz[c]);
            }
        }
    };
    if (slot < p.rows) fetch(slot);
    for (int64_t row = slot; row < p.rows; row += p.slots) {
        float u[CH][kV], e[CH][kV], z[CH][kV], x[CH][kV];
        float sq = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                u[c][v] = nu[c][v];
                e[c][v] = ne[c][v];
                z[c][v] = nz[c][v];
                x[c][v] = nx[c][v];
            }
        // the next row's loads are in flight while this one is worked on
        if (row + p.slots < p.rows) fetch(row + p.slots);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int n = p.size - (c * lanes + lane) * kV;
            if (n <= 0) continue;
            if constexpr (MODE != kResidual) {
#pragma unroll
                for (int v = 0; v < kV; ++v) u[c][v] = MODE == kGateFirst ? x[c][v] * silu(z[c][v]) : x[c][v];
            }
#pragma unroll
            for (int v = 0; v < kV; ++v)
                if (v < n) sq = fmaf(u[c][v], u[c][v], sq);
        }
        const float r = 1.f / sqrtf(team_sum<TEAM>(sq, red[0]) / (float)p.size + p.eps);
        float dot = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int n = p.size - (c * lanes + lane) * kV;
            if (n <= 0) continue;
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                if (v >= n) continue;
                const float hat = u[c][v] * r;
                if constexpr (MODE == kGateAfter) {
                    const float s = sigmoid(z[c][v]), d = e[c][v];
                    e[c][v] = d * z[c][v] * s;
                    z[c][v] = d * hat * w[c][v] * silu_slope(z[c][v], s);       // dz
                }
                dw[c][v] = fmaf(e[c][v], hat, dw[c][v]);
                e[c][v] *= w[c][v];
                dot = fmaf(e[c][v], hat, dot);
            }
        }
        dot = team_sum<TEAM>(dot, red[1]) / (float)p.size;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = (c * lanes + lane) * kV, n = p.size - i;
            if (n <= 0) continue;
            float du[kV];
#pragma unroll
            for (int v = 0; v < kV; ++v) du[v] = r * (e[c][v] - u[c][v] * r * dot);
            if constexpr (MODE == kResidual) {
                if (p.dstream) {
#pragma unroll
                    for (int v = 0; v < kV; ++v) du[v] += z[c][v];
                }
                store_part<STREAM>(p.dz + row * p.D + i, n, du);
                if (p.scale) {
#pragma unroll
                    for (int v = 0; v < kV; ++v) {
                        ds[c][v] = fmaf(du[v], x[c][v], ds[c][v]);
                        du[v] *= g[c][v];
                    }
                    store_part<STREAM>(p.dx + row * p.D + i, n, du);
                }
            } else {
                if constexpr (MODE == kGateFirst) {
                    float dz[kV];
#pragma unroll
                    for (int v = 0; v < kV; ++v) {
                        const float s = sigmoid(z[c][v]);
                        dz[v] = du[v] * x[c][v] * silu_slope(z[c][v], s);
                        du[v] *= z[c][v] * s;
                    }
                    store_part<STREAM>(p.dz + row * p.D + c0 + i, n, dz);
                } else {
                    store_part<STREAM>(p.dz + row * p.D + c0 + i, n, z[c]);
                }
                store_part<STREAM>(p.dx + row * p.D + c0 + i, n, du);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = (c * lanes + lane) * kV, n = p.size - i;
        if (n <= 0) continue;
        store_part(p.part + slot * p.part_stride + c0 + i, n, dw[c]);
        if (MODE == kResidual && p.scale) store_part(p.part_scale + slot * p.part_stride + c0 + i, n, ds[c]);
    }
}

template <typename TX, typename TO, int MODE, int TEAM, int CH>
__global__ __launch_bounds__(TEAM ? 256 : 1024, backward_waves(TEAM, CH)) void norm_backward_kernel(NormParams p) {
    if (p.stream) norm_backward<TX, TO, MODE, TEAM, CH, true>(p);
    else norm_backward<TX, TO, MODE, TEAM, CH, false>(p);
}

// Lanes per team and packs per lane for a group of `size` channels: a wave or less up to
// 1024 channels, which needs no barrier.  Above, forward, four waves with up to eight packs
// a lane (5120 channels in four waves of five packs: 150 us for 16384 rows of the gated norm,
// in ten waves of two 192, in ten persistent waves with the next row's loads ahead 175);
// backward, just enough waves with one or two packs (2560 channels in ten waves of one pack:
// 174 us for the residual norm's 16384 rows, in five waves of two 297).  Past 8192 channels
// 16 waves with more packs.
struct Team {
    int team, lanes, ch;
};
static Team team_of(int64_t size, bool backward) {
    for (int lanes = 8; lanes <= 32; lanes *= 2)
        if (size <= 4 * lanes) return {lanes, lanes, 1};
    if (size <= 1024) return {64, 64, (int)((size + 255) / 256)};
    if (size > 8192) return {0, 1024, size <= 16384 ? 4 : 8};
    if (!backward) return {256, 256, (int)((size + 1023) / 1024)};
    const int ch = size <= 4096 ? 1 : 2;
    return {0, (int)((size + 256 * ch - 1) / (256 * ch)) * 64, ch};
}
// Teams per group in the backward: as many as stay on the chip together, but at least 8
// rows each, so that the partial sums stay small beside the rows.  (What adding them takes is
// not counted: see column_sums_kernel for narrow rows.)
static int64_t slots_of(int64_t size, int64_t groups, int64_t rows) {
    const Team t = team_of(size, true);
    const int64_t waves = backward_waves(t.team, t.ch);
    const int64_t teams = t.team ? 1024 * 64 * waves / t.lanes : 256 * std::max<int64_t>(1, 4 * waves / (t.lanes / 64));
    return std::max<int64_t>(1, std::min((teams + groups - 1) / groups, (rows + 7) / 8));
}

template <typename TX, typename TO, int MODE, int TEAM, int CH>
static void launch_one(bool backward, const NormParams& p, int lanes, hipStream_t s) {
    const int64_t units = (backward ? p.slots : p.rows) * p.groups, per = TEAM ? 256 / (TEAM ? TEAM : 1) : 1;
    const dim3 grid((unsigned)((units + per - 1) / per)), block(TEAM ? 256 : lanes);
    if (backward) {
        if constexpr (TEAM < 256) hipLaunchKernelGGL((norm_backward_kernel<TX, TO, MODE, TEAM, CH>), grid, block, 0, s, p);
    } else if constexpr (TEAM != 0 || CH > 2) {
        hipLaunchKernelGGL((norm_forward_kernel<TX, TO, MODE, TEAM, CH>), grid, block, 0, s, p);
    }
}
template <typename TX, typename TO, int MODE> static hipError_t launch_norm(bool backward, const NormParams& p, hipStream_t s) {
    const Team t = team_of(p.size, backward);
#define SSD_NORM_CASE(L, C) \
    if (t.team == L && t.ch == C) launch_one<TX, TO, MODE, L, C>(backward, p, t.lanes, s);
    SSD_NORM_CASE(8, 1) SSD_NORM_CASE(16, 1) SSD_NORM_CASE(32, 1)
    SSD_NORM_CASE(64, 1) SSD_NORM_CASE(64, 2) SSD_NORM_CASE(64, 3) SSD_NORM_CASE(64, 4)
    SSD_NORM_CASE(256, 2) SSD_NORM_CASE(256, 3) SSD_NORM_CASE(256, 4) SSD_NORM_CASE(256, 5) SSD_NORM_CASE(256, 6)
    SSD_NORM_CASE(256, 7) SSD_NORM_CASE(256, 8)
    SSD_NORM_CASE(0, 1) SSD_NORM_CASE(0, 2) SSD_NORM_CASE(0, 4) SSD_NORM_CASE(0, 8)
#undef SSD_NORM_CASE
    return hipGetLastError();
}

}  // namespace ssd

namespace {

using namespace ssd_host;

constexpr int64_t kMaxDim = int64_t(1) << 31;
constexpr int64_t kMaxGroup = 32768;

int validate(const ssd_norm_problem_t* p, bool gated) {
    if (!p) return SSD_ERR_NULL_POINTER;
    if (p->rows < 0 || p->channels <= 0 || p->group_size <= 0 || p->channels % p->group_size != 0 ||
        p->ldx < p->channels || p->ldz < p->channels)
        return SSD_ERR_BAD_SHAPE;
    if (p->rows >= kMaxDim || p->channels >= kMaxDim || p->ldx >= kMaxDim || p->ldz >= kMaxDim) return SSD_ERR_BAD_SHAPE;
    if (!(p->eps >= 0.f) || p->eps > 1e30f) return SSD_ERR_BAD_SHAPE;
    if ((p->dtype != SSD_DTYPE_BF16 && p->dtype != SSD_DTYPE_F32) ||
        (p->x_dtype != SSD_DTYPE_BF16 && p->x_dtype != SSD_DTYPE_F32))
        return SSD_ERR_UNSUPPORTED;
    if (p->reserved != 0 || p->group_size > kMaxGroup) return SSD_ERR_UNSUPPORTED;
    if (gated) {
        if (p->flags & ~uint32_t(SSD_NORM_GATE_FIRST)) return SSD_ERR_UNSUPPORTED;
        if (p->x_dtype == SSD_DTYPE_BF16 && p->dtype == SSD_DTYPE_F32) return SSD_ERR_UNSUPPORTED;
    } else {
        if (p->flags != 0 || p->x_dtype != p->dtype || p->group_size != p->channels) return SSD_ERR_UNSUPPORTED;
    }
    // a launch holds fewer than 2^32 lanes
    if (double(std::max<int64_t>(1, p->rows)) * (p->channels / p->group_size) * ssd::team_of(p->group_size, false).lanes >= 4e9)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

int64_t slots_of(const ssd_norm_problem_t* p) {
    return ssd::slots_of(p->group_size, p->channels / p->group_size, p->rows);
}
// A single team per group writes dw and dscale themselves.
int64_t backward_bytes(const ssd_norm_problem_t* p, bool scaled) {
    return p->rows == 0 || slots_of(p) == 1 ? 0 : align256(slots_of(p) * p->channels * 4 * (scaled ? 2 : 1));
}

int64_t span(int64_t rows, int64_t ld, int64_t cols, int64_t e) { return rows > 0 ? ((rows - 1) * ld + cols) * e : 0; }

// out_size: bytes of an element of the largest output.
ssd::NormParams params_of(const ssd_norm_problem_t* p, int64_t out_size) {
    ssd::NormParams n{};
    n.rows = p->rows;
    n.D = p->channels;
    n.ldx = p->ldx;
    n.ldz = p->ldz;
    n.size = (int)p->group_size;
    n.groups = (int)(p->channels / p->group_size);
    n.eps = p->eps;
    n.stream = p->rows * p->channels * out_size > ssd::kStreamBytes;
    return n;
}

hipError_t run_gated(const ssd_norm_problem_t* p, bool backward, const ssd::NormParams& n, hipStream_t s) {
    const bool first = (p->flags & SSD_NORM_GATE_FIRST) != 0;
    if (p->dtype == SSD_DTYPE_F32)
        return first ? ssd::launch_norm<float, float, ssd::kGateFirst>(backward, n, s)
                     : ssd::launch_norm<float, float, ssd::kGateAfter>(backward, n, s);
    if (p->x_dtype == SSD_DTYPE_F32)
        return first ? ssd::launch_norm<float, __bf16, ssd::kGateFirst>(backward, n, s)
                     : ssd::launch_norm<float, __bf16, ssd::kGateAfter>(backward, n, s);
    return first ? ssd::launch_norm<__bf16, __bf16, ssd::kGateFirst>(backward, n, s)
                 : ssd::launch_norm<__bf16, __bf16, ssd::kGateAfter>(backward, n, s);
}
hipError_t run_residual(const ssd_norm_problem_t* p, bool backward, const ssd::NormParams& n, hipStream_t s) {
    return p->dtype == SSD_DTYPE_BF16 ? ssd::launch_norm<__bf16, __bf16, ssd::kResidual>(backward, n, s)
                                      : ssd::launch_norm<float, float, ssd::kResidual>(backward, n, s);
}

int done(const char* what, const ssd_norm_problem_t* p, hipError_t e) {
    if (log_enabled())
        std::fprintf(stderr, "[ssd] %s dtype=%d rows=%lld channels=%lld group=%lld -> %s\n", what, p->dtype,
                     (long long)p->rows, (long long)p->channels, (long long)p->group_size, hipGetErrorString(e));
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

// Where the teams' sums go, and their sums over teams.
void place_sums(const ssd_norm_problem_t* p, ssd::NormParams* n, float* dweight, float* dscale, void* workspace) {
    n->slots = slots_of(p);
    const bool direct = n->slots == 1;
    n->part = direct ? dweight : static_cast<float*>(workspace);
    n->part_scale = direct ? dscale : n->part + p->channels;
    n->part_stride = p->channels * (dscale ? 2 : 1);
}
hipError_t finish(const ssd_norm_problem_t* p, const ssd::NormParams& n, float* dweight, float* dscale, hipStream_t s) {
    if (n.slots == 1) return hipSuccess;
    ssd::ColumnSums c{};
    c.part = n.part;
    c.out = dweight;
    c.out2 = dscale;
    c.split = p->channels;
    c.rows = n.slots;
    c.cols = c.split2 = n.part_stride;
    return ssd::launch_column_sums(c, s);
}

}  // namespace

extern "C" {

int ssd_gated_norm_forward(const ssd_norm_problem_t* p, const void* x, const void* z, const float* weight, void* out,
                           void* stream) {
    const int v = validate(p, true);
    if (v != SSD_OK) return v;
    if (!weight || (p->rows > 0 && (!x || !z || !out))) return SSD_ERR_NULL_POINTER;
    const int64_t ex = elem_size(p->x_dtype), e = elem_size(p->dtype), cb = p->channels * 4;
    if (misaligned(x, ex) || misaligned(z, e) || misaligned(out, e) || misaligned(weight, 4)) return SSD_ERR_ALIGNMENT;
    const Buf ins[] = {{x, span(p->rows, p->ldx, p->channels, ex)}, {z, span(p->rows, p->ldz, p->channels, e)}, {weight, cb}};
    const Buf outs[] = {{out, p->rows * p->channels * e}};
    const int a = check_alias(ins, 3, outs, 1);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    if (p->rows == 0) return SSD_OK;
    ssd::NormParams n = params_of(p, e);
    n.x = x;
    n.z = z;
    n.w = weight;
    n.out = out;
    return done("gated norm", p, run_gated(p, false, n, static_cast<hipStream_t>(stream)));
}

size_t ssd_gated_norm_backward_workspace_size(const ssd_norm_problem_t* p) {
    return validate(p, true) == SSD_OK ? (size_t)backward_bytes(p, false) : 0;
}

int ssd_gated_norm_backward(const ssd_norm_problem_t* p, const void* x, const void* z, const float* weight,
                            const float* dout, float* dx, float* dz, float* dweight, void* workspace,
                            size_t workspace_bytes, void* stream) {
    const int v = validate(p, true);
    if (v != SSD_OK) return v;
    if (!weight || !dweight || (p->rows > 0 && (!x || !z || !dout || !dx || !dz))) return SSD_ERR_NULL_POINTER;
    const int64_t wsb = backward_bytes(p, false);
    if (wsb > 0 && !workspace) return SSD_ERR_WORKSPACE;
    const int64_t ex = elem_size(p->x_dtype), e = elem_size(p->dtype), cb = p->channels * 4, f = p->rows * cb;
    if (misaligned(x, ex) || misaligned(z, e) || misaligned(weight, 4) || misaligned(dout, 4) || misaligned(dx, 4) ||
        misaligned(dz, 4) || misaligned(dweight, 4) || misaligned(workspace, 256))
        return SSD_ERR_ALIGNMENT;
    if ((int64_t)workspace_bytes < wsb) return SSD_ERR_WORKSPACE;
    const Buf ins[] = {{x, span(p->rows, p->ldx, p->channels, ex)}, {z, span(p->rows, p->ldz, p->channels, e)}, {weight, cb}, {dout, f}};
    const Buf outs[] = {{dx, f}, {dz, f}, {dweight, cb}, {workspace, wsb}};
    const int a = check_alias(ins, 4, outs, 4);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (p->rows == 0) return done("gated norm backward", p, ssd::launch_fill(dweight, p->channels, s));
    ssd::NormParams n = params_of(p, 4);
    n.x = x;
    n.z = z;
    n.w = weight;
    n.dout = dout;
    n.dx = dx;
    n.dz = dz;
    place_sums(p, &n, dweight, nullptr, workspace);
    hipError_t r = run_gated(p, true, n, s);
    if (r == hipSuccess) r = finish(p, n, dweight, nullptr, s);
    return done("gated norm backward", p, r);
}

int ssd_residual_norm_forward(const ssd_norm_problem_t* p, const void* x, const float* residual, const float* weight,
                              const float* scale, void* out, float* residual_out, void* stream) {
    const int v = validate(p, false);
    if (v != SSD_OK) return v;
    if (!weight || (p->rows > 0 && (!x || !out || !residual_out))) return SSD_ERR_NULL_POINTER;
    const int64_t e = elem_size(p->dtype), cb = p->channels * 4, f = p->rows * cb;
    if (misaligned(x, e) || misaligned(out, e) || misaligned(residual, 4) || misaligned(weight, 4) ||
        misaligned(scale, 4) || misaligned(residual_out, 4))
        return SSD_ERR_ALIGNMENT;
    // the stream may be updated in place: a lane reads its channels before it writes them
    const bool in_place = residual == residual_out && p->ldz == p->channels;
    const Buf ins[] = {{x, span(p->rows, p->ldx, p->channels, e)}, {weight, cb}, {scale, cb},
                       {in_place ? nullptr : residual, span(p->rows, p->ldz, p->channels, 4)}};
    const Buf outs[] = {{out, p->rows * p->channels * e}, {residual_out, f}};
    const int a = check_alias(ins, 4, outs, 2);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    if (p->rows == 0) return SSD_OK;
    ssd::NormParams n = params_of(p, 4);
    n.x = x;
    n.z = residual;
    n.w = weight;
    n.scale = scale;
    n.out = out;
    n.res = residual_out;
    return done("residual norm", p, run_residual(p, false, n, static_cast<hipStream_t>(stream)));
}

size_t ssd_residual_norm_backward_workspace_size(const ssd_norm_problem_t* p, int scaled) {
    return validate(p, false) == SSD_OK ? (size_t)backward_bytes(p, scaled != 0) : 0;
}

int ssd_residual_norm_backward(const ssd_norm_problem_t* p, const void* x, const float* residual_out,
                               const float* weight, const float* scale, const float* dout, const float* dresidual_out,
                               float* dx, float* dresidual, float* dweight, float* dscale, void* workspace,
                               size_t workspace_bytes, void* stream) {
    const int v = validate(p, false);
    if (v != SSD_OK) return v;
    if (!weight || !dweight || (scale && !dscale) ||
        (p->rows > 0 && (!residual_out || !dout || !dresidual || (scale && (!x || !dx)))))
        return SSD_ERR_NULL_POINTER;
    const int64_t wsb = backward_bytes(p, scale != nullptr);
    if (wsb > 0 && !workspace) return SSD_ERR_WORKSPACE;
    const int64_t e = elem_size(p->dtype), cb = p->channels * 4, f = p->rows * cb;
    if (misaligned(x, e) || misaligned(residual_out, 4) || misaligned(weight, 4) || misaligned(scale, 4) ||
        misaligned(dout, 4) || misaligned(dresidual_out, 4) || misaligned(dx, 4) || misaligned(dresidual, 4) ||
        misaligned(dweight, 4) || misaligned(dscale, 4) || misaligned(workspace, 256))
        return SSD_ERR_ALIGNMENT;
    if ((int64_t)workspace_bytes < wsb) return SSD_ERR_WORKSPACE;
    const Buf ins[] = {{scale ? x : nullptr, span(p->rows, p->ldx, p->channels, e)}, {residual_out, f}, {weight, cb}, {scale, cb}, {dout, f}, {dresidual_out, f}};
    const Buf outs[] = {{scale ? dx : nullptr, f}, {dresidual, f}, {dweight, cb}, {scale ? dscale : nullptr, cb}, {workspace, wsb}};
    const int a = check_alias(ins, 6, outs, 5);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (p->rows == 0) {
        hipError_t r = ssd::launch_fill(dweight, p->channels, s);
        if (r == hipSuccess && scale) r = ssd::launch_fill(dscale, p->channels, s);
        return done("residual norm backward", p, r);
    }
    ssd::NormParams n = params_of(p, 4);
    n.x = x;
    n.w = weight;
    n.scale = scale;
    n.res = const_cast<float*>(residual_out);
    n.dout = dout;
    n.dstream = dresidual_out;
    n.dx = dx;
    n.dz = dresidual;
    place_sums(p, &n, dweight, scale ? dscale : nullptr, workspace);
    hipError_t r = run_residual(p, true, n, s);
    if (r == hipSuccess) r = finish(p, n, dweight, scale ? dscale : nullptr, s);
    return done("residual norm backward", p, r);
}

}  // extern "C"
