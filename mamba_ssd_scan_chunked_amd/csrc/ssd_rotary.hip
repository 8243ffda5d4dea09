// Root-mean-square norm of B and C per head with the rotation by position, and its
// gradients.  C entries of include/ssd.h.
//
//   v = u r w,  r = 1 / sqrt(mean(u^2) + eps);   (p, q) -> (p cos - q sin, p sin + q cos).
// Gradients: e = the rotation's transpose of dout;  hat = u r;
//   du = r (e w - hat mean(e w hat)),   dw = sum over tokens and heads of e hat.
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
    float* part;                     // (teams, 2, N) sums of dw
    int64_t tokens, seqlen, ld[2];
    int heads[2];
    int N, R;
    float eps;
    int interleaved;
};

// cos and sin of position times freq.  The angle, in revolutions, is formed in fp64 (31 bits of
// position times 24 of freq leave 2^-22 of a radian at the far end) and reduced to half a
// revolution before it is rounded to fp32.
__device__ inline void turn_of(int64_t position, float freq, float* c, float* s) {
    const double rev = (double)position * ((double)freq * 0.15915494309189535);
    sincospif(2.f * (float)(rev - rint(rev)), s, c);
}

// A wave per (token, head): lane l holds pairs l, l + 64, ... and the channels behind them.
template <typename T, bool BACK> __global__ __launch_bounds__(64) void rotary_kernel(RotaryParams p) {
    const int lane = threadIdx.x, all = p.heads[0] + p.heads[1];
    float* dw = p.part ? p.part + (int64_t)blockIdx.x * 2 * p.N : nullptr;
    if constexpr (BACK)
        for (int c = lane; c < 2 * p.N; c += 64) dw[c] = 0.f;
    for (int64_t unit = blockIdx.x; unit < p.tokens * all; unit += gridDim.x) {
        const int64_t t = unit / all;
        int head = (int)(unit % all);
        const int k = head >= p.heads[0];
        if (k) head -= p.heads[0];
        const T* u = (const T*)p.u[k] + t * p.ld[k] + (int64_t)head * p.N;
        const int64_t o = (t * p.heads[k] + head) * p.N;
        const int64_t position = p.positions ? p.positions[t] : t % p.seqlen;
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
                        dw[k * p.N + c] += e * h;
                        if (pair) dw[k * p.N + c2] += e2 * h2;
                    } else {
                        p.du[k][o + c] = r * (e * w - h * dot);
                        if (pair) p.du[k][o + c2] = r * (e2 * w2 - h2 * dot);
                    }
                }
            }
        }
    }
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
    return SSD_OK;
}

int64_t teams_of(const ssd_rotary_problem_t* p) {
    return std::min<int64_t>(4096, p->tokens * (p->b_heads + p->c_heads));
}
int64_t backward_bytes(const ssd_rotary_problem_t* p) { return align256(teams_of(p) * 2 * p->headdim * 4); }

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
                            const float* cw, const float* freqs, const int32_t* positions) {
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
    ssd::RotaryParams r = params_of(p, B, C, b_weight, c_weight, freqs, positions);
    r.out[0] = B_out;
    r.out[1] = C_out;
    const dim3 grid((unsigned)teams_of(p));
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (p->dtype == SSD_DTYPE_BF16) hipLaunchKernelGGL((ssd::rotary_kernel<__bf16, false>), grid, dim3(64), 0, st, r);
    else hipLaunchKernelGGL((ssd::rotary_kernel<float, false>), grid, dim3(64), 0, st, r);
    return done("forward", p, hipGetLastError());
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
    ssd::RotaryParams r = params_of(p, B, C, b_weight, c_weight, freqs, positions);
    r.dout[0] = dB_out;
    r.dout[1] = dC_out;
    r.du[0] = dB;
    r.du[1] = dC;
    r.part = static_cast<float*>(workspace);
    const dim3 grid((unsigned)teams_of(p));
    if (p->dtype == SSD_DTYPE_BF16) hipLaunchKernelGGL((ssd::rotary_kernel<__bf16, true>), grid, dim3(64), 0, st, r);
    else hipLaunchKernelGGL((ssd::rotary_kernel<float, true>), grid, dim3(64), 0, st, r);
    hipError_t q = hipGetLastError();
    if (q == hipSuccess) {
        ssd::ColumnSums cs{};
        cs.part = r.part;
        cs.out = db_weight;
        cs.out2 = dc_weight;
        cs.split = p->headdim;
        cs.rows = teams_of(p);
        cs.cols = cs.split2 = 2 * p->headdim;
        q = ssd::launch_column_sums(cs, st);
    }
    return done("backward", p, q);
}

}  // extern "C"
