// The gated linear recurrence: whole sequences, their gradients, and the single-token step.
// C entries of include/ssd.h.
//
//   s = sigmoid(r),  L = A s,  a = e^L,  m = 1 - a,  beta = sqrt(1 - a^2) = sqrt(m (2 - m)),
//   h_t = h_{t-1} - m h_{t-1} + beta sigmoid(i) x,      y = h  or  h silu(z).
#include "ssd.h"

#include <algorithm>
#include <cstdio>

#include "block_common.hpp"
#include "block_host.hpp"

namespace ssd {

struct RecurrenceParams {
    const void *x, *r, *i, *z;
    const float *A_log, *init;
    const int32_t* seq_idx;
    void* y;
    float* fin;
    const float *dy, *dfin;
    float *dx, *dr, *di, *dz, *dinit;
    float *part, *states;
    int64_t batch, T, D, nseqs, ldx, ldr, ldi, ldz;
};

// -exp(A_log), kept finite so that A times a gate of 0 is 0.
__device__ inline float rate_of(float a_log) { return -fminf(expf(a_log), 1e30f); }

// m = 1 - e^L for L <= 0.  Near 0 the difference would cancel (and a long memory is a matter of
// m, not of a): there m = -L (1 + L/2 + L^2/6 + ...), a polynomial fitted to the definition on
// [-1/4, 0] by interpolation at Chebyshev points (relative error 3e-9).
__device__ inline float one_minus_exp(float L) {
    float q = fmaf(0.007513605989515781f, L, 0.04149065539240837f);
    q = fmaf(q, L, 0.16665108501911163f);
    q = fmaf(q, L, 0.4999995231628418f);
    q = fmaf(q, L, 1.f);
    const float far = 1.f - __builtin_amdgcn_exp2f(L * kLog2e);
    return L > -0.25f ? -L * q : far;
}

struct Decay {
    float s, L, m, beta;
};
__device__ inline Decay decay_of(float r, float A) {
    Decay d;
    d.s = sigmoid(r);
    d.L = A * d.s;
    d.m = one_minus_exp(d.L);
    d.beta = __builtin_amdgcn_sqrtf(d.m * (2.f - d.m));
    return d;
}

template <typename T> __device__ inline float at(const void* p, int64_t i) { return (float)((const T*)p)[i]; }

// A thread per (row, channel) walks the row.
template <typename T> __global__ __launch_bounds__(64) void recurrence_forward_kernel(RecurrenceParams p) {
    const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
    if (c >= p.D) return;
    const float A = rate_of(p.A_log[c]);
    int64_t seq = b;
    float h = 0.f;
    for (int64_t t = 0; t < p.T; ++t) {
        const int64_t n = b * p.T + t;
        bool fresh = t == 0;
        if (p.seq_idx) {
            const int64_t id = clamp_id(p.seq_idx[n], p.nseqs);
            fresh = fresh || id != seq;
            seq = id;
        }
        if (fresh) h = p.init ? p.init[seq * p.D + c] : 0.f;
        const Decay d = decay_of(at<T>(p.r, n * p.ldr + c), A);
        h += fmaf(-d.m, h, d.beta * sigmoid(at<T>(p.i, n * p.ldi + c)) * at<T>(p.x, n * p.ldx + c));
        if (p.states) p.states[n * p.D + c] = h;
        if (p.y) ((T*)p.y)[n * p.D + c] = (T)(p.z ? h * silu(at<T>(p.z, n * p.ldz + c)) : h);
        if (p.fin && (t + 1 == p.T || (p.seq_idx && clamp_id(p.seq_idx[n + 1], p.nseqs) != seq))) p.fin[seq * p.D + c] = h;
    }
}

template <typename T> __global__ __launch_bounds__(64) void recurrence_backward_kernel(RecurrenceParams p) {
    const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
    if (c >= p.D) return;
    const float A = rate_of(p.A_log[c]);
    float q = 0.f, dA = 0.f;
    for (int64_t t = p.T - 1; t >= 0; --t) {
        const int64_t n = b * p.T + t;
        int64_t seq = b;
        bool fresh = t == 0, last = t + 1 == p.T;
        if (p.seq_idx) {
            seq = clamp_id(p.seq_idx[n], p.nseqs);
            fresh = fresh || clamp_id(p.seq_idx[n - 1], p.nseqs) != seq;
            last = last || clamp_id(p.seq_idx[n + 1], p.nseqs) != seq;
        }
        if (last) q = p.dfin ? p.dfin[seq * p.D + c] : 0.f;
        const float before = fresh ? (p.init ? p.init[seq * p.D + c] : 0.f) : p.states[(n - 1) * p.D + c];
        float g = p.dy[n * p.D + c];
        if (p.z) {
            const float z = at<T>(p.z, n * p.ldz + c), s = sigmoid(z);
            p.dz[n * p.D + c] = g * p.states[n * p.D + c] * silu_slope(z, s);
            g *= z * s;
        }
        g += q;
        const Decay d = decay_of(at<T>(p.r, n * p.ldr + c), A);
        const float iv = at<T>(p.i, n * p.ldi + c), si = sigmoid(iv), x = at<T>(p.x, n * p.ldx + c), u = si * x;
        const float a = 1.f - d.m, ratio = d.beta > 0.f ? d.L / d.beta : 0.f;
        const float M = g * (d.L * a * before - u * a * a * ratio);
        p.dx[n * p.D + c] = g * d.beta * si;
        p.di[n * p.D + c] = g * d.beta * u * sigmoid(-iv);
        p.dr[n * p.D + c] = M * sigmoid(-at<T>(p.r, n * p.ldr + c));
        dA += M;
        q = g - d.m * g;
        if (fresh && p.dinit) p.dinit[seq * p.D + c] = q;
    }
    p.part[b * p.D + c] = dA;
}

}  // namespace ssd

namespace {

using namespace ssd_host;

constexpr int64_t kMaxDim = int64_t(1) << 31;

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
    if (p->batch >= 65536) return SSD_ERR_UNSUPPORTED;
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

int64_t forward_bytes(const ssd_recurrence_problem_t*) { return 0; }
int64_t backward_bytes(const ssd_recurrence_problem_t* p) {
    return empty(p) ? 0 : align256(p->batch * p->seqlen * p->channels * 4) + align256(p->batch * p->channels * 4);
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
    return c;
}

int done(const char* what, const ssd_recurrence_problem_t* p, hipError_t e) {
    if (log_enabled())
        std::fprintf(stderr, "[ssd] recurrence %s dtype=%d batch=%lld T=%lld D=%lld -> %s\n", what, p->dtype,
                     (long long)p->batch, (long long)p->seqlen, (long long)p->channels, hipGetErrorString(e));
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

dim3 grid_of(const ssd_recurrence_problem_t* p) { return dim3((unsigned)((p->channels + 63) / 64), (unsigned)p->batch); }

hipError_t run_forward(const ssd_recurrence_problem_t* p, const ssd::RecurrenceParams& c, hipStream_t s) {
    if (p->dtype == SSD_DTYPE_BF16)
        hipLaunchKernelGGL((ssd::recurrence_forward_kernel<__bf16>), grid_of(p), dim3(64), 0, s, c);
    else
        hipLaunchKernelGGL((ssd::recurrence_forward_kernel<float>), grid_of(p), dim3(64), 0, s, c);
    return hipGetLastError();
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
    return done("forward", p, run_forward(p, c, st));
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
    return done("step", p, run_forward(p, c, static_cast<hipStream_t>(stream)));
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
    c.states = static_cast<float*>(workspace);
    e2 = run_forward(p, c, st);
    if (e2 != hipSuccess) return done("backward", p, e2);
    c.dy = dy;
    c.dfin = dfinal;
    c.dx = dx;
    c.dr = dr;
    c.di = di;
    c.dz = dz;
    c.dinit = dinit;
    c.part = c.states + align256(p->batch * p->seqlen * p->channels * 4) / 4;
    // ids that do not occur keep a zero gradient
    if (seq_idx && dinit) e2 = ssd::launch_fill(dinit, n.state / 4, st);
    if (e2 == hipSuccess) {
        if (p->dtype == SSD_DTYPE_BF16)
            hipLaunchKernelGGL((ssd::recurrence_backward_kernel<__bf16>), grid_of(p), dim3(64), 0, st, c);
        else
            hipLaunchKernelGGL((ssd::recurrence_backward_kernel<float>), grid_of(p), dim3(64), 0, st, c);
        e2 = hipGetLastError();
    }
    if (e2 == hipSuccess) {
        ssd::ColumnSums cs{};
        cs.part = c.part;
        cs.out = dA_log;
        cs.rows = p->batch;
        cs.cols = cs.split = cs.split2 = p->channels;
        e2 = ssd::launch_column_sums(cs, st);
    }
    return done("backward", p, e2);
}

}  // extern "C"
