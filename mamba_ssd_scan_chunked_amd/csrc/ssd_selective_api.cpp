// Host side of the selective scan's entry points (declared in include/ssd.h): argument
// checks, the workspace layouts and the launches.  Every check runs before the first HIP
// call.
#include "ssd.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "block_host.hpp"
#include "selective.hpp"

namespace {

using namespace ssd_host;

constexpr int64_t kMaxDim = int64_t(1) << 31;
// Segments are whole tiles of the kernels that walk them.
constexpr int64_t kForwardTile = 32, kBackwardTile = 8;

int64_t blocks_of(const ssd_selective_problem_t* p) { return (p->channels / p->ngroups + 63) / 64; }

// Segments per row.  A row's 64-channel blocks give `items` workgroups' worth of work; a row
// is cut to fill the chip.  Forward, a cut adds the local pass (nearly the scan again): on
// an MI355X (2048 tokens, 16 states, bf16) 10 items take 160 us whole and 38 us in segments
// of 64 tokens, 80 items 158 and 93, 160 items 190 and 158, 240 items 188 and 221; 80 items
// of 512 tokens 44 and 40, 16 items of 300 tokens 30 and 32.  The borders are those of 16
// states; whole and as the rule has it, 2048 tokens: 8 states 80 items 124 and 65, 160 items 145
// and 112, 192 items 146 and 122; 32 states 207 and 157, 277 and 290, 277 and 321; 64 states 321
// and 253, 462 and 496, 462 and 559 (from 160 items on these lose by the cut).  Backward, the local pass is
// needed for its checkpoints anyway and the segments only add to it: 10 items 1356 us whole
// and 69 us in segments of 32 tokens, 80 items 1416 and 279, 320 items 1748 and (12 segments)
// 947, 640 items 2232 and (six) 1780.  Rows stay whole where they alone fill four fifths of
// their rounds of resident workgroups (1024 tokens, whole and in segments: 16 states, of 768
// resident, 1280 items 1684 and 1776 us, 960 items 1493 and 1346; 64 states, of 256, 240
// items 1221 and 1306, 480 items 2228 and 2511, 320 items 2177 and 1628).
struct Segments {
    int64_t n, len;
};
Segments segments_of(const ssd_selective_problem_t* p, bool backward) {
    const int64_t tile = backward ? kBackwardTile : kForwardTile;
    const int64_t tiles = std::max<int64_t>(1, (p->seqlen + tile - 1) / tile);
    const int64_t items = std::max<int64_t>(1, p->batch * p->ngroups * blocks_of(p));
    int64_t n = 1;
    if (p->segments > 0) {
        n = p->segments;
    } else if (backward) {
        // whole rounds of the reverse pass's workgroups, as many as stay on the chip together
        const int64_t resident = p->dstate == 8 ? 1536 : (p->dstate == 16 ? 768 : (p->dstate == 32 ? 512 : 256));
        const double whole = double(items) / double(resident);
        if (whole < 0.8 * std::ceil(whole)) {
            const int64_t rounds = std::max<int64_t>(1, std::min<int64_t>(5, p->seqlen / 32 * items / resident));
            n = std::min(rounds * resident / items, p->seqlen / 32);
        }
    } else if (items <= 192 && p->seqlen >= 512) {
        n = std::min(4096 / items, p->seqlen / 64);
    }
    n = std::max<int64_t>(1, std::min(n, tiles));
    const int64_t per = (tiles + n - 1) / n;
    return {(tiles + per - 1) / per, per * tile};
}

// `step`: for the single token, whose kernel takes each element's offset in 64 bits.
int validate(const ssd_selective_problem_t* p, bool step = false) {
    if (!p) return SSD_ERR_NULL_POINTER;
    if (p->batch < 0 || p->seqlen < 0 || p->channels <= 0 || p->dstate <= 0 || p->ngroups <= 0 || p->nseqs < 0 ||
        p->segments < 0)
        return SSD_ERR_BAD_SHAPE;
    if (p->batch >= kMaxDim || p->seqlen >= kMaxDim || p->channels >= kMaxDim || p->nseqs >= kMaxDim)
        return SSD_ERR_BAD_SHAPE;
    if (p->channels % p->ngroups != 0) return SSD_ERR_BAD_SHAPE;
    if (p->dtype != SSD_DTYPE_BF16 && p->dtype != SSD_DTYPE_F32) return SSD_ERR_UNSUPPORTED;
    if (p->dstate != 8 && p->dstate != 16 && p->dstate != 32 && p->dstate != 64) return SSD_ERR_UNSUPPORTED;
    if ((p->flags & ~uint32_t(SSD_FLAG_DT_SOFTPLUS)) || p->reserved != 0) return SSD_ERR_UNSUPPORTED;
    const int64_t gn = p->ngroups * p->dstate;
    for (int64_t ld : {p->ldx, p->lddt, p->ldz})
        if (ld < p->channels || ld >= kMaxDim) return SSD_ERR_BAD_SHAPE;
    for (int64_t ld : {p->ldb, p->ldc})
        if (ld < gn || ld >= kMaxDim) return SSD_ERR_BAD_SHAPE;
    // a tile is addressed with 32-bit byte offsets
    const int64_t widest = std::max({p->ldx, p->lddt, p->ldz, p->ldb, p->ldc, p->channels});
    if ((step ? p->channels : widest) >= int64_t(1) << 25) return SSD_ERR_UNSUPPORTED;
    // sizes stay far from int64 overflow, and every launch below 2^32 threads
    const double tokens = double(p->batch) * double(p->seqlen), states = double(p->channels) * p->dstate;
    if (tokens * states > 1e17 || tokens * double(widest) > 4e17 || double(p->nseqs) * states > 1e17 ||
        tokens * gn * double(blocks_of(p)) > 1e17)
        return SSD_ERR_BAD_SHAPE;
    const double items = double(p->batch) * double(p->ngroups) * double(blocks_of(p));
    const double most = std::max(segments_of(p, false).n, segments_of(p, true).n);
    if (items * most * 512 >= 4e9 || double(p->batch) * states >= 4e9 || tokens * gn / 4 >= 4e9)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

struct SelSizes {
    int64_t x, dt, z, b, c, y, f, a, d, state, seq, bc;
};
SelSizes sel_sizes(const ssd_selective_problem_t* p) {
    SelSizes s;
    const int64_t bt = p->batch * p->seqlen, e = elem_size(p->dtype), gn = p->ngroups * p->dstate;
    auto span = [&](int64_t ld, int64_t cols) { return bt > 0 ? ((bt - 1) * ld + cols) * e : 0; };
    s.x = span(p->ldx, p->channels);
    s.dt = span(p->lddt, p->channels);
    s.z = span(p->ldz, p->channels);
    s.b = span(p->ldb, gn);
    s.c = span(p->ldc, gn);
    s.y = bt * p->channels * e;
    s.f = bt * p->channels * 4;
    s.bc = bt * gn * 4;
    s.a = p->channels * p->dstate * 4;
    s.d = p->channels * 4;
    s.state = p->nseqs * s.a;
    s.seq = bt * 4;
    return s;
}

// Regions of the workspaces, in bytes from their start.
struct ForwardSpace {
    int64_t step, total;             // seg_state at 0
};
ForwardSpace forward_space(const ssd_selective_problem_t* p) {
    const int64_t n = p->batch * (segments_of(p, false).n - 1) * p->channels;
    ForwardSpace w;
    w.step = align256(n * p->dstate * 4);
    w.total = n > 0 && p->seqlen > 0 ? w.step + align256(n * 4) : 0;
    return w;
}
struct BackwardSpace {
    int64_t step, grad, ckpt, ckpt_step, part_b, part_c, sums, total;
};
BackwardSpace backward_space(const ssd_selective_problem_t* p) {
    BackwardSpace w{};
    if (p->batch == 0 || p->seqlen == 0) return w;
    const Segments sg = segments_of(p, true);
    const int64_t n = p->batch * (sg.n - 1) * p->channels, tile = ssd::sel_ckpt_tile();
    const int64_t tiles = p->batch * ((p->seqlen + tile - 1) / tile) * p->channels;
    const int64_t bc = align256(blocks_of(p) * p->batch * p->seqlen * p->ngroups * p->dstate * 4);
    w.step = align256(n * p->dstate * 4);
    w.grad = w.step + align256(n * 4);
    w.ckpt = w.grad + align256(n * p->dstate * 4);
    w.ckpt_step = w.ckpt + align256(tiles * p->dstate * 4);
    // a single channel block per group writes dB and dC themselves
    w.part_b = w.ckpt_step + align256(tiles * 4);
    w.part_c = w.part_b + (blocks_of(p) > 1 ? bc : 0);
    w.sums = w.part_c + (blocks_of(p) > 1 ? bc : 0);
    w.total = w.sums + align256(p->batch * sg.n * p->channels * (p->dstate + 2) * 4);
    return w;
}

ssd::SelParams params_of(const ssd_selective_problem_t* p, bool backward) {
    ssd::SelParams s{};
    const Segments sg = segments_of(p, backward);
    s.batch = p->batch;
    s.T = p->seqlen;
    s.D = p->channels;
    s.G = p->ngroups;
    s.nseqs = p->nseqs;
    s.ldx = p->ldx;
    s.lddt = p->lddt;
    s.ldz = p->ldz;
    s.ldb = p->ldb;
    s.ldc = p->ldc;
    s.seg_len = sg.len;
    s.nseg = (int)sg.n;
    s.per_group = (int)(p->channels / p->ngroups);
    s.blocks = (int)blocks_of(p);
    s.softplus = (p->flags & SSD_FLAG_DT_SOFTPLUS) ? 1 : 0;
    return s;
}

template <typename T> T* at(void* base, int64_t off) { return reinterpret_cast<T*>(static_cast<char*>(base) + off); }

int done(const char* what, const ssd_selective_problem_t* p, int64_t segs, hipError_t e) {
    if (log_enabled())
        std::fprintf(stderr, "[ssd] selective %s dtype=%d batch=%lld T=%lld D=%lld N=%lld G=%lld segments=%lld -> %s\n",
                     what, p->dtype, (long long)p->batch, (long long)p->seqlen, (long long)p->channels,
                     (long long)p->dstate, (long long)p->ngroups, (long long)segs, hipGetErrorString(e));
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

}  // namespace

extern "C" {

size_t ssd_selective_workspace_size(const ssd_selective_problem_t* p) {
    return validate(p) == SSD_OK ? (size_t)forward_space(p).total : 0;
}
size_t ssd_selective_backward_workspace_size(const ssd_selective_problem_t* p) {
    return validate(p) == SSD_OK ? (size_t)backward_space(p).total : 0;
}

int ssd_selective_forward(const ssd_selective_problem_t* p, const void* x, const void* dt, const float* dt_bias,
                          const float* A_log, const void* B, const void* C, const float* D, const void* z,
                          const float* init_state, const int32_t* seq_idx, void* y, float* final_state, void* workspace,
                          size_t workspace_bytes, void* stream) {
    const int v = validate(p);
    if (v != SSD_OK) return v;
    const bool empty = p->batch == 0 || p->seqlen == 0;
    if (!A_log || (!empty && (!x || !dt || !B || !C || !y))) return SSD_ERR_NULL_POINTER;
    const int q = check_sequences(p, seq_idx);
    if (q != SSD_OK) return q;
    const ForwardSpace ws = forward_space(p);
    if (ws.total > 0 && !workspace) return SSD_ERR_WORKSPACE;
    const uintptr_t e = (uintptr_t)elem_size(p->dtype);
    if (misaligned(x, e) || misaligned(dt, e) || misaligned(B, e) || misaligned(C, e) || misaligned(z, e) ||
        misaligned(y, e) || misaligned(dt_bias, 4) || misaligned(A_log, 4) || misaligned(D, 4) ||
        misaligned(init_state, 4) || misaligned(seq_idx, 4) || misaligned(final_state, 4) || misaligned(workspace, 256))
        return SSD_ERR_ALIGNMENT;
    if ((int64_t)workspace_bytes < ws.total) return SSD_ERR_WORKSPACE;
    const SelSizes s = sel_sizes(p);
    const Buf in[] = {{x, s.x}, {dt, s.dt}, {dt_bias, s.d}, {A_log, s.a}, {B, s.b}, {C, s.c}, {D, s.d}, {z, s.z},
                      {init_state, s.state}, {seq_idx, s.seq}};
    const Buf out[] = {{y, s.y}, {final_state, s.state}, {workspace, ws.total}};
    const int a = check_alias(in, 10, out, 3);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (empty) {
        // no token: each row's final state is its initial state
        if (seq_idx || !final_state) return SSD_OK;
        return done("forward", p, 0, ssd::launch_copy(final_state, init_state, s.state / 4, st));
    }
    ssd::SelParams k = params_of(p, false);
    k.x = x;
    k.dt = dt;
    k.B = B;
    k.C = C;
    k.z = z;
    k.A_log = A_log;
    k.skip = D;
    k.dt_bias = dt_bias;
    k.init = init_state;
    k.seq_idx = seq_idx;
    k.y = y;
    k.fin = final_state;
    hipError_t r = hipSuccess;
    if (k.nseg > 1) {
        k.seg_state = at<float>(workspace, 0);
        k.seg_step = at<float>(workspace, ws.step);
        r = ssd::launch_sel_local(k, p->dtype, p->dstate, st);
        if (r == hipSuccess) r = ssd::launch_sel_combine(k, p->dstate, false, st);
    }
    if (r == hipSuccess) r = ssd::launch_sel_forward(k, p->dtype, p->dstate, st);
    return done("forward", p, k.nseg, r);
}

int ssd_selective_step(const ssd_selective_problem_t* p, const void* x, const void* dt, const float* dt_bias,
                       const float* A_log, const void* B, const void* C, const float* D, const void* z,
                       const float* state, float* state_out, void* y, void* stream) {
    if (!p) return SSD_ERR_NULL_POINTER;
    if (p->seqlen != 1 || p->nseqs != p->batch) return SSD_ERR_BAD_SHAPE;
    const int v = validate(p, true);
    if (v != SSD_OK) return v;
    if (!A_log || (p->batch > 0 && (!x || !dt || !B || !C || !state || !state_out || !y))) return SSD_ERR_NULL_POINTER;
    const uintptr_t e = (uintptr_t)elem_size(p->dtype);
    if (misaligned(x, e) || misaligned(dt, e) || misaligned(B, e) || misaligned(C, e) || misaligned(z, e) ||
        misaligned(y, e) || misaligned(dt_bias, 4) || misaligned(A_log, 4) || misaligned(D, 4) || misaligned(state, 4) ||
        misaligned(state_out, 4))
        return SSD_ERR_ALIGNMENT;
    const SelSizes s = sel_sizes(p);
    const Buf in[] = {{x, s.x}, {dt, s.dt}, {dt_bias, s.d}, {A_log, s.a}, {B, s.b}, {C, s.c}, {D, s.d}, {z, s.z},
                      {state == state_out ? nullptr : state, s.state}};
    const Buf out[] = {{y, s.y}, {state_out, s.state}};
    const int a = check_alias(in, 9, out, 2);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    if (p->batch == 0) return SSD_OK;
    ssd::SelParams k = params_of(p, false);
    k.x = x;
    k.dt = dt;
    k.B = B;
    k.C = C;
    k.z = z;
    k.A_log = A_log;
    k.skip = D;
    k.dt_bias = dt_bias;
    k.init = state;
    k.fin = state_out;
    k.y = y;
    return done("step", p, 1, ssd::launch_sel_step(k, p->dtype, p->dstate, static_cast<hipStream_t>(stream)));
}

int ssd_selective_backward(const ssd_selective_problem_t* p, const void* x, const void* dt, const float* dt_bias,
                           const float* A_log, const void* B, const void* C, const float* D, const void* z,
                           const float* init_state, const int32_t* seq_idx, const float* dy, const float* dfinal,
                           float* dx, float* ddt, float* dA_log, float* dB, float* dC, float* dD, float* dz,
                           float* dinit, float* ddt_bias, void* workspace, size_t workspace_bytes, void* stream) {
    const int v = validate(p);
    if (v != SSD_OK) return v;
    const bool empty = p->batch == 0 || p->seqlen == 0;
    if (!A_log || !dA_log || (!empty && (!x || !dt || !B || !C || !dy || !dx || !ddt || !dB || !dC || (z && !dz))))
        return SSD_ERR_NULL_POINTER;
    const int q = check_sequences(p, seq_idx);
    if (q != SSD_OK) return q;
    const BackwardSpace ws = backward_space(p);
    if (ws.total > 0 && !workspace) return SSD_ERR_WORKSPACE;
    const uintptr_t e = (uintptr_t)elem_size(p->dtype);
    if (misaligned(x, e) || misaligned(dt, e) || misaligned(B, e) || misaligned(C, e) || misaligned(z, e) ||
        misaligned(dt_bias, 4) || misaligned(A_log, 4) || misaligned(D, 4) || misaligned(init_state, 4) ||
        misaligned(seq_idx, 4) || misaligned(dy, 4) || misaligned(dfinal, 4) || misaligned(dx, 4) || misaligned(ddt, 4) ||
        misaligned(dA_log, 4) || misaligned(dB, 4) || misaligned(dC, 4) || misaligned(dD, 4) || misaligned(dz, 4) ||
        misaligned(dinit, 4) || misaligned(ddt_bias, 4) || misaligned(workspace, 256))
        return SSD_ERR_ALIGNMENT;
    if ((int64_t)workspace_bytes < ws.total) return SSD_ERR_WORKSPACE;
    const SelSizes s = sel_sizes(p);
    const Buf in[] = {{x, s.x}, {dt, s.dt}, {dt_bias, s.d}, {A_log, s.a}, {B, s.b}, {C, s.c}, {D, s.d}, {z, s.z},
                      {init_state, s.state}, {seq_idx, s.seq}, {dy, s.f}, {dfinal, s.state}};
    const Buf out[] = {{dx, s.f}, {ddt, s.f}, {dA_log, s.a}, {dB, s.bc}, {dC, s.bc}, {dD, s.d}, {z ? dz : nullptr, s.f},
                       {dinit, s.state}, {ddt_bias, s.d}, {workspace, ws.total}};
    const int a = check_alias(in, 12, out, 10);
    if (a != SSD_OK) return a;
    const int d = check_device();
    if (d != SSD_OK) return d;
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t r = hipSuccess;
    if (empty) {
        // no token: nothing reaches the parameters, and each row's final state is its initial state
        r = ssd::launch_fill(dA_log, s.a / 4, st);
        if (r == hipSuccess) r = ssd::launch_fill(dD, s.d / 4, st);
        if (r == hipSuccess) r = ssd::launch_fill(ddt_bias, s.d / 4, st);
        if (r == hipSuccess && dinit) r = ssd::launch_copy(dinit, seq_idx ? nullptr : dfinal, s.state / 4, st);
        return done("backward", p, 0, r);
    }
    ssd::SelParams k = params_of(p, true);
    k.x = x;
    k.dt = dt;
    k.B = B;
    k.C = C;
    k.z = z;
    k.A_log = A_log;
    k.skip = D;
    k.dt_bias = dt_bias;
    k.init = init_state;
    k.seq_idx = seq_idx;
    k.dy = dy;
    k.dfin = dfinal;
    k.dx = dx;
    k.ddt = ddt;
    k.dz = dz;
    k.dinit = dinit;
    k.seg_state = at<float>(workspace, 0);
    k.seg_step = at<float>(workspace, ws.step);
    k.seg_grad = at<float>(workspace, ws.grad);
    k.ckpt = at<float>(workspace, ws.ckpt);
    k.ckpt_step = at<float>(workspace, ws.ckpt_step);
    k.part_b = k.blocks > 1 ? at<float>(workspace, ws.part_b) : dB;
    k.part_c = k.blocks > 1 ? at<float>(workspace, ws.part_c) : dC;
    k.part_sums = at<float>(workspace, ws.sums);
    // ids that do not occur keep a zero gradient
    if (seq_idx && dinit) r = ssd::launch_fill(dinit, s.state / 4, st);
    if (r == hipSuccess) r = ssd::launch_sel_locals(k, p->dtype, p->dstate, st);
    if (r == hipSuccess && k.nseg > 1) r = ssd::launch_sel_combine(k, p->dstate, true, st);
    if (r == hipSuccess) r = ssd::launch_sel_reverse(k, p->dtype, p->dstate, st);
    if (r == hipSuccess && k.blocks > 1) r = ssd::launch_sel_group_sums(k, p->dstate, dB, dC, st);
    if (r == hipSuccess) {
        ssd::ColumnSums c{};
        c.part = k.part_sums;
        c.out = dA_log;
        c.out2 = dD;
        c.out3 = ddt_bias;
        c.rows = p->batch * k.nseg;
        c.cols = p->channels * (p->dstate + 2);
        c.split = p->channels * p->dstate;
        c.split2 = c.split + p->channels;
        r = ssd::launch_column_sums(c, st);
    }
    return done("backward", p, k.nseg, r);
}

}  // extern "C"
