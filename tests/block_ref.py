"""Plain 64-bit forms of the operators around the scan, on CPU tensors, one sequence at
a time, and the comparison that the tests use.

Tolerances count roundings.  U32 = 2^-24 and U16 = 2^-8 are the half steps of fp32 and
bf16.  An output is held to  half step of its type * |ref| + n * U32 * scale,  `scale`
being the sum of the magnitudes of the terms that the output is a sum of, and n the
number of fp32 roundings that a term can pass through: that many roundings of terms of
that size are the most that any order of summation can lose, to first order."""
import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8


def half_step(dtype):
    return U16 if dtype == torch.bfloat16 else U32


def check(got, ref, scale, n, what):
    ref, scale = ref.double(), torch.as_tensor(scale).double()
    err = (got.detach().cpu().double() - ref).abs()
    bound = half_step(got.dtype) * ref.abs() + n * U32 * scale
    assert torch.isfinite(got).all(), "%s has non-finite values" % what
    worst = float((err / bound.clamp(min=1e-300)).max()) if err.numel() else 0.0
    assert worst <= 1.0, "%s: error %.2f times its bound" % (what, worst)


def silu(v):
    return v * torch.sigmoid(v)


def sequences(b, T, lens):
    """[(row, first token, length)] by sequence id; lens None: a sequence per row."""
    if lens is None:
        return [(r, 0, T) for r in range(b)]
    out = []
    for r, row in enumerate(lens):
        t = 0
        for n in row:
            out.append((r, t, n))
            t += n
        assert t == T
    return out


def ids_of(b, T, lens):
    if lens is None:
        return None
    seq = torch.zeros(b, T, dtype=torch.int32)
    for k, (r, t, n) in enumerate(sequences(b, T, lens)):
        seq[r, t:t + n] = k
    return seq


def conv(x, w, bias, init, lens, act):
    """(y, final) of the causal convolution in the inputs' own precision."""
    b, T, D = x.shape
    K = w.shape[1]
    y, final = [], []
    for k, (r, t, n) in enumerate(sequences(b, T, lens)):
        line = torch.cat([init[k], x[r, t:t + n]])
        pre = sum(line[i:i + n] * w[:, i] for i in range(K))
        if bias is not None:
            pre = pre + bias
        y.append(silu(pre) if act else pre)
        final.append(line[n:])
    return torch.cat(y).view(b, T, D), torch.stack(final)


def gated(x, z, w, size, eps, first):
    u = x * silu(z) if first else x
    g = u.unflatten(-1, (-1, size))
    out = (g / torch.sqrt((g * g).mean(-1, keepdim=True) + eps)).flatten(-2) * w
    return out if first else out * silu(z)


def residual(x, res, w, scale, eps):
    u = x if scale is None else x * scale
    u = u if res is None else res + u
    return u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps) * w, u


def leaves(*ts):
    return [None if t is None else t.detach().double().clone().requires_grad_() for t in ts]


def scan(x, dt, A_log, B, C, D, z, init, bias, soft, lens):
    """(y, final) of the selective scan in the inputs' own precision; B, C (b,T,G,N)."""
    b, T, Dc = x.shape
    G, N = B.shape[2:]
    A = -torch.exp(A_log)
    rep = Dc // G
    ys, final = [], []
    for k, (r, t0, n) in enumerate(sequences(b, T, lens)):
        h = init[k]
        for t in range(t0, t0 + n):
            step = dt[r, t] + bias
            if soft:
                step = torch.logaddexp(step, torch.zeros_like(step))
            Bt, Ct = B[r, t].repeat_interleave(rep, 0), C[r, t].repeat_interleave(rep, 0)
            h = torch.exp(step[:, None] * A) * h + (step * x[r, t])[:, None] * Bt
            y = (h * Ct).sum(-1) + D * x[r, t]
            ys.append(y * silu(z[r, t]) if z is not None else y)
        final.append(h)
    return torch.stack(ys).view(b, T, Dc), torch.stack(final)


def scan_sizes(x, dt, A_log, B, C, D, z, init, bias, soft, lens):
    """The same map over magnitudes, with every factor's derivative counted positive: its
    values and autograd gradients are the sums of magnitudes that the scan's are sums of.
    x, B, C, D, z and init come as leaves holding magnitudes (z: the gate's value is taken
    from ``z`` itself, which may be signed)."""
    b, T, Dc = x.shape
    G, N = B.shape[2:]
    A = torch.exp(A_log)
    rep = Dc // G
    ys, final = [], []
    for k, (r, t0, n) in enumerate(sequences(b, T, lens)):
        h = init[k]
        for t in range(t0, t0 + n):
            step = dt[r, t] + bias
            if soft:
                step = torch.logaddexp(step, torch.zeros_like(step))
            arg = step[:, None] * A
            decay = torch.exp(-arg).detach() * torch.exp(arg - arg.detach())
            Bt, Ct = B[r, t].repeat_interleave(rep, 0), C[r, t].repeat_interleave(rep, 0)
            h = decay * h + (step * x[r, t])[:, None] * Bt
            y = (h * Ct).sum(-1) + D * x[r, t]
            if z is not None:
                zt = z[r, t]
                # silu's slope is below 1.1
                y = y * (silu(zt).abs().detach() + 1.1 * (zt - zt.detach()))
            ys.append(y)
        final.append(h)
    return torch.stack(ys).view(b, T, Dc), torch.stack(final)
