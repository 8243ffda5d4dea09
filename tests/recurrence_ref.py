"""The gated linear recurrence and the norm with rotation in 64 bits, on CPU tensors, with
the error that their 32-bit forms may have.

The bounds count roundings, U32 = 2^-24 being half a step of fp32, to first order.  A decay
a = 1 - m is known to (N_M m + 2) U32: m = 1 - e^L passes through the sigmoid, the rate, their
product and the difference (20 roundings at most, relative to m).  An input beta sigmoid(i) x
passes 30, a state two in each step and one or two more in the products of decays that carry it
across a cut, so with H the same recurrence over magnitudes
    E_t = a E_{t-1} + U32 ((N_M m) H_{t-1} + 4 H_t + N_U |u_t|),
and each level of a tree of cuts adds roundings of H_t itself, below 20 in all.  Backwards the
same holds for the gradient that reaches a state, over dy.

A gate of bf16 activations takes e^-v with the exponent v log2(e) rounded to fp32, which moves it
by |v| roundings (half a step of a number near v is at most |v| 2^-24): N_M and the gates' own
factors have |r| and |i| more there, beta half of |r| (|v| beyond 100 is as 100: the sigmoid is
below FLUSH or 1 there).

Underflow: a sigmoid below FLUSH = 2^-126, fp32's smallest normal number, may count as 0.  That
moves silu(z) by FLUSH |z|, sigmoid(i) x by FLUSH |x|, and, beta being sqrt(2 |A| sigmoid(r))
there, beta and |L| / beta by at most sqrt(2 |A| FLUSH), 1.5e-19 sqrt |A|: terms of that size times
what they multiply are added (a bound of relative roundings alone would ask for more than fp32's
range holds: silu(-95) = -5e-40)."""
import torch

import block_ref as ref
from block_ref import U32

N_M, N_U, N_TREE = 20, 30, 20
FLUSH = 2.0 ** -126


def check(got, want, bound, what):
    """Half a step of the output's type, and the bound."""
    assert torch.isfinite(got).all(), "%s has non-finite values" % what
    want = want.detach().double()
    err = (got.detach().cpu().double() - want).abs()
    room = ref.half_step(got.dtype) * want.abs() * (1 + 1e-6) + bound.detach().double() + FLUSH
    if not err.numel():
        return
    at = int((err / room).argmax())
    got, want, err, room = (t.reshape(-1)[at].item() for t in (got, want, err, room))
    assert err <= room, "%s: error %.2f times its bound at flat index %d: %g, should be %g" % (what, err / room, at, got, want)


def parts(x, r, i, A_log):
    L = -torch.exp(A_log) * torch.sigmoid(r)
    beta = torch.sqrt(-torch.expm1(2 * L))
    return L, torch.exp(L), -torch.expm1(L), beta, beta * torch.sigmoid(i) * x


def argument(v, bf16):
    return v.abs().clamp(max=100) if bf16 else torch.zeros_like(v)


def lost_beta(A_log):
    return torch.sqrt(2 * FLUSH * torch.exp(A_log))


def forward(x, r, i, A_log, z, init, lens, bf16=False):
    """(y, final, bound of y, bound of final, states, their magnitudes, their errors), 64 bits."""
    b, T, D = x.shape
    L, a, m, beta, u = parts(x, r, i, A_log)
    n_m, n_u = N_M + argument(r, bf16), N_U + argument(r, bf16) / 2 + argument(i, bf16)
    lost = FLUSH * x.abs() + lost_beta(A_log) * (torch.sigmoid(i) * x).abs()
    hs, Hs, Es = (torch.zeros(b, T, D, dtype=torch.double) for _ in range(3))
    final, fin_e = [], []
    for k, (row, t0, n) in enumerate(ref.sequences(b, T, lens)):
        h, H, E = init[k], init[k].abs(), torch.zeros(D, dtype=torch.double)
        for t in range(t0, t0 + n):
            E = a[row, t] * E + U32 * n_m[row, t] * m[row, t] * H
            h, H = a[row, t] * h + u[row, t], a[row, t] * H + u[row, t].abs()
            E = E + U32 * (4 * H + n_u[row, t] * u[row, t].abs()) + lost[row, t]
            hs[row, t], Hs[row, t], Es[row, t] = h, H, E
        final.append(h)
        fin_e.append(E + N_TREE * U32 * H)
    Es = Es + N_TREE * U32 * Hs
    gate = torch.ones_like(x) if z is None else ref.silu(z)
    bound = Es * gate.abs() + (0 if z is None else U32 * (12 + argument(z, bf16)) * (hs * gate).abs() + FLUSH * (hs * z).abs())
    return hs * gate, torch.stack(final), bound, torch.stack(fin_e), hs, Hs, Es


def backward(x, r, i, A_log, dy, z, init, dfinal, lens, bf16=False):
    """{name: (gradient, bound)}, 64 bits, from the formulas."""
    b, T, D = x.shape
    _, _, _, _, hs, Hs, Es = forward(x, r, i, A_log, z, init, lens, bf16)
    nr, ni = argument(r, bf16), argument(i, bf16)
    L, a, m, beta, _ = parts(x, r, i, A_log)
    si, s = torch.sigmoid(i), torch.sigmoid(r)
    v = si * x
    out = {}
    gy, gn, gl = dy, torch.ones_like(dy), torch.zeros_like(dy)
    if z is not None:
        sz = torch.sigmoid(z)
        slope, wide = sz * (1 + z * (1 - sz)), sz * (1 + z.abs() * (1 - sz))
        out["dz"] = (dy * hs * slope, dy.abs() * (Es * slope.abs() + hs.abs() * (U32 * (20 + argument(z, bf16)) * wide + FLUSH * (1 + z.abs()))))
        gy, gn, gl = dy * z * sz, 12 + argument(z, bf16), FLUSH * (dy * z).abs()
    g, G, EG = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    before, Hb, Eb = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    dinit, dinit_e = torch.zeros_like(init), torch.zeros_like(init)
    for k, (row, t0, n) in enumerate(ref.sequences(b, T, lens)):
        if n == 0:
            dinit[k] = dfinal[k]
            continue
        q, Q, E = dfinal[k], dfinal[k].abs(), torch.zeros(D, dtype=torch.double)
        for t in range(t0 + n - 1, t0 - 1, -1):
            own = gy[row, t]
            g[row, t], G[row, t] = own + q, own.abs() + Q
            EG[row, t] = E + U32 * ((gn[row, t] + 4) * own.abs() + 4 * Q) + gl[row, t]
            q, Q = a[row, t] * g[row, t], a[row, t] * G[row, t]
            E = a[row, t] * EG[row, t] + U32 * ((N_M + nr[row, t]) * m[row, t] + 2) * G[row, t]
            first = t == t0
            before[row, t] = init[k] if first else hs[row, t - 1]
            Hb[row, t] = init[k].abs() if first else Hs[row, t - 1]
            Eb[row, t] = 0 if first else Es[row, t - 1]
        dinit[k], dinit_e[k] = q, E + N_TREE * U32 * Q
    EG = EG + N_TREE * U32 * G
    ratio = torch.where(beta > 0, L / beta, torch.zeros_like(L))
    lost = lost_beta(A_log)
    out["dx"] = (g * beta * si, (EG + U32 * (40 + nr / 2 + ni) * G) * beta * si + G * (lost * si + FLUSH))
    out["di"] = (g * beta * v * (1 - si),
                 (EG + U32 * (50 + nr / 2 + 2 * ni) * G) * (beta * v * (1 - si)).abs() + G * ((lost * v * (1 - si)).abs() + 2 * FLUSH * x.abs()))
    M = g * (L * a * before - v * a * a * ratio)
    ea = U32 * ((N_M + nr) * m + 2)                                            # of a
    size = L.abs() * a * Hb + v.abs() * a * a * ratio.abs()
    M_e = EG * size + G * (U32 * (40 + 2 * nr + ni) * size + L.abs() * (a * Eb + ea * Hb) + v.abs() * ratio.abs() * 2 * a * ea)
    M_e = M_e + G * (lost * v.abs() + FLUSH * (torch.exp(A_log) * Hb + x.abs()))
    out["dr"] = (M * (1 - s), (M_e + U32 * (12 + nr) * M.abs()) * (1 - s) + FLUSH * M.abs())
    out["dA_log"] = (M.sum((0, 1)), M_e.sum((0, 1)) + (b * T + 20) * U32 * M.abs().sum((0, 1)))
    out["dinit"] = (dinit, dinit_e)
    return out


# ------------------------------------------------------------------ norm with rotation
def rotate(v, freqs, positions, interleaved, transposed=False):
    """Pairs of the first 2 len(freqs) channels of v (tokens, heads, N) turned; 64 bits."""
    R = 2 * freqs.numel()
    angle = positions.double()[:, None, None] * freqs.double()
    c, s = torch.cos(angle), torch.sin(angle) * (-1 if transposed else 1)
    p, q = (v[..., 0:R:2], v[..., 1:R:2]) if interleaved else (v[..., :R // 2], v[..., R // 2:R])
    p, q = p * c - q * s, p * s + q * c
    turned = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    return torch.cat([turned, v[..., R:]], -1)


def both_of_pair(v, R, interleaved):
    """|p| + |q| at both places of a pair: the sizes that a turned value is a sum of."""
    if interleaved:
        turned = v[..., :R].unflatten(-1, (-1, 2)).sum(-1, keepdim=True).expand(*v.shape[:-1], R // 2, 2).flatten(-2)
    else:
        half = v[..., :R // 2] + v[..., R // 2:R]
        turned = torch.cat([half, half], -1)
    return torch.cat([turned, v[..., R:]], -1)


def turn_error(freqs, positions):
    """Error of a cosine or sine: the angle reduced in 64 bits (three roundings of it), then
    rounded to 32 (half a revolution at most), then the function's own four roundings."""
    return 8 * U32 + 3 * 2.0 ** -53 * float(positions.abs().max() if positions.numel() else 0) * float(
        freqs.abs().max() if freqs.numel() else 0)


def norm_depth(N):
    """Roundings of a sum over a head: at most N / 4 in a lane, then six steps."""
    return N // 4 + 6
