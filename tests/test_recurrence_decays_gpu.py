"""The gated linear recurrence with fast decays: what a decay a = e^L << 1 multiplies (the state
that a token passes on, dinit, and dr and dA_log, which are proportional to a) is right relative
to itself, not only to 1.

The bounds are those of recurrence_ref with another one for the decay.  L carries N_M roundings
(with |r| more for the gates of bf16 activations), so e^L is known to a (N_M |L| + 2) U32, the
exponential's own step being 2 of them; two more for the product that uses it.  Above L = -1 the
form for long memories is as good: a = 1 - m with m known to N_M roundings of m, a |L| <= m.  A
decay or a product of decays below FLUSH may count as 0."""
import math

import pytest
import torch

import block_ref as ref
import recurrence_ref as rr
from block_ref import U32

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FLUSH = rr.FLUSH


def announce(msg):
    print("[case] " + msg, flush=True)


def make(dt, b, T, rates, shift, spread, lens=None, seed=0):
    """rates: A_log of the channels; r is shift + spread * normal.  Every third channel's input gate is
    closed, so its states are products of decays."""
    g = torch.Generator().manual_seed(seed + 13 * T + len(rates))
    D, n = len(rates), len(ref.sequences(b, T, lens))
    q = {"x": torch.randn(b, T, D, generator=g), "r": shift + spread * torch.randn(b, T, D, generator=g),
         "i": torch.randn(b, T, D, generator=g)}
    q["i"][..., ::3] = -100.0
    q = {k: v.to(TYPES[dt]) for k, v in q.items()}
    q.update(A_log=torch.tensor(rates), init=torch.randn(n, D, generator=g), dy=torch.randn(b, T, D, generator=g),
             dfinal=torch.randn(n, D, generator=g), ids=ref.ids_of(b, T, lens), lens=lens, n=n)
    return q


def reference(q):
    """{name: (value, bound)} of y, final and the gradients, 64 bits."""
    bf16 = q["x"].dtype == torch.bfloat16
    x, r, i, A_log, init, dy, dfinal = (q[k].double() for k in ("x", "r", "i", "A_log", "init", "dy", "dfinal"))
    b, T, D = x.shape
    L, a, m, beta, u = rr.parts(x, r, i, A_log)
    nr, ni = rr.argument(r, bf16), rr.argument(i, bf16)
    n_m = rr.N_M + nr
    ea = U32 * torch.where(L > -1, n_m * m + 4, a * (n_m * L.abs() + 4)) + FLUSH
    s, si = torch.sigmoid(r), torch.sigmoid(i)
    v = si * x
    may_shut = (r < -80) & (s > 0)                                    # a gate that may count as 0
    tiny = torch.where(may_shut, rr.lost_beta(A_log), 0.0)
    lost = FLUSH * x.abs() + tiny * v.abs()
    n_u = rr.N_U + nr / 2 + ni
    zero = torch.zeros_like(x)
    hs, Hs, Es, before, Hb, Eb, g, G, EG = (zero.clone() for _ in range(9))
    out = {k: (torch.zeros_like(init), torch.zeros_like(init)) for k in ("final", "dinit")}
    for k, (row, t0, n) in enumerate(ref.sequences(b, T, q["lens"])):
        h, H, E = init[k], init[k].abs(), torch.zeros(D, dtype=torch.double)
        for t in range(t0, t0 + n):
            before[row, t], Hb[row, t], Eb[row, t] = h, H, E
            E = a[row, t] * E + ea[row, t] * H
            h, H = a[row, t] * h + u[row, t], a[row, t] * H + u[row, t].abs()
            E = E + U32 * (4 * H + n_u[row, t] * u[row, t].abs()) + lost[row, t] + FLUSH
            hs[row, t], Hs[row, t], Es[row, t] = h, H, E
        out["final"][0][k], out["final"][1][k] = h, E + rr.N_TREE * U32 * H + FLUSH * (1 + init[k].abs())
        p, P, E = dfinal[k], dfinal[k].abs(), torch.zeros(D, dtype=torch.double)
        for t in range(t0 + n - 1, t0 - 1, -1):
            g[row, t], G[row, t] = dy[row, t] + p, dy[row, t].abs() + P
            EG[row, t] = E + U32 * (4 * dy[row, t].abs() + 4 * P)
            p, P = a[row, t] * g[row, t], a[row, t] * G[row, t]
            E = a[row, t] * EG[row, t] + ea[row, t] * G[row, t] + U32 * 2 * P + FLUSH
        out["dinit"][0][k], out["dinit"][1][k] = p, E + rr.N_TREE * U32 * P + FLUSH
    Es = Es + rr.N_TREE * U32 * Hs
    Eb = Eb + rr.N_TREE * U32 * Hb
    EG = EG + rr.N_TREE * U32 * G
    out["y"] = (hs, Es)
    ratio = torch.where(beta > 0, L / beta, 0.0)
    out["dx"] = (g * beta * si, (EG + U32 * (40 + nr / 2 + ni) * G) * beta * si + G * (tiny * si + FLUSH))
    di = beta * v * (1 - si)
    out["di"] = (g * di, (EG + U32 * (50 + nr / 2 + 2 * ni) * G) * di.abs() + G * ((tiny * v * (1 - si)).abs() + 2 * FLUSH * x.abs()))
    M = g * (L * a * before - v * a * a * ratio)
    size = L.abs() * a * Hb + v.abs() * a * a * ratio.abs()
    M_e = EG * size + G * (U32 * (40 + 2 * nr + ni) * size + L.abs() * (a * Eb + ea * Hb) + v.abs() * ratio.abs() * 2 * a * ea)
    M_e = M_e + G * (tiny * v.abs() + FLUSH * (torch.where(may_shut, torch.exp(A_log), 1.0) * Hb + x.abs()))
    out["dr"] = (M * (1 - s), (M_e + U32 * (12 + nr) * M.abs()) * (1 - s) + FLUSH * M.abs())
    out["dA_log"] = (M.sum((0, 1)), M_e.sum((0, 1)) + (b * T + 20) * U32 * M.abs().sum((0, 1)))
    return out


def check(ssd, q):
    want = reference(q)
    d = {k: v.cuda() if torch.is_tensor(v) else v for k, v in q.items()}
    y, final = ssd.gated_recurrence(d["x"], d["r"], d["i"], d["A_log"], None, d["init"], d["ids"], q["n"])
    rr.check(y, *want["y"], "y")
    rr.check(final, *want["final"], "final")
    got = ssd.gated_recurrence_backward(d["x"], d["r"], d["i"], d["A_log"], d["dy"], init_state=d["init"],
                                        dfinal=d["dfinal"], seq_idx=d["ids"], nseqs=q["n"])
    for k, v in got.items():
        rr.check(v, *want[k], k)
    if q["x"].shape[1] == 1 and q["lens"] is None:
        state = torch.empty_like(d["init"])
        y = ssd.gated_recurrence_step(d["x"][:, 0], d["r"][:, 0], d["i"][:, 0], d["A_log"], d["init"], state_out=state)
        rr.check(y[:, None], *want["y"], "y of a step")
        rr.check(state, *want["final"], "state of a step")


SIZES = [(2, 1, None), (2, 43, None), (1, 300, None), (2, 300, [[1, 150, 149], [290, 10]])]
SIZE_IDS = ["step", "tile", "tiles", "packed"]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=SIZE_IDS)
@pytest.mark.parametrize("shift", [2.0, 4.0])
def test_fast_decays(dt, size, shift):
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence fast decays %s %s %s" % (dt, size, shift))
    rates = [math.log(v) for v in (1, 2, 4, 6, 8, 10, 12, 14, 16, 20, 24, 28, 32, 40, 60, 80, 100, 0.1, 0.01)]
    check(ssd, make(dt, size[0], size[1], rates, shift, 1.0, size[2]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=SIZE_IDS)
def test_large_rates_with_nearly_closed_gates(dt, size):
    """A_log from 60 to 76 where A sigmoid(r) is around 1: neither factor is near it."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence large rates %s %s" % (dt, size))
    rates = [60.0 + k for k in range(17)]
    q = make(dt, size[0], size[1], rates, 0.0, 1.0, size[2])
    q["r"] = (q["r"].float() - q["A_log"]).to(q["r"].dtype)
    check(ssd, q)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_largest_rates(dt):
    """A_log counts as at most 88: beyond it an open gate forgets everything, a closed one nothing."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence largest rates %s" % dt)
    q = make(dt, 1, 40, [70.0, 88.0, 88.5, 100.0, 1e30, math.inf], 2.0, 1.0)
    q["r"][:, 20:] = -math.inf
    q["init"], q["x"] = q["init"] * 1000, q["x"] * 256               # times the rate alone past fp32's range
    capped = dict(q, A_log=q["A_log"].clamp(max=88))
    check(ssd, capped)
    d = {k: v.cuda() if torch.is_tensor(v) else v for k, v in q.items()}
    both = [ssd.gated_recurrence(d["x"], d["r"], d["i"], A, None, d["init"]) for A in (d["A_log"], capped["A_log"].cuda())]
    assert torch.equal(both[0][0], both[1][0]) and torch.equal(both[0][1], both[1][1])
    both = [ssd.gated_recurrence_backward(d["x"], d["r"], d["i"], A, d["dy"], init_state=d["init"], dfinal=d["dfinal"])
            for A in (d["A_log"], capped["A_log"].cuda())]
    assert all(torch.equal(both[0][k], both[1][k]) and torch.isfinite(both[0][k]).all() for k in both[0])
