"""The recurrence and the norm with rotation run together with the operators around them: an SSD
layer whose B and C are normed and rotated, then a layer of the gated recurrence."""
import pytest
import torch

import block_ref as ref
import recurrence_ref as rr

pytestmark = pytest.mark.gpu

EPS = 1e-5
H, P, N, G, M, D = 4, 32, 64, 2, 48, 96          # heads, their channels, states, groups; stream, recurrence


def announce(msg):
    print("[case] " + msg, flush=True)


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)      # noqa: E731
    W = H * P + 2 * G * N
    return {"pre1": 1 + 0.1 * r(M), "win1": r(M, H * P + W) / M ** 0.5, "conv1": r(W, 4) / 2, "cb1": r(W) * 0.1,
            "bw": 1 + 0.1 * r(N), "cw": 1 + 0.1 * r(N), "A1": torch.rand(H, generator=g) * 2, "skip": r(H), "dtb": r(H) - 1,
            "gate": 1 + 0.1 * r(H * P), "wout1": r(H * P, M) / (H * P) ** 0.5,
            "pre2": 1 + 0.1 * r(M), "win2": r(M, 4 * D) / M ** 0.5, "conv2": r(D, 4) / 2, "cb2": r(D) * 0.1,
            "A2": torch.rand(D, generator=g) * 3 - 4, "wout2": r(D, M) / D ** 0.5,
            "freqs": (10000.0 ** (-torch.arange(N // 2).double() / (N // 2))).float()}


def step_sizes(w, h):
    return h[..., :H].float() * 0.5                  # any function of the token will do


def prompt(ssd, w, x, stream, positions, ids=None, n=None, states=(None,) * 4):
    """x (b,T,M) through both layers: (output, stream, four states)."""
    b, T = x.shape[:2]
    conv1, ssm, conv2, rec = states
    h, stream = ssd.residual_norm(x, stream, w["pre1"], eps=EPS)
    proj = h @ w["win1"].to(h.dtype)
    dt = step_sizes(w, h)
    xbc, conv1 = ssd.causal_conv(proj[..., H * P:], w["conv1"], w["cb1"], conv1, ids, n)
    xs, B, C = xbc.split([H * P, G * N, G * N], -1)
    B, C = ssd.rotary_norm(B.unflatten(-1, (G, N)), C.unflatten(-1, (G, N)), w["bw"], w["cw"], w["freqs"], positions, eps=EPS)
    y, ssm = ssd.forward(xs.reshape(b, T, H, P), dt, w["A1"], B, C, w["skip"], init_state=ssm, seq_idx=ids, nseqs=n,
                         dt_scales_x=True, dt_bias=w["dtb"], dt_softplus=True)
    y = ssd.gated_norm(y.flatten(-2), proj[..., :H * P], w["gate"], eps=EPS)
    h, stream = ssd.residual_norm(y @ w["wout1"].to(y.dtype), stream, w["pre2"], eps=EPS)
    proj = h @ w["win2"].to(h.dtype)
    xc, conv2 = ssd.causal_conv(proj[..., :D], w["conv2"], w["cb2"], conv2, ids, n)
    y, rec = ssd.gated_recurrence(xc, proj[..., D:2 * D], proj[..., 2 * D:3 * D], w["A2"], proj[..., 3 * D:], rec, ids, n)
    return y @ w["wout2"].to(y.dtype), stream, (conv1, ssm, conv2, rec)


def token(ssd, w, x, stream, positions, states):
    """One token per row, x (b,M); the states are updated in place."""
    conv1, ssm, conv2, rec = states
    h, stream = ssd.residual_norm(x, stream, w["pre1"], eps=EPS)
    proj = h @ w["win1"].to(h.dtype)
    dt = step_sizes(w, h)
    xbc = ssd.causal_conv_step(proj[:, H * P:], w["conv1"], w["cb1"], conv1)
    xs, B, C = xbc.split([H * P, G * N, G * N], -1)
    B, C = ssd.rotary_norm(B.unflatten(-1, (G, N)), C.unflatten(-1, (G, N)), w["bw"], w["cw"], w["freqs"], positions, eps=EPS)
    y = ssd.step(xs.reshape(-1, H, P), dt, w["A1"], B, C, w["skip"], ssm, dt_scales_x=True, dt_bias=w["dtb"], dt_softplus=True)
    y = ssd.gated_norm(y.reshape(-1, H * P), proj[:, :H * P], w["gate"], eps=EPS)
    h, stream = ssd.residual_norm(y @ w["wout1"].to(y.dtype), stream, w["pre2"], eps=EPS)
    proj = h @ w["win2"].to(h.dtype)
    xc = ssd.causal_conv_step(proj[:, :D], w["conv2"], w["cb2"], conv2)
    y = ssd.gated_recurrence_step(xc, proj[:, D:2 * D], proj[:, 2 * D:3 * D], w["A2"], rec, z=proj[:, 3 * D:])
    return y @ w["wout2"].to(y.dtype), stream


def plain(w, x, stream, positions, lens):
    """The same in 64 bits on the CPU."""
    b, T = x.shape[:2]
    n = len(ref.sequences(b, T, lens))
    zero = lambda *s: torch.zeros(n, *s, dtype=torch.double)      # noqa: E731
    h, stream = ref.residual(x, stream, w["pre1"], None, EPS)
    proj = h @ w["win1"]
    xbc, _ = ref.conv(proj[..., H * P:], w["conv1"], w["cb1"], zero(3, H * P + 2 * G * N), lens, True)
    xs, B, C = xbc.split([H * P, G * N, G * N], -1)
    out = []
    for u, k in ((B, "bw"), (C, "cw")):
        u = u.reshape(b * T, G, N)
        v = u / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS) * w[k]
        out.append(rr.rotate(v, w["freqs"], positions.reshape(-1), False).view(b, T, G, N).repeat_interleave(H // G, 2))
    B, C = out
    dt = torch.nn.functional.softplus(h[..., :H] * 0.5 + w["dtb"])
    xs = xs.reshape(b, T, H, P)
    ys, s = torch.zeros(b, T, H, P, dtype=torch.double), None
    for r, t0, m in ref.sequences(b, T, lens):
        s = torch.zeros(H, P, N, dtype=torch.double)
        for t in range(t0, t0 + m):
            s = torch.exp(-dt[r, t] * torch.exp(w["A1"]))[:, None, None] * s + \
                (dt[r, t][:, None] * xs[r, t])[..., None] * B[r, t][:, None]
            ys[r, t] = (s * C[r, t][:, None]).sum(-1) + w["skip"][:, None] * xs[r, t]
    y = ref.gated(ys.flatten(-2), proj[..., :H * P], w["gate"], H * P, EPS, True)
    h, stream = ref.residual(y @ w["wout1"], stream, w["pre2"], None, EPS)
    proj = h @ w["win2"]
    xc, _ = ref.conv(proj[..., :D], w["conv2"], w["cb2"], zero(3, D), lens, True)
    y = rr.forward(xc, proj[..., D:2 * D], proj[..., 2 * D:3 * D], w["A2"], proj[..., 3 * D:], zero(D), lens)[0]
    return y @ w["wout2"], stream


@pytest.mark.parametrize("dt_", ["bf16", "f32"])
def test_prompt_then_tokens(dt_):
    """A prompt followed by single tokens equals the whole prompt, packed rows their sequences run
    alone, and both the 64-bit form."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrent layers %s" % dt_)
    b, T, K = 2, 150, 6
    cpu = weights(1)
    w = {k: v.cuda() for k, v in cpu.items()}
    g = torch.Generator().manual_seed(2)
    typ = torch.bfloat16 if dt_ == "bf16" else torch.float32
    x = torch.randn(b, T + K, M, generator=g).to(typ).cuda()
    res = torch.randn(b, T + K, M, generator=g).cuda()
    pos = (torch.arange(T + K, dtype=torch.int32) + torch.tensor([[0], [70000]], dtype=torch.int32)).cuda()
    whole, stream, states1 = prompt(ssd, w, x, res, pos)
    out, _, states = prompt(ssd, w, x[:, :T], res[:, :T], pos[:, :T].contiguous())
    outs = [out]
    for t in range(T, T + K):
        outs.append(token(ssd, w, x[:, t], res[:, t], pos[:, t].contiguous(), states)[0][:, None])
    # bf16: a dozen roundings of 2^-8 on the way through both layers, in the scan's products too,
    # each of the size of what it rounds: 2^-3 of the largest output covers 32 of them.  fp32: the
    # scan's 1e-5 and a few hundred roundings of 2^-24 per product: 2^-12.
    tol = 2.0 ** -3 if dt_ == "bf16" else 2.0 ** -12
    size = float(whole.float().abs().max())
    assert float((torch.cat(outs, 1).float() - whole.float()).abs().max()) <= tol * size
    for a, c in zip(states, states1):
        assert float((a - c).abs().max()) <= tol * float(c.abs().max())

    wide = {k: v.double() for k, v in cpu.items()}
    want, wants = plain(wide, x.cpu().double(), res.cpu().double(), pos.cpu(), None)
    assert float((whole.cpu().double() - want).abs().max()) <= tol * float(want.abs().max())
    assert float((stream.cpu().double() - wants).abs().max()) <= tol * float(wants.abs().max())

    lens = [[50, 106], [1, 155]]
    ids = ref.ids_of(b, T + K, lens).cuda()
    place = torch.cat([torch.arange(m, dtype=torch.int32) for row in lens for m in row]).view(b, T + K).cuda()
    packed, _, states = prompt(ssd, w, x, res, place, ids, 4)
    for k, (r, t, m) in enumerate(ref.sequences(b, T + K, lens)):
        o, _, s = prompt(ssd, w, x[r:r + 1, t:t + m], res[r:r + 1, t:t + m], None)
        assert float((o[0].float() - packed[r, t:t + m].float()).abs().max()) <= tol * size
        for one, all_ in zip(s, states):
            assert float((one[0] - all_[k]).abs().max()) <= tol * float(all_.abs().max())


def test_gradients():
    """residual_norm -> causal_conv -> gated_recurrence, and rotary_norm -> forward, forwards and
    backwards in fp32, against autograd through the 64-bit forms."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrent layers, gradients")
    b, T = 2, 90
    lens = [[40, 50], [1, 89]]
    n = 4
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g)      # noqa: E731
    p = {"h": r(b, T, M), "res": r(b, T, M), "pre": 1 + 0.1 * r(M), "win": r(M, 4 * D) / M ** 0.5, "conv": r(D, 4) / 2,
         "cb": r(D) * 0.1, "A": torch.rand(D, generator=g) * 3 - 4}
    dout, dres = r(b, T, D), r(b, T, M)
    ids = ref.ids_of(b, T, lens).cuda()
    q = {k: v.cuda() for k, v in p.items()}
    normed, stream = ssd.residual_norm(q["h"], q["res"], q["pre"], eps=EPS)
    proj = normed @ q["win"]
    xc, _ = ssd.causal_conv(proj[..., :D], q["conv"], q["cb"], seq_idx=ids, nseqs=n)
    args = (xc, proj[..., D:2 * D], proj[..., 2 * D:3 * D], q["A"])
    y, _ = ssd.gated_recurrence(*args, z=proj[..., 3 * D:], seq_idx=ids, nseqs=n)
    s = ssd.gated_recurrence_backward(*args, dout.cuda(), z=proj[..., 3 * D:], seq_idx=ids, nseqs=n)
    c = ssd.causal_conv_backward(proj[..., :D], q["conv"], s["dx"], q["cb"], seq_idx=ids, nseqs=n)
    dproj = torch.cat([c["dx"], s["dr"], s["di"], s["dz"]], -1)
    f = ssd.residual_norm_backward(q["h"], stream, q["pre"], dproj @ q["win"].t(), dres.cuda(), eps=EPS)
    got = {"h": f["dx"], "res": f["dresidual"], "pre": f["dweight"], "win": normed.flatten(0, 1).t() @ dproj.flatten(0, 1),
           "conv": c["dweight"], "cb": c["dbias"], "A": s["dA_log"]}
    v = dict(zip(p, ref.leaves(*p.values())))
    normed, stream = ref.residual(v["h"], v["res"], v["pre"], None, EPS)
    proj = normed @ v["win"]
    xc, _ = ref.conv(proj[..., :D], v["conv"], v["cb"], torch.zeros(n, 3, D, dtype=torch.double), lens, True)
    L = -torch.exp(v["A"]) * torch.sigmoid(proj[..., D:2 * D])
    a, u = torch.exp(L), torch.sqrt(-torch.expm1(2 * L)) * torch.sigmoid(proj[..., 2 * D:3 * D]) * xc
    rows = []
    for row, t0, m in ref.sequences(b, T, lens):
        h = torch.zeros(D, dtype=torch.double)
        for t in range(t0, t0 + m):
            h = a[row, t] * h + u[row, t]
            rows.append(h)
    yr = torch.stack(rows).view(b, T, D) * ref.silu(proj[..., 3 * D:])
    grads = dict(zip(v, torch.autograd.grad((yr * dout.double()).sum() + (stream * dres.double()).sum(), list(v.values()))))
    # five products and operators in fp32, each within a few hundred roundings (2^-24) of the
    # largest value that it handles: 2^-13 of the largest gradient covers 2048 of them
    assert float((y.cpu().double() - yr.detach()).abs().max()) <= 2.0 ** -13 * float(yr.detach().abs().max())
    for k, want in grads.items():
        assert float((got[k].cpu().double() - want).abs().max()) <= 2.0 ** -13 * float(want.abs().max()), k

    # the rotation before the scan: L = <dy, y>, the scan's dB and dC through rotary_norm_backward
    q = {"B": r(b, T, G, N), "C": r(b, T, G, N), "bw": 1 + 0.1 * r(N), "cw": 1 + 0.1 * r(N)}
    x, dt, A, dy = r(b, T, H, P), torch.rand(b, T, H, generator=g) * 0.2, torch.rand(H, generator=g), r(b, T, H, P)
    freqs = weights(1)["freqs"]
    pos = torch.cat([torch.arange(m, dtype=torch.int32) for row in lens for m in row]).view(b, T)
    d = [t.cuda() for t in (q["B"], q["C"], q["bw"], q["cw"], freqs)]
    B, C = ssd.rotary_norm(*d, positions=pos.cuda(), eps=EPS)
    s = ssd.backward(x.cuda(), dt.cuda(), A.cuda(), B, C, dy.cuda(), seq_idx=ids, nseqs=n)
    got = ssd.rotary_norm_backward(*d, s["dB"], s["dC"], positions=pos.cuda(), eps=EPS)
    v = dict(zip(q, ref.leaves(*q.values())))
    out = []
    for k, wk in (("B", "bw"), ("C", "cw")):
        u = v[k].reshape(b * T, G, N)
        out.append(rr.rotate(u / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS) * v[wk], freqs, pos.reshape(-1), False)
                   .view(b, T, G, N).repeat_interleave(H // G, 2))
    loss = 0.0
    for row, t0, m in ref.sequences(b, T, lens):
        h = torch.zeros(H, P, N, dtype=torch.double)
        for t in range(t0, t0 + m):
            h = torch.exp(-dt[row, t].double() * torch.exp(A.double()))[:, None, None] * h + \
                x[row, t].double()[..., None] * out[0][row, t][:, None]
            loss = loss + ((h * out[1][row, t][:, None]).sum(-1) * dy[row, t].double()).sum()
    grads = dict(zip(v, torch.autograd.grad(loss, list(v.values()))))
    for k, name in (("B", "dB"), ("C", "dC"), ("bw", "db_weight"), ("cw", "dc_weight")):
        want = grads[k]
        assert float((got[name].cpu().double() - want).abs().max()) <= 2.0 ** -13 * float(want.abs().max()), k
