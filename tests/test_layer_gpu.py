"""The operators run together as a Mamba layer uses them: prompt, single tokens, gradients."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

EPS = 1e-5


def announce(msg):
    print("[case] " + msg, flush=True)


def weights(H, P, N, G, seed):
    g = torch.Generator().manual_seed(seed)
    D, W = H * P, H * P + 2 * G * N
    return {"conv": torch.randn(W, 4, generator=g) / 2, "cbias": torch.randn(W, generator=g) * 0.1,
            "A_log": torch.rand(H, generator=g) * 2, "D": torch.randn(H, generator=g), "bias": torch.randn(H, generator=g) - 1,
            "norm": 1 + 0.1 * torch.randn(D, generator=g), "pre": 1 + 0.1 * torch.randn(24, generator=g)}


def mamba2_prompt(ssd, w, proj, dt, H, P, N, G, ids, n, conv0, state0):
    """Projection rows (b,T, D + D+2GN): gate z, then the convolved x, B, C."""
    b, T = proj.shape[:2]
    D = H * P
    xbc, conv = ssd.causal_conv(proj[..., D:], w["conv"], w["cbias"], conv0, ids, n)
    x, B, C = xbc.split([D, G * N, G * N], -1)
    y, state = ssd.forward(x.reshape(b, T, H, P), dt, w["A_log"], B.reshape(b, T, G, N), C.reshape(b, T, G, N), w["D"],
                           init_state=state0, seq_idx=ids, nseqs=n, dt_scales_x=True, dt_bias=w["bias"], dt_softplus=True)
    return ssd.gated_norm(y.flatten(-2), proj[..., :D], w["norm"], group_size=D // G, eps=EPS), conv, state


@pytest.mark.parametrize("dt_", ["bf16", "f32"])
def test_mamba2_prompt_then_tokens(dt_):
    """A prompt followed by single tokens equals the whole prompt, and packed rows equal
    their sequences run alone."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("mamba2 layer %s" % dt_)
    H, P, N, G, b, T, K = 4, 32, 64, 2, 2, 50, 6
    D = H * P
    typ = torch.bfloat16 if dt_ == "bf16" else torch.float32
    w = {k: v.cuda() for k, v in weights(H, P, N, G, 1).items()}
    g = torch.Generator().manual_seed(2)
    proj = torch.randn(b, T + K, 2 * D + 2 * G * N, generator=g).to(typ).cuda()
    dt = torch.randn(b, T + K, H, generator=g).cuda()
    whole, conv1, state1 = mamba2_prompt(ssd, w, proj, dt, H, P, N, G, None, None, None, None)
    out, conv, state = mamba2_prompt(ssd, w, proj[:, :T], dt[:, :T], H, P, N, G, None, None, None, None)
    outs = [out]
    for t in range(T, T + K):
        row = proj[:, t]
        xbc = ssd.causal_conv_step(row[:, D:], w["conv"], w["cbias"], conv)
        x, B, C = xbc.split([D, G * N, G * N], -1)
        y = ssd.step(x.reshape(b, H, P), dt[:, t], w["A_log"], B.reshape(b, G, N), C.reshape(b, G, N), w["D"], state,
                     dt_scales_x=True, dt_bias=w["bias"], dt_softplus=True)
        outs.append(ssd.gated_norm(y.reshape(b, 1, D), row[:, None, :D], w["norm"], group_size=D // G, eps=EPS))
    got = torch.cat(outs, 1)
    assert torch.equal(conv, conv1)
    # the scan's own tolerances (2e-2 and 1e-5 of the largest value) carry over to its norm
    tol = 2e-2 if dt_ == "bf16" else 1e-5
    assert float((got.float() - whole.float()).abs().max()) <= 2 * tol * float(whole.float().abs().max())
    assert float((state - state1).abs().max()) <= tol * float(state1.abs().max())

    ids = ref.ids_of(b, T + K, [[20, 36], [1, 55]]).cuda()
    packed, conv, state = mamba2_prompt(ssd, w, proj, dt, H, P, N, G, ids, 4, None, None)
    for k, (r, t, n) in enumerate(ref.sequences(b, T + K, [[20, 36], [1, 55]])):
        o, c, s = mamba2_prompt(ssd, w, proj[r:r + 1, t:t + n], dt[r:r + 1, t:t + n], H, P, N, G, None, None, None, None)
        assert float((o[0].float() - packed[r, t:t + n].float()).abs().max()) <= 2 * tol * float(packed.float().abs().max())
        assert torch.equal(c[0], conv[k])
        assert float((s[0] - state[k]).abs().max()) <= tol * float(state.abs().max())


def test_mamba1_layer_gradients():
    """residual_norm -> projection -> causal_conv -> selective_scan with its gate, forwards and
    backwards in fp32, against autograd through the 64-bit forms."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("mamba1 layer gradients")
    b, T, M, D, N, R = 2, 30, 24, 40, 16, 3
    lens = [[12, 18], [1, 29]]
    n = 4
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g)      # noqa: E731
    p = {"h": r(b, T, M), "res": r(b, T, M), "pre": r(M), "win": r(M, 2 * D) / M ** 0.5, "conv": r(D, 4) / 2, "cb": r(D),
         "wx": r(D, R + 2 * N) / D ** 0.5, "wdt": r(R, D), "A_log": torch.rand(D, N, generator=g), "skip": r(D), "bias": r(D)}
    dout, dres = r(b, T, D), r(b, T, M)
    ids = ref.ids_of(b, T, lens).cuda()
    q = {k: v.cuda() for k, v in p.items()}

    normed, stream = ssd.residual_norm(q["h"], q["res"], q["pre"], eps=EPS)
    proj = normed @ q["win"]
    xc, _ = ssd.causal_conv(proj[..., :D], q["conv"], q["cb"], seq_idx=ids, nseqs=n)
    dbc = xc @ q["wx"]
    low, B, C = dbc[..., :R], dbc[..., R:R + N].unflatten(-1, (1, N)), dbc[..., R + N:].unflatten(-1, (1, N))
    dt = low @ q["wdt"]
    kw = dict(D=q["skip"], z=proj[..., D:], seq_idx=ids, nseqs=n, dt_bias=q["bias"], dt_softplus=True)
    y, _ = ssd.selective_scan(xc, dt, q["A_log"], B, C, **kw)

    s = ssd.selective_scan_backward(xc, dt, q["A_log"], B, C, dout.cuda(), **kw)
    dlow = s["ddt"] @ q["wdt"].t()
    ddbc = torch.cat([dlow, s["dB"].flatten(-2), s["dC"].flatten(-2)], -1)
    c = ssd.causal_conv_backward(proj[..., :D], q["conv"], s["dx"] + ddbc @ q["wx"].t(), q["cb"], seq_idx=ids, nseqs=n)
    dproj = torch.cat([c["dx"], s["dz"]], -1)
    f = ssd.residual_norm_backward(q["h"], stream, q["pre"], dproj @ q["win"].t(), dres.cuda(), eps=EPS)
    got = {"h": f["dx"], "res": f["dresidual"], "pre": f["dweight"], "win": normed.flatten(0, 1).t() @ dproj.flatten(0, 1),
           "conv": c["dweight"], "cb": c["dbias"], "wx": xc.flatten(0, 1).t() @ ddbc.flatten(0, 1),
           "wdt": low.flatten(0, 1).t() @ s["ddt"].flatten(0, 1), "A_log": s["dA_log"], "skip": s["dD"], "bias": s["ddt_bias"]}

    v = dict(zip(p, ref.leaves(*p.values())))
    normed, stream = ref.residual(v["h"], v["res"], v["pre"], None, EPS)
    proj = normed @ v["win"]
    zero = torch.zeros(n, 3, D, dtype=torch.double)
    xc, _ = ref.conv(proj[..., :D], v["conv"], v["cb"], zero, lens, True)
    dbc = xc @ v["wx"]
    B, C = dbc[..., R:R + N].unflatten(-1, (1, N)), dbc[..., R + N:].unflatten(-1, (1, N))
    yr, _ = ref.scan(xc, dbc[..., :R] @ v["wdt"], v["A_log"], B, C, v["skip"], proj[..., D:],
                     torch.zeros(n, D, N, dtype=torch.double), v["bias"], True, lens)
    grads = dict(zip(v, torch.autograd.grad((yr * dout.double()).sum() + (stream * dres.double()).sum(), list(v.values()))))
    # seven products and operators in fp32, each within a few hundred roundings (2^-24) of
    # the largest value that it handles: 2^-13 of the largest gradient covers 2048 of them
    assert float((y.cpu().double() - yr.detach()).abs().max()) <= 2.0 ** -13 * float(yr.detach().abs().max())
    for k, want in grads.items():
        assert float((got[k].cpu().double() - want).abs().max()) <= 2.0 ** -13 * float(want.abs().max()), k
