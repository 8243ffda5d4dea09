"""The gated norm and the residual norm with their gradients against their 64-bit forms."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def announce(msg):
    print("[case] " + msg, flush=True)


def gpu(v):
    return v.cuda() if torch.is_tensor(v) else v


def depth(size):
    """Roundings of a sum over a group: at most 32 terms in a lane, six steps in a wave,
    sixteen waves."""
    return min(size, 32) + 6 + 16


# x type, z and out type, rows, channels, group
GATED = [
    ("f32", "bf16", 5, 128, 128), ("f32", "f32", 5, 128, 128), ("bf16", "bf16", 3, 64, 64),
    ("f32", "bf16", 300, 48, 16), ("f32", "f32", 7, 1, 1), ("bf16", "bf16", 9, 105, 35), ("f32", "f32", 33, 264, 33),
    ("f32", "bf16", 4, 514, 257), ("f32", "f32", 2, 1023, 1023), ("f32", "bf16", 3, 5120, 5120),
    ("f32", "bf16", 2, 5120, 640), ("bf16", "bf16", 2, 8191, 8191), ("f32", "f32", 2, 9001, 9001),
    ("f32", "bf16", 2, 32768, 32768), ("f32", "f32", 1000, 8, 4),
]


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("case", GATED, ids=lambda c: "%s-%s-%dx%d-g%d" % c)
def test_gated(case, first):
    import mamba_ssd_scan_chunked_amd as ssd
    tx, tz, M, D, size = case
    announce("gated norm %s first=%s" % (case, first))
    g = torch.Generator().manual_seed(D + M)
    x, z = torch.randn(M, D, generator=g).to(TYPES[tx]), torch.randn(M, D, generator=g).to(TYPES[tz])
    w, dout = torch.randn(D, generator=g), torch.randn(M, D, generator=g)
    out = ssd.gated_norm(gpu(x), gpu(z), gpu(w), group_size=size, eps=EPS, gate_first=first)
    lv = ref.leaves(x, z, w)
    want = ref.gated(*lv, size, EPS, first)
    assert out.dtype == TYPES[tz]
    # every factor of the product: gate 6 roundings, rms depth/2 + 4, products 4
    n = depth(size)
    ref.check(out, want.detach(), want.detach().abs(), n + 14, "out")
    got = ssd.gated_norm_backward(gpu(x), gpu(z), gpu(w), gpu(dout), group_size=size, eps=EPS, gate_first=first)
    grads = torch.autograd.grad((want * dout.double()).sum(), lv)
    # du = r (e w - hat mean(e w hat)): two terms, each a product of factors as above; the
    # mean's terms by their magnitudes.  The gate's slope is below 1.1 and its terms' sizes below 2 + |z|.
    xd, zd, wd, dd = (t.detach().double() for t in (x, z, w, dout))
    gate = ref.silu(zd)
    u = xd * gate if first else xd
    e = dd if first else dd * gate
    r = 1 / torch.sqrt((u * u).unflatten(-1, (-1, size)).mean(-1) + EPS).repeat_interleave(size, -1)
    hat = u * r
    mean = (e * wd * hat).abs().unflatten(-1, (-1, size)).mean(-1).repeat_interleave(size, -1)
    du = r * ((e * wd).abs() + hat.abs() * mean)
    slope = 2 + zd.abs()
    ref.check(got["dx"], grads[0], du * (gate.abs() if first else 1), 4 * n + 40, "dx")
    ref.check(got["dz"], grads[1], (du * xd.abs() if first else (dd * hat * wd).abs()) * slope, 4 * n + 40, "dz")
    # rows: at least 8 in a team, then the teams 16 at a time
    ref.check(got["dweight"], grads[2], (e * hat).abs().sum(0), n + 20 + M, "dweight")


# type, rows, channels, residual given, scale given
RESIDUAL = [
    ("bf16", 4, 2560, True, False), ("f32", 4, 2560, True, True), ("bf16", 33, 77, False, True), ("f32", 3, 7, False, False),
    ("bf16", 1, 1, True, True), ("bf16", 700, 130, True, True), ("f32", 2, 12000, True, False), ("bf16", 9, 1024, True, True),
]


@pytest.mark.parametrize("case", RESIDUAL, ids=lambda c: "%s-%dx%d%s%s" % (c[:3] + ("-res" if c[3] else "", "-scale" if c[4] else "")))
def test_residual(case):
    import mamba_ssd_scan_chunked_amd as ssd
    dt, M, D, has_res, has_scale = case
    announce("residual norm %s" % (case,))
    g = torch.Generator().manual_seed(D + M)
    x = torch.randn(M, D, generator=g).to(TYPES[dt])
    res = torch.randn(M, D, generator=g) if has_res else None
    scale = torch.randn(D, generator=g) if has_scale else None
    w, dout, dres = torch.randn(D, generator=g), torch.randn(M, D, generator=g), torch.randn(M, D, generator=g)
    out, stream = ssd.residual_norm(gpu(x), gpu(res), gpu(w), scale=gpu(scale), eps=EPS)
    lv = ref.leaves(x, res, w, scale)
    want, u = ref.residual(*lv, EPS)
    terms = (x.double() * (1 if scale is None else scale.double())).abs() + (0 if res is None else res.double().abs())
    assert stream.dtype == torch.float32
    ref.check(stream, u.detach(), terms, 1, "residual_out")
    n = depth(D)
    r = 1 / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS).detach()
    # the stream's own rounding is relative to its two terms
    ref.check(out, want.detach(), terms * r * w.abs().double(), 2 * n + 10, "out")

    # gradients from the stream as it was rounded, which is what the call is given
    for later in (None, dres):
        got = ssd.residual_norm_backward(gpu(x), stream, gpu(w), gpu(dout), dresidual_out=gpu(later), scale=gpu(scale), eps=EPS)
        s, wl = ref.leaves(stream.cpu(), w)
        loss = (ref.residual(s, None, wl, None, EPS)[0] * dout.double()).sum()
        ds, dw = torch.autograd.grad(loss, (s, wl))
        hat = (s * r).detach()
        e = (dout * w).double()
        size = r * (e.abs() + hat.abs() * (e * hat).abs().mean(-1, keepdim=True))
        if later is not None:
            ds, size = ds + later.double(), size + later.double().abs()
        ref.check(got["dresidual"], ds, size, 3 * n + 30, "dresidual")
        ref.check(got["dweight"], dw, (dout.double() * hat).abs().sum(0), n + 20 + M, "dweight")
        if scale is None:
            assert got["dx"] is got["dresidual"] and "dscale" not in got
        else:
            ref.check(got["dx"], ds * scale.double(), size * scale.double().abs(), 3 * n + 31, "dx")
            ref.check(got["dscale"], (ds * x.double()).sum(0), (size * x.double().abs()).sum(0), 3 * n + 31 + M, "dscale")


def test_gradients_against_differences():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("norm differences")
    g = torch.Generator().manual_seed(3)
    base = [torch.randn(4, 24, generator=g), torch.randn(4, 24, generator=g), torch.randn(24, generator=g)]
    dout = torch.randn(4, 24, generator=g)
    for first in (True, False):
        got = ssd.gated_norm_backward(*[gpu(t) for t in base], gpu(dout), group_size=8, eps=EPS, gate_first=first)
        for i, name in enumerate(("dx", "dz", "dweight")):
            v, h = torch.randn(base[i].shape, generator=g).double(), 1e-5
            lo, hi = [t.double() for t in base], [t.double() for t in base]
            lo[i], hi[i] = lo[i] - h * v, hi[i] + h * v
            slope = float(((ref.gated(*hi, 8, EPS, first) - ref.gated(*lo, 8, EPS, first)) * dout.double()).sum()) / (2 * h)
            along = got[name].cpu().double() * v
            assert abs(float(along.sum()) - slope) <= 1e-5 * float(along.abs().sum()), name


def test_rows_of_zeros_and_in_place_stream():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("norm zeros, in place")
    z = torch.zeros(3, 40, device="cuda")
    w = torch.ones(40, device="cuda")
    assert not bool(ssd.gated_norm(z, z, w).any())
    g = ssd.gated_norm_backward(z, z, w, torch.ones_like(z))
    assert all(bool(torch.isfinite(t).all()) for t in g.values())
    x, res = torch.randn(6, 100, device="cuda").to(torch.bfloat16), torch.randn(6, 100, device="cuda")
    w = torch.randn(100, device="cuda")
    out0, new0 = ssd.residual_norm(x, res, w)
    stream = res.clone()
    out, new = ssd.residual_norm(x, stream, w, residual_out=stream)
    assert new is stream and torch.equal(stream, new0) and torch.equal(out, out0)


def test_slices_shapes_and_empty():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("norm slices")
    wide = torch.randn(2, 30, 211, device="cuda").to(torch.bfloat16)
    x, w = torch.randn(2, 30, 90, device="cuda"), torch.randn(90, device="cuda")
    z = wide[..., 17:107]
    a = ssd.gated_norm(x, z, w, group_size=45)
    assert a.shape == x.shape and torch.equal(a, ssd.gated_norm(x, z.contiguous(), w, group_size=45))
    g, h = (ssd.gated_norm_backward(x, v, w, x, group_size=45) for v in (z, z.contiguous()))
    assert all(torch.equal(g[k], h[k]) for k in g)
    out, res = ssd.residual_norm(z, None, w)
    assert torch.equal(out, ssd.residual_norm(z.contiguous(), None, w)[0]) and torch.equal(res, z.float())
    e = torch.empty(0, 90, device="cuda")
    assert ssd.gated_norm(e, e, w).shape == e.shape
    assert not bool(ssd.gated_norm_backward(e, e, w, e)["dweight"].any())
    g = ssd.residual_norm_backward(e, e, w, e, scale=w)
    assert not bool(g["dweight"].any()) and not bool(g["dscale"].any())


def test_graph_replays_equal_eager():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("norm graph")
    x, z = torch.randn(200, 640, device="cuda"), torch.randn(200, 640, device="cuda").to(torch.bfloat16)
    w, sc, d = torch.randn(640, device="cuda"), torch.randn(640, device="cuda"), torch.randn(200, 640, device="cuda")

    def run():
        out, res = ssd.residual_norm(z, x, w, scale=sc)
        g = ssd.gated_norm_backward(x, z, w, d, group_size=64)
        h = ssd.residual_norm_backward(z, res, w, d, d, scale=sc)
        return [ssd.gated_norm(x, z, w, group_size=64), out, res] + list(g.values()) + list(h.values())

    eager = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for _ in range(3):
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(outs, eager))


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows equal a call of their own."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("norm many rows")
    M, D, tail = 420000, 5376, 5
    x = torch.randn(4000, D, device="cuda").repeat(105, 1)
    z, w = x.to(torch.bfloat16), torch.randn(D, device="cuda")
    assert torch.equal(ssd.gated_norm(x, z, w)[-tail:], ssd.gated_norm(x[-tail:], z[-tail:], w))
    out, res = ssd.residual_norm(z, x, w)
    out1, res1 = ssd.residual_norm(z[-tail:], x[-tail:], w)
    assert torch.equal(out[-tail:], out1) and torch.equal(res[-tail:], res1)
    del out
    g = ssd.residual_norm_backward(z, res, w, x)
    assert torch.equal(g["dx"][-tail:], ssd.residual_norm_backward(z[-tail:], res1, w, x[-tail:])["dx"])


def test_arguments_are_checked():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("norm arguments")
    x, w = torch.zeros(6, 8, device="cuda"), torch.ones(8, device="cuda")
    h = x.bfloat16()
    for kind, f in (
            (TypeError, lambda: ssd.gated_norm(x.half(), x, w)), (TypeError, lambda: ssd.gated_norm(x, x.half(), w)),
            (TypeError, lambda: ssd.gated_norm(x, x, w.bfloat16())), (ValueError, lambda: ssd.gated_norm(x, x[:5], w)),
            (ValueError, lambda: ssd.gated_norm(x, x, w[:7])), (ValueError, lambda: ssd.gated_norm(x, x.cpu(), w)),
            (ssd.SSDError, lambda: ssd.gated_norm(x, x, w, group_size=3)), (ssd.SSDError, lambda: ssd.gated_norm(x, x, w, group_size=0)),
            (ssd.SSDError, lambda: ssd.gated_norm(h, x, w)), (ssd.SSDError, lambda: ssd.gated_norm(x, x, w, eps=-1.0)),
            (ssd.SSDError, lambda: ssd.gated_norm(x, x.clone(), w, out=x)), (TypeError, lambda: ssd.gated_norm(x, h, w, out=x.clone())),
            (ValueError, lambda: ssd.gated_norm_backward(x, x, w, x[:5])), (TypeError, lambda: ssd.residual_norm(x, h, w)),
            (ValueError, lambda: ssd.residual_norm(x, x[:5], w)), (ValueError, lambda: ssd.residual_norm(x, x, w, scale=w[:7])),
            (ValueError, lambda: ssd.residual_norm(x, x, w, residual_out=x[:5])),
            (ValueError, lambda: ssd.residual_norm(x[0, 0], None, w)),
            (ValueError, lambda: ssd.residual_norm_backward(x[0, 0], x[0, 0], w, x[0, 0])),
            (ValueError, lambda: ssd.residual_norm_backward(x, x[:5], w, x)),
            (TypeError, lambda: ssd.residual_norm_backward(x, x, w, x, dresidual_out=h))):
        with pytest.raises(kind):
            f()


def test_outputs_larger_than_the_caches():
    """Rows are independent, so those of a call whose fp32 outputs pass 32 MB (bf16 ones do not)
    equal those of a call below it, however either stores them."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("norms, outputs above and below 32 MB")
    D, M, few = 1030, 8400, 700
    assert M * D * 2 < 32 << 20 < M * D * 4
    g = torch.Generator(device="cuda").manual_seed(11)
    x, z, res, dout = (torch.randn(M, D, device="cuda", generator=g) for _ in range(4))
    w, scale = (torch.randn(D, device="cuda", generator=g) for _ in range(2))
    z = z.bfloat16()
    for first in (True, False):
        kw = dict(group_size=D // 2, gate_first=first)
        a, c = ssd.gated_norm_backward(x, z, w, dout, **kw), ssd.gated_norm_backward(x[:few], z[:few], w, dout[:few], **kw)
        assert torch.equal(a["dx"][:few], c["dx"]) and torch.equal(a["dz"][:few], c["dz"])
    a, c = ssd.residual_norm(z, res, w, scale), ssd.residual_norm(z[:few], res[:few], w, scale)
    assert torch.equal(a[0][:few], c[0]) and torch.equal(a[1][:few], c[1])
    ga, gc = (ssd.residual_norm_backward(z[:m], s, w, dout[:m], scale=scale) for m, s in ((M, a[1]), (few, c[1])))
    assert torch.equal(ga["dx"][:few], gc["dx"]) and torch.equal(ga["dresidual"][:few], gc["dresidual"])
