"""Gates over the whole range of their argument: sigmoid's exponential leaves fp32 below
-88.72, where silu and its slope are 0 to fp32, and the type's largest values are finite."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ROWS = 40


def announce(msg):
    print("[case] " + msg, flush=True)


def values(dt):
    """(ROWS, channels) values of the type: [-110, 110] in steps of 1/40, the border where e^-v
    leaves fp32 in steps of 1/1000, and far values up to the type's largest."""
    top = torch.finfo(TYPES[dt]).max
    far = torch.tensor([-1e4, 1e4, -1e30, 1e30, -top, top])
    v = torch.cat([torch.linspace(-110, 110, 8801), torch.linspace(-89.5, -87, 2501), far])
    v = torch.cat([v, torch.zeros(-v.numel() % ROWS)])
    return v.view(-1, ROWS).t().contiguous().to(TYPES[dt])


def gate(v):
    """silu, its slope and the sigmoid in 64 bits."""
    v = v.double()
    s = torch.sigmoid(v)
    return v * s, s * (1 + v * (1 - s)), s


def check(got, want, s, scale, n, what):
    """As ref.check, but where the sigmoid is below fp32's normal range (2^-126, a factor of
    two left for its own error) what it is a factor of may be anything between its value
    and zero."""
    got, scale = got.detach().cpu(), scale.double()
    assert torch.isfinite(got).all(), "%s: %d values are not finite" % (what, int((~torch.isfinite(got)).sum()))
    err = (got.double() - want).abs()
    bound = ref.half_step(got.dtype) * want.abs() + n * ref.U32 * scale
    bound = torch.where(s < 2.0 ** -125, 1.01 * want.abs(), bound)
    worst = float((err / bound.clamp(min=1e-300)).max())
    assert worst <= 1.0, "%s: error %.2f times its bound" % (what, worst)


# Roundings of the gate: the exponential 2 (the instruction) and 3 (its remainder), the sum 1,
# the reciprocal 2, the product 1; a bf16 result takes the plain exponential, whose argument
# is off by 2 U32 |v| (the product and log2 e; |v| up to 110, past which it is 0 or 1).
def value_roundings(v):
    return 12 + 2 * v.double().abs().clamp(max=110)


# The slope s (1 + v (1 - s)): s passes 9 roundings in each place and the rest 4; its terms are s and v s.
SLOPE = 32


def slope_size(v, s):
    return s * (1 + v.double().abs().clamp(max=110))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_convolution(dt):
    import mamba_ssd_scan_chunked_amd as ssd
    announce("conv gate %s" % dt)
    v = values(dt)
    D = v.shape[1]
    want, slope, s = gate(v)
    w = torch.tensor([0.0, 1.0]).repeat(D, 1).cuda()          # pre = the token itself
    x = v.cuda()[None]
    y, _ = ssd.causal_conv(x, w)
    check(y[0], want, s, value_roundings(v) * want.abs(), 1, "y")
    y = ssd.causal_conv_step(x[0], w, None, torch.zeros(ROWS, 1, D, device="cuda"))
    check(y, want, s, value_roundings(v) * want.abs(), 1, "y of a step")
    g = ssd.causal_conv_backward(x, w, torch.ones(1, ROWS, D, device="cuda"))
    check(g["dx"][0], slope, s, slope_size(v, s), SLOPE, "dx")
    assert all(bool(torch.isfinite(t).all()) for t in g.values())


@pytest.mark.parametrize("segments", [1, 2])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_selective_scan(dt, segments):
    import mamba_ssd_scan_chunked_amd as ssd
    announce("selective gate %s segments=%d" % (dt, segments))
    v = values(dt)
    D, N = v.shape[1], 8
    want, slope, s = gate(v)
    typ = TYPES[dt]
    x, step = torch.ones(1, ROWS, D, dtype=typ, device="cuda"), torch.full((1, ROWS, D), 0.5, dtype=typ, device="cuda")
    B = torch.zeros(1, ROWS, 1, N, dtype=typ, device="cuda")
    A, skip, z = torch.zeros(D, N, device="cuda"), torch.ones(D, device="cuda"), v.cuda()[None]
    y, _ = ssd.selective_scan(x, step, A, B, B, skip, z, segments=segments)
    check(y[0], want, s, value_roundings(v) * want.abs(), 1, "y")
    y = ssd.selective_step(x[0], step[0], A, B[0], B[0], skip, torch.zeros(ROWS, D, N, device="cuda"), z[0])
    check(y, want, s, value_roundings(v) * want.abs(), 1, "y of a step")
    g = ssd.selective_scan_backward(x, step, A, B, B, torch.ones(1, ROWS, D, device="cuda"), skip, z, segments=segments)
    check(g["dz"][0], slope, s, slope_size(v, s), SLOPE, "dz")
    check(g["dx"][0], want, s, value_roundings(v) * want.abs(), 1, "dx")
    assert all(bool(torch.isfinite(t).all()) for t in g.values())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gate_after_the_norm(dt):
    import mamba_ssd_scan_chunked_amd as ssd
    announce("gated norm, gate after, %s" % dt)
    v = values(dt)
    D = v.shape[1] // 4 * 4
    v = v[:, :D].contiguous()
    want, slope, s = gate(v)
    one = torch.ones(ROWS, D, device="cuda")                 # a norm of ones is 1 exactly
    args = (one, v.cuda(), one[0].contiguous())
    out = ssd.gated_norm(*args, group_size=4, eps=0.0, gate_first=False)
    check(out, want, s, value_roundings(v) * want.abs(), 1, "out")
    g = ssd.gated_norm_backward(*args, one, group_size=4, eps=0.0, gate_first=False)
    check(g["dz"], slope, s, slope_size(v, s), SLOPE, "dz")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gate_before_the_norm(dt):
    """Groups that are half closed (gates in [-110, -87]), and groups that are closed altogether."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("gated norm, gate first, %s" % dt)
    M, D, size, eps = 64, 64, 32, 1e-5
    g = torch.Generator().manual_seed(1)
    x, z = torch.randn(M, D, generator=g), torch.randn(M, D, generator=g)
    z[:, ::2] = -87 - 23 * torch.rand(M, D // 2, generator=g)
    z[: M // 2, :size] = -87 - 23 * torch.rand(M // 2, size, generator=g)
    z = z.to(TYPES[dt])
    w, dout = torch.randn(D, generator=g), torch.randn(M, D, generator=g)
    lv = ref.leaves(x, z, w)
    want = ref.gated(*lv, size, eps, True)
    dx, dz, dw = torch.autograd.grad((want * dout.double()).sum(), lv)
    args = (x.cuda(), z.cuda(), w.cuda())
    out = ssd.gated_norm(*args, group_size=size, eps=eps)
    # a closed gate is at most 110 e^-87 = 2e-36; a zero in its place moves out by that times |x| r |w|
    n = min(size, 32) + 6 + 16 + 14
    tiny = 1e-30 / ref.U32
    ref.check(out, want.detach(), want.detach().abs() * (1 if dt == "f32" else 3) + tiny, n, "out")
    got = ssd.gated_norm_backward(*args, dout.cuda(), group_size=size, eps=eps)
    gates = ref.silu(z.double())
    u = x.double() * gates
    r = 1 / torch.sqrt((u * u).unflatten(-1, (-1, size)).mean(-1) + eps).repeat_interleave(size, -1)
    e, hat = (dout * w).double(), u * r
    mean = (e * hat).abs().unflatten(-1, (-1, size)).mean(-1).repeat_interleave(size, -1)
    du = r * (e.abs() + hat.abs() * mean)
    ref.check(got["dx"], dx, du * gates.abs() + tiny, 4 * n + 40, "dx")
    # the slope's terms are at most s (1 + |v|), which is as small where the gate is closed
    s = torch.sigmoid(z.double())
    ref.check(got["dz"], dz, du * x.double().abs() * 2 * slope_size(z, s) + tiny, 4 * n + 40, "dz")
    ref.check(got["dweight"], dw, (dout.double() * hat).abs().sum(0) + tiny, n + 20 + M, "dweight")
