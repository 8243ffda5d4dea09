"""What the operators around the scan refuse, on the host before any HIP call."""
import ctypes

import pytest

import mamba_ssd_scan_chunked_amd as ssd

A = 0x10000000          # made-up device addresses, far apart: never read
STEP = 0x10000000


def call(name, p, order, workspace=None, **over):
    lib = ssd.load_library()
    vals = {k: A + STEP * (i + 1) for i, k in enumerate(order)}
    vals.update(over)
    args = [vals[k] for k in order]
    if workspace is not None:
        args += list(workspace)
    return getattr(lib, name)(ctypes.byref(p), *args, None)


CONV = dict(batch=2, seqlen=10, channels=64, width=4)
FWD = ["x", "weight", "bias", "init", "seq", "y", "final"]
BWD = ["x", "weight", "bias", "init", "seq", "dy", "dfinal", "dx", "dweight", "dbias", "dinit"]
STP = ["x", "weight", "bias", "state", "state_out", "y"]


def conv(**kw):
    return ssd.conv_problem(**{**CONV, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), 2), (dict(seqlen=-1), 2), (dict(channels=0), 2), (dict(nseqs=-1), 2), (dict(ldx=63), 2),
    (dict(batch=1 << 31), 2), (dict(seqlen=1 << 31), 2), (dict(channels=1 << 31), 2), (dict(ldx=1 << 31), 2),
    (dict(width=1), 3), (dict(width=5), 3), (dict(dtype=2), 3),
    (dict(batch=1 << 20, nseqs=1 << 20, seqlen=1 << 20, channels=64), 3),
])
def test_conv_problems(kw, code):
    assert call("ssd_conv_forward", conv(**kw), FWD) == code
    assert ssd.conv_backward_workspace_size(conv(**kw)) == 0


def test_conv_pointers():
    p = conv(nseqs=3)
    for k in ("x", "weight", "y"):
        assert call("ssd_conv_forward", p, FWD, **{k: None}) == 1
    assert call("ssd_conv_forward", p, FWD, seq=None) == 2                 # nseqs must be the batch
    assert call("ssd_conv_forward", conv(nseqs=0), FWD) == 2
    for k, a in (("x", 1), ("y", 1), ("weight", 2), ("bias", 2), ("init", 2), ("seq", 2), ("final", 2)):
        assert call("ssd_conv_forward", p, FWD, **{k: A + 9 * STEP + a}) == 4
    for a, b in (("y", "x"), ("y", "init"), ("final", "init"), ("final", "x"), ("y", "final"), ("y", "seq"), ("final", "weight")):
        same = A + 20 * STEP
        assert call("ssd_conv_forward", p, FWD, **{a: same, b: same}) == 6
    p.reserved = 1
    assert call("ssd_conv_forward", p, FWD) == 3
    p.reserved, p.flags = 0, 2
    assert call("ssd_conv_forward", p, FWD) == 3
    assert ssd.load_library().ssd_conv_forward(None, *[None] * 8) == 1


def test_conv_backward_pointers():
    p = conv(nseqs=3)
    n = ssd.conv_backward_workspace_size(p)
    assert n > 0 and n % 256 == 0 and ssd.conv_backward_workspace_size(conv(seqlen=0)) == 0
    assert ssd.conv_backward_workspace_size(conv(batch=1, seqlen=4)) == 0           # one run
    ws = (A + 40 * STEP, n)
    for k in ("x", "weight", "dy", "dx", "dweight"):
        assert call("ssd_conv_backward", p, BWD, ws, **{k: None}) == 1
    assert call("ssd_conv_backward", p, BWD, (None, 0)) == 5
    assert call("ssd_conv_backward", p, BWD, (A + 40 * STEP, n - 1)) == 5
    assert call("ssd_conv_backward", p, BWD, (A + 40 * STEP + 64, n)) == 4
    same = A + 20 * STEP
    for a, b in (("dx", "x"), ("dx", "dy"), ("dinit", "dfinal"), ("dinit", "init"), ("dweight", "weight"), ("dbias", "bias"),
                 ("dx", "dinit")):
        assert call("ssd_conv_backward", p, BWD, ws, **{a: same, b: same}) == 6
    assert call("ssd_conv_backward", p, BWD, (same, n), dx=same) == 6


def test_conv_step_pointers():
    p = conv(seqlen=1)
    assert call("ssd_conv_step", conv(seqlen=2), STP) == 2
    assert call("ssd_conv_step", conv(seqlen=1, nseqs=3), STP) == 2
    assert call("ssd_conv_step", conv(seqlen=1, batch=1 << 20, channels=1 << 12), STP) == 3      # 2^32 threads
    for k in ("x", "weight", "state", "state_out", "y"):
        assert call("ssd_conv_step", p, STP, **{k: None}) == 1
    assert call("ssd_conv_step", p, STP, state_out=A + 4 * STEP + 4) == 6   # state shifted by a channel
    assert call("ssd_conv_step", p, STP, y=A + 4 * STEP) == 6


NORM = dict(rows=4, channels=64, group_size=32)
GF, GB = ["x", "z", "weight", "out"], ["x", "z", "weight", "dout", "dx", "dz", "dweight"]
RF = ["x", "res", "weight", "scale", "out", "res_out"]
RB = ["x", "res_out", "weight", "scale", "dout", "dres_out", "dx", "dres", "dweight", "dscale"]


def norm(**kw):
    return ssd.norm_problem(**{**NORM, **kw})


def stream(**kw):
    return ssd.norm_problem(**{**dict(rows=4, channels=64, x_dtype=ssd.DTYPE_BF16), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 2), (dict(channels=0, group_size=1), 2), (dict(group_size=0), 2), (dict(group_size=48), 2),
    (dict(ldx=63), 2), (dict(ldz=63), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2), (dict(rows=1 << 31), 2),
    (dict(x_dtype=5), 3), (dict(dtype=5), 3), (dict(x_dtype=1, dtype=0), 3),
    (dict(channels=40000, group_size=40000), 3), (dict(rows=1 << 24, channels=4096, group_size=4096), 3), (dict(channels=1 << 30, group_size=1), 3),
])
def test_norm_problems(kw, code):
    assert call("ssd_gated_norm_forward", norm(**kw), GF) == code
    assert ssd.gated_norm_backward_workspace_size(norm(**kw)) == 0


def test_gated_norm_pointers():
    p = norm()
    for k in GF:
        assert call("ssd_gated_norm_forward", p, GF, **{k: None}) == 1
    assert call("ssd_gated_norm_forward", p, GF, x=A + 2) == 4 and call("ssd_gated_norm_forward", p, GF, z=A + 1) == 4
    for k in ("x", "z", "weight"):
        assert call("ssd_gated_norm_forward", p, GF, out=A, **{k: A}) == 6
    assert ssd.gated_norm_backward_workspace_size(p) == 0                          # few rows: one team per group
    p = norm(rows=40)
    n = ssd.gated_norm_backward_workspace_size(p)
    ws = (A + 40 * STEP, n)
    assert n > 0 and call("ssd_gated_norm_backward", p, GB, (None, 0)) == 5
    for k in GB:
        assert call("ssd_gated_norm_backward", p, GB, ws, **{k: None}) == 1
    for a, b in (("dx", "x"), ("dz", "z"), ("dx", "dout"), ("dx", "dz"), ("dweight", "weight")):
        assert call("ssd_gated_norm_backward", p, GB, ws, **{a: A, b: A}) == 6
    p.flags = 2
    assert call("ssd_gated_norm_forward", p, GF) == 3


def test_residual_norm_pointers():
    p = stream()
    assert call("ssd_residual_norm_forward", norm(x_dtype=1), RF) == 3            # groups
    assert call("ssd_residual_norm_forward", stream(x_dtype=0), RF) == 3
    for k in ("x", "weight", "out", "res_out"):
        assert call("ssd_residual_norm_forward", p, RF, **{k: None}) == 1
    assert call("ssd_residual_norm_forward", p, RF, res_out=A, res=A + 4) == 6     # shifted
    assert call("ssd_residual_norm_forward", stream(ldz=80), RF, res_out=A, res=A) == 6
    assert call("ssd_residual_norm_forward", p, RF, out=A, x=A) == 6
    assert ssd.residual_norm_backward_workspace_size(p, True) == 0
    p = stream(rows=40)
    n = ssd.residual_norm_backward_workspace_size(p, True)
    assert n == 2 * ssd.residual_norm_backward_workspace_size(p, False) > 0
    ws = (A + 40 * STEP, n)
    for k in ("x", "res_out", "weight", "dout", "dx", "dres", "dweight", "dscale"):
        assert call("ssd_residual_norm_backward", p, RB, ws, **{k: None}) == 1
    assert call("ssd_residual_norm_backward", p, RB, (A + 40 * STEP, n - 1)) == 5
    for a, b in (("dx", "x"), ("dres", "res_out"), ("dres", "dout"), ("dres", "dres_out"), ("dx", "dres"), ("dscale", "scale")):
        assert call("ssd_residual_norm_backward", p, RB, ws, **{a: A, b: A}) == 6


def test_binding_refuses_on_the_cpu():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    for f in (lambda: ssd.causal_conv(x, w), lambda: ssd.causal_conv_backward(x, w, x),
              lambda: ssd.causal_conv_step(x[:, 0], w, None, torch.zeros(1, 3, 8)), lambda: ssd.gated_norm(x, x, w[:, 0]),
              lambda: ssd.gated_norm_backward(x, x, w[:, 0], x), lambda: ssd.residual_norm(x, x, w[:, 0]),
              lambda: ssd.residual_norm_backward(x, x, w[:, 0], x), lambda: ssd.selective_scan(x, x, w, x, x),
              lambda: ssd.selective_scan_backward(x, x, w, x, x, x), lambda: ssd.selective_step(x, x, w, x, x, None, x)):
        with pytest.raises(ValueError):
            f()


SEL = dict(batch=2, seqlen=40, channels=64, dstate=16)
SF = ["x", "dt", "dt_bias", "A_log", "B", "C", "D", "z", "init", "seq", "y", "final"]
SB = ["x", "dt", "dt_bias", "A_log", "B", "C", "D", "z", "init", "seq", "dy", "dfinal", "dx", "ddt", "dA_log", "dB", "dC",
      "dD", "dz", "dinit", "ddt_bias"]
SS = ["x", "dt", "dt_bias", "A_log", "B", "C", "D", "z", "state", "state_out", "y"]
NONE = (None, 0)


def sel(**kw):
    return ssd.selective_problem(**{**SEL, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), 2), (dict(seqlen=-1), 2), (dict(channels=0), 2), (dict(dstate=0), 2), (dict(ngroups=0), 2),
    (dict(ngroups=3), 2), (dict(segments=-1), 2), (dict(nseqs=-1), 2), (dict(seqlen=1 << 31), 2),
    (dict(ldx=63), 2), (dict(lddt=63), 2), (dict(ldz=63), 2), (dict(ldb=15), 2), (dict(ldc=15), 2), (dict(ldx=1 << 31), 2),
    (dict(dtype=3), 3), (dict(dstate=12), 3), (dict(dstate=128), 3),
    # a tile is addressed with 32-bit byte offsets
    (dict(ldx=1 << 25), 3), (dict(lddt=1 << 25), 3), (dict(ldz=1 << 25), 3), (dict(ldb=1 << 25), 3), (dict(ldc=1 << 25), 3),
    (dict(channels=1 << 25), 3),
    (dict(batch=1 << 30, nseqs=1 << 30, seqlen=1 << 30), 2), (dict(nseqs=1 << 30, channels=1 << 24, dstate=64), 2),
    (dict(batch=1 << 20, nseqs=1 << 20, channels=1 << 14), 3),
])
def test_selective_problems(kw, code):
    assert call("ssd_selective_forward", sel(**kw), SF, NONE) == code
    assert ssd.selective_workspace_size(sel(**kw)) == 0 and ssd.selective_backward_workspace_size(sel(**kw)) == 0


def test_selective_workspaces():
    assert ssd.selective_workspace_size(sel(seqlen=16)) == 0                       # one tile: not cut
    assert ssd.selective_workspace_size(sel(batch=8, channels=8192)) == 0          # the channels fill the chip
    p = sel(seqlen=100, segments=3)                                                # 4 tiles of 32: two segments
    assert ssd.selective_workspace_size(p) == 2 * 64 * 16 * 4 + 2 * 64 * 4
    assert ssd.selective_backward_workspace_size(sel(seqlen=0)) == 0
    n = ssd.selective_workspace_size(p)
    p.nseqs = 3
    assert call("ssd_selective_forward", p, SF, NONE) == 5
    assert call("ssd_selective_forward", p, SF, (A + 40 * STEP, n - 1)) == 5
    assert call("ssd_selective_forward", p, SF, (A + 40 * STEP + 16, n)) == 4
    assert call("ssd_selective_forward", p, SF, (A, n), y=A + 30 * STEP, x=A) == 6


def test_selective_pointers():
    p = sel(nseqs=3, segments=1)
    for k in ("x", "dt", "A_log", "B", "C", "y"):
        assert call("ssd_selective_forward", p, SF, NONE, **{k: None}) == 1
    assert call("ssd_selective_forward", p, SF, NONE, seq=None) == 2
    assert call("ssd_selective_forward", sel(nseqs=0, segments=1), SF, NONE) == 2
    for k in ("x", "dt", "B", "C", "z", "y"):
        assert call("ssd_selective_forward", p, SF, NONE, **{k: A + 30 * STEP + 1}) == 4
    same = A + 30 * STEP
    for a, b in (("y", "x"), ("y", "dt"), ("y", "z"), ("y", "B"), ("final", "init"), ("final", "A_log"), ("y", "final")):
        assert call("ssd_selective_forward", p, SF, NONE, **{a: same, b: same}) == 6
    p.flags = 1
    assert call("ssd_selective_forward", p, SF, NONE) == 3
    p.flags, p.reserved = 0, 1
    assert call("ssd_selective_forward", p, SF, NONE) == 3


def test_selective_backward_pointers():
    p = sel(nseqs=3)
    n = ssd.selective_backward_workspace_size(p)
    ws = (A + 40 * STEP, n)
    assert n > 0
    for k in ("x", "dt", "A_log", "B", "C", "dy", "dx", "ddt", "dA_log", "dB", "dC", "dz"):
        assert call("ssd_selective_backward", p, SB, ws, **{k: None}) == 1
    assert call("ssd_selective_backward", p, SB, NONE) == 5
    assert call("ssd_selective_backward", p, SB, (A + 40 * STEP, n - 1)) == 5
    same = A + 30 * STEP
    for a, b in (("dx", "dy"), ("ddt", "dt"), ("dB", "B"), ("dC", "dB"), ("dinit", "dfinal"), ("dz", "z"), ("dA_log", "A_log"),
                 ("dD", "D"), ("ddt_bias", "dt_bias")):
        assert call("ssd_selective_backward", p, SB, ws, **{a: same, b: same}) == 6


def test_selective_step_pointers():
    p = sel(seqlen=1)
    assert call("ssd_selective_step", sel(), SS) == 2 and call("ssd_selective_step", sel(seqlen=1, nseqs=3), SS) == 2
    for k in ("x", "dt", "A_log", "B", "C", "state", "state_out", "y"):
        assert call("ssd_selective_step", p, SS, **{k: None}) == 1
    assert call("ssd_selective_step", p, SS, state_out=A + 9 * STEP + 4) == 6
    assert call("ssd_selective_step", p, SS, y=A + 9 * STEP) == 6
