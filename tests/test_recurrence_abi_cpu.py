"""What the gated linear recurrence and the norm with rotation refuse, on the host before any HIP call."""
import ctypes

import pytest
import torch

import mamba_ssd_scan_chunked_amd as ssd

A = 0x10000000          # made-up device addresses, far apart: never read
STEP = 0x10000000


def call(name, p, order, workspace=None, **over):
    vals = {k: A + STEP * (i + 1) for i, k in enumerate(order)}
    vals.update(over)
    args = [vals[k] for k in order]
    if workspace is not None:
        args += list(workspace)
    return getattr(ssd.load_library(), name)(ctypes.byref(p), *args, None)


REC = dict(batch=2, seqlen=600, channels=64)
FWD = ["x", "r", "i", "A_log", "z", "init", "seq", "y", "final"]
BWD = ["x", "r", "i", "A_log", "z", "init", "seq", "dy", "dfinal", "dx", "dr", "di", "dA_log", "dz", "dinit"]
STP = ["x", "r", "i", "A_log", "z", "state", "state_out", "y"]


def rec(**kw):
    return ssd.recurrence_problem(**{**REC, **kw})


def room(p, back=False):
    n = (ssd.recurrence_backward_workspace_size if back else ssd.recurrence_workspace_size)(p)
    return (A + 40 * STEP if n else None, n)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), 2), (dict(seqlen=-1), 2), (dict(channels=0), 2), (dict(nseqs=-1), 2), (dict(ldx=63), 2),
    (dict(ldr=63), 2), (dict(ldi=0), 2), (dict(ldz=-64), 2), (dict(batch=1 << 31), 2), (dict(seqlen=1 << 31), 2),
    (dict(channels=1 << 31), 2), (dict(ldr=1 << 31), 2), (dict(dtype=2), 3), (dict(nseqs=1 << 31), 2),
    (dict(batch=1 << 30, nseqs=1 << 30, seqlen=1 << 30), 2), (dict(batch=1 << 20, nseqs=1 << 20, seqlen=1 << 20), 3),
])
def test_recurrence_problems(kw, code):
    p = rec(**kw)
    assert ssd.recurrence_workspace_size(p) == 0 and ssd.recurrence_backward_workspace_size(p) == 0
    assert call("ssd_recurrence_forward", p, FWD, (None, 0)) == code
    assert call("ssd_recurrence_backward", p, BWD, (None, 0)) == code


def test_recurrence_pointers():
    p = rec(nseqs=3)
    ws = room(p)
    for k in ("x", "r", "i", "A_log", "y"):
        assert call("ssd_recurrence_forward", p, FWD, ws, **{k: None}) == 1
    assert call("ssd_recurrence_forward", p, FWD, ws, seq=None) == 2            # nseqs must be the batch
    assert call("ssd_recurrence_forward", rec(nseqs=0), FWD, ws) == 2
    for k, a in (("x", 1), ("r", 1), ("i", 1), ("z", 1), ("y", 1), ("A_log", 2), ("init", 2), ("seq", 2), ("final", 2)):
        assert call("ssd_recurrence_forward", p, FWD, ws, **{k: A + 30 * STEP + a}) == 4
    same = A + 20 * STEP
    for a, b in (("y", "x"), ("y", "r"), ("y", "z"), ("final", "init"), ("final", "A_log"), ("y", "final"), ("y", "seq")):
        assert call("ssd_recurrence_forward", p, FWD, ws, **{a: same, b: same}) == 6
    if ws[1]:
        assert call("ssd_recurrence_forward", p, FWD, (None, 0)) == 5
        assert call("ssd_recurrence_forward", p, FWD, (ws[0], ws[1] - 1)) == 5
        assert call("ssd_recurrence_forward", p, FWD, (ws[0] + 64, ws[1])) == 4
        assert call("ssd_recurrence_forward", p, FWD, (same, ws[1]), y=same) == 6
        assert call("ssd_recurrence_forward", p, FWD, (same, ws[1]), x=same) == 6
    p.flags = 1
    assert call("ssd_recurrence_forward", p, FWD, ws) == 3
    assert ssd.load_library().ssd_recurrence_forward(None, *[None] * 10, 0, None) == 1
    assert ssd.recurrence_workspace_size(rec(seqlen=0)) == 0 and ssd.recurrence_backward_workspace_size(rec(seqlen=0)) == 0
    assert ssd.recurrence_workspace_size(rec(seqlen=1)) == 0


def test_recurrence_backward_pointers():
    p = rec(nseqs=3)
    ws = room(p, True)
    assert ws[1] > 0 and ws[1] % 256 == 0
    for k in ("x", "r", "i", "A_log", "dy", "dx", "dr", "di", "dA_log", "dz"):
        assert call("ssd_recurrence_backward", p, BWD, ws, **{k: None}) == 1
    assert call("ssd_recurrence_backward", p, BWD, (None, 0)) == 5
    assert call("ssd_recurrence_backward", p, BWD, (ws[0], ws[1] - 1)) == 5
    assert call("ssd_recurrence_backward", p, BWD, (ws[0] + 64, ws[1])) == 4
    for k in ("dy", "dfinal", "dx", "dr", "di", "dA_log", "dz", "dinit"):
        assert call("ssd_recurrence_backward", p, BWD, ws, **{k: A + 30 * STEP + 2}) == 4
    same = A + 20 * STEP
    for a, b in (("dx", "x"), ("dr", "dy"), ("di", "i"), ("dz", "z"), ("dinit", "dfinal"), ("dinit", "init"),
                 ("dA_log", "A_log"), ("dx", "dr"), ("di", "dz"), ("dinit", "dx")):
        assert call("ssd_recurrence_backward", p, BWD, ws, **{a: same, b: same}) == 6
    assert call("ssd_recurrence_backward", p, BWD, (same, ws[1]), dx=same) == 6


def test_recurrence_step_pointers():
    p = rec(seqlen=1)
    assert call("ssd_recurrence_step", rec(seqlen=2), STP) == 2
    assert call("ssd_recurrence_step", rec(seqlen=1, nseqs=3), STP) == 2
    assert call("ssd_recurrence_step", rec(seqlen=1, batch=1 << 15, channels=1 << 17), STP) == 3      # 2^32 threads
    for k in ("x", "r", "i", "A_log", "state", "state_out", "y"):
        assert call("ssd_recurrence_step", p, STP, **{k: None}) == 1
    assert call("ssd_recurrence_step", p, STP, state_out=A + 6 * STEP + 4) == 6     # state shifted by a channel
    assert call("ssd_recurrence_step", p, STP, y=A + 6 * STEP) == 6


ROT = dict(tokens=20, b_heads=2, c_heads=4, headdim=64, rotary_dim=32)
RF = ["B", "C", "bw", "cw", "freqs", "positions", "B_out", "C_out"]
RB = ["B", "C", "bw", "cw", "freqs", "positions", "dB_out", "dC_out", "dB", "dC", "dbw", "dcw"]


def rot(**kw):
    return ssd.rotary_problem(**{**ROT, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), 2), (dict(tokens=1 << 31), 2), (dict(b_heads=0), 2), (dict(c_heads=0), 2), (dict(headdim=0, rotary_dim=0), 2),
    (dict(rotary_dim=-2), 2), (dict(rotary_dim=31), 2), (dict(rotary_dim=66), 2), (dict(seqlen=0), 2), (dict(ldb=127), 2),
    (dict(ldc=255), 2), (dict(ldb=1 << 31), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2), (dict(headdim=1025), 3),
    (dict(dtype=2), 3), (dict(b_heads=1 << 31), 2), (dict(seqlen=(1 << 31) + 1), 2),
])
def test_rotary_problems(kw, code):
    assert ssd.rotary_norm_backward_workspace_size(rot(**kw)) == 0
    assert call("ssd_rotary_norm_forward", rot(**kw), RF) == code
    assert call("ssd_rotary_norm_backward", rot(**kw), RB, (None, 0)) == code


def test_rotary_pointers():
    p = rot()
    for k in ("B", "C", "bw", "cw", "freqs", "B_out", "C_out"):
        assert call("ssd_rotary_norm_forward", p, RF, **{k: None}) == 1
    for k, a in (("B", 1), ("C", 1), ("B_out", 1), ("C_out", 1), ("bw", 2), ("cw", 2), ("freqs", 2), ("positions", 2)):
        assert call("ssd_rotary_norm_forward", p, RF, **{k: A + 30 * STEP + a}) == 4
    same = A + 20 * STEP
    for a, b in (("B_out", "B"), ("B_out", "C"), ("C_out", "C"), ("B_out", "C_out"), ("C_out", "freqs"), ("B_out", "positions"),
                 ("C_out", "cw")):
        assert call("ssd_rotary_norm_forward", p, RF, **{a: same, b: same}) == 6
    p.flags = 2
    assert call("ssd_rotary_norm_forward", p, RF) == 3
    p.flags, p.reserved = 1, 1
    assert call("ssd_rotary_norm_forward", p, RF) == 3
    p = rot(tokens=5000)
    n = ssd.rotary_norm_backward_workspace_size(p)
    assert n > 0 and n % 256 == 0
    ws = (A + 40 * STEP, n)
    for k in ("B", "C", "bw", "cw", "freqs", "dB_out", "dC_out", "dB", "dC", "dbw", "dcw"):
        assert call("ssd_rotary_norm_backward", p, RB, ws, **{k: None}) == 1
    assert call("ssd_rotary_norm_backward", p, RB, (None, 0)) == 5
    assert call("ssd_rotary_norm_backward", p, RB, (ws[0], n - 1)) == 5
    assert call("ssd_rotary_norm_backward", p, RB, (ws[0] + 64, n)) == 4
    for a, b in (("dB", "B"), ("dC", "dC_out"), ("dB", "dC"), ("dbw", "dcw"), ("dbw", "bw")):
        assert call("ssd_rotary_norm_backward", p, RB, ws, **{a: same, b: same}) == 6
    assert call("ssd_rotary_norm_backward", p, RB, (same, n), dC=same) == 6


def test_tensors_must_be_on_a_gpu():
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError):
        ssd.gated_recurrence(x, x, x, x[0, 0])
    with pytest.raises(ValueError):
        ssd.gated_recurrence_step(x[0], x[0], x[0], x[0, 0], x[0])
    b = torch.zeros(2, 3, 1, 8)
    with pytest.raises(ValueError):
        ssd.rotary_norm(b, b, b[0, 0, 0], b[0, 0, 0], torch.ones(4))
