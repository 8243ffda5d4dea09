"""The selective scan (whole rows, gradients, single tokens) against its 64-bit form."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def announce(msg):
    print("[case] " + msg, flush=True)


def gpu(v):
    return v.cuda() if torch.is_tensor(v) else v


def make(dt, b, T, D, N, G=1, lens=None, state=True, gate=True, soft=True, skip=True, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g)

    typ = TYPES[dt]
    n = len(ref.sequences(b, T, lens))
    q = {"x": normal(b, T, D).to(typ), "B": (normal(b, T, G, N) / N ** 0.5).to(typ), "C": normal(b, T, G, N).to(typ),
         "A_log": torch.rand(D, N, generator=g) * 3 - 1, "D": normal(D) if skip else None,
         "z": normal(b, T, D).to(typ) if gate else None, "init": normal(n, D, N) if state else None,
         "dy": normal(b, T, D), "dfinal": normal(n, D, N) if state else None, "ids": ref.ids_of(b, T, lens),
         "lens": lens, "n": n, "soft": soft}
    if soft:
        q["dt"], q["bias"] = (normal(b, T, D) - 1).to(typ), normal(D)
    else:
        q["dt"], q["bias"] = (torch.rand(b, T, D, generator=g) * 0.5).to(typ), None
    return q


def more(q, **kw):
    return dict(D=gpu(q["D"]), z=gpu(q["z"]), init_state=gpu(q["init"]), seq_idx=gpu(q["ids"]),
                nseqs=q["n"] if q["ids"] is not None else None, dt_bias=gpu(q["bias"]), dt_softplus=q["soft"], **kw)


def forward(q, **kw):
    import mamba_ssd_scan_chunked_amd as ssd
    return ssd.selective_scan(*[gpu(q[k]) for k in ("x", "dt", "A_log", "B", "C")], **more(q, **kw))


def backward(q, **kw):
    import mamba_ssd_scan_chunked_amd as ssd
    return ssd.selective_scan_backward(*[gpu(q[k]) for k in ("x", "dt", "A_log", "B", "C", "dy")],
                                       dfinal=gpu(q["dfinal"]), **more(q, **kw))


ORDER = ("x", "dt", "A_log", "B", "C", "D", "z", "init", "bias")
NAMES = ("dx", "ddt", "dA_log", "dB", "dC", "dD", "dz", "dinit", "ddt_bias")


def full(q):
    """The nine inputs in 64 bits, zeros for those not given (z stays None)."""
    D, N = q["A_log"].shape
    d = {**q, "D": torch.zeros(D) if q["D"] is None else q["D"], "bias": torch.zeros(D) if q["bias"] is None else q["bias"],
         "init": torch.zeros(q["n"], D, N) if q["init"] is None else q["init"]}
    return [None if d[k] is None else d[k].double() for k in ORDER]


def reference(q, grads=False):
    """(values, sizes): y and final, or the gradients by name, and the sums of magnitudes."""
    values = full(q)
    sizes = [v if v is None or k in ("dt", "A_log", "bias", "z") else v.abs() for k, v in zip(ORDER, values)]
    out = []
    for f, args in ((ref.scan, values), (ref.scan_sizes, sizes)):
        lv = ref.leaves(*args)
        y, final = f(*lv, q["soft"], q["lens"])
        if not grads:
            out.append((y.detach(), final.detach()))
            continue
        dy = q["dy"].double()
        dfin = torch.zeros_like(final) if q["dfinal"] is None else q["dfinal"].double()
        if f is ref.scan_sizes:
            dy, dfin = dy.abs(), dfin.abs()
        loss = (y * dy).sum() + (final * dfin).sum()
        wanted = [(k, t) for k, t in zip(NAMES, lv) if t is not None]
        out.append(dict(zip([k for k, _ in wanted], torch.autograd.grad(loss, [t for _, t in wanted]))))
    return out


def longest(q):
    return max(n for _, _, n in ref.sequences(*q["x"].shape[:2], q["lens"]))


CASES = [
    # dtype, rows, tokens, channels, N, G, lengths, state, gate, softplus, skip
    ("bf16", 2, 37, 64, 16, 1, None, True, True, True, True),
    ("f32", 2, 37, 64, 16, 1, None, True, True, True, True),
    ("f32", 1, 1, 5, 8, 1, None, True, True, True, True),
    ("bf16", 1, 1, 130, 16, 1, None, False, False, False, False),
    ("f32", 1, 16, 65, 8, 1, None, True, False, True, False),
    ("f32", 1, 17, 66, 32, 3, None, False, True, True, True),
    ("bf16", 2, 50, 30, 64, 2, None, True, True, False, True),
    ("f32", 1, 45, 129, 16, 1, [[1, 1, 2, 12, 16, 13]], True, True, True, True),
    ("bf16", 2, 40, 70, 32, 2, [[7, 33], [1, 38, 1]], True, True, True, True),
    ("f32", 2, 33, 20, 64, 1, [[8, 8, 17], [33]], False, False, True, True),
    ("f32", 1, 24, 10, 8, 2, [[8, 8, 8]], True, True, False, True),
]
IDS = ["%s-b%d-T%d-D%d-N%d-G%d-%s" % (c[:6] + ("packed" if c[6] else "rows",)) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    announce("selective forward %s" % (case,))
    q = make(*case)
    (yr, fr), (ys, fs) = reference(q)
    y, f = forward(q)
    # per token a term passes the decay (argument, exp2 and the rate's own roundings: 6) and
    # two more roundings; then the read-out, the gate (8)
    n = 8 * longest(q)
    ref.check(y, yr, ys, n + q["A_log"].shape[1] + 12, "y")
    ref.check(f, fr, fs, n + 8, "final")


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    announce("selective backward %s" % (case,))
    q = make(*case, seed=1)
    grads, sizes = reference(q, grads=True)
    got = backward(q)
    assert set(got) == set(grads)
    # a term passes the tokens of its sequence forwards and backwards, 8 roundings each, the
    # gate and its slope, and a sum: over states, channels (64 in a wave, then blocks) or tokens
    b, T, D = q["x"].shape
    extra = {"dB": 6 + D // 64 + 1, "dC": 6 + D // 64 + 1, "dA_log": T + b, "dD": T + b, "ddt_bias": T + b}
    for k in grads:
        ref.check(got[k], grads[k], sizes[k], 16 * longest(q) + q["A_log"].shape[1] + 40 + extra.get(k, 0), k)


@pytest.mark.parametrize("segments", [1, 2, 3, 7])
@pytest.mark.parametrize("lens", [None, [[16, 1, 31, 52], [99, 1]]])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_segments(segments, lens, dt):
    announce("selective segments %d %s %s" % (segments, lens, dt))
    q = make(dt, 2, 100, 70, 16, 1, lens, seed=2)
    (yr, fr), (ys, fs) = reference(q)
    y, f = forward(q, segments=segments)
    n = 8 * longest(q)
    ref.check(y, yr, ys, n + 40, "y")
    ref.check(f, fr, fs, n + 20, "final")
    grads, sizes = reference(q, grads=True)
    got = backward(q, segments=segments)
    for k in grads:
        ref.check(got[k], grads[k], sizes[k], 2 * n + 200, k)


def test_segments_with_larger_states():
    announce("selective segments N=32, 64")
    for N, D in ((32, 40), (64, 65)):
        q = make("f32", 1, 70, D, N, 1, [[20, 50]], seed=3)
        grads, sizes = reference(q, grads=True)
        got = backward(q, segments=3)
        for k in grads:
            ref.check(got[k], grads[k], sizes[k], 16 * 50 + 200, k)


@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_many_rows(N):
    """More than three 64-channel workgroups for every compute unit: the wider shape."""
    announce("selective many rows N=%d" % N)
    q = make("f32", 800, 3, 20, N, 1, seed=16)
    (yr, fr), (ys, fs) = reference(q)
    y, f = forward(q)
    ref.check(y, yr, ys, 8 * 3 + N + 12, "y")
    ref.check(f, fr, fs, 8 * 3 + 8, "final")


def test_gradients_against_differences():
    announce("selective differences")
    q = make("f32", 1, 24, 12, 8, 2, [[5, 1, 18]], seed=4)
    got = backward(q)
    base = full(q)

    def loss(args):
        y, f = ref.scan(*args, q["soft"], q["lens"])
        return float((y * q["dy"].double()).sum() + (f * q["dfinal"].double()).sum())

    g = torch.Generator().manual_seed(5)
    for i, name in enumerate(NAMES):
        v, h = torch.randn(base[i].shape, generator=g).double(), 1e-5
        lo, hi = list(base), list(base)
        lo[i], hi[i] = base[i] - h * v, base[i] + h * v
        slope = (loss(hi) - loss(lo)) / (2 * h)
        along = got[name].cpu().double() * v
        # differences: h^2 of the third derivative and 2^-52 |loss| / h; the kernel: fp32 gradients
        assert abs(float(along.sum()) - slope) <= 2e-5 * float(along.abs().sum()), name


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("in_place", [False, True])
def test_steps_continue_a_prompt(dt, N, in_place):
    import mamba_ssd_scan_chunked_amd as ssd
    announce("selective steps %s N=%d" % (dt, N))
    q = make(dt, 3, 20, 38, N, 2, seed=6)
    d = {k: gpu(v) for k, v in q.items()}
    (yr, fr), (ys, fs) = reference(q)
    head = {k: v[:, :13] if torch.is_tensor(v) and v.dim() > 2 and k not in ("init", "dfinal") else v for k, v in q.items()}
    _, state = forward(head)
    for t in range(13, 20):
        args = [d[k][:, t] if k not in ("A_log",) else d[k] for k in ("x", "dt", "A_log", "B", "C")]
        kw = dict(z=d["z"][:, t], dt_bias=d["bias"], dt_softplus=True)
        if in_place:
            y = ssd.selective_step(*args, d["D"], state, **kw)
        else:
            old, new = state.clone(), torch.empty_like(state)
            y = ssd.selective_step(*args, d["D"], state, state_out=new, **kw)
            assert torch.equal(state, old)
            state = new
        ref.check(y, yr[:, t], ys[:, t], 8 * 20 + N + 12, "y of a step")
    ref.check(state, fr, fs, 8 * 20 + 8, "state")


def test_long_steps_and_extreme_decays():
    """A_log and step sizes at the ends of fp32: decays of exactly 0 and 1."""
    announce("selective extremes")
    q = make("f32", 1, 21, 9, 8, 1, seed=7)
    q["A_log"][0], q["A_log"][1] = 100.0, -200.0
    q["dt"][0, :, 2] = 80.0
    q["dt"][0, :, 3] = -100.0
    (yr, fr), (ys, fs) = reference({**q, "A_log": q["A_log"].clamp(max=80.0)})
    y, f = forward(q)
    ref.check(y, yr, ys, 8 * 21 + 20, "y")
    ref.check(f, fr, fs, 8 * 21 + 8, "final")
    assert all(bool(torch.isfinite(v).all()) for k, v in backward(q).items() if k != "dA_log")


def test_slices_are_read_in_place():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("selective slices")
    q = make("bf16", 2, 30, 48, 16, 2, seed=8)
    s = dict(q)
    for k in ("x", "dt", "z"):
        wide = torch.randn(2, 30, 131).to(torch.bfloat16)
        wide[:, :, 33:81] = q[k]
        s[k] = wide.cuda()[:, :, 33:81]
    wide = torch.cat([q["B"].flatten(-2), q["C"].flatten(-2), torch.zeros(2, 30, 3, dtype=torch.bfloat16)], -1).cuda()
    s["B"], s["C"] = wide[..., :32].unflatten(-1, (2, 16)), wide[..., 32:64].unflatten(-1, (2, 16))
    a, c = forward(q), forward(s)
    assert all(torch.equal(u, v) for u, v in zip(a, c))
    a, c = backward(q), backward(s)
    assert all(torch.equal(a[k], c[k]) for k in a)


@pytest.mark.parametrize("segments", [0, 3])
def test_bad_values_stay_in_their_sequence(segments):
    announce("selective no leak")
    lens = [[20, 44, 16]]
    q = make("f32", 1, 80, 66, 16, 1, lens, seed=9)
    clean, cleang = forward(q, segments=segments), backward(q, segments=segments)
    for bad in (float("inf"), float("nan")):
        for k in ("x", "dt", "B", "dy"):
            r = dict(q)
            r[k] = q[k].clone()
            r[k][:, 20:64] = bad
            y, f = forward(r, segments=segments)
            g = backward(r, segments=segments)
            for lo, hi in ((0, 20), (64, 80)):
                assert torch.equal(y[:, lo:hi], clean[0][:, lo:hi]), (bad, k)
                for name in ("dx", "ddt", "dB", "dC", "dz"):
                    assert torch.equal(g[name][:, lo:hi], cleang[name][:, lo:hi]), (bad, k, name)
            assert torch.equal(f[[0, 2]], clean[1][[0, 2]])
            assert torch.equal(g["dinit"][[0, 2]], cleang["dinit"][[0, 2]])


def test_absent_sequences_and_empty_rows():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("selective absent ids")
    q = make("f32", 1, 6, 10, 8, 1, seed=10)
    ids = torch.tensor([[1, 1, 3, 3, 3, 3]], dtype=torch.int32)
    r = {**q, "ids": ids, "n": 5, "init": torch.randn(5, 10, 8), "dfinal": torch.randn(5, 10, 8)}
    f = torch.full((5, 10, 8), 7.0).cuda()
    forward(r, final_state=f)
    assert bool((f[[0, 2, 4]] == 7).all()) and not bool((f[[1, 3]] == 7).any())
    g = backward(r)
    assert bool((g["dinit"][[0, 2, 4]] == 0).all()) and bool((g["dinit"][[1, 3]] != 0).any())
    e = {**q, "x": q["x"][:, :0], "dt": q["dt"][:, :0], "B": q["B"][:, :0], "C": q["C"][:, :0], "z": q["z"][:, :0],
         "dy": q["dy"][:, :0]}
    y, f = forward(e)
    assert y.shape == (1, 0, 10) and torch.equal(f.cpu(), q["init"])
    g = backward(e)
    assert torch.equal(g["dinit"].cpu(), q["dfinal"]) and not any(bool(g[k].any()) for k in ("dA_log", "dD", "ddt_bias"))


def test_graph_replays_equal_eager():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("selective graph")
    lens = [[40, 3, 100], [143]]
    q = make("bf16", 2, 143, 70, 16, 1, lens, seed=11)
    d = {k: gpu(v) for k, v in q.items()}
    kw = more(d, segments=3)
    state = d["init"][:2].contiguous()

    def run(s):
        y, f = ssd.selective_scan(*[d[k] for k in ("x", "dt", "A_log", "B", "C")], **kw)
        g = ssd.selective_scan_backward(*[d[k] for k in ("x", "dt", "A_log", "B", "C", "dy")], dfinal=d["dfinal"], **kw)
        yt = ssd.selective_step(*[d[k][:, 0] for k in ("x", "dt")], d["A_log"], d["B"][:, 0], d["C"][:, 0], d["D"], s,
                                z=d["z"][:, 0], dt_bias=d["bias"], dt_softplus=True)
        return [y, f, yt] + [g[k] for k in sorted(g)]

    eager_state = state.clone()
    eager = run(eager_state)
    torch.cuda.synchronize()
    graph_state = state.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(graph_state)
    for _ in range(3):
        for t in outs:
            t.fill_(float("nan"))
        graph_state.copy_(state)
        torch.cuda.synchronize()
        graph.replay()
        run(state.clone())
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(outs, eager)) and torch.equal(graph_state, eager_state)


def test_another_stream():
    announce("selective stream")
    q = make("f32", 2, 300, 50, 16, seed=12)
    y0, f0 = forward(q)
    g0 = backward(q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        d = {k: gpu(v) for k, v in q.items()}
        torch.cuda.synchronize()
        y, f = forward(d, stream=handle)
        g = backward(d, stream=handle)
        s.synchronize()
        assert torch.equal(y, y0) and torch.equal(f, f0) and all(torch.equal(g[k], g0[k]) for k in g)


def test_long_row_is_split_and_agrees():
    announce("selective long row")
    q = make("f32", 1, 3000, 64, 16, 1, seed=13)
    q["A_log"] = q["A_log"] - 2.0
    y, f = forward(q)
    y1, f1 = forward(q, segments=1)
    # 3000 tokens of eight roundings each at most, in either
    ref.check(y, y1.cpu(), y1.abs().max().item() * 4, 2 * 8 * 64, "y")
    ref.check(f, f1.cpu(), f1.abs().max().item() * 4, 2 * 8 * 64, "final")
    g, g1 = backward(q), backward(q, segments=1)
    for k in g:
        ref.check(g[k], g1[k].cpu(), g1[k].abs().max().item() * 4, 2 * 8 * 64, k)


def test_masked_tokens_leave_the_state_alone():
    """A step that softplus maps to zero (dt of -inf, or the type's lowest value) masks its token."""
    announce("selective masked tokens")
    for dt in ("f32", "bf16"):
        for low in (float("-inf"), torch.finfo(TYPES[dt]).min):
            q = make(dt, 2, 40, 33, 16, 1, seed=14)
            q["dt"][0, 3:30], q["dt"][1] = low, low
            y, f = forward(q)
            g = backward(q)
            assert bool(torch.isfinite(y).all()) and torch.equal(f[1].cpu(), q["init"][1])
            assert all(bool(torch.isfinite(v).all()) for v in g.values())
            assert not bool(g["ddt"][0, 3:30].any()) and torch.equal(g["dinit"][1].cpu(), check_dinit(q, 1))
            short = {**q, **{k: torch.cat([q[k][:1, :3], q[k][:1, 30:]], 1) for k in ("x", "dt", "B", "C", "z", "dy")},
                     "init": q["init"][:1], "dfinal": q["dfinal"][:1], "n": 1}
            _, f1 = forward(short)
            ref.check(f[:1], f1.double().cpu(), f1.abs().double().cpu() + 4, 8 * 13, "final")


def check_dinit(q, row):
    """dL/dinit of a row whose steps are all zero: its state is its initial state throughout."""
    g = (q["dy"][row] * ref.silu(q["z"][row].float())).double()                  # (T, D)
    want = torch.einsum("td,tn->dn", g, q["C"][row, :, 0].double()) + q["dfinal"][row].double()
    got = backward(q)["dinit"][row].cpu()
    size = torch.einsum("td,tn->dn", g.abs(), q["C"][row, :, 0].double().abs()) + q["dfinal"][row].double().abs()
    ref.check(got, want, size, 40 + 12, "dinit of a masked row")
    return got


def test_offsets_past_32_bits():
    """A row of more than 2^31 elements: its last tokens equal a run of their own from the state
    that the steps' decay leaves (steps of 30 forget everything before)."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("selective long row")
    T, D, N, tail = 264000, 8192, 8, 50
    x = torch.randn(1, 4000, D, device="cuda").to(torch.bfloat16).repeat(1, 66, 1)
    dt = torch.full((1, T, D), -3.0, dtype=torch.bfloat16, device="cuda")
    dt[:, -tail] = 200.0
    B = torch.randn(1, T, 1, N, device="cuda").to(torch.bfloat16)
    A_log = torch.zeros(D, N, device="cuda")
    y, f = ssd.selective_scan(x, dt, A_log, B, B, dt_softplus=True)
    y1, f1 = ssd.selective_scan(x[:, -tail:], dt[:, -tail:], A_log, B[:, -tail:], B[:, -tail:], dt_softplus=True)
    # the same products in kernels of other shapes: sums of eight terms in another order.  Both
    # sides are rounded to bf16: |a - b| <= |a - v| + |v - w| + |w - b| with a half step each
    # for the first and the last, so the bound has two half steps where check() counts one
    one, whole = y1.cpu().double(), y[:, -tail:].cpu().double()
    bound = 2 * ref.U16 * one.abs() + 16 * ref.U32 * (one.abs() + 8 * 200.0)
    assert bool(((whole - one).abs() <= bound).all())
    ref.check(f, f1.cpu().double(), f1.cpu().double().abs(), 8, "final")


def test_arguments_are_checked():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("selective arguments")
    q = make("f32", 2, 6, 8, 8, 1, seed=15)
    d = {k: gpu(v) for k, v in q.items()}

    def call(x=d["x"], dt=d["dt"], A=d["A_log"], B=d["B"], C=d["C"], **kw):
        return ssd.selective_scan(x, dt, A, B, C, **kw)

    for kind, f in (
            (TypeError, lambda: call(x=d["x"].half())), (TypeError, lambda: call(dt=d["dt"].bfloat16())),
            (TypeError, lambda: call(B=d["B"].bfloat16())), (TypeError, lambda: call(z=d["z"].bfloat16())),
            (TypeError, lambda: call(A=d["A_log"].bfloat16())), (ValueError, lambda: call(dt=d["dt"][:, :5])),
            (ValueError, lambda: call(A=d["A_log"][:7])), (ValueError, lambda: call(B=d["B"][:, :5], C=d["C"][:, :5])),
            (ValueError, lambda: call(C=d["C"][:, :5])), (ValueError, lambda: call(z=d["z"].cpu())),
            (ValueError, lambda: call(init_state=d["init"][:1])), (ValueError, lambda: call(nseqs=5)),
            (ValueError, lambda: call(D=d["D"][:7])), (ValueError, lambda: call(y=torch.zeros(2, 6, 9, device="cuda"))),
            (ValueError, lambda: call(final_state=d["init"][:1])),
            (ssd.SSDError, lambda: call(segments=-1)), (ssd.SSDError, lambda: call(y=d["x"])),
            (ssd.SSDError, lambda: call(init_state=d["init"], final_state=d["init"])),
            (ssd.SSDError, lambda: call(A=d["A_log"][:, :5].contiguous(), B=d["B"][..., :5], C=d["C"][..., :5])),
            (ValueError, lambda: ssd.selective_scan_backward(d["x"], d["dt"], d["A_log"], d["B"], d["C"], d["dy"][:1])),
            (ValueError, lambda: ssd.selective_scan_backward(d["x"], d["dt"], d["A_log"], d["B"], d["C"], d["dy"],
                                                             workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))),
            (ValueError, lambda: ssd.selective_step(d["x"][:, 0], d["dt"][:, 0], d["A_log"], d["B"][:, 0], d["C"][:, 0], None, d["init"][:1]))):
        with pytest.raises(kind):
            f()


@pytest.mark.parametrize("soft", [True, False])
def test_bad_steps_stay_in_their_sequence_across_segments(soft):
    """Segments of 32 tokens; the bad sequence starts in the middle of the second, which the
    sequence before reaches from the first."""
    announce("selective no leak across segments softplus=%s" % soft)
    q = make("f32", 1, 96, 66, 16, 1, [[40, 40, 16]], soft=soft, seed=17)
    clean, cleang = forward(q, segments=3), backward(q, segments=3)
    for bad in (float("nan"), float("-inf"), float("inf")):
        r = {**q, "dt": q["dt"].clone()}
        r["dt"][:, 50:55] = bad
        y, f = forward(r, segments=3)
        g = backward(r, segments=3)
        for lo, hi in ((0, 40), (80, 96)):
            assert torch.equal(y[:, lo:hi], clean[0][:, lo:hi]), bad
            for name in ("dx", "ddt", "dB", "dC", "dz"):
                assert torch.equal(g[name][:, lo:hi], cleang[name][:, lo:hi]), (bad, name)
        assert torch.equal(f[[0, 2]], clean[1][[0, 2]]) and torch.equal(g["dinit"][[0, 2]], cleang["dinit"][[0, 2]])


def test_last_tokens_of_long_prompts():
    """A step on ``hidden[:, -1]``: rows are a whole prompt apart, here 2^25 elements and more."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("selective step, rows 2^25 elements apart")
    b, T, D, N = 2, 8192, 5120, 16
    wide = torch.randn(b, T, D, device="cuda", dtype=torch.bfloat16)
    x, dt, z = (wide[:, -k] for k in (1, 2, 3))
    B, C = (wide[:, -k, :N].unflatten(-1, (1, N)) for k in (4, 5))
    assert all(t.stride(0) >= 1 << 25 for t in (x, dt, z, B, C))
    A, skip = torch.rand(D, N, device="cuda"), torch.randn(D, device="cuda")
    state = torch.randn(b, D, N, device="cuda")
    other = state.clone()
    y = ssd.selective_step(x, dt, A, B, C, skip, state, z, dt_softplus=True)
    want = ssd.selective_step(*[t.contiguous() for t in (x, dt, A, B, C)], skip, other, z.contiguous(), dt_softplus=True)
    assert torch.equal(y, want) and torch.equal(state, other)


def test_far_apart_tokens_are_copied():
    """The prompt calls read tokens up to 2^25 elements apart in place; past that they are copied."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("selective prompt, tokens 2^25 elements apart")
    T, D, N, ld = 9, 70, 8, 1 << 25
    wide = torch.zeros((T - 1) * ld + D, dtype=torch.bfloat16, device="cuda")
    far = wide.as_strided((1, T, D), (T * ld, ld, 1))
    far.copy_(torch.randn(1, T, D))
    B = far[..., :N].unflatten(-1, (1, N))
    A, dy = torch.rand(D, N, device="cuda"), torch.randn(1, T, D, device="cuda")
    y, f = ssd.selective_scan(far, far, A, B, B, z=far, dt_softplus=True)
    g = ssd.selective_scan_backward(far, far, A, B, B, dy, z=far, dt_softplus=True)
    x, B = far.contiguous(), B.contiguous()
    y1, f1 = ssd.selective_scan(x, x, A, B, B, z=x, dt_softplus=True)
    g1 = ssd.selective_scan_backward(x, x, A, B, B, dy, z=x, dt_softplus=True)
    assert torch.equal(y, y1) and torch.equal(f, f1) and all(torch.equal(g[k], g1[k]) for k in g)


def test_shapes_of_a_step():
    """B and C of a step are (b,G,N) both, not merely of as many values."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("selective step shapes")
    q = make("f32", 2, 1, 16, 8, 2, seed=18)
    d = {k: gpu(v[:, 0] if k in ("x", "dt", "B", "C") else v) for k, v in q.items() if k in ("x", "dt", "A_log", "B", "C", "init")}
    for C in (d["C"].transpose(1, 2), d["C"].reshape(2, 1, 16), d["C"].reshape(2, 16), d["C"][0, 0], d["C"][:1]):
        with pytest.raises(ValueError):
            ssd.selective_step(d["x"], d["dt"], d["A_log"], d["B"], C, None, d["init"].clone())
