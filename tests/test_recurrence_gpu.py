"""The gated linear recurrence (whole rows, gradients, single tokens) against its 64-bit form."""
import pytest
import torch

import block_ref as ref
import recurrence_ref as rr

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def announce(msg):
    print("[case] " + msg, flush=True)


def gpu(v):
    return v.cuda() if torch.is_tensor(v) else v


def make(dt, b, T, D, lens=None, state=True, gate=True, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * T + D)
    n = len(ref.sequences(b, T, lens))

    def act(std=1.0):
        return (torch.randn(b, T, D, generator=g) * std).to(TYPES[dt])

    # memories from a token to a thousand
    return {"x": act(), "r": act(2.0), "i": act(), "z": act() if gate else None,
            "A_log": torch.rand(D, generator=g) * 8 - 6, "init": torch.randn(n, D, generator=g) if state else None,
            "dy": torch.randn(b, T, D, generator=g), "dfinal": torch.randn(n, D, generator=g) if state else None,
            "ids": ref.ids_of(b, T, lens), "lens": lens, "n": n}


def forward(ssd, q, **kw):
    return ssd.gated_recurrence(gpu(q["x"]), gpu(q["r"]), gpu(q["i"]), gpu(q["A_log"]), gpu(q["z"]), gpu(q["init"]),
                                gpu(q["ids"]), q["n"], **kw)


def backward(ssd, q, **kw):
    return ssd.gated_recurrence_backward(gpu(q["x"]), gpu(q["r"]), gpu(q["i"]), gpu(q["A_log"]), gpu(q["dy"]),
                                         gpu(q["z"]), gpu(q["init"]), gpu(q["dfinal"]), gpu(q["ids"]), q["n"], **kw)


def wide(q):
    w = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in q.items()}
    for k in ("init", "dfinal"):
        if w[k] is None:
            w[k] = torch.zeros(q["n"], q["x"].shape[2], dtype=torch.double)
    return w


def check_forward(ssd, q, got=None):
    y, f = forward(ssd, q) if got is None else got
    assert y.dtype == q["x"].dtype and f.dtype == torch.float32
    w = wide(q)
    want, final, ey, ef = rr.forward(w["x"], w["r"], w["i"], w["A_log"], w["z"], w["init"], q["lens"], q["x"].dtype == torch.bfloat16)[:4]
    rr.check(y, want, ey, "y")
    rr.check(f, final, ef, "final")


def check_backward(ssd, q, got=None):
    got = backward(ssd, q) if got is None else got
    w = wide(q)
    want = rr.backward(w["x"], w["r"], w["i"], w["A_log"], w["dy"], w["z"], w["init"], w["dfinal"], q["lens"],
                       q["x"].dtype == torch.bfloat16)
    assert set(got) == set(want)
    for k in want:
        assert got[k].dtype == torch.float32
        rr.check(got[k], *want[k], k)


CASES = [
    # dtype, rows, tokens, channels, sequence lengths, initial state, gate
    ("bf16", 2, 130, 64, None, True, True), ("f32", 2, 130, 64, None, True, True),
    ("bf16", 1, 1, 40, None, True, True), ("f32", 1, 1, 1, None, False, False),
    ("f32", 3, 2, 5, None, True, False), ("bf16", 1, 97, 7, None, True, False),         # fewer channels than a vector
    ("f32", 1, 300, 3, None, False, True), ("bf16", 2, 75, 1029, None, False, False),   # odd rows
    ("bf16", 3, 33, 9, None, True, True), ("f32", 2, 31, 65, None, True, True),
    ("bf16", 1, 257, 72, None, True, False), ("f32", 1, 513, 8, None, True, False),
    ("bf16", 1, 1025, 96, None, True, True), ("f32", 2, 2049, 6, None, False, True),    # many tiles
    ("f32", 1, 67, 131, [[1, 1, 1, 2, 3, 4, 5, 18, 31, 1]], True, True),
    ("bf16", 2, 70, 72, [[64, 6], [1, 2, 67]], True, True),
    ("bf16", 1, 600, 33, [[3, 61, 64, 72, 255, 145]], False, True),
    ("f32", 2, 300, 24, [[300], [2, 1, 297]], True, False),
    ("f32", 1, 1300, 68, [[1, 127, 128, 256, 257, 1, 530]], True, True),
    ("bf16", 1, 5000, 16, None, True, False),
]
IDS = ["%s-b%d-T%d-D%d-%s%s%s" % (c[0], c[1], c[2], c[3], "packed" if c[4] else "rows", "" if c[5] else "-nostate",
                                  "-gate" if c[6] else "") for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence forward %s" % (case,))
    check_forward(ssd, make(*case))


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence backward %s" % (case,))
    check_backward(ssd, make(*case))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", list(range(1, 20)) + [31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 385])
def test_lengths(T, dt):
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence length %d %s" % (T, dt))
    q = make(dt, 2, T, 24, None if T < 3 else [[T], [T - 2, 2]])
    check_forward(ssd, q)
    check_backward(ssd, q)


def test_gradients_against_differences():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence differences")
    q = make("f32", 2, 70, 12, [[40, 30], [1, 69]])
    w = wide(q)
    got = backward(ssd, q)

    def loss(v):
        y, f = rr.forward(v["x"], v["r"], v["i"], v["A_log"], v["z"], v["init"], q["lens"])[:2]
        return float((y * w["dy"]).sum() + (f * w["dfinal"]).sum())

    g = torch.Generator().manual_seed(1)
    for name in ("x", "r", "i", "z", "A_log", "init"):
        along = torch.randn(w[name].shape, generator=g).double()
        lo, hi, h = dict(w), dict(w), 1e-5
        lo[name], hi[name] = w[name] - h * along, w[name] + h * along
        slope = (loss(hi) - loss(lo)) / (2 * h)
        part = got["d" + name].cpu().double() * along
        # differences of step h are off by h^2 and by 2^-52 / h of the loss's terms
        assert abs(float(part.sum()) - slope) <= 1e-5 * float(part.abs().sum()), name


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("in_place", [False, True])
def test_steps_continue_a_prompt(dt, in_place):
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence steps %s" % dt)
    for b, D in ((3, 100), (1, 7), (2, 264)):
        q = make(dt, b, 40, D)
        d = {k: gpu(v) for k, v in q.items()}
        whole, final = forward(ssd, q)
        y, state = ssd.gated_recurrence(d["x"][:, :30], d["r"][:, :30], d["i"][:, :30], d["A_log"], d["z"][:, :30], d["init"])
        ys, fresh = [y], torch.empty_like(state)
        for t in range(30, 40):
            old = state.clone()
            kw = {} if in_place else {"state_out": fresh}
            ys.append(ssd.gated_recurrence_step(d["x"][:, t], d["r"][:, t], d["i"][:, t], d["A_log"], state,
                                                z=d["z"][:, t], **kw)[:, None])
            if not in_place:
                assert torch.equal(state, old)
                state, fresh = fresh, state
        check_forward(ssd, q, (torch.cat(ys, 1), state))
        check_forward(ssd, q, (whole, final))


def test_extreme_gates():
    """Gates over their whole range, the type's lowest and infinite values among them: a closed
    recurrence gate keeps the state as it is, a closed input gate adds nothing."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence extreme gates")
    for dt in ("bf16", "f32"):
        low = torch.finfo(TYPES[dt]).min
        q = make(dt, 1, 64, 40)
        vals = torch.tensor([low, -1e30, -200.0, -95.0, -88.0, -60.0, -20.0, -1.0, 0.0, 1.0, 20.0, 90.0, 1e30, -low])
        for k, shift in (("r", 0), ("i", 3), ("z", 5)):
            q[k] = vals[(torch.arange(64)[:, None] + shift + torch.arange(40)) % len(vals)][None].to(TYPES[dt]).contiguous()
        q["z"] = q["z"].clamp(-1e4, 1e4)
        check_forward(ssd, q)
        check_backward(ssd, q)
        q["r"][:] = float("-inf")
        q["z"] = None
        y, f = forward(ssd, q)
        assert torch.equal(f.cpu(), q["init"]) and torch.equal(y.cpu(), q["init"][:, None].to(TYPES[dt]).expand_as(q["x"]))
        got = backward(ssd, q)
        for k in ("dx", "dr", "di", "dA_log"):
            assert not got[k].any(), k
        q["r"][:] = float("inf")
        q["i"][:] = float("-inf")
        y, f = forward(ssd, q)
        assert torch.isfinite(y.float()).all()
        got = backward(ssd, q)
        assert not got["di"].any() and not got["dx"].any() and not got["dr"].any()


def test_long_memory():
    """Decays of 1 - 1e-6 over thousands of tokens: 1 - a and not a sets the result."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence long memory")
    for T in (100, 3000):
        q = make("f32", 1, T, 16, gate=False)
        q["A_log"] = torch.linspace(-30, -4, 16)
        check_forward(ssd, q)
        check_backward(ssd, q)


def test_bad_values_stay_in_their_sequence():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence bad values")
    lens = [[90, 210, 300, 100], [400, 300]]
    for bad in (float("nan"), float("inf")):
        for dt in ("f32", "bf16"):
            q = make(dt, 2, 700, 24, lens, gate=False)
            clean_y, clean_f = forward(ssd, q)
            clean = backward(ssd, q)
            q["x"][0, 150, 3] = bad
            y, f = forward(ssd, q)
            got = backward(ssd, q)
            keep = torch.ones(2, 700, 24, dtype=torch.bool)
            keep[0, 150:300, 3] = False                      # before it, and other channels, nothing changes
            assert torch.equal(y.cpu()[keep], clean_y.cpu()[keep]) and not torch.isfinite(y.cpu()[0, 150, 3])
            ok = torch.ones(6, 24, dtype=torch.bool)
            ok[1, 3] = False
            assert torch.equal(f.cpu()[ok], clean_f.cpu()[ok])
            for k in ("dx", "dr", "di"):
                rest = torch.ones(2, 700, 24, dtype=torch.bool)
                rest[0, 90:300, 3] = False
                assert torch.equal(got[k].cpu()[rest], clean[k].cpu()[rest]), k
            q["x"][0, 150, 3] = 0
            q["dy"][0, 150, 3] = bad
            got = backward(ssd, q)
            rest = torch.ones(2, 700, 24, dtype=torch.bool)
            rest[0, 90:151, 3] = False                       # a gradient reaches earlier tokens of its sequence
            clean = backward(ssd, dict(q, dy=q["dy"].nan_to_num(0, 0, 0)))
            for k in ("dx", "dr", "di"):
                assert torch.equal(got[k].cpu()[rest], clean[k].cpu()[rest]), k
            assert torch.isfinite(got["dinit"].cpu()[[0, 2, 3, 4, 5]]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nan_is_not_lost(dt):
    """A NaN in any input shows from its token on, and only in its channel."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence NaN %s" % dt)
    for T in (1, 40, 700):
        q = make(dt, 1, T, 24)
        clean_y, clean_f = forward(ssd, q)
        clean = backward(ssd, q)
        t = T // 2
        for name in ("x", "r", "i", "z", "A_log", "init"):
            bad = dict(q, **{name: q[name].clone()})
            bad[name][(0, t, 5) if name in "xriz" else (5 if name == "A_log" else (0, 5))] = float("nan")
            y, f = forward(ssd, bad)
            g = backward(ssd, bad)
            others = torch.arange(24) != 5
            assert torch.equal(y.cpu()[..., others], clean_y.cpu()[..., others]), name
            assert torch.equal(f.cpu()[:, others], clean_f.cpu()[:, others]), name
            for k in clean:
                assert torch.equal(g[k].cpu()[..., others], clean[k].cpu()[..., others]), (name, k)
            first = t if name in "xriz" else 0
            assert torch.isnan(y.cpu()[0, first, 5]) and torch.equal(y.cpu()[0, :first], clean_y.cpu()[0, :first]), name
            if name != "z":
                assert torch.isnan(f.cpu()[0, 5]), name


def test_absent_sequences_and_empty_rows():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence absent sequences")
    q = make("f32", 1, 300, 20, [[150, 0, 150]])
    final = torch.full((3, 20), 7.0, device="cuda")
    y, f = forward(ssd, q, final_state=final)
    assert f is final and (f[1] == 7.0).all()                # not written
    want = rr.forward(*[wide(q)[k] for k in ("x", "r", "i", "A_log", "z", "init")], q["lens"])
    rr.check(y, want[0], want[2], "y")
    rr.check(f[[0, 2]], want[1][[0, 2]], want[3][[0, 2]], "final")
    assert not backward(ssd, q)["dinit"][1].any()
    for b, T in ((2, 0), (0, 5), (0, 0)):
        q = make("bf16", b, T, 20)
        y, f = forward(ssd, q)
        assert y.shape == (b, T, 20) and torch.equal(f.cpu(), q["init"])
        got = backward(ssd, q)
        assert torch.equal(got["dinit"].cpu(), q["dfinal"]) and not got["dA_log"].any() and got["dx"].shape == (b, T, 20)
    y, f = forward(ssd, dict(make("f32", 2, 0, 20), init=None))
    assert not f.any()


def test_slices_are_read_in_place():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence slices")
    for dt, D in (("bf16", 70), ("f32", 64), ("bf16", 5)):
        q = make(dt, 2, 200, D)
        wide_ = torch.full((2, 200, 4 * D + 3), float("nan"), dtype=TYPES[dt], device="cuda")
        s = dict(q)
        for k, name in enumerate(("x", "r", "i", "z")):
            s[name] = wide_[..., 1 + k * D:1 + (k + 1) * D]
            s[name].copy_(q[name])
        for a, b in zip(forward(ssd, q), forward(ssd, s)):
            assert torch.equal(a, b)
        got, want = backward(ssd, s), backward(ssd, q)
        for k in want:
            assert torch.equal(got[k], want[k]), k
        # orders that no distance between tokens describes are copied
        turned = {k: gpu(q[k]).transpose(0, 1).contiguous().transpose(0, 1) for k in ("x", "r", "i", "z")}
        for a, b in zip(forward(ssd, dict(q, **turned)), forward(ssd, q)):
            assert torch.equal(a, b)
        token = {k: s[k][:, 3] for k in ("x", "r", "i", "z")}
        state = gpu(torch.randn(2, D))
        a = ssd.gated_recurrence_step(token["x"], token["r"], token["i"], gpu(q["A_log"]), state.clone(), z=token["z"])
        b = ssd.gated_recurrence_step(*[token[k].contiguous() for k in ("x", "r", "i")], gpu(q["A_log"]), state.clone(),
                                      z=token["z"].contiguous())
        assert torch.equal(a, b)


def test_results_repeat():
    """The same call gives the same bits, alone and beside another one."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence repeats")
    q = make("bf16", 2, 3000, 200, [[1000, 2000], [1, 2999]])
    d = {k: gpu(v) for k, v in q.items()}
    y0, f0 = forward(ssd, d)
    g0 = backward(ssd, d)
    torch.cuda.synchronize()
    others = [torch.cuda.Stream() for _ in range(2)]
    for s in others:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        results = []
        for s in others:
            results.append((forward(ssd, d, stream=s), backward(ssd, d, stream=s)))
        torch.cuda.synchronize()
        for (y, f), g in results:
            assert torch.equal(y, y0) and torch.equal(f, f0)
            for k in g0:
                assert torch.equal(g[k], g0[k]), k


def test_graph_replays_equal_eager():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence graph")
    q = make("bf16", 2, 1500, 136, [[700, 800], [1500]])
    s = {k: gpu(v) for k, v in q.items()}
    p = ssd.recurrence_problem(2, 1500, 136, 3)
    ws = torch.empty(max(ssd.recurrence_workspace_size(p), ssd.recurrence_backward_workspace_size(p), 1), dtype=torch.uint8,
                     device="cuda")
    token = {k: s[k][:, 0].contiguous() for k in ("x", "r", "i", "z")}
    state = gpu(torch.randn(2, 136))

    def work():
        # both directions share a workspace
        y, f = forward(ssd, s, workspace=ws)
        g = backward(ssd, s, workspace=ws)
        step = ssd.gated_recurrence_step(token["x"], token["r"], token["i"], s["A_log"], state, z=token["z"])
        return [y, f, step] + [g[k] for k in sorted(g)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for k in range(4):
        new = make("bf16", 2, 1500, 136, q["lens"], seed=50 + k)
        for name in ("x", "r", "i", "z", "dy", "init", "dfinal"):
            s[name].copy_(new[name])
        for name in token:
            token[name].copy_(s[name][:, 0])
        state.copy_(new["dfinal"][:2])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        state.copy_(new["dfinal"][:2])
        for a, b in zip(got, work()):
            assert torch.equal(a, b)


def test_another_stream():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence stream")
    q = make("f32", 2, 400, 48)
    d = {k: gpu(v) for k, v in q.items()}
    y0, f0 = forward(ssd, d)
    g0 = backward(ssd, d)
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream, 0):
        y, f = forward(ssd, d, stream=s)
        g = backward(ssd, d, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.equal(f, f0) and all(torch.equal(g[k], g0[k]) for k in g0)


def test_offsets_past_32_bits():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence far offsets")
    ld, T, D = (1 << 30) + 5, 5, 40                          # the last token starts past 2^32 elements
    big = torch.empty(4 * ld + D, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((1, T, D), (T * ld, ld, 1))
    q = make("bf16", 1, T, D, gate=False)
    x.copy_(q["x"])
    a = ssd.gated_recurrence(x, x, x, gpu(q["A_log"]), init_state=gpu(q["init"]))
    c = x.contiguous()
    b = ssd.gated_recurrence(c, c, c, gpu(q["A_log"]), init_state=gpu(q["init"]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = ssd.gated_recurrence_backward(x, x, x, gpu(q["A_log"]), gpu(q["dy"]))
    gb = ssd.gated_recurrence_backward(c, c, c, gpu(q["A_log"]), gpu(q["dy"]))
    assert all(torch.equal(ga[k], gb[k]) for k in gb)
    del big, x
    # outputs past 2^32 bytes: whole rows of the last of them
    b_, T, D = 9, 4000, 60000
    x = torch.randn(1, T, D, device="cuda").to(torch.bfloat16).expand(b_, T, D).contiguous()
    A = torch.rand(D, device="cuda") * 4 - 4
    y, f = ssd.gated_recurrence(x, x, x, A)
    y1, f1 = ssd.gated_recurrence(x[-1:], x[-1:], x[-1:], A)
    assert torch.equal(f[-1], f1[0]) and torch.equal(y[-1], y1[0]) and torch.equal(y[0], y1[0])


def test_many_rows():
    """More rows than a launch has in a second dimension; chains of one tile and of several."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence many rows")
    for b, T, D in ((70000, 2, 4), (3000, 70, 8), (600, 300, 5)):
        one = make("f32", 3, T, D)
        big = {k: (v.repeat(b // 3, *[1] * (v.dim() - 1)) if torch.is_tensor(v) and v.dim() > 1 and v.shape[0] == 3 else v)
               for k, v in one.items()}
        big["n"] = big["x"].shape[0]
        y, f = forward(ssd, big)
        y3, f3 = forward(ssd, one)
        m = b // 3
        assert torch.equal(y.view(m, 3, T, D), y3.expand(m, 3, T, D)) and torch.equal(f.view(m, 3, D), f3.expand(m, 3, D))
        g, g3 = backward(ssd, big), backward(ssd, one)
        for k in ("dx", "dr", "di", "dz"):
            assert torch.equal(g[k].view(m, 3, T, D), g3[k].expand(m, 3, T, D)), k
        assert torch.equal(g["dinit"].view(m, 3, D), g3["dinit"].expand(m, 3, D))


def test_outputs_larger_than_the_caches():
    """Outputs stored past the caches are the same values."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence large outputs")
    for dt, b, T, D in (("bf16", 3, 3000, 2050), ("f32", 2, 3000, 1500)):
        q = make(dt, 1, T, 50, gate=True)
        wide_ = {k: gpu(v).repeat(*([b] + [1] * (v.dim() - 2) + [D // 50])) if torch.is_tensor(v) and v.dim() > 1 else v
                 for k, v in q.items()}
        wide_["A_log"] = q["A_log"].repeat(D // 50)
        wide_["n"] = b
        y, f = forward(ssd, wide_)
        assert y.numel() * y.element_size() > 32 << 20
        y1, f1 = forward(ssd, q)
        assert torch.equal(y.unflatten(-1, (-1, 50)), y1.unsqueeze(2).expand(b, T, D // 50, 50))
        assert torch.equal(f.view(b, -1, 50), f1[:, None].expand(b, D // 50, 50))
        g, g1 = backward(ssd, wide_), backward(ssd, q)
        for k in ("dx", "dr", "di", "dz"):
            assert torch.equal(g[k].unflatten(-1, (-1, 50)), g1[k].unsqueeze(2).expand(b, T, D // 50, 50)), k


def test_sequence_ids_out_of_range_stay_in_memory():
    """Ids beyond the states are clamped: values undefined, memory safe."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence ids out of range")
    q = make("f32", 1, 200, 20, [[100, 100]])
    guard = torch.full((4, 20), 3.0, device="cuda")
    q["ids"] = torch.where(torch.arange(200)[None] < 100, -5, 1000).int()
    y, f = forward(ssd, q, final_state=guard[1:3])
    assert (guard[0] == 3.0).all() and (guard[3] == 3.0).all() and torch.isfinite(y).all()
    assert all(torch.isfinite(t).all() for t in backward(ssd, q).values())


def test_arguments_are_checked():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("recurrence arguments")
    q = {k: gpu(v) for k, v in make("bf16", 2, 10, 16).items()}
    good = [q["x"], q["r"], q["i"], q["A_log"]]
    for at, bad, err in ((0, q["x"].half(), TypeError), (0, q["x"].cpu(), ValueError), (0, q["x"][0], ValueError),
                         (1, q["r"].float(), TypeError), (1, q["r"][:, :9], ValueError), (2, q["i"].cpu(), ValueError),
                         (3, q["A_log"].double(), TypeError), (3, q["A_log"][:15], ValueError)):
        args = list(good)
        args[at] = bad
        with pytest.raises(err):
            ssd.gated_recurrence(*args)
        with pytest.raises(err):
            ssd.gated_recurrence_backward(*args, q["dy"])
    for kw, err in (({"z": q["z"].float()}, TypeError), ({"init_state": q["init"][:1]}, ValueError),
                    ({"init_state": q["init"].double()}, TypeError), ({"nseqs": 3}, ValueError),
                    ({"seq_idx": torch.zeros(2, 10, dtype=torch.int32, device="cuda")}, ValueError),
                    ({"seq_idx": torch.zeros(2, 10, dtype=torch.int64, device="cuda"), "nseqs": 1}, TypeError),
                    ({"y": torch.empty(2, 10, 16, device="cuda")}, TypeError),
                    ({"y": torch.empty(2, 10, 32, dtype=torch.bfloat16, device="cuda")[..., ::2]}, ValueError),
                    ({"final_state": torch.empty(3, 16, device="cuda")}, ValueError),
                    ({"init_state": q["init"], "final_state": q["init"]}, ssd.SSDError),
                    ({"y": q["x"]}, ssd.SSDError)):
        with pytest.raises(err):
            ssd.gated_recurrence(*good, **kw)
    with pytest.raises(TypeError):
        ssd.gated_recurrence_backward(*good, q["dy"].bfloat16())
    with pytest.raises(ValueError):
        ssd.gated_recurrence_backward(*good, q["dy"], dfinal=q["dfinal"][:1])
    token = [t[:, 0] for t in good[:3]]
    with pytest.raises(ValueError):
        ssd.gated_recurrence_step(q["x"], *token[1:], q["A_log"], q["init"])
    with pytest.raises(ValueError):
        ssd.gated_recurrence_step(*token, q["A_log"], q["init"][:, ::2])
    with pytest.raises(ssd.SSDError):
        ssd.gated_recurrence_step(*token, q["A_log"], q["init"], state_out=q["init"].view(-1)[:32].view(2, 16),
                                  y=q["x"].view(-1)[:32].view(2, 16))
