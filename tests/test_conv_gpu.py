"""The causal convolution (whole rows, gradients, single tokens) against its 64-bit form."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def announce(msg):
    print("[case] " + msg, flush=True)


def make(dt, b, T, D, K, lens=None, state=True, bias=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = len(ref.sequences(b, T, lens))
    return {"x": torch.randn(b, T, D, generator=g).to(TYPES[dt]), "w": torch.randn(D, K, generator=g) / K ** 0.5,
            "bias": torch.randn(D, generator=g) if bias else None,
            "init": torch.randn(n, K - 1, D, generator=g) if state else None,
            "dy": torch.randn(b, T, D, generator=g), "dfinal": torch.randn(n, K - 1, D, generator=g) if state else None,
            "ids": ref.ids_of(b, T, lens), "lens": lens, "n": n, "K": K}


def gpu(v):
    return v.cuda() if torch.is_tensor(v) else v


def zero_state(q):
    return torch.zeros(q["n"], q["K"] - 1, q["x"].shape[2]) if q["init"] is None else q["init"]


CASES = [
    # dtype, rows, tokens, channels, K, sequence lengths, initial state, bias, silu
    ("bf16", 2, 130, 64, 4, None, True, True, True),
    ("f32", 2, 130, 64, 4, None, True, True, True),
    ("bf16", 1, 1, 40, 4, None, True, True, True),             # one token
    ("f32", 3, 2, 5, 4, None, True, False, False),             # fewer tokens than taps, one tail vector
    ("f32", 1, 300, 3, 3, None, False, True, True),            # fewer channels than a vector
    ("bf16", 1, 97, 7, 2, None, True, True, False),
    ("bf16", 2, 75, 1029, 3, None, False, False, True),        # odd channels: unaligned rows
    ("f32", 1, 67, 131, 4, [[1, 1, 1, 2, 3, 4, 5, 18, 31, 1]], True, True, True),
    ("bf16", 2, 70, 72, 4, [[64, 6], [1, 2, 67]], True, True, True),
    ("bf16", 1, 200, 33, 2, [[3, 61, 64, 72]], False, True, True),
    ("f32", 2, 40, 24, 3, [[40], [2, 1, 37]], True, True, False),
    ("bf16", 1, 5000, 16, 4, None, True, True, True),          # many runs of one row
]
IDS = ["%s-b%d-T%d-D%d-K%d-%s%s" % (c[0], c[1], c[2], c[3], c[4], "packed" if c[5] else "rows", "" if c[6] else "-nostate")
       for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    import mamba_ssd_scan_chunked_amd as ssd
    dt, b, T, D, K, lens, state, bias, act = case
    announce("conv forward %s" % (case,))
    q = make(dt, b, T, D, K, lens, state, bias)
    y, f = ssd.causal_conv(gpu(q["x"]), gpu(q["w"]), gpu(q["bias"]), gpu(q["init"]), gpu(q["ids"]),
                           q["n"] if lens else None, silu=act)
    args = [t if t is None else t.double() for t in (q["x"], q["w"], q["bias"], zero_state(q))]
    yr, fr = ref.conv(*args, lens, act)
    # each of K + 1 terms of pre passes K roundings; silu has slope below 1.1 and eight of its own
    size, _ = ref.conv(args[0].abs(), args[1].abs(), None if args[2] is None else args[2].abs(), args[3].abs(), lens, False)
    ref.check(y, yr, size, 1.1 * K + 8, "y")
    assert torch.equal(f.cpu().double(), fr), "the final state holds inputs: no rounding"


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    import mamba_ssd_scan_chunked_amd as ssd
    dt, b, T, D, K, lens, state, bias, act = case
    announce("conv backward %s" % (case,))
    q = make(dt, b, T, D, K, lens, state, bias, seed=1)
    got = ssd.causal_conv_backward(gpu(q["x"]), gpu(q["w"]), gpu(q["dy"]), gpu(q["bias"]), gpu(q["init"]),
                                   gpu(q["dfinal"]), gpu(q["ids"]), q["n"] if lens else None, silu=act)
    bias_in = torch.zeros(D) if q["bias"] is None else q["bias"]
    lv = ref.leaves(q["x"], q["w"], bias_in, zero_state(q))
    y, f = ref.conv(*lv, lens, act)
    dfin = torch.zeros_like(f) if q["dfinal"] is None else q["dfinal"].double()
    grads = torch.autograd.grad((y * q["dy"].double()).sum() + (f * dfin).sum(), lv)
    # magnitudes: the gradient of the same sums with every factor's magnitude and silu's
    # slope at its most, 1.1.  g = dy silu'(pre): pre is off by K U32 size(pre) and silu''
    # is below 0.5; size(pre) stays below 16 at these inputs, so 8 K roundings, eight of the
    # slope itself and K of the sum.  Sums over tokens add at most 64 in a run, then the
    # runs, 16 at a time over 16 waves.
    av = ref.leaves(*[t.detach().abs() for t in lv])
    ya, fa = ref.conv(*av, lens, False)
    assert float(ya.detach().max()) < 16
    scales = torch.autograd.grad((1.1 * ya * q["dy"].double().abs()).sum() + (fa * dfin.abs()).sum(), av)
    runs = b * ((T + 3) // 4)
    for name, r, s, extra in zip(("dx", "dweight", "dbias", "dinit"), grads, scales, (0, 96 + runs / 16, 96 + runs / 16, 0)):
        ref.check(got[name], r, s, 9 * K + 8 + extra, name)


def test_gradients_against_differences():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("conv differences")
    lens = [[1, 2, 30, 7]]
    q = make("f32", 1, 40, 12, 4, lens, seed=5)
    got = ssd.causal_conv_backward(gpu(q["x"]), gpu(q["w"]), gpu(q["dy"]), gpu(q["bias"]), gpu(q["init"]),
                                   gpu(q["dfinal"]), gpu(q["ids"]), q["n"])
    base = [q[k].double() for k in ("x", "w", "bias", "init")]

    def loss(args):
        y, f = ref.conv(*args, lens, True)
        return float((y * q["dy"].double()).sum() + (f * q["dfinal"].double()).sum())

    g = torch.Generator().manual_seed(6)
    for i, name in enumerate(("dx", "dweight", "dbias", "dinit")):
        v = torch.randn(base[i].shape, generator=g).double()
        h = 1e-5
        lo, hi = list(base), list(base)
        lo[i], hi[i] = base[i] - h * v, base[i] + h * v
        slope = (loss(hi) - loss(lo)) / (2 * h)
        along = float((got[name].cpu().double() * v).sum())
        # differences: h^2 times the third derivative, and 2^-52 |loss| / h; the kernel: fp32 gradients
        assert abs(along - slope) <= 1e-5 * float((got[name].cpu().double() * v).abs().sum()), name


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("in_place", [False, True])
def test_steps_continue_a_prompt(dt, K, in_place):
    import mamba_ssd_scan_chunked_amd as ssd
    announce("conv steps %s K=%d" % (dt, K))
    q = make(dt, 3, 20, 37, K, seed=2)
    d = {k: gpu(v) for k, v in q.items()}
    y, f = ssd.causal_conv(d["x"], d["w"], d["bias"], d["init"])
    _, state = ssd.causal_conv(d["x"][:, :13], d["w"], d["bias"], d["init"])
    for t in range(13, 20):
        if in_place:
            yt = ssd.causal_conv_step(d["x"][:, t], d["w"], d["bias"], state)
        else:
            old, new = state.clone(), torch.empty_like(state)
            yt = ssd.causal_conv_step(d["x"][:, t], d["w"], d["bias"], state, state_out=new)
            assert torch.equal(state, old)
            state = new
        # the same K products, summed in one order in both kernels
        ref.check(yt, y[:, t].cpu(), y[:, t].cpu().abs() + 8, 2 * K + 8, "y of a step")
    assert torch.equal(state, f)


def test_slices_are_read_in_place():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("conv slices")
    q = make("bf16", 2, 50, 48, 4, seed=3)
    wide = torch.randn(2, 50, 131, device="cuda").to(torch.bfloat16)
    wide[:, :, 33:81] = q["x"].cuda()
    part = wide[:, :, 33:81]
    y, f = ssd.causal_conv(part, gpu(q["w"]), gpu(q["bias"]), gpu(q["init"]))
    y0, f0 = ssd.causal_conv(gpu(q["x"]), gpu(q["w"]), gpu(q["bias"]), gpu(q["init"]))
    assert torch.equal(y, y0) and torch.equal(f, f0)
    a = ssd.causal_conv_backward(part, gpu(q["w"]), gpu(q["dy"]), gpu(q["bias"]), gpu(q["init"]))
    c = ssd.causal_conv_backward(gpu(q["x"]), gpu(q["w"]), gpu(q["dy"]), gpu(q["bias"]), gpu(q["init"]))
    assert all(torch.equal(a[k], c[k]) for k in c)
    # transposed activations and rows in another order are copied first
    t = q["x"].cuda().transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(ssd.causal_conv(t, gpu(q["w"]), gpu(q["bias"]), gpu(q["init"]))[0], y0)
    one = torch.ones(1, 1, 48, device="cuda", dtype=torch.bfloat16).expand(2, 50, 48)
    assert torch.equal(ssd.causal_conv(one, gpu(q["w"]))[0], ssd.causal_conv(one.contiguous(), gpu(q["w"]))[0])


def test_bad_values_stay_in_their_sequence():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("conv no leak")
    lens = [[5, 1, 40, 18]]
    q = make("f32", 1, 64, 20, 4, lens, seed=4)
    d = {k: gpu(v) for k, v in q.items()}
    clean = ssd.causal_conv(d["x"], d["w"], d["bias"], d["init"], d["ids"], q["n"])
    cleang = ssd.causal_conv_backward(d["x"], d["w"], d["dy"], d["bias"], d["init"], d["dfinal"], d["ids"], q["n"])
    for bad in (float("inf"), float("nan")):
        x, dy = d["x"].clone(), d["dy"].clone()
        x[0, 6:46], dy[0, 6:46] = bad, bad
        y, f = ssd.causal_conv(x, d["w"], d["bias"], d["init"], d["ids"], q["n"])
        for lo, hi in ((0, 6), (46, 64)):
            assert torch.equal(y[:, lo:hi], clean[0][:, lo:hi])
        assert torch.equal(f[[0, 1, 3]], clean[1][[0, 1, 3]])
        g = ssd.causal_conv_backward(x, d["w"], dy, d["bias"], d["init"], d["dfinal"], d["ids"], q["n"])
        for lo, hi in ((0, 6), (46, 64)):
            assert torch.equal(g["dx"][:, lo:hi], cleang["dx"][:, lo:hi])
        assert torch.equal(g["dinit"][[0, 1, 3]], cleang["dinit"][[0, 1, 3]])


def test_absent_sequences_and_empty_rows():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("conv absent ids")
    q = make("f32", 1, 6, 10, 4, None, seed=7)
    ids = torch.tensor([[1, 1, 3, 3, 3, 3]], dtype=torch.int32).cuda()
    init, dfin = torch.randn(5, 3, 10).cuda(), torch.randn(5, 3, 10).cuda()
    f = torch.full((5, 3, 10), 7.0).cuda()
    ssd.causal_conv(gpu(q["x"]), gpu(q["w"]), None, init, ids, 5, final_state=f)
    assert bool((f[[0, 2, 4]] == 7).all()) and not bool((f[[1, 3]] == 7).any())
    g = ssd.causal_conv_backward(gpu(q["x"]), gpu(q["w"]), gpu(q["dy"]), None, init, dfin, ids, 5)
    assert bool((g["dinit"][[0, 2, 4]] == 0).all()) and bool((g["dinit"][[1, 3]] != 0).any())
    x = torch.empty(2, 0, 10, device="cuda")
    init, dfin = init[:2].contiguous(), dfin[:2].contiguous()
    y, f = ssd.causal_conv(x, gpu(q["w"]), None, init)
    assert y.shape == x.shape and torch.equal(f, init)
    g = ssd.causal_conv_backward(x, gpu(q["w"]), x, None, init, dfin)
    assert torch.equal(g["dinit"], dfin) and not bool(g["dweight"].any()) and not bool(g["dbias"].any())
    g = ssd.causal_conv_backward(x, gpu(q["w"]), x)
    assert not bool(g["dinit"].any())
    y, f = ssd.causal_conv(torch.empty(0, 4, 10, device="cuda"), gpu(q["w"]))
    assert y.shape == (0, 4, 10) and f.shape == (0, 3, 10)
    assert ssd.causal_conv_step(x[:0, 0:0].reshape(0, 10), gpu(q["w"]), None, init[:0]).shape == (0, 10)


def test_graph_replays_equal_eager():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("conv graph")
    lens = [[40, 3, 100], [143]]
    q = make("bf16", 2, 143, 64, 4, lens, seed=8)
    d = {k: gpu(v) for k, v in q.items()}
    state = d["init"][:2].contiguous()

    def run(s):
        y, f = ssd.causal_conv(d["x"], d["w"], d["bias"], d["init"], d["ids"], q["n"])
        g = ssd.causal_conv_backward(d["x"], d["w"], d["dy"], d["bias"], d["init"], d["dfinal"], d["ids"], q["n"])
        return [y, f, ssd.causal_conv_step(d["x"][:, 0], d["w"], d["bias"], s)] + [g[k] for k in sorted(g)]

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
    import mamba_ssd_scan_chunked_amd as ssd
    announce("conv stream")
    q = make("f32", 2, 300, 50, 4, seed=9)
    d = {k: gpu(v) for k, v in q.items()}
    y0, f0 = ssd.causal_conv(d["x"], d["w"], d["bias"], d["init"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        y, f = ssd.causal_conv(d["x"].transpose(1, 2).contiguous().transpose(1, 2), d["w"], d["bias"], d["init"])
        torch.cuda.synchronize()
        y, f = ssd.causal_conv(d["x"], d["w"], d["bias"], d["init"], stream=handle)
        s.synchronize()
        assert torch.equal(y, y0) and torch.equal(f, f0)


def test_offsets_past_32_bits():
    """A row of more than 2^31 elements: its last tokens equal a run of their own."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("conv long row")
    T, D, tail = 420000, 5376, 40
    x = torch.randn(1, 4096, D, device="cuda").to(torch.bfloat16).repeat(1, 103, 1)[:, :T]
    w, b = torch.randn(D, 4, device="cuda"), torch.randn(D, device="cuda")
    y, f = ssd.causal_conv(x, w, b)
    y1, f1 = ssd.causal_conv(x[:, -tail:], w, b, x[:, -tail - 3:-tail].float().contiguous())
    assert torch.equal(y[:, -tail:], y1) and torch.equal(f, f1)
    del y
    dy = torch.zeros(1, T, D, device="cuda")
    dy[:, -tail:] = torch.randn(1, tail, D, device="cuda")
    g = ssd.causal_conv_backward(x, w, dy, b)
    g1 = ssd.causal_conv_backward(x[:, -tail:], w, dy[:, -tail:], b, x[:, -tail - 3:-tail].float().contiguous())
    assert torch.equal(g["dx"][:, -tail:], g1["dx"]) and torch.equal(g["dx"][:, -tail - 3:-tail], g1["dinit"])


def test_arguments_are_checked():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("conv arguments")
    x, w = torch.zeros(2, 5, 8, device="cuda"), torch.zeros(8, 4, device="cuda")
    ok = dict(init_state=torch.zeros(2, 3, 8, device="cuda"))
    for kind, f in (
            (TypeError, lambda: ssd.causal_conv(x.half(), w)), (TypeError, lambda: ssd.causal_conv(x, w.bfloat16())),
            (ValueError, lambda: ssd.causal_conv(x, w[:7])), (ValueError, lambda: ssd.causal_conv(x, w, w[:, 0][:7])),
            (ValueError, lambda: ssd.causal_conv(x, w.cpu())), (ValueError, lambda: ssd.causal_conv(x[0], w)),
            (ValueError, lambda: ssd.causal_conv(x, w, init_state=ok["init_state"][:1])),
            (ValueError, lambda: ssd.causal_conv(x, w, nseqs=3)),
            (ValueError, lambda: ssd.causal_conv(x, w, seq_idx=torch.zeros(2, 5, dtype=torch.int32, device="cuda"))),
            (TypeError, lambda: ssd.causal_conv(x, w, seq_idx=torch.zeros(2, 5, device="cuda"), nseqs=2)),
            (ValueError, lambda: ssd.causal_conv(x, w, y=torch.zeros(2, 8, 5, device="cuda").transpose(1, 2))),
            (TypeError, lambda: ssd.causal_conv(x, w, y=x.bfloat16())),
            (ValueError, lambda: ssd.causal_conv(x, w, final_state=torch.zeros(2, 4, 8, device="cuda"))),
            (ValueError, lambda: ssd.causal_conv_step(x[:, 0], w, None, torch.zeros(2, 8, 3, device="cuda").transpose(1, 2))),
            (ValueError, lambda: ssd.causal_conv_backward(x, w, x[:1])), (TypeError, lambda: ssd.causal_conv_backward(x, w, x.half())),
            (ssd.SSDError, lambda: ssd.causal_conv(x, w[:, :1])), (ssd.SSDError, lambda: ssd.causal_conv(x, w, y=x)),
            (ssd.SSDError, lambda: ssd.causal_conv(x, w, final_state=ok["init_state"], **ok)),
            (ValueError, lambda: ssd.causal_conv_backward(torch.zeros(8, 300, 8, device="cuda"), w, torch.zeros(8, 300, 8, device="cuda"),
                                                          workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(kind):
            f()


LONG = [
    # dtype, rows, tokens, channels, K.  Forward runs of 10 and 20 tokens (a round of four waves a
    # SIMD over the 64 and 72 workgroups of channels and rows), backward of 25 and 27 (three
    # waves a SIMD over 128 and 72).
    ("bf16", 16, 600, 2048, 4), ("f32", 8, 1111, 2052, 3),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "%s-b%d-T%d-D%d-K%d" % c)
def test_packed_rows_in_long_runs(case):
    """Runs of several groups of four tokens: sequences that start and end in any token of a
    group and of a run, several of them in a run, and some over several runs."""
    import mamba_ssd_scan_chunked_amd as ssd
    dt, b, T, D, K = case
    announce("conv long runs %s" % (case,))
    g = torch.Generator().manual_seed(T)
    lens = []
    for _ in range(b):
        row, left = [], T
        while left:
            longest = (3, 12, 200)[int(torch.randint(3, (1,), generator=g))]
            row.append(min(left, 1 + int(torch.randint(longest, (1,), generator=g))))
            left -= row[-1]
        lens.append(row)
    q = make(dt, b, T, D, K, lens, True, True, seed=T)
    d = {k: gpu(v) for k, v in q.items()}
    runs = ssd.conv_backward_workspace_size(ssd.conv_problem(b, T, D, K, q["n"], ssd.DTYPE_BF16 if dt == "bf16" else ssd.DTYPE_F32)) \
        // (D * (K + 1) * 4)
    assert T * b >= 24 * runs, "backward runs are shorter than this test is about"
    y, f = ssd.causal_conv(d["x"], d["w"], d["bias"], d["init"], d["ids"], q["n"])
    args = [d[k].double() for k in ("x", "w", "bias", "init")]
    yr, fr = ref.conv(*args, lens, True)
    size, _ = ref.conv(*[t.abs() for t in args], lens, False)
    # as in test_forward
    ref.check(y, yr.cpu(), size.cpu(), 1.1 * K + 8, "y")
    assert torch.equal(f.double(), fr)

    got = ssd.causal_conv_backward(d["x"], d["w"], d["dy"], d["bias"], d["init"], d["dfinal"], d["ids"], q["n"])
    lv = [t.detach().requires_grad_() for t in args]
    y, f = ref.conv(*lv, lens, True)
    grads = torch.autograd.grad((y * d["dy"].double()).sum() + (f * d["dfinal"].double()).sum(), lv)
    av = [t.detach().abs().requires_grad_() for t in args]
    ya, fa = ref.conv(*av, lens, False)
    scales = torch.autograd.grad((1.1 * ya * d["dy"].double().abs()).sum() + (fa * d["dfinal"].double().abs()).sum(), av)
    # as in test_backward, with K U32 size(pre) / 2 from the slope's argument for the largest size here
    n = K * float(ya.detach().max()) / 2 + K + 8
    for name, r, s, extra in zip(("dx", "dweight", "dbias", "dinit"), grads, scales, (0, 96 + runs / 16, 96 + runs / 16, 0)):
        ref.check(got[name], r.cpu(), s.cpu(), n + extra, name)


def test_far_apart_rows_are_copied():
    """Rows 2^31 elements apart and more are copied first."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("conv, rows 2^31 elements apart")
    D, ld = 40, 1 << 31
    wide = torch.empty(ld + D, dtype=torch.bfloat16, device="cuda")
    far = wide.as_strided((2, D), (ld, 1))
    far.copy_(torch.randn(2, D))
    x, w = far.contiguous(), torch.randn(D, 4, device="cuda")
    state = torch.randn(2, 3, D, device="cuda")
    other = state.clone()
    assert torch.equal(ssd.causal_conv_step(far, w, None, state), ssd.causal_conv_step(x, w, None, other))
    assert torch.equal(state, other)
    assert torch.equal(ssd.causal_conv(far[:, None], w)[0], ssd.causal_conv(x[:, None], w)[0])
    weight = torch.ones(D, device="cuda")
    assert torch.equal(ssd.gated_norm(far, far, weight), ssd.gated_norm(x, x, weight))
    a, c = ssd.residual_norm(far, None, weight), ssd.residual_norm(x, None, weight)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
