"""The norm of B and C with the rotation by position, and its gradients, against the 64-bit form."""
import pytest
import torch

import block_ref as ref
import recurrence_ref as rr
from block_ref import U32

pytestmark = pytest.mark.gpu

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def announce(msg):
    print("[case] " + msg, flush=True)


def gpu(v):
    return v.cuda() if torch.is_tensor(v) else v


def make(dt, b, T, G, H, N, R, positions="far", seed=0):
    g = torch.Generator().manual_seed(seed + 11 * T + N + R)
    q = {"B": torch.randn(b, T, G, N, generator=g).to(TYPES[dt]), "C": (torch.randn(b, T, H, N, generator=g) * 3).to(TYPES[dt]),
         "b_weight": torch.randn(N, generator=g), "c_weight": torch.randn(N, generator=g),
         "freqs": (10000.0 ** (-torch.arange(R // 2).double() / max(1, R // 2))).float(),
         "dB": torch.randn(b, T, G, N, generator=g), "dC": torch.randn(b, T, H, N, generator=g), "positions": None}
    if positions == "far":
        q["positions"] = torch.randint(-70000, 3000000, (b, T), generator=g, dtype=torch.int32)
    return q


def names(q):
    return [gpu(q[k]) for k in ("B", "C", "b_weight", "c_weight", "freqs")]


def forward(ssd, q, pairs, **kw):
    return ssd.rotary_norm(*names(q), positions=gpu(q["positions"]), interleaved=pairs, eps=EPS, **kw)


def backward(ssd, q, pairs, **kw):
    return ssd.rotary_norm_backward(*names(q), gpu(q["dB"]), gpu(q["dC"]), positions=gpu(q["positions"]),
                                    interleaved=pairs, eps=EPS, **kw)


def check(ssd, q, pairs):
    B, C = forward(ssd, q, pairs)
    got = backward(ssd, q, pairs)
    assert set(got) == {"dB", "dC", "db_weight", "dc_weight"}
    b, T = q["B"].shape[:2]
    N, R = q["B"].shape[-1], 2 * q["freqs"].numel()
    positions = (torch.arange(T).expand(b, T) if q["positions"] is None else q["positions"]).reshape(-1)
    turn = rr.turn_error(q["freqs"], positions)
    n = rr.norm_depth(N)
    for k, out in (("B", B), ("C", C)):
        assert out.dtype == q[k].dtype and out.shape == q[k].shape and out.is_contiguous()
        u = q[k].double().reshape(-1, q[k].shape[2], N)
        w, d = q[k.lower() + "_weight"].double(), q["d" + k].double().reshape(u.shape)
        r = 1 / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS)
        v = u * r * w
        want = rr.rotate(v, q["freqs"], positions, pairs).view(out.shape)
        # r: half the sum's roundings and four; three products, the turn's two and its sum
        size = rr.both_of_pair(v.abs(), R, pairs).view(out.shape)
        rr.check(out, want, ((n / 2 + 10) * U32 + turn) * size, k)
        # gradients: e turned back, e w, the mean of e w hat, their difference
        e = rr.rotate(d, q["freqs"], positions, pairs, transposed=True)
        es = rr.both_of_pair(d.abs(), R, pairs)
        e_err = (3 * U32 + turn) * es
        hat = u * r
        mean = (e * w * hat).mean(-1, keepdim=True)
        du = r * (e * w - hat * mean)
        sizes = (es * w.abs() * hat.abs()).mean(-1, keepdim=True)
        room = r * (e_err * w.abs() + (n + 12) * U32 * es * w.abs()
                    + hat.abs() * ((e_err * w.abs() * hat.abs()).mean(-1, keepdim=True) + (3 * n + 20) * U32 * sizes))
        rr.check(got["d" + k], du.view(out.shape), room.view(out.shape), "d" + k)
        terms = es * hat.abs()
        rr.check(got["d" + k.lower() + "_weight"], (e * hat).sum((0, 1)),
                 ((e_err * hat.abs()) + (n / 2 + 8) * U32 * terms).sum((0, 1))
                 + (u.shape[0] * u.shape[1] + 20) * U32 * terms.sum((0, 1)), "d%s_weight" % k)


CASES = [
    # dtype, rows, tokens, heads of B and C, N, R, positions
    ("bf16", 2, 65, 1, 1, 128, 128, "far"), ("f32", 2, 65, 1, 1, 128, 128, "far"),
    ("bf16", 1, 1, 1, 1, 128, 128, "far"), ("f32", 3, 1, 2, 4, 64, 64, None),
    ("bf16", 1, 200, 8, 32, 64, 64, "far"), ("bf16", 2, 33, 2, 2, 256, 256, None), ("f32", 2, 33, 2, 6, 256, 128, "far"),
    ("bf16", 2, 17, 3, 6, 80, 40, "far"), ("f32", 2, 17, 3, 6, 80, 40, "far"),
    ("bf16", 2, 9, 3, 3, 96, 96, "far"), ("bf16", 1, 31, 1, 2, 72, 36, None), ("f32", 1, 31, 5, 5, 100, 50, "far"),
    ("bf16", 1, 11, 2, 2, 7, 6, "far"), ("f32", 1, 11, 2, 3, 1, 0, "far"), ("bf16", 2, 5, 1, 1, 2, 2, None),
    ("bf16", 2, 40, 2, 2, 128, 0, None),                                    # no rotation
    ("f32", 1, 7, 1, 3, 33, 2, "far"), ("bf16", 1, 13, 1, 1, 1024, 1024, "far"), ("f32", 1, 13, 2, 1, 1000, 998, None),
    ("bf16", 1, 6, 80, 1, 128, 64, "far"), ("f32", 1, 9, 1, 1, 512, 512, "far"), ("bf16", 3, 700, 1, 1, 16, 16, None),
    ("bf16", 1, 9, 1, 2, 192, 192, "far"), ("bf16", 1, 9, 3, 2, 320, 160, "far"), ("f32", 1, 5, 2, 2, 6, 4, None),
]


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s-%dx%d-G%d-H%d-N%d-R%d-%s" % c)
def test_norm_and_rotation(case, pairs):
    import mamba_ssd_scan_chunked_amd as ssd
    announce("rotary norm %s interleaved=%s" % (case, pairs))
    check(ssd, make(*case), pairs)


def test_many_tokens():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("rotary norm, many tokens")
    for case in (("bf16", 2, 3001, 2, 4, 64, 64, None), ("f32", 1, 5003, 1, 1, 128, 64, "far"), ("bf16", 1, 9001, 1, 1, 32, 32, "far")):
        check(ssd, make(*case), False)


def test_gradients_against_differences():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("rotary norm differences")
    for pairs in (False, True):
        q = make("f32", 1, 6, 2, 3, 24, 16)
        got = backward(ssd, q, pairs)
        w = {k: v.double() for k, v in q.items() if k != "freqs" and k != "positions"}

        def loss(v):
            total = 0.0
            for k in ("B", "C"):
                u = v[k].reshape(-1, v[k].shape[2], 24)
                hat = u / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS)
                out = rr.rotate(hat * v[k.lower() + "_weight"], q["freqs"], q["positions"].reshape(-1), pairs)
                total += float((out * w["d" + k].view(u.shape)).sum())
            return total

        g = torch.Generator().manual_seed(2)
        for name in ("B", "C", "b_weight", "c_weight"):
            along, h = torch.randn(w[name].shape, generator=g).double(), 1e-5
            lo, hi = dict(w), dict(w)
            lo[name], hi[name] = w[name] - h * along, w[name] + h * along
            part = got["d" + name].cpu().double() * along
            slope = (loss(hi) - loss(lo)) / (2 * h)
            assert abs(float(part.sum()) - slope) <= 1e-5 * float(part.abs().sum()), name


def test_far_positions():
    """Angles of the farthest positions: still those of the exact product position * freq."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("rotary norm far positions")
    q = make("f32", 1, 8, 1, 1, 64, 64)
    q["positions"] = torch.tensor([[0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 999999937]], dtype=torch.int32)
    for pairs in (False, True):
        check(ssd, q, pairs)


def test_relative_positions():
    """What the rotation is for: <C_t, B_s> depends on t - s only."""
    import mamba_ssd_scan_chunked_amd as ssd
    announce("rotary norm relative positions")
    q = make("f32", 1, 50, 1, 1, 64, 64)
    products = []
    for start in (0, 1000, 123456):
        q["positions"] = (torch.arange(50, dtype=torch.int32) + start)[None]
        B, C = (t.cpu().double()[0, :, 0] for t in forward(ssd, q, False))
        products.append(C @ B.t())
    size = float((C.norm(dim=-1).max() * B.norm(dim=-1).max()))
    # both vectors carry (depth / 2 + 10 + turn) roundings of their length
    turn = rr.turn_error(q["freqs"], q["positions"])
    bound = 2 * 2 * ((rr.norm_depth(64) / 2 + 12) * U32 + turn) * 2 * size
    assert float((products[0] - products[1]).abs().max()) <= bound and float((products[0] - products[2]).abs().max()) <= bound


def test_rows_of_zeros_and_extremes():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("rotary norm zeros")
    q = make("bf16", 1, 4, 2, 2, 32, 32)
    q["B"].zero_()
    B, C = forward(ssd, q, False)
    got = backward(ssd, q, False)
    assert not B.any() and all(torch.isfinite(t).all() for t in got.values()) and not got["db_weight"].any()
    # a bad head stays in its own head
    clean = forward(ssd, q, False)[1]
    q["C"][0, 1, 1, 3] = float("nan")
    C = forward(ssd, q, False)[1]
    keep = torch.ones(1, 4, 2, 32, dtype=torch.bool)
    keep[0, 1, 1] = False
    assert torch.equal(C.cpu()[keep], clean.cpu()[keep]) and torch.isnan(C.cpu()[0, 1, 1]).all()


def test_slices_shapes_and_empty():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("rotary norm slices")
    for dt, N, R in (("bf16", 128, 128), ("f32", 20, 10), ("bf16", 9, 4)):
        q = make(dt, 2, 70, 2, 3, N, R)
        wide = torch.full((2, 70, 5 * N + 7), float("nan"), dtype=TYPES[dt], device="cuda")
        s = dict(q)
        s["B"], s["C"] = wide[..., 3:3 + 2 * N].unflatten(-1, (2, N)), wide[..., 3 + 2 * N:3 + 5 * N].unflatten(-1, (3, N))
        s["B"].copy_(q["B"])
        s["C"].copy_(q["C"])
        for a, b in zip(forward(ssd, s, True), forward(ssd, q, True)):
            assert torch.equal(a, b)
        got, want = backward(ssd, s, True), backward(ssd, q, True)
        assert all(torch.equal(got[k], want[k]) for k in want)
        # heads before tokens in memory: copied
        t = dict(q, B=gpu(q["B"]).transpose(1, 2).contiguous().transpose(1, 2))
        assert torch.equal(forward(ssd, t, False)[0], forward(ssd, q, False)[0])
        # single tokens (b, G, N) at their own positions
        one = dict(q, B=gpu(q["B"])[:, 5], C=gpu(q["C"])[:, 5], positions=q["positions"][:, 5].contiguous())
        for a, b in zip(forward(ssd, one, False), forward(ssd, q, False)):
            assert torch.equal(a, b[:, 5])
    # without positions: the index along the dimension before the heads
    q = make("f32", 3, 8, 1, 1, 16, 16, None)
    a = forward(ssd, q, False)[0]
    b = forward(ssd, dict(q, positions=torch.arange(8, dtype=torch.int32).expand(3, 8)), False)[0]
    assert torch.equal(a, b)
    for b_, T in ((0, 4), (2, 0)):
        q = make("bf16", b_, T, 2, 2, 16, 16)
        B, C = forward(ssd, q, False)
        got = backward(ssd, q, False)
        assert B.shape == (b_, T, 2, 16) and not got["db_weight"].any() and not got["dc_weight"].any()


def test_graph_replays_equal_eager():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("rotary norm graph")
    s = {k: gpu(v) for k, v in make("bf16", 2, 900, 2, 4, 128, 128).items()}
    p = ssd.rotary_problem(1800, 2, 4, 128, 128)
    ws = torch.empty(max(1, ssd.rotary_norm_backward_workspace_size(p)), dtype=torch.uint8, device="cuda")

    def work():
        g = backward(ssd, s, False, workspace=ws)
        return list(forward(ssd, s, False)) + [g[k] for k in sorted(g)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for k in range(4):
        new = make("bf16", 2, 900, 2, 4, 128, 128, seed=90 + k)
        for name in ("B", "C", "dB", "dC", "positions"):
            s[name].copy_(new[name])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for a, b in zip(got, work()):
            assert torch.equal(a, b)


def test_results_repeat_on_other_streams():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("rotary norm streams")
    s = {k: gpu(v) for k, v in make("f32", 2, 700, 1, 2, 64, 64).items()}
    want, g0 = forward(ssd, s, False), backward(ssd, s, False)
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream, 0):
        out, g = forward(ssd, s, False, stream=stream), backward(ssd, s, False, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and all(torch.equal(g[k], g0[k]) for k in g0)


def test_offsets_past_32_bits():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("rotary norm far offsets")
    ld = (1 << 30) + 3
    big = torch.empty(4 * ld + 64, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((5, 1, 64), (ld, 64, 1))
    q = make("bf16", 1, 5, 1, 1, 64, 64)
    x.copy_(q["B"][0])
    args = [gpu(q[k]) for k in ("b_weight", "c_weight", "freqs")]
    a, b = ssd.rotary_norm(x, x, *args), ssd.rotary_norm(x.contiguous(), x.contiguous(), *args)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    del big, x
    T = (1 << 25) + 11                                      # outputs past 2^32 bytes
    B = torch.randn(1, 1, 64, device="cuda").to(torch.bfloat16).expand(T, 1, 64).contiguous()
    positions = torch.full((T,), 77, dtype=torch.int32, device="cuda")
    out = ssd.rotary_norm(B, B[:, :, :], *args, positions=positions)[1]
    assert torch.equal(out, out[:1].expand_as(out))


def test_arguments_are_checked():
    import mamba_ssd_scan_chunked_amd as ssd
    announce("rotary norm arguments")
    q = {k: gpu(v) for k, v in make("bf16", 2, 10, 2, 4, 16, 16).items()}
    good = names(q)
    for at, bad, err in ((0, q["B"].half(), TypeError), (0, q["B"].cpu(), ValueError), (0, q["B"][0, 0], ValueError),
                         (1, q["C"].float(), TypeError), (1, q["C"][:, :9], ValueError), (1, q["C"][..., :8], ValueError),
                         (1, q["C"].cpu(), ValueError), (2, q["b_weight"].double(), TypeError), (3, q["c_weight"][:8], ValueError),
                         (4, q["freqs"][None], ValueError), (4, torch.ones(9, device="cuda"), ssd.SSDError),
                         (4, q["freqs"].double(), TypeError)):
        args = list(good)
        args[at] = bad
        with pytest.raises(err):
            ssd.rotary_norm(*args)
        with pytest.raises(err):
            ssd.rotary_norm_backward(*args, q["dB"], q["dC"])
    for kw, err in (({"positions": q["positions"].long()}, TypeError), ({"positions": q["positions"][0]}, ValueError),
                    ({"eps": -1.0}, ssd.SSDError), ({"B_out": torch.empty_like(q["C"])}, ValueError),
                    ({"B_out": q["B"]}, ssd.SSDError), ({"C_out": q["C"].float()}, TypeError)):
        with pytest.raises(err):
            ssd.rotary_norm(*good, **kw)
    with pytest.raises(TypeError):
        ssd.rotary_norm_backward(*good, q["dB"].bfloat16(), q["dC"])
    with pytest.raises(ValueError):
        ssd.rotary_norm_backward(*good, q["dB"], q["dB"])
    big = torch.zeros(1, 1, 1, 1025, device="cuda")
    w = torch.ones(1025, device="cuda")
    with pytest.raises(ssd.SSDError):
        ssd.rotary_norm(big, big, w, w, torch.ones(4, device="cuda"))
