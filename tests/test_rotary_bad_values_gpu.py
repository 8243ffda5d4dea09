"""Infinite and NaN values of the norm with rotation stay where the formulas put them: a channel
behind the rotated ones meets no other one, a rotated one its pair only."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# whole packs of 8, 4, 2 and 1 channels, two packs a lane, and heads without packs
SIZES = [(128, 64), (64, 32), (80, 40), (72, 36), (100, 50), (96, 32), (36, 18), (20, 10), (1000, 8), (33, 2), (7, 4)]


def announce(msg):
    print("[case] " + msg, flush=True)


def make(dt, N, R):
    g = torch.Generator().manual_seed(N + R)
    r = lambda *s: torch.randn(*s, generator=g).cuda()      # noqa: E731
    tokens, G, H = 9, 2, 3
    return {"B": r(tokens, G, N).to(TYPES[dt]), "C": r(tokens, H, N).to(TYPES[dt]), "b_weight": r(N), "c_weight": r(N),
            "freqs": r(R // 2), "dB": r(tokens, G, N), "dC": r(tokens, H, N)}


def passes(ssd, q, pairs):
    args = [q[k] for k in ("B", "C", "b_weight", "c_weight", "freqs")]
    B, C = ssd.rotary_norm(*args, interleaved=pairs)
    return dict(ssd.rotary_norm_backward(*args, q["dB"], q["dC"], interleaved=pairs), B=B, C=C)


def partner(c, R, pairs):
    """The channels that a value of channel c reaches through the rotation."""
    if c >= R:
        return [c]
    if pairs:
        return [c, c ^ 1]
    return [c, (c + R // 2) % R]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("N,R", SIZES)
def test_bad_values_stay_in_their_channel(N, R, pairs, dt):
    import mamba_ssd_scan_chunked_amd as ssd
    announce("rotary norm, bad values N=%d R=%d %s interleaved=%s" % (N, R, dt, pairs))
    q = make(dt, N, R)
    clean = passes(ssd, q, pairs)
    for c in sorted({0, R - 1, R, R + (N - R) // 2, N - 1}):
        reached = torch.zeros(N, dtype=torch.bool, device="cuda")
        reached[partner(c, R, pairs)] = True
        for bad in (float("nan"), float("inf")):
            # a weight: outputs of its channel in every head; the weights' gradients hold no weight
            got = passes(ssd, dict(q, b_weight=q["b_weight"].index_fill(0, torch.tensor([c], device="cuda"), bad)), pairs)
            assert torch.equal(got["B"][..., ~reached], clean["B"][..., ~reached]), (c, bad)
            assert not torch.isfinite(got["B"][..., c]).any(), (c, bad)
            for k in ("C", "dC", "db_weight", "dc_weight"):
                assert torch.equal(got[k], clean[k]), (k, c, bad)
            # a gradient of one token and head: all of that head's, and its channel's weight
            d = q["dC"].clone()
            d[4, 1, c] = bad
            got = passes(ssd, dict(q, dC=d), pairs)
            assert torch.equal(got["dc_weight"][~reached], clean["dc_weight"][~reached]), (c, bad)
            assert not torch.isfinite(got["dc_weight"][c]), (c, bad)
            others = torch.ones(9, 3, dtype=torch.bool, device="cuda")
            others[4, 1] = False
            assert torch.equal(got["dC"][others], clean["dC"][others]), (c, bad)
            for k in ("B", "C", "dB", "db_weight"):
                assert torch.equal(got[k], clean[k]), (k, c, bad)
