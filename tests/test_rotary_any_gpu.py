"""The norm with rotation of heads that no packs fit, over more heads and tokens than a launch has
workgroups: each workgroup adds many of them to its sums of the weights' gradients."""
import pytest

import test_rotary_gpu as rotary

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("case", [("bf16", 1, 700, 2, 3, 33, 32, "far"), ("f32", 2, 500, 1, 2, 7, 4, None),
                                  ("f32", 1, 400, 1, 2, 199, 100, "far"), ("bf16", 1, 900, 1, 1, 5, 0, None)],
                         ids=lambda c: "%s-N%d-R%d" % (c[0], c[5], c[6]))
def test_many_heads_without_packs(case, pairs):
    import mamba_ssd_scan_chunked_amd as ssd
    rotary.announce("rotary norm without packs %s interleaved=%s" % (case, pairs))
    rotary.check(ssd, rotary.make(*case), pairs)
