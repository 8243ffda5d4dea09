"""The binding's dealings with the library and with strides, without a GPU."""
import ctypes

import pytest

import mamba_ssd_scan_chunked_amd as ssd
from mamba_ssd_scan_chunked_amd import block


class Older:
    """The library as it was before the operators around the scan, or of another version."""

    def __init__(self, version):
        self._lib, self._version = ctypes.CDLL(ssd.library_path()), version

    def __getattr__(self, name):
        if name == "ssd_version":
            class Version:
                restype = None

                def __call__(this):
                    return self._version
            return Version()
        if name.startswith(("ssd_conv", "ssd_selective", "ssd_gated", "ssd_residual")):
            raise AttributeError("undefined symbol: " + name)
        return getattr(self._lib, name)


@pytest.mark.parametrize("version", [5, 4])
def test_an_older_library_asks_for_a_rebuild(monkeypatch, version):
    older = Older(version)
    monkeypatch.setattr(ssd, "_lib", None)
    monkeypatch.setattr(ssd.ctypes, "CDLL", lambda path: older)
    with pytest.raises(ImportError, match="rebuild it"):
        ssd.load_library()
    assert ssd._lib is None


def test_a_step_takes_rows_any_distance_apart():
    """The step has no tile, so the prompt calls' bound on its offsets is not its own.  A batch
    of no rows gets past every check (and, without a device, no further)."""
    lib = ssd.load_library()
    far = dict(batch=0, seqlen=1, channels=64, dstate=16)
    for k in ("ldx", "lddt", "ldz", "ldb", "ldc"):
        for ld, codes in (((1 << 25), (0, 8)), ((1 << 31) - 1, (0, 8)), (1 << 31, (2,))):
            p = ssd.selective_problem(**far, **{k: ld})
            args = [0x10000000 * (i + 1) for i in range(11)]
            assert lib.ssd_selective_step(ctypes.byref(p), *args, None) in codes, (k, ld)
            assert ssd.selective_workspace_size(p) == 0


def test_rows_further_apart_than_a_kernel_reads_are_copied():
    torch = pytest.importorskip("torch")
    wide = torch.zeros(4 * 100)
    t = wide.as_strided((4, 8), (100, 1))
    same, ld = block._rows(t, 101)
    assert same is t and ld == 100
    copy, ld = block._rows(t, 100)
    assert copy.is_contiguous() and ld == 8 and torch.equal(copy, t)
