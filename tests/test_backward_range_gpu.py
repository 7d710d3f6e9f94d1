"""The scan's gradients at the edges of what the call accepts.

Tolerances as derived in tests/test_backward_gpu.py.
"""
import pytest
import torch

from tests.test_backward_gpu import BF16, TOL_F32_TC, TOL_TC, _check, _scan_got, _scan_problem, _scan_want

pytestmark = pytest.mark.gpu

ssd = pytest.importorskip("ssd_scan_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ssd.load_library()
    yield
    assert ssd.ssd_read_device_error() == ssd.SSD_OK


@pytest.mark.parametrize("S", [40, 200])
@pytest.mark.parametrize("log2", [0, 36])
def test_large_finite_rows_give_finite_gradients(S, log2):
    """x and dy times 2^36: x . dy near 2^75, with rows that decay by 2^56 over
    32 of them.  Every gradient the formulas give stays below 2^100."""
    H, P, N, G = 8, 64, 128, 2
    t = _scan_problem(2, S, H, P, N, G, BF16, seed=21, softplus=False)
    gen = torch.Generator(device="cuda").manual_seed(22)
    t["dt"] = 1.15 + 0.1 * torch.rand(2, S, H, generator=gen, device="cuda")
    t["A"] = -torch.ones(H, device="cuda")
    k = 2.0 ** log2
    t["xbc"][..., :H * P] *= k
    t["dy"] *= k
    t["h0"] *= k
    t["dhS"] *= k
    before = ssd.ssd_launch_counts()["scan_backward_tc"]
    kw = dict(softplus=False, bias=False)
    got, want = _scan_got(t, H, P, N, G, **kw), _scan_want(t, H, P, N, G, **kw)
    assert ssd.ssd_launch_counts()["scan_backward_tc"] == before + 1
    x = H * P
    _check(got.dxbc[..., :x], want["dxbc"][..., :x], TOL_TC, "dx")
    _check(got.dxbc[..., x:], want["dxbc"][..., x:], TOL_TC, "dB | dC")
    for n in ("ddt", "dA", "dD", "dssm_state"):
        _check(getattr(got, n), want[n], TOL_F32_TC, n)
