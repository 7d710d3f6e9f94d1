"""The gated norm's gradients of tiny rows, with an eps of nothing or next to
nothing: 1 / rms is finite, its square is not.

Tolerances as derived in tests/test_backward_gpu.py.  y^2 below the smallest
normal number is off by up to 2^-150: relative to 2^-132, 2^-18 an element,
which over the 256 and more of a group's mean is 2^-22.
"""
import pytest
import torch

from tests import backward_ref as ref
from tests.test_backward_gpu import BF16, F32, TOL_F32, TOL_ROW, _check, _norm_problem

pytestmark = pytest.mark.gpu

ssd = pytest.importorskip("ssd_scan_gb300")

# a warp, a vector a thread, and a CTA that reads twice, in either type
SHAPES = [(F32, 512, 2), (BF16, 512, 2), (F32, 2048, 1), (BF16, 4096, 1), (F32, 4096, 1), (BF16, 8192, 1)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ssd.load_library()
    yield
    assert ssd.ssd_read_device_error() == ssd.SSD_OK


def _hold(got, want, act):
    row = TOL_F32 if act == F32 else TOL_ROW
    _check(got.dy, want["dy"], row, "dy")
    _check(got.dz, want["dz"], row, "dz")
    _check(got.dweight, want["dweight"], TOL_F32, "dweight")


@pytest.mark.parametrize("act,C,G", SHAPES)
def test_tiny_rows_without_eps(act, C, G):
    y, z, do, w = _norm_problem(2, 9, C, act, seed=3)
    y = y * 2.0 ** -67  # 2 randn before: a mean square of 2^-132
    assert bool(torch.isfinite(ssd.gated_group_rmsnorm(y, z, w, ngroups=G, eps=0.0)).all())
    _hold(ssd.gated_group_rmsnorm_backward(do, y, z, w, ngroups=G, eps=0.0), ref.norm_backward(do, y, z, w, G, 0.0), act)


@pytest.mark.parametrize("act,C,G", SHAPES)
def test_zero_rows_with_a_tiny_eps(act, C, G):
    eps = 2.0 ** -133
    y, z, do, w = _norm_problem(2, 9, C, act, seed=4)
    y[:, 2:5] = 0
    assert bool(torch.isfinite(ssd.gated_group_rmsnorm(y, z, w, ngroups=G, eps=eps)).all())
    _hold(ssd.gated_group_rmsnorm_backward(do, y, z, w, ngroups=G, eps=eps), ref.norm_backward(do, y, z, w, G, eps), act)
