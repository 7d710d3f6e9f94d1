"""The tensor-core gradients of the scan where a CTA walks many heads and the
states kernel takes two heads a CTA: what the large calls run on, compared in
value with the formulas in 64 bits.

Tolerances as derived in tests/test_backward_gpu.py, but for dA where its rows
cancel.  dA is one number a head, the sum over rows and state elements (p, n)
of dt_t exp(a_t) lam_t h_{t-1}.  On the tensor cores h and lam are each off by
two roundings to two bf16, 2^-16 of the element at most, 2^-16 / sqrt(3) in
the root mean square: four of them in quadrature, 2^-16 * 2 / sqrt(3) of a
product.  At worst an element's error is the same in every row, and those of
different elements are independent, so the sum is off by that times the 2-norm
over (p, n) of sum_t |dt_t exp(a_t) lam_t h_{t-1}|; four times that for the
tail.
"""
import pytest
import torch

from tests.test_backward_gpu import BF16, _scan_check, _scan_got, _scan_problem, _scan_want

pytestmark = pytest.mark.gpu

ssd = pytest.importorskip("ssd_scan_gb300")

P, N = 64, 128
DA_TOL = 4 * 2 / 3 ** 0.5 * 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ssd.load_library()
    yield
    assert ssd.ssd_read_device_error() == ssd.SSD_OK


def _split(B, S, H, G):
    """The CTAs that share the heads of a (chunk, group), from the workspace:
    their shares of dB | dC are what is left of it."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    units = B * H * -(-S // 128)
    fixed = up(units * 1412 * 4) + 2 * up(units * 2 * N * P * 2) + up(B * -(-S // 128) * 3 * H * 4)
    shares = ssd.ssd_chunk_scan_backward_workspace_size(ssd.dims(B, S, H, P, N, G), ssd.SSD_BF16) - fixed
    one = B * S * 2 * G * N * 4
    assert shares >= 0 and shares - shares // one * one < 256
    return max(1, shares // one)


def _dA_scale(t, H, G, softplus=True, bias=True):
    """[H]: the 2-norm over (p, n) of sum_t |dt_t exp(a_t) lam_t h_{t-1}|, the
    root of the sum of squares over sequences."""
    f = lambda k: t[k].double()  # noqa: E731
    B, S = t["dt"].shape[:2]
    x, b, c = f("xbc").split([H * P, G * N, G * N], -1)
    x = x.reshape(B, S, H, P)
    heads = lambda v: v.reshape(B, S, G, 1, N).expand(B, S, G, H // G, N).reshape(B, S, H, N)  # noqa: E731
    b, c, dt = heads(b), heads(c), f("dt")
    if softplus:
        v = dt + f("dt_bias") if bias else dt
        dt = torch.logaddexp(v, torch.zeros_like(v))
    a = dt * f("A")
    e = torch.exp(torch.clamp(a, max=0.0))[..., None, None]
    h = [f("h0")]
    for k in range(S):
        h.append(e[:, k] * h[-1] + (dt[:, k, :, None] * x[:, k])[..., None] * b[:, k, :, None])
    lam, total = f("dhS"), torch.zeros_like(h[0])
    for k in reversed(range(S)):
        lam = lam + f("dy")[:, k, :, :, None] * c[:, k, :, None]
        total += torch.where(a[:, k] > 0, 0.0, dt[:, k].abs())[..., None, None] * (e[:, k] * lam * h[k]).abs()
        lam = e[:, k] * lam
    return total.square().sum((0, 2, 3)).sqrt()


@pytest.mark.parametrize("B,S,H,G,per,last", [
    (1, 2048, 128, 8, 16, 16),  # a group's heads in one CTA
    (1, 700, 128, 2, 6, 4),     # split, the last CTA with fewer heads
    (2, 1030, 64, 4, 8, 8),
    (2, 300, 66, 2, 3, 3),      # an odd number of heads; groups that do not pair up
    (4, 2000, 9, 1, 5, 4),
    (1, 5000, 8, 1, 3, 2),      # many chunks
])
def test_scan_gradients_of_many_heads_a_cta(B, S, H, G, per, last):
    split, R = _split(B, S, H, G), H // G
    assert (-(-R // split), R - (split - 1) * -(-R // split)) == (per, last)
    before = ssd.ssd_launch_counts()["scan_backward_tc"]
    t = _scan_problem(B, S, H, P, N, G, BF16, seed=50 + H)
    got = _scan_got(t, H, P, N, G)
    assert ssd.ssd_launch_counts()["scan_backward_tc"] == before + 1
    _scan_check(got, _scan_want(t, H, P, N, G), BF16, True)


@pytest.mark.parametrize("B,S,H,G", [(2, 150, 8, 2), (1, 300, 128, 8), (3, 129, 7, 7)])
def test_tensor_core_sums_of_given_dt(B, S, H, G):
    """dt as given, zero and rising rows among it: dA a head at a time, zeros
    for a dt_bias that the forward ignores."""
    before = ssd.ssd_launch_counts()["scan_backward_tc"]
    t = _scan_problem(B, S, H, P, N, G, BF16, softplus=False, seed=60 + H)
    t["dt"][:, 3::7] *= -1
    got = _scan_got(t, H, P, N, G, softplus=False)
    want = _scan_want(t, H, P, N, G, softplus=False, bias=False)
    assert ssd.ssd_launch_counts()["scan_backward_tc"] == before + 1
    _scan_check(got, want, BF16, True, ("dxbc", "ddt", "dD", "dssm_state"))
    off = (got.dA.double() - want["dA"]).abs() / _dA_scale(t, H, G, softplus=False)
    assert float(off.max()) <= DA_TOL, f"{float(off.max()):.3e}"
    assert float(got.ddt_bias.abs().max()) == 0.0


@pytest.mark.parametrize("B,S,H,G", [(1, 100, 8, 2), (2, 1111, 16, 1), (1, 2048, 128, 8), (2, 33, 7, 1)])
def test_tensor_core_dA_a_head_at_a_time(B, S, H, G):
    t = _scan_problem(B, S, H, P, N, G, BF16, seed=70 + H)
    got, want = _scan_got(t, H, P, N, G), _scan_want(t, H, P, N, G)
    off = (got.dA.double() - want["dA"]).abs() / _dA_scale(t, H, G)
    assert float(off.max()) <= DA_TOL, f"{float(off.max()):.3e}"


@pytest.mark.parametrize("B,S,H,G", [(1, 1, 2, 1), (1, 2, 8, 2), (2, 127, 4, 4), (2, 129, 5, 5), (3, 513, 4, 1), (1, 290, 6, 2)])
def test_few_heads_are_as_exact_as_fp32_rows(B, S, H, G):
    """bf16 calls that the fp32 pipes take: held to their tolerances, rising and
    zero rows of a given dt among them."""
    before = ssd.ssd_launch_counts()["scan_backward_simt"]
    t = _scan_problem(B, S, H, P, N, G, BF16, seed=80 + S)
    _scan_check(_scan_got(t, H, P, N, G), _scan_want(t, H, P, N, G), BF16, False)
    t = _scan_problem(B, S, H, P, N, G, BF16, softplus=False, seed=S)
    t["dt"][:, 3::7] *= -1
    kw = dict(softplus=False, bias=False)
    got, want = _scan_got(t, H, P, N, G, **kw), _scan_want(t, H, P, N, G, **kw)
    _scan_check(got, want, BF16, False, ("dxbc", "ddt", "dD", "dssm_state"))
    if S > 1:
        _scan_check(got, want, BF16, False, ("dA",))
    assert ssd.ssd_launch_counts()["scan_backward_simt"] == before + 2
