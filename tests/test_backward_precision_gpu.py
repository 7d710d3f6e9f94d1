"""How exact the tensor-core gradients' fp32 outputs are, in the 2-norm against
64 bits, beyond the tolerances of tests/test_backward_gpu.py.

The initial state's gradient: the walk over the chunks multiplies all 24 bits
of the scaled rows, so a term carries the exponential (2^-22), the factor and
the product (2^-24 each), and its way into the sum: 8 steps of the tensor
pipe at the sum's size, which cut off up to 2^-23 each, and a rounding a chunk.
In quadrature 2^-22 sqrt(1 + 8 / 4) and the roundings: under 2^-21 = 4.8e-7,
twice that allowed.

Gradients inside a chunk: the decay between two rows is the product of two
exponentials (2^-22 each) of double-float differences, x . dy and C . B are sums
of the tensor pipe (4 and 8 steps, 2^-23), and the sums over rows in fp32 trees
of up to 12 roundings: 2^-22 sqrt(2 + 3) and the roundings, under 6e-7; 1e-6
allowed.
"""
import pytest
import torch

from tests.test_backward_gpu import BF16, _scan_got, _scan_problem, _scan_want

pytestmark = pytest.mark.gpu

ssd = pytest.importorskip("ssd_scan_gb300")

P, N = 64, 128


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ssd.load_library()
    yield
    assert ssd.ssd_read_device_error() == ssd.SSD_OK


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("B,S,H,G", [(1, 128, 8, 2), (2, 300, 8, 1), (2, 1111, 16, 1), (1, 700, 128, 8)])
def test_initial_state_gradient(B, S, H, G):
    t = _scan_problem(B, S, H, P, N, G, BF16, seed=100 + S)
    t["dhS"] *= 0.0  # all of it from the rows
    got, want = _scan_got(t, H, P, N, G), _scan_want(t, H, P, N, G)
    assert _off(got.dssm_state, want["dssm_state"]) <= 2 * 2.0 ** -21


@pytest.mark.parametrize("decay", [0.02, 0.3, 1.1])
def test_gradients_inside_a_chunk(decay):
    """Decays of exp(-decay) a row: 2^-51 over a block of 32 rows at most."""
    B, S, H, G = 4, 128, 16, 2
    t = _scan_problem(B, S, H, P, N, G, BF16, seed=110, softplus=False)
    gen = torch.Generator(device="cuda").manual_seed(111)
    t["dt"] = 1 + 0.05 * torch.rand(B, S, H, generator=gen, device="cuda")
    t["A"] = -decay * (0.9 + 0.1 * torch.rand(H, generator=gen, device="cuda"))
    kw = dict(state=False, softplus=False, bias=False)
    before = ssd.ssd_launch_counts()["scan_backward_tc"]
    got, want = _scan_got(t, H, P, N, G, **kw), _scan_want(t, H, P, N, G, **kw)
    assert ssd.ssd_launch_counts()["scan_backward_tc"] == before + 1
    assert _off(got.ddt, want["ddt"]) <= 1e-6


def test_gradients_beside_a_cliff():
    """One row in 32 decays by 2^-58, the others hardly: the factors that a
    pair's decay is split into are 2^58 and 2^-58 on one side of it, and their
    exponents' last bits 2^-18."""
    B, S, H, G = 4, 128, 16, 2
    t = _scan_problem(B, S, H, P, N, G, BF16, seed=120, softplus=False)
    gen = torch.Generator(device="cuda").manual_seed(121)
    t["dt"] = 0.01 * (1 + torch.rand(B, S, H, generator=gen, device="cuda"))
    t["dt"][:, 31::32] = 40.0 + 0.2 * torch.rand(B, S // 32, H, generator=gen, device="cuda")
    t["xbc"][:, 31::32, :H * P] = 0  # else these rows' dt makes up all of the gradients
    t["A"] = -torch.ones(H, device="cuda")
    kw = dict(state=False, softplus=False, bias=False)
    got, want = _scan_got(t, H, P, N, G, **kw), _scan_want(t, H, P, N, G, **kw)
    assert _off(got.ddt, want["ddt"]) <= 1e-6
