"""The scan's gradients at the edges of what the call accepts.

Tolerances as derived in tests/test_backward_gpu.py.
"""
import ctypes
import threading

import pytest
import torch

from tests.test_backward_gpu import BF16, F32, TOL_F32_TC, TOL_TC, _check, _scan_check, _scan_got, _scan_problem, _scan_want

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


def test_threads_with_shapes_of_their_own():
    """Calls from several threads, whose kernels need different amounts of
    shared memory: each gets what it gets alone.  The C calls alone, so that
    they meet; 4 threads whose first kernel needs 75 or 50 KB, 4 with 13 KB."""
    lib = ssd.load_library()
    shapes = 2 * [(1, 4, 1, 480, 64, 1), (1, 4, 2, 16, 16, 1), (1, 4, 1, 128, 256, 1), (1, 4, 1, 32, 16, 1)]
    jobs = []
    for k, (B, S, H, P, N, G) in enumerate(shapes):
        t = _scan_problem(B, S, H, P, N, G, F32, seed=30 + k)
        want = _scan_got(t, H, P, N, G)
        out = ssd.ScanGrads(*(torch.empty_like(v) for v in want))
        d = ssd.dims(B, S, H, P, N, G)
        ws = torch.empty(ssd.ssd_chunk_scan_backward_workspace_size(d, ssd.SSD_F32), dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        ptrs = [t[n].data_ptr() for n in ("xbc", "dt", "dt_bias", "A", "D", "h0", "dy", "dhS")] + [v.data_ptr() for v in out]
        args = [ctypes.byref(d), ssd.SSD_F32, ssd.SSD_DT_SOFTPLUS, *ptrs, ws.data_ptr(), ws.numel(), stream.cuda_stream]
        jobs.append((args, t, ws, stream, out, want))
    torch.cuda.synchronize()
    status = [set() for _ in jobs]

    def work(k):
        for _ in range(3000):
            status[k].add(lib.ssd_chunk_scan_backward(*jobs[k][0]))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(jobs))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert all(st == {ssd.SSD_OK} for st in status), status
    for *_, out, want in jobs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("act", [F32, BF16])
@pytest.mark.parametrize("S,H,P,G", [(1, 2, 64, 1), (45, 4, 64, 2), (70, 3, 16, 1), (33, 2, 4, 2)])
def test_scan_gradients_of_states_of_512(S, H, P, G, act):
    """The widest state that the forward takes, as it takes it."""
    N = 512
    t = _scan_problem(2, S, H, P, N, G, act, seed=40)
    ssd.chunk_scan(t["xbc"], t["dt"], t["A"], nheads=H, headdim=P, dstate=N, ngroups=G)
    _scan_check(_scan_got(t, H, P, N, G), _scan_want(t, H, P, N, G), act, False)


@pytest.mark.parametrize("act", [F32, BF16])
@pytest.mark.parametrize("S,H,P,N,G", [(37, 1, 512, 32, 1), (16, 2, 1024, 16, 2), (50, 3, 500, 64, 1), (50, 2, 500, 64, 1), (1, 1, 640, 8, 1)])
def test_scan_gradients_of_wide_heads(S, H, P, N, G, act):
    """Head sizes whose chunks have 16 rows, the last one partly filled; a head
    size that is not a multiple of the columns a warp takes."""
    if act == BF16 and (H * P + 2 * G * N) % 8:
        pytest.skip("rows of whole 16-byte vectors")
    t = _scan_problem(2, S, H, P, N, G, act, seed=41)
    ssd.chunk_scan(t["xbc"], t["dt"], t["A"], nheads=H, headdim=P, dstate=N, ngroups=G)
    _scan_check(_scan_got(t, H, P, N, G), _scan_want(t, H, P, N, G), act, False)


@pytest.mark.parametrize("B,S,H,G", [(40, 32, 8, 2), (500, 3, 8, 1), (17, 2, 32, 8), (100, 20, 24, 3)])
def test_large_batches_of_short_sequences_on_the_tensor_cores(B, S, H, G):
    """Few rows a sequence, many in all; the fp32 pipes keep calls of up to 32 rows."""
    P, N = 64, 128
    before = ssd.ssd_launch_counts()
    t = _scan_problem(B, S, H, P, N, G, BF16, seed=90 + S)
    _scan_check(_scan_got(t, H, P, N, G), _scan_want(t, H, P, N, G), BF16, True)
    few = _scan_problem(32 // S, S, H, P, N, G, BF16, seed=91)
    _scan_check(_scan_got(few, H, P, N, G), _scan_want(few, H, P, N, G), BF16, False)
    after = ssd.ssd_launch_counts()
    assert [after[k] - before[k] for k in ("scan_backward_tc", "scan_backward_simt")] == [1, 1]
