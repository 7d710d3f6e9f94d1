"""The forward row-exact scan and the decode step called by several threads at
once, each with a shape whose kernel needs another amount of shared memory: the
C calls alone, so that they meet."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

ssd = pytest.importorskip("ssd_scan_gb300")

BF16, F32 = torch.bfloat16, torch.float32
CALLS = 3000


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ssd.load_library()
    yield
    assert ssd.ssd_read_device_error() == ssd.SSD_OK


def _rows(B, S, H, P, N, G, act, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return dict(xbc=r(B, S, H * P + 2 * G * N).to(act), dt=r(B, S, H), A=-torch.rand(H, generator=gen, device="cuda") - 0.1,
                state=0.1 * r(B, H, P, N))


def _all_at_once(call, jobs):
    """call(*args) CALLS times in a thread per job; every status."""
    status = [set() for _ in jobs]

    def work(k):
        for _ in range(CALLS):
            status[k].add(call(*jobs[k]))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(jobs))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    return set().union(*status)


def test_row_exact_scans():
    lib, jobs, held = ssd.load_library(), [], []
    # one kernel form (32 state elements a thread): 4 threads that need 74 KB, 4 that need 41
    for k, (P, N, G) in enumerate(4 * [(64, 256, 1), (256, 32, 1)]):
        H = 2
        t = _rows(1, 4, H, P, N, G, F32, k)
        want, wstate, _ = ssd.chunk_scan(t["xbc"], t["dt"], t["A"], nheads=H, headdim=P, dstate=N, ngroups=G, ssm_state=t["state"])
        y, state, d, stream = torch.empty_like(want), torch.empty_like(wstate), ssd.dims(1, 4, H, P, N, G), torch.cuda.Stream()
        ptr = lambda v: v.data_ptr()  # noqa: E731
        jobs.append((ctypes.byref(d), ssd.SSD_F32, ssd.SSD_DT_SOFTPLUS, ptr(t["xbc"]), None, None, None, None, ptr(t["dt"]), None,
                     ptr(t["A"]), None, None, ptr(t["state"]), ptr(y), ptr(state), None, 0, stream.cuda_stream))
        held.append((t, d, stream, y, want, state, wstate))
    torch.cuda.synchronize()
    assert _all_at_once(lib.ssd_chunk_scan, jobs) == {ssd.SSD_OK}
    for _, _, _, y, want, state, wstate in held:
        assert torch.equal(y, want) and torch.equal(state, wstate)


def test_decode_steps():
    lib, jobs, held = ssd.load_library(), [], []
    # 4 threads whose kernels need some 20 KB, 4 of 1 KB
    for k, (H, P, N) in enumerate(4 * [(64, 64, 128), (2, 8, 16)]):
        t = _rows(2, 1, H, P, N, 1, BF16, k)
        d, slots = ssd.dims(2, 1, H, P, N, 1), torch.arange(2, dtype=torch.int32, device="cuda")
        y, pool, stream = torch.empty(2, 1, H, P, dtype=BF16, device="cuda"), t["state"].clone(), torch.cuda.Stream()
        ptr = lambda v: v.data_ptr()  # noqa: E731
        jobs.append((ctypes.byref(d), ssd.SSD_BF16, ssd.SSD_DT_SOFTPLUS, ptr(t["xbc"]), None, None, None, ptr(t["dt"]), None,
                     ptr(t["A"]), None, None, ptr(slots), 2, ptr(pool), ptr(y), stream.cuda_stream))
        held.append((t, d, slots, y, pool, stream))
    torch.cuda.synchronize()
    assert _all_at_once(lib.ssd_decode_step, jobs) == {ssd.SSD_OK}
    for t, d, slots, y, pool, _ in held:
        other, last = t["state"].clone(), torch.empty_like(y)
        for _ in range(CALLS):
            ssd.ssd_decode_step(d, ssd.SSD_BF16, ssd.SSD_DT_SOFTPLUS, t["xbc"], None, None, None, t["dt"], None, t["A"], None, None, slots, 2, other, last)
        assert torch.equal(pool, other) and torch.equal(y, last)
