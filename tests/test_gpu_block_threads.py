"""The block calls from several host threads at once."""
import ctypes
import threading
import time

import pytest
import torch

from tests import _block_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from __graft_entry__ import build_library
    build_library()
    import paged_kv_cache_136_gb300 as pa
    pa.pa_device_errors(clear=True)
    return pa


def _run(threads):
    """Run the functions at once; raise what any of them raised."""
    errors, gate = [], threading.Barrier(len(threads))

    def go(f):
        try:
            torch.cuda.set_device(0)
            gate.wait(timeout=60)
            f()
        except BaseException as e:  # handed to the test
            errors.append(e)

    ts = [threading.Thread(target=go, args=(f,)) for f in threads]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    if errors:
        raise errors[0]


class _Decode:
    """One problem: its inputs, its reference, its own stream and workspace."""

    def __init__(self, pa, i, lens, h, hkv, d, bs, dtype):
        tables, nb = R.make_tables(lens, bs, seed=i)
        self.pool, self.scales = R.make_pool(nb, bs, hkv, d, dtype, True, seed=i)
        self.q = torch.randn(len(lens), h, d, generator=R.gen(i, "cuda"), device="cuda").to(dtype)
        self.tables, self.sl, self.bs, self.msl = tables, R.ints(lens), bs, max(lens)
        self.out, self.stream = torch.zeros_like(self.q), torch.cuda.Stream()
        self.ws = torch.empty(pa.pa_block_decode_workspace_size(h, hkv, d), dtype=torch.uint8,
                              device="cuda")
        self.ref = R.ref_decode(self.q, self.pool, self.scales, tables, self.sl, bs, 0.1)

    def check(self):
        R.check_decode(self.out, self.ref, True, True)


# other numbers of warps and types, each looked up when it is first met
PROBLEMS = [([900, 70], 3, 3, 64, 16, torch.float16), ([30, 1200], 10, 5, 128, 32, torch.bfloat16),
            ([2500], 14, 7, 64, 32, torch.bfloat16), ([64, 5, 800], 12, 6, 128, 16, torch.float16),
            ([3100, 1], 8, 1, 128, 16, torch.bfloat16), ([17] * 9, 32, 16, 64, 16, torch.float16)]


def test_c_calls_from_many_threads(pa):
    """Through the C entry, which no lock of the interpreter orders."""
    P, I = ctypes.c_void_p, ctypes.c_int
    fn = ctypes.CDLL(pa.lib_path()).pa_decode_fp8_block
    fn.restype = I
    fn.argtypes = [P] * 7 + [I] * 7 + [ctypes.c_float] + [I] * 2 + [P, ctypes.c_size_t, P]
    runs = [_Decode(pa, i, *PROBLEMS[i % len(PROBLEMS)]) for i in range(12)]
    torch.cuda.synchronize()

    def calls(r):
        b, h, d = r.q.shape
        nb, hkv = r.pool.shape[1], r.pool.shape[3]
        for _ in range(50):
            st = fn(r.out.data_ptr(), None, r.q.data_ptr(), r.pool.data_ptr(), r.scales.data_ptr(),
                    r.tables.data_ptr(), r.sl.data_ptr(), b, h, hkv, d, r.bs, nb,
                    r.tables.shape[1], 0.1, int(r.q.dtype == torch.bfloat16), r.msl,
                    r.ws.data_ptr(), r.ws.numel(), r.stream.cuda_stream)
            assert st == 0

    _run([lambda r=r: calls(r) for r in runs])
    torch.cuda.synchronize()
    assert pa.pa_device_errors(clear=True) == 0
    for r in runs:
        r.check()


def test_a_launch_that_waits_stops_no_other_thread(pa):
    """A stream whose queue is full makes the launching thread wait; another
    thread of the interpreter runs on meanwhile."""
    hkv, d, bs = 2, 64, 16
    tables, nb = R.make_tables([bs], bs)
    pool, scales = R.make_pool(nb, bs, hkv, d, torch.float16, True)
    bounds = torch.zeros(nb, hkv, 2, d, dtype=torch.int8, device="cuda")
    bsc = torch.zeros(nb, hkv, device="cuda")
    args = (bounds, bsc, pool, tables, R.ints([bs]), R.starts([bs]), bs, bs)
    pa.pa_update_block_bounds(*args, kv_scales=scales)
    torch.cuda.synchronize()
    stream, done, gaps = torch.cuda.Stream(), threading.Event(), []

    def watch():
        last = time.perf_counter()
        while not done.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    t = threading.Thread(target=watch)
    t.start()
    try:
        with torch.cuda.stream(stream):
            torch.cuda._sleep(1_000_000_000)           # about half a second
        for _ in range(4000):                          # more than a queue holds
            pa.pa_update_block_bounds(*args, kv_scales=scales, stream=stream)
    finally:
        done.set()
        t.join()
    torch.cuda.synchronize()
    # a thread that has the lock gives it up every 5 ms; a wait for the whole
    # sleep with the lock held shows as one gap of hundreds
    assert max(gaps) < 0.2


def test_binding_calls_from_many_threads(pa):
    runs = [_Decode(pa, i, *PROBLEMS[i % len(PROBLEMS)]) for i in range(12)]
    torch.cuda.synchronize()

    def calls(r):
        for _ in range(50):
            pa.pa_decode_fp8_block(r.out, r.q, r.pool, r.scales, r.tables, r.sl, 0.1, r.bs, r.msl,
                                   r.ws, stream=r.stream)

    _run([lambda r=r: calls(r) for r in runs])
    torch.cuda.synchronize()
    assert pa.pa_device_errors(clear=True) == 0
    for r in runs:
        r.check()
