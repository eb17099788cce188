"""The device-side failure paths of the projection and the recurrence, made to run without faulting or hanging the GPU: a call
with an injected stall issues only so many loads, or hands no state on, and caps every wait at a short count of polls.  A
wait that depends on what is missing runs out, the status word says which, every CTA drains and exits, and the next ordinary
call on the same workspace is right."""
import ctypes

import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd

pytestmark = pytest.mark.gpu

BF, F4, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TIMEOUT, ROUNDS = 5, 1 << 14


def status(work):
    from mamba_ssd_chunked_scan_gb300 import _lib
    where = ctypes.c_uint32(0)
    return _lib.lib.ssd_check_status_where(work.data_ptr(), torch.cuda.current_stream().cuda_stream, ctypes.byref(where)), where.value


# rows, columns, contraction, operands, loads issued by each CTA, plan: none, a few, more than there are stages (the stages come back)
@pytest.mark.parametrize("m,n,k,kind,loads,plan", [
    (300, 520, 2048, BF, 0, "cta"), (300, 520, 2048, BF, 3, "cta"), (300, 520, 8192, E4, 11, "cta"), (1426, 8088, 1600, BF, 5, "cta"),
    (8, 20000, 2560, BF, 0, "T"), (8, 20000, 2560, E4, 12, "T"), (8, 2560, 5120, E4, 1, "T"),
    (8943, 1609, 2336, BF, 0, "pair"), (8943, 1609, 2336, BF, 3, "pair"), (8943, 1609, 2336, BF, 9, "pair"), (8943, 1609, 2336, BF, 50, "pair"),
    (5373, 2563, 2960, BF, 7, "pair"), (2534, 7848, 4240, E4, 0, "pair"), (2534, 7848, 4240, E4, 6, "pair")])
def test_stalled_projection(m, n, k, kind, loads, plan):
    from mamba_ssd_chunked_scan_gb300 import _lib
    lib, code = _lib.lib, _lib.SSD_E4M3 if kind is E4 else _lib.SSD_BF16
    q = _lib.linear_plan(m, n, k, code)
    assert plan == ("T" if q.transposed else "pair" if q.tile_rows == 256 else "cta")
    g = torch.Generator(device="cuda").manual_seed(m)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, w, bias, res = r(m, k).to(kind), r(n, k).to(kind), r(n), r(m, n).to(BF)
    scales = (torch.rand(m, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")) if kind is E4 else (None, None)
    want = ssd.linear(x, w, bias, res, x_scales=scales[0], w_scales=scales[1])
    p = _lib.LinearParams(m, k, n, k, code, 0)
    work = torch.empty(lib.ssd_linear_workspace_size(p), dtype=torch.uint8, device="cuda")
    y = torch.full((m, n), 77.0, dtype=BF, device="cuda")
    args = [ctypes.byref(p), x.data_ptr(), w.data_ptr(), *(s.data_ptr() if s is not None else None for s in scales), bias.data_ptr(),
            res.data_ptr(), y.data_ptr(), None, work.data_ptr(), work.numel()]
    st = torch.cuda.current_stream().cuda_stream
    assert lib.ssd_linear_fault_inject(*args, loads, ROUNDS, st) == 0
    got = status(work)
    assert got[0] == TIMEOUT and 61 <= got[1] <= 64, got   # a wait of the work itself, not of its drain
    assert status(work) == (0, 0)
    if loads < 2 and q.splits == 1:
        assert (y == 77).all()   # of sums that are not whole nothing is written
    assert lib.ssd_linear(*args, st) == 0
    assert status(work) == (0, 0) and torch.equal(y, want)


@pytest.mark.parametrize("width,docs", [(2048, False), (2048, True), (1533, False), (1533, True)])
@pytest.mark.parametrize("dtype", [BF, F4])
@pytest.mark.parametrize("loads", [0, 2, -1])   # none; some; all, but no tile hands its map on
def test_stalled_recurrence(width, docs, dtype, loads):
    from mamba_ssd_chunked_scan_gb300 import _lib
    lib, L = _lib.lib, 6000
    gen = torch.Generator(device="cuda").manual_seed(width)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    g, x = (r(1, L, width) + 3).to(dtype), r(1, L, width).to(dtype)
    cu = torch.tensor([0, 1, 700, 5000, L], dtype=torch.int32, device="cuda") if docs else None
    n = 4 if docs else 1
    init, fin, y = r(n, width), torch.empty(n, width, device="cuda"), torch.empty_like(x)
    want = ssd.gate_scan(g, x, init, cu, return_final_states=True)
    p = _lib.GateScanParams(1, L, width, width, width, n if docs else 0, _lib.SSD_BF16 if dtype is BF else _lib.SSD_F32)
    work = torch.empty(lib.ssd_gate_scan_workspace_size(p), dtype=torch.uint8, device="cuda")
    args = [ctypes.byref(p), g.data_ptr(), x.data_ptr(), init.data_ptr(), cu.data_ptr() if docs else None, y.data_ptr(), fin.data_ptr(),
            work.data_ptr(), work.numel()]
    st = torch.cuda.current_stream().cuda_stream
    assert lib.ssd_gate_scan_fault_inject(*args, loads, ROUNDS, st) == 0
    got = status(work)
    assert got[0] == TIMEOUT and 51 <= got[1] <= 56, got
    assert status(work) == (0, 0)
    assert lib.ssd_gate_scan(*args, st) == 0
    assert status(work) == (0, 0) and torch.equal(y, want[0]) and torch.equal(fin, want[1])


def test_limits_count_from_the_end_of_earlier_launches():
    """A launch that starts while a long one before it still runs does not count that time against its own waits: with caps far
    below the earlier launch's time, and everything loaded, the calls are ordinary ones."""
    from mamba_ssd_chunked_scan_gb300 import _lib
    lib = _lib.lib
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    # the sum of many rows' gradients of eight columns: one CTA adds the shares, for tens of milliseconds, and the rest of the GPU is free
    tall, small = torch.ones(1 << 29, 8, dtype=BF, device="cuda"), torch.ones(8, 8, dtype=BF, device="cuda")
    long = lambda: ssd.linear_bwd(tall, tall, small, want_dx=False, want_dw=False, want_dbias=True)
    assert (long()["dbias"] == 1 << 29).all()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    long()
    b.record()
    torch.cuda.synchronize()
    print("the call before: %.1f ms" % a.elapsed_time(b))

    for m, n, k in ((8, 2560, 256), (300, 520, 2048)):
        x, w = r(m, k).to(BF), r(n, k).to(BF)
        want, y = ssd.linear(x, w), torch.empty(m, n, dtype=BF, device="cuda")
        p = _lib.LinearParams(m, k, n, k, _lib.SSD_BF16, 0)
        work = torch.empty(lib.ssd_linear_workspace_size(p), dtype=torch.uint8, device="cuda")
        long()
        assert lib.ssd_linear_fault_inject(ctypes.byref(p), x.data_ptr(), w.data_ptr(), None, None, None, None, y.data_ptr(), None,
                                           work.data_ptr(), work.numel(), 0x7fffffff, 4096, st) == 0
        assert status(work) == (0, 0) and torch.equal(y, want), (m, n, k)
    for width in (256, 255):
        g, x = r(1, 2000, width).to(BF), r(1, 2000, width).to(BF)
        want, y = ssd.gate_scan(g, x), torch.empty_like(x)
        p = _lib.GateScanParams(1, 2000, width, width, width, 0, _lib.SSD_BF16)
        work = torch.empty(lib.ssd_gate_scan_workspace_size(p), dtype=torch.uint8, device="cuda")
        long()
        assert lib.ssd_gate_scan_fault_inject(ctypes.byref(p), g.data_ptr(), x.data_ptr(), None, None, y.data_ptr(), None,
                                              work.data_ptr(), work.numel(), 0x7fffffff, 4096, st) == 0
        assert status(work) == (0, 0) and torch.equal(y, want), width
