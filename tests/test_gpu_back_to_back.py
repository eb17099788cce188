"""Calls that follow one another with nothing between them, on buffers that are rewritten each time.

A launch may start while the one before it ends; whatever it reads has to be what that one and all before it
wrote.  Each chain runs once with the stream synchronised after every call and once without; the results
have to be the same bit for bit."""
import ctypes

import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd

pytestmark = pytest.mark.gpu

BF, F4, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
ROUNDS = 24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def chain(step, outputs):
    """The outputs of every round, without a wait between any two calls and then with one after each."""
    both = []
    for wait in (False, True):
        torch.cuda.synchronize()
        got = []
        for k in range(ROUNDS):
            step(k, torch.cuda.synchronize if wait else lambda: None)
            got.append([t.clone() for t in outputs()])
        torch.cuda.synchronize()
        both.append(got)
    for k, (a, b) in enumerate(zip(*both)):
        for j, (u, v) in enumerate(zip(a, b)):
            assert torch.equal(u, v), (k, j)


# products whose contraction is split: rows of x, columns, contraction.  Few rows are computed transposed; an odd number
# of columns takes the residual element by element.
@pytest.mark.parametrize("m,n,k", [(8, 2560, 5120), (40, 1001, 5120), (200, 520, 5120), (200, 515, 5120)])
@pytest.mark.parametrize("kind", [BF, E4])
def test_split_product_on_rewritten_buffers(m, n, k, kind):
    from mamba_ssd_chunked_scan_gb300 import _lib
    lib = _lib.lib
    e4 = kind is E4
    p = _lib.LinearParams(m, k, n, k, _lib.SSD_E4M3 if e4 else _lib.SSD_BF16, 0)
    nbytes = lib.ssd_linear_workspace_size(p)
    assert nbytes > 256   # it has parts to join
    g = gen(m + n)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    rows = [(r(m, k) * 3).to(kind) for _ in range(3)]
    w = (r(n, k) / k ** 0.5).to(kind) if not e4 else r(n, k).to(kind)
    scales = [(torch.rand(m, generator=g, device="cuda") + 0.5, (torch.rand(n, generator=g, device="cuda") + 0.5) / k ** 0.5) for _ in range(4)]
    biases = [r(n) for _ in range(5)]
    x, xs, ws, bias = rows[0].clone(), scales[0][0].clone(), scales[0][1].clone(), biases[0].clone()
    res = torch.zeros(m, n, dtype=BF, device="cuda")   # each call's result is the next one's residual
    y = torch.empty_like(res)
    work = torch.empty(nbytes, dtype=torch.uint8, device="cuda")

    def call(residual, out):
        rc = lib.ssd_linear(ctypes.byref(p), x.data_ptr(), w.data_ptr(), xs.data_ptr() if e4 else None, ws.data_ptr() if e4 else None,
                            bias.data_ptr(), residual.data_ptr(), out.data_ptr(), None, work.data_ptr(), nbytes,
                            torch.cuda.current_stream().cuda_stream)
        assert rc == 0

    def step(i, wait):
        if i == 0:
            res.zero_()
        x.copy_(rows[i % 3])
        xs.copy_(scales[i % 4][0])
        ws.copy_(scales[i % 4][1])
        bias.copy_(biases[i % 5])
        wait()
        call(res, y)
        wait()
        call(y, res)   # nothing but the library's launches between the two
        wait()
        res.mul_(0.25)
        wait()

    chain(step, lambda: (y, res))


def test_norm_scales_feed_a_split_product():
    """e4m3 rows and scales written by the norm's launch, read by the product and by its join."""
    m, n, k = 8, 2560, 5120
    g = gen(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    xs, weight = [r(m, k).mul_(1 + j).to(BF) for j in range(4)], torch.rand(k, generator=g, device="cuda") + 0.5
    w, ws = r(n, k).to(E4), torch.rand(n, generator=g, device="cuda") / k ** 0.5
    x, out = xs[0].clone(), []

    def step(i, wait):
        x.copy_(xs[i % 4])
        wait()
        nrm = ssd.add_norm(x, weight, out_dtype=E4)
        wait()
        out[:] = [ssd.linear(nrm["out"], w, x_scales=nrm["scales"], w_scales=ws)]
        wait()

    chain(step, lambda: out)


# batch, tokens, width, documents: one tile, several, rows off 16-byte alignment, documents whose states the main warps read
@pytest.mark.parametrize("batch,seqlen,width,docs", [(3, 100, 64, None), (2, 1500, 128, None), (2, 1500, 61, None), (1, 1500, 128, [1, 200, 3, 1296]),
                                                     (1, 1500, 61, [700, 1, 1, 798])])
@pytest.mark.parametrize("dtype", [BF, F4])
def test_recurrence_on_rewritten_states(batch, seqlen, width, docs, dtype):
    """The final states of one call, copied over its initial states, are the next one's."""
    g = gen(seqlen + width)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    gates, xs = [(r(batch, seqlen, width) + 3).to(dtype) for _ in range(3)], [r(batch, seqlen, width).to(dtype) for _ in range(2)]
    dy = r(batch, seqlen, width).to(dtype)
    n = len(docs) if docs else batch
    cu = torch.tensor([sum(docs[:k]) for k in range(n + 1)], dtype=torch.int32, device="cuda") if docs else None
    start, dstart = r(n, width), r(n, width)
    init, dfin, out = start.clone(), dstart.clone(), []

    def step(i, wait):
        if i == 0:
            init.copy_(start)
            dfin.copy_(dstart)
        wait()
        y, fin = ssd.gate_scan(gates[i % 3], xs[i % 2], init, cu, return_final_states=True)
        wait()
        got = ssd.gate_scan_bwd(gates[i % 3], xs[i % 2], y, dy, init, dfin, cu)
        wait()
        # from one call to the next without anything between: a step updates the states in place
        again = ssd.gate_scan(gates[i % 3], xs[i % 2], fin, cu, return_final_states=True)
        wait()
        ssd.gate_scan_step(again[1], gates[i % 3][0, :1].expand(n, width).contiguous(), xs[i % 2][0, :1].expand(n, width).contiguous())
        wait()
        last = ssd.gate_scan(gates[i % 3], xs[i % 2], again[1], cu)
        wait()
        init.copy_(fin)
        dfin.copy_(got["dinit"] + 1)
        wait()
        out[:] = [y, fin, got["dg"], got["dx"], got["dinit"], again[0], again[1], last]

    chain(step, lambda: out)
