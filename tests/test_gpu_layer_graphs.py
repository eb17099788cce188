"""The operators around the scan in CUDA graphs and on a stream of their own: the same bits as called one by one."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd

pytestmark = pytest.mark.gpu

BF, F4, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def calls():
    """One layer's forward and backward, and a decoding step: every launch that the operators have, parts and their joins among them."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    m, width, inner = 700, 640, 1280
    d, s, weight = r(1, m, width).to(BF), r(1, m, width), torch.rand(width, generator=gen, device="cuda") + 0.5
    w_in, b_in, w_out = (r(2 * inner, width) / 25).to(BF), r(2 * inner), (r(width, inner) / 35).to(BF)
    q_in, sc_in = r(2 * inner, width).to(E4), torch.rand(2 * inner, generator=gen, device="cuda") / 25
    dd, ds, state, tok, toks = r(1, m, width).to(BF), r(1, m, width), r(8, inner), r(8, width).to(BF), r(8, width)

    def layer():
        n = ssd.add_norm(d, weight, s, return_rstd=True)
        gx = ssd.linear(n["out"], w_in, b_in)
        g, x = gx[..., :inner], gx[..., inner:]
        h, fin = ssd.gate_scan(g, x, None, return_final_states=True)
        y, pre = ssd.linear(h, w_out, act="silu", return_pre=True)
        out = ssd.linear_bwd(dd, h, w_out, pre, act="silu", want_dbias=True)
        gb = ssd.gate_scan_bwd(g, x, h, out["dx"])
        inp = ssd.linear_bwd(torch.cat([gb["dg"], gb["dx"]], -1), n["out"], w_in)
        nb = ssd.add_norm_bwd(inp["dx"], n["residual"], weight, n["rstd"], ds)
        q = ssd.add_norm(tok, weight, toks, out_dtype=E4)
        one = ssd.linear(q["out"], q_in, b_in, x_scales=q["scales"], w_scales=sc_in)
        after = torch.empty_like(state)
        h1 = ssd.gate_scan_step(state, one[:, :inner], one[:, inner:], state_out=after)
        return [n["out"], n["residual"], n["rstd"], gx, h, fin, y, pre, out["dx"], out["dw"], out["dbias"], gb["dg"], gb["dx"], inp["dx"],
                inp["dw"], nb["dx"], nb["dresidual"], nb["dweight"], q["out"].view(torch.uint8), q["scales"], one, h1, after,
                ssd.linear(h1, w_out)]

    return layer


def test_captured_in_a_graph():
    layer = calls()
    want = layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), k


def test_on_a_stream_of_its_own():
    layer = calls()
    want = layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [layer() for _ in range(3)]
    side.synchronize()
    for g in got:
        for k, (a, b) in enumerate(zip(g, want)):
            assert torch.equal(a, b), k
