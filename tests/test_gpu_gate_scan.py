"""The gated recurrence, its gradient and its single-token form on the GPU against the formula in 64 bits,
walked token by token.

Bounds.  With U = 2^-24: exp(-g) carries the rounding of its argument (|g| log2 e U) and a few units of
the function; a and 1 - a add a reciprocal and a product; a token's step and the composition of
tiles' maps round a handful of times per token.  So token t adds at most U (12 + 4 |g_t|) H_t to the error,
H_t = a_t H_{t-1} + (1 - a_t) |x_t| being the recurrence of the magnitudes, and what came before decays
with a_t.  The adjoint obeys the same with its own magnitudes.  The gradient of g sees h_{t-1} from an
output rounded to y's type at some tokens, whose error decays as H does."""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
OUT = {torch.float32: U, torch.bfloat16: 2.0 ** -8 * 1.01}
BF, F4 = torch.bfloat16, torch.float32


def offsets(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def make(batch, seqlen, width, dtype, seed, pad=0, off=0, spread=2.0):
    """Gate logits and inputs as column ranges of one matrix of 2 * width + pad columns, `off` columns in."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    if pad or off:
        both = torch.zeros(batch, seqlen, 2 * width + pad, dtype=dtype, device="cuda")
        g, x = both[..., off:off + width], both[..., off + width:off + 2 * width]
        g.copy_(r(batch, seqlen, width) * spread + 3)
        x.copy_(r(batch, seqlen, width))
    else:
        g, x = (r(batch, seqlen, width) * spread + 3).to(dtype), r(batch, seqlen, width).to(dtype)
    return g, x, r


def walk(g, x, init, cu):
    """h, the state before each token, the magnitudes H and the error bound E of h, in 64 bits."""
    g, x = g.double(), x.double()
    a, m = torch.sigmoid(g), torch.sigmoid(-g)
    h, before, H, E = (torch.zeros_like(x) for _ in range(4))
    starts = {0: None} if cu is None else {t: d for d, t in enumerate(cu.tolist()[:-1])}
    z = torch.zeros_like(x[:, 0])
    for t in range(x.shape[1]):
        if t in starts:
            d = starts[t]
            last = z if init is None else (init.double() if d is None else init[d].double()[None])
            Hl, El = last.abs(), z
        before[:, t] = last
        last = a[:, t] * last + m[:, t] * x[:, t]
        Hl = a[:, t] * Hl + m[:, t] * x[:, t].abs()
        El = a[:, t] * El + U * (12 + 4 * g[:, t].abs().clamp(max=100)) * Hl
        h[:, t], H[:, t], E[:, t] = last, Hl, El
    return a, m, h, before, H, E


def walk_back(g, a, dy, dfin, cu):
    g, dy = g.double(), dy.double()
    L = dy.shape[1]
    ends = {L - 1: None} if cu is None else {t - 1: d for d, t in enumerate(cu.tolist()[1:])}
    lam, Lm, E = (torch.zeros_like(dy) for _ in range(3))
    z = torch.zeros_like(dy[:, 0])
    for t in range(L - 1, -1, -1):
        if t in ends:
            d = ends[t]
            mu = z if dfin is None else (dfin.double() if d is None else dfin[d].double()[None])
            Mm, Em = mu.abs(), z
        lam[:, t] = dy[:, t] + mu
        Lm[:, t] = dy[:, t].abs() + Mm
        E[:, t] = Em + 2 * U * Lm[:, t]
        mu, Mm = a[:, t] * lam[:, t], a[:, t] * Lm[:, t]
        # a = 1 - (1 - a) in the adjoint's chain: off by at most U
        Em = a[:, t] * E[:, t] + U * (12 + 4 * g[:, t].abs().clamp(max=100)) * Mm + U * Lm[:, t]
    return lam, Lm, E, mu, Em


def close(got, want, bound, what):
    assert torch.isfinite(got).all(), what
    worst = ((got.double() - want).abs() / (bound + 1e-30)).max().item()
    assert worst <= 1, (what, worst)


# batch, tokens, width, columns beyond two halves, first column, documents
CASES = [
    (1, 1, 1, 0, 0, None), (3, 1, 40, 0, 0, None), (2, 2, 65, 0, 0, None), (5, 15, 66, 0, 0, None), (2, 16, 64, 6, 2, None),
    (1, 17, 129, 3, 1, None), (2, 127, 128, 0, 0, None), (2, 128, 130, 2, 0, None), (3, 129, 63, 0, 0, None),
    (1, 300, 200, 5, 3, None), (2, 2048, 72, 0, 0, None), (1, 2049, 70, 8, 4, None), (1, 4500, 33, 0, 0, None),
    (1, 8, 50, 0, 0, [1, 1, 1, 5]), (1, 300, 64, 0, 0, [128, 1, 127, 44]), (1, 2300, 61, 0, 0, [3, 1, 700, 15, 16, 1, 1, 1500, 63]),
    (1, 4300, 64, 4, 2, [4299, 1]), (1, 2100, 48, 0, 0, [1] * 200 + [1900]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:5])) + ("d%d" % len(c[5]) if c[5] else ""))
@pytest.mark.parametrize("dtype", [BF, F4])
@pytest.mark.parametrize("states", [False, True])
def test_sequences(case, dtype, states):
    batch, seqlen, width, pad, off, docs = case
    g, x, r = make(batch, seqlen, width, dtype, seqlen + width, pad, off)
    cu = offsets(docs) if docs else None
    n = len(docs) if docs else batch
    init = r(n, width) if states else None
    dy = r(batch, seqlen, width).to(dtype)
    dfin = r(n, width) if states else None
    y, fin = ssd.gate_scan(g, x, init, cu, return_final_states=True, check_status=True)
    a, m, h, before, H, E = walk(g, x, init, cu)
    close(y, h, OUT[dtype] * h.abs() + E, "y")
    at = [t - 1 for t in cu.tolist()[1:]] if docs else None
    close(fin, h[0, at] if docs else h[:, -1], E[0, at] if docs else E[:, -1], "final states")

    got = ssd.gate_scan_bwd(g, x, y, dy, init, dfin, cu, want_dinit=True, check_status=True)
    assert got["dg"].stride() == g.stride() and got["dx"].stride() == x.stride()
    lam, Lm, EL, mu, Em = walk_back(g, a, dy, dfin, cu)
    gate = U * (8 + 4 * g.double().abs())
    close(got["dx"], m * lam, OUT[dtype] * (m * lam).abs() + m * EL + gate * m * Lm, "dx")
    starts = torch.zeros(seqlen, dtype=torch.bool, device="cuda")
    starts[[0] if cu is None else cu.tolist()[:-1]] = True
    Hb = torch.cat([torch.zeros_like(H[:, :1]), H[:, :-1]], 1)
    Eb = torch.cat([torch.zeros_like(E[:, :1]), E[:, :-1]], 1)
    Hb[:, starts], Eb[:, starts] = before[:, starts].abs(), 0
    eh = Eb + OUT[dtype] * (Hb + Eb)
    dg = lam * (before - x.double()) * a * m
    near = (Hb + x.double().abs()) * a * m
    close(got["dg"], dg, OUT[dtype] * dg.abs() + EL * near + Lm * a * m * eh + 2 * gate * Lm * near, "dg")
    if docs:
        first = cu.tolist()[:-1]
        mus, bound = (a * lam)[0, first], (a * EL + U * (12 + 4 * g.double().abs()) * a * Lm + U * Lm)[0, first]
    else:
        mus, bound = mu, Em
    close(got["dinit"], mus, bound, "dinit")


# rows off 16-byte alignment fall into classes by their shift: fewer rows than classes, batch rows that start in any of
# them, strides of every shift
@pytest.mark.parametrize("batch,seqlen,width,pad,off", [
    (1, 1, 1, 0, 0), (1, 3, 5, 0, 0), (3, 1, 63, 0, 0), (1, 7, 64, 3, 1), (5, 9, 65, 0, 0), (9, 129, 3, 1, 1), (3, 131, 70, 2, 2),
    (2, 127, 128, 4, 4), (4, 66, 66, 6, 3), (2, 258, 191, 5, 5), (1, 1030, 12, 1, 0)])
@pytest.mark.parametrize("dtype", [BF, F4])
def test_rows_of_every_shift(batch, seqlen, width, pad, off, dtype):
    test_sequences((batch, seqlen, width, pad, off, None), dtype, True)


def test_gradients_against_differences():
    g, x, r = make(2, 150, 6, F4, 4)
    init, dy, dfin = r(2, 6), r(2, 150, 6), r(2, 6)
    y = ssd.gate_scan(g, x, init)
    got = ssd.gate_scan_bwd(g, x, y, dy, init, dfin)

    def value(gg, xx, ii):
        h = walk(gg, xx, ii, None)[2]
        return (h * dy.double()).sum() + (h[:, -1] * dfin.double()).sum()

    for name, t, d in (("dg", 0, r(2, 150, 6)), ("dx", 1, r(2, 150, 6)), ("dinit", 2, r(2, 6))):
        at = [g.double(), x.double(), init.double()]
        up, down = list(at), list(at)
        up[t], down[t] = at[t] + 1e-4 * d.double(), at[t] - 1e-4 * d.double()
        slope = (value(*up) - value(*down)) / 2e-4
        terms = got[name].double() * d.double()
        assert abs(terms.sum() - slope) <= 2e-5 * terms.abs().sum(), name


def test_gates_at_their_limits():
    """Logits of either type's lowest and highest value, and infinities: a is 0 or 1 and nothing else turns NaN."""
    for dtype in (BF, F4):
        low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
        g = torch.zeros(1, 40, 64, device="cuda", dtype=dtype)
        g[0, 5], g[0, 11], g[0, 20], g[0, 30] = low, high, float("-inf"), float("inf")
        x = torch.randn(1, 40, 64, device="cuda").to(dtype)
        y = ssd.gate_scan(g, x)
        assert torch.isfinite(y).all()
        for t in (5, 20):   # 1 - a = e / (1 + e), two roundings of one
            assert ((y[0, t].double() - x[0, t].double()).abs() <= 2 * OUT[dtype] * x[0, t].double().abs() + 1e-30).all()
        assert torch.equal(y[0, 11], y[0, 10]) and torch.equal(y[0, 30], y[0, 29])
        got = ssd.gate_scan_bwd(g, x, y, torch.ones_like(x))
        for t in (5, 11, 20, 30):
            assert (got["dg"][0, t].float().abs() < 1e-30).all()
        assert (got["dx"][0, [11, 30]].float().abs() < 1e-30).all() and torch.isfinite(got["dx"]).all()


def test_nan_stays_in_its_channel_and_after_its_token():
    g, x, r = make(1, 300, 70, F4, 8)
    x[0, 140, 3] = float("nan")
    y = ssd.gate_scan(g, x)
    bad = y.isnan()
    assert bad[0, 140:, 3].all() and bad.sum() == 160
    g[0, 200, 9] = float("nan")
    assert ssd.gate_scan(g, x).isnan()[0, 200:, 9].all()


def test_documents_do_not_touch_each_other():
    lens = [130, 1, 250, 16, 300]
    g, x, r = make(1, sum(lens), 66, BF, 12)
    init, cu = r(5, 66), offsets(lens)
    y, fin = ssd.gate_scan(g, x, init, cu, return_final_states=True)
    g2, x2 = g.clone(), x.clone()
    x2[0, 131:381] = 7
    g2[0, 131:381] = -1
    y2, fin2 = ssd.gate_scan(g2, x2, init, cu, return_final_states=True)
    keep = [0, 1, 3, 4]
    assert torch.equal(fin[keep], fin2[keep]) and torch.equal(y[0, :131], y2[0, :131]) and torch.equal(y[0, 381:], y2[0, 381:])


def test_carried_state_repeats_and_streams():
    g, x, r = make(2, 5000, 96, F4, 2)
    y, fin = ssd.gate_scan(g, x, return_final_states=True)
    for _ in range(3):
        again = ssd.gate_scan(g, x, return_final_states=True)
        assert torch.equal(again[0], y) and torch.equal(again[1], fin)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = ssd.gate_scan(g, x, return_final_states=True, stream=s)
    s.synchronize()
    assert torch.equal(other[0], y)
    # in two calls, the state carried: the same up to the bound of either
    a = ssd.gate_scan(g[:, :1700].contiguous(), x[:, :1700].contiguous(), return_final_states=True)
    b = ssd.gate_scan(g[:, 1700:].contiguous(), x[:, 1700:].contiguous(), a[1], return_final_states=True)
    E = walk(g, x, None, None)[5]
    close(torch.cat([a[0], b[0]], 1), y.double(), 2 * E, "two calls")


def test_captured_in_a_graph():
    g, x, r = make(1, 3000, 64, BF, 6)
    want = ssd.gate_scan(g, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ssd.gate_scan(g, x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ssd.gate_scan(g, x)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("batch,width,pad,off", [(1, 1, 0, 0), (7, 64, 0, 0), (3, 65, 1, 1), (64, 5120, 0, 0), (5, 100, 4, 4), (2, 130, 6, 2)])
@pytest.mark.parametrize("dtype", [BF, F4])
def test_step(batch, width, pad, off, dtype):
    g, x, r = make(batch, 1, width, dtype, batch + width, pad, off)
    g, x = g[:, 0], x[:, 0]
    state = r(batch, width)
    before = state.clone()
    out = torch.empty_like(state)
    y2 = ssd.gate_scan_step(state, g, x, state_out=out)
    assert torch.equal(state, before)
    y = ssd.gate_scan_step(state, g, x)
    assert torch.equal(out, state) and torch.equal(y, y2)
    a, m, h, _, H, E = walk(g[:, None], x[:, None], before, None)
    close(state, h[:, 0], E[:, 0], "state")
    close(y, h[:, 0], OUT[dtype] * h[:, 0].abs() + E[:, 0], "y")


def test_steps_follow_a_prefill():
    g, x, r = make(3, 140, 128, F4, 31)
    y, fin = ssd.gate_scan(g, x, return_final_states=True)
    _, state = ssd.gate_scan(g[:, :130].contiguous(), x[:, :130].contiguous(), return_final_states=True)
    E = walk(g, x, None, None)[5]
    for t in range(130, 140):
        out = ssd.gate_scan_step(state, g[:, t], x[:, t])
        close(out, y[:, t].double(), 2 * E[:, t], t)
    close(state, fin.double(), 2 * E[:, -1], "state")


def test_offsets_that_break_their_rule_are_reported():
    g, x, r = make(1, 400, 64, F4, 1)
    for cu in ([0, 200, 200, 400], [0, 300, 100, 400], [5, 400], [0, 399], [0, 500], [-7, 400]):
        with pytest.raises(ssd.SSDError):
            ssd.gate_scan(g, x, None, torch.tensor(cu, dtype=torch.int32, device="cuda"), return_final_states=True, check_status=True)
    ssd.gate_scan(g, x, None, offsets([100, 300]), check_status=True)


def test_tensors_refused():
    g, x, r = make(2, 20, 64, BF, 1)
    cu = offsets([10, 10])
    for bad in (lambda: ssd.gate_scan(g.half(), x.half()),):
        with pytest.raises(TypeError):
            bad()
    y = ssd.gate_scan(g, x)
    for bad in (lambda: ssd.gate_scan(g[0], x[0]), lambda: ssd.gate_scan(g, x[:1]), lambda: ssd.gate_scan(g, x.float()),
                lambda: ssd.gate_scan(g.cpu(), x), lambda: ssd.gate_scan(g[..., ::2], x[..., ::2]),
                lambda: ssd.gate_scan(g.transpose(0, 1), x.transpose(0, 1)),
                lambda: ssd.gate_scan(g[:1], x[:1], None, cu.long()), lambda: ssd.gate_scan(g, x, r(3, 64)),
                lambda: ssd.gate_scan(g, x, r(2, 64).to(BF)), lambda: ssd.gate_scan_bwd(g, x, y, y[:, :19]),
                lambda: ssd.gate_scan_bwd(g, x, y, y, dg=torch.empty(2, 20, 70, dtype=BF, device="cuda")[..., :64])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ssd.gate_scan(g, x, None, cu), lambda: ssd.gate_scan(g[:, :0], x[:, :0])):
        with pytest.raises(ssd.SSDError):
            bad()
    state = r(2, 64)
    for bad in (lambda: ssd.gate_scan_step(state[:1], g[:, 0], x[:, 0]), lambda: ssd.gate_scan_step(state, g[:, 0], x),
                lambda: ssd.gate_scan_step(state.double(), g[:, 0], x[:, 0])):
        with pytest.raises(ValueError):
            bad()
