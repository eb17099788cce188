"""The operators around the scan, as they are measured: residual RMS norm, projection, gated recurrence.

Each case is one call of a layer built around a recurrent mixer: the pre-norm that also carries the
residual stream (optionally leaving e4m3 rows for an 8-bit projection), the projection with its
epilogue, the gated linear recurrence, and the backward passes that training needs.  Widths and
lengths are those of the library's own workloads (16,384 tokens of 5120 inner channels, 65,536
tokens of 2048, 32,768 packed tokens in 37 documents) or generic.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
AMAX_MIN = 1e-30
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1, "none": 0}


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step's pre-norm for 8 sequences, written in 8 bits for the projection
        dict(name="norm_decode_e4m3", op="norm", rows=8, width=2560, dtype="bf16", residual="f32", out="e4m3", train=False),
        # a training forward's pre-norm: 8 x 2048 tokens, the residual stream kept in 32 bits
        dict(name="norm_train", op="norm", rows=16384, width=2560, dtype="bf16", residual="f32", out="bf16", train=True),
        # its gradient, at a ragged number of tokens
        dict(name="norm_bwd", op="norm_bwd", rows=12289, width=2560, dtype="bf16", residual="f32"),
        # the input projection of one decoding step of 8 sequences, 8-bit weights
        dict(name="linear_decode_e4m3", op="linear", m=8, n=10240, k=2560, dtype="e4m3", act="none", bias=False, residual=False, train=False),
        # the input projection of a training forward: gates and inputs of 5120 channels
        dict(name="linear_train", op="linear", m=16384, n=10240, k=2560, dtype="bf16", act="none", bias=True, residual=False, train=False),
        # an output projection onto the residual of a ragged prefill, in 8 bits
        dict(name="linear_prefill_e4m3", op="linear", m=4099, n=2560, k=5120, dtype="e4m3", act="none", bias=False, residual=True, train=False),
        # the gradients of a projection with its activation: 4 x 2048 tokens
        dict(name="linear_bwd_silu", op="linear_bwd", m=8192, n=5120, k=2560, act="silu", bias=True),
        # a long context in one row, with the state carried in and out
        dict(name="scan_long", op="scan", batch=1, seqlen=65536, width=2048, docs=0, dtype="bf16", states=True, strided=True),
        # packed documents of an odd total, each from its own state, an odd width
        dict(name="scan_packed", op="scan", batch=1, seqlen=32767, width=1533, docs=37, dtype="bf16", states=True, strided=False),
        # the recurrence's gradient in a training step: 8 x 2048 tokens of 5120 channels
        dict(name="scan_bwd", op="scan_bwd", batch=8, seqlen=2048, width=5120, docs=0, dtype="bf16", states=False, strided=True),
        # the same in 32 bits over one longer, ragged row
        dict(name="scan_bwd_f32", op="scan_bwd", batch=1, seqlen=10001, width=2048, docs=0, dtype="f32", states=True, strided=False),
        # one decoding step of 64 sequences
        dict(name="scan_step", op="step", batch=64, width=5120, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "norm_bwd", "linear", "linear", "linear_bwd", "scan", "scan", "scan_bwd", "step"))
    if op in ("norm", "norm_bwd"):
        width = _log_int(rng, 24, 8192)
        if rng.random() < 0.6:
            width = -(-width // 8) * 8
        rows = _log_int(rng, 1, min(20000, 42_000_000 // width))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        c = dict(op=op, rows=rows, width=width, dtype=dtype, residual=rng.choice(("f32", "bf16", "none") if dtype == "bf16" else ("f32", "none")))
        if op == "norm":
            c["out"] = rng.choice((dtype, "e4m3"))
            c["train"] = rng.random() < 0.5
        return c
    if op in ("linear", "linear_bwd"):
        n = _log_int(rng, 33, 10240)
        k = _log_int(rng, 2, 320) * 16
        top = int(min(16384, 3.4e11 // (n * k)))
        act = rng.choice(("none", "silu", "gelu"))
        if op == "linear":
            return dict(op=op, m=_log_int(rng, 1, top), n=n, k=k, dtype=rng.choice(("bf16", "e4m3")), act=act,
                        bias=rng.random() < 0.5, residual=rng.random() < 0.5, train=rng.random() < 0.3)
        return dict(op=op, m=_log_int(rng, 16, max(16, top // 2)), n=n, k=k, act=act, bias=rng.random() < 0.5)
    width = _log_int(rng, 40, 5120)
    if rng.random() < 0.7:
        width = -(-width // 8) * 8
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "step":
        return dict(op=op, batch=_log_int(rng, 1, 512), width=width, dtype=dtype)
    seqlen = _log_int(rng, 1, min(65536, 80_000_000 // width))
    batch = _log_int(rng, 1, max(1, min(16, 80_000_000 // (width * seqlen))))
    docs = 0
    if rng.random() < 0.3:
        docs, batch = _log_int(rng, 1, max(1, min(seqlen, 200))), 1
    return dict(op=op, batch=batch, seqlen=seqlen, width=width, docs=docs, dtype=dtype, states=rng.random() < 0.5, strided=rng.random() < 0.4)


# ----------------------------------------------------------------------------------------- inputs

def _normal(gen, *shape, scale=1.0, shift=0.0, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).add_(shift).to(dtype)


def _e4m3_rows(v):
    """Rows of e4m3 numbers and the scale of each."""
    scale = v.abs().amax(-1).clamp(min=AMAX_MIN) / E4M3_MAX
    return (v / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _offsets(docs, total, seed):
    """docs documents of geometric-like lengths, at least one token each, total tokens in all."""
    r = np.random.RandomState(seed % (1 << 31))
    share = r.exponential(size=docs)
    lengths = 1 + np.floor(share / share.sum() * (total - docs)).astype(np.int64)
    lengths[-1] += total - lengths.sum()
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def _gates(gen, case):
    """Gate logits and inputs: two halves of one projection's rows, or tensors of their own."""
    b, n, d = case["batch"], case.get("seqlen", 1), case["width"]
    dt = DTYPES[case["dtype"]]
    shape = (b, n) if "seqlen" in case else (b,)
    if case.get("strided"):
        both = torch.empty(*shape, 2 * d, dtype=dt, device="cuda")
        both[..., :d] = _normal(gen, *shape, d, scale=2.0, shift=3.0, dtype=dt)
        both[..., d:] = _normal(gen, *shape, d, dtype=dt)
        return both[..., :d], both[..., d:]
    return _normal(gen, *shape, d, scale=2.0, shift=3.0, dtype=dt), _normal(gen, *shape, d, dtype=dt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    op, s = case["op"], dict(case)
    if op in ("norm", "norm_bwd"):
        rows, width, dt = case["rows"], case["width"], DTYPES[case["dtype"]]
        s["weight"] = _normal(gen, width, scale=0.2, shift=1.0)
        # a residual stream has a few channels far larger than the rest
        loud = 1.0 + 20.0 * (torch.rand(width, generator=gen, device="cuda") < 0.01)
        x = _normal(gen, rows, width, dtype=dt)
        res = None if case["residual"] == "none" else (_normal(gen, rows, width, scale=3.0) * loud).to(DTYPES[case["residual"]])
        if op == "norm":
            s.update(x=x, res=res)
            return s
        h = x if res is None else res
        s.update(h=h, rstd=1.0 / torch.sqrt((h.float() ** 2).mean(-1) + EPS), dout=_normal(gen, rows, width, dtype=dt),
                 dres=None if res is None else _normal(gen, rows, width, dtype=res.dtype))
        return s
    if op in ("linear", "linear_bwd"):
        m, n, k = case["m"], case["n"], case["k"]
        x = _normal(gen, m, k)
        w = _normal(gen, n, k, scale=1.0 / math.sqrt(k))
        bias = _normal(gen, n, scale=0.5) if case["bias"] else None
        if op == "linear":
            s["bias"] = bias
            s["res"] = _normal(gen, m, n, scale=2.0, dtype=torch.bfloat16) if case["residual"] else None
            if case["dtype"] == "e4m3":
                s["x"], s["xs"] = _e4m3_rows(x)
                s["w"], s["ws"] = _e4m3_rows(w)
            else:
                s.update(x=x.to(torch.bfloat16), w=w.to(torch.bfloat16), xs=None, ws=None)
            return s
        s.update(x=x.to(torch.bfloat16), w=w.to(torch.bfloat16), dy=_normal(gen, m, n, dtype=torch.bfloat16),
                 pre=None if case["act"] == "none" else _normal(gen, m, n, dtype=torch.bfloat16))
        return s
    s["g"], s["x"] = _gates(gen, case)
    b, d = case["batch"], case["width"]
    if op == "step":
        s["state"] = _normal(gen, b, d, scale=0.5)
        return s
    s["cu"] = _offsets(case["docs"], case["seqlen"], seed) if case["docs"] else None
    rows = case["docs"] or b
    s["init"] = _normal(gen, rows, d, scale=0.5) if case["states"] else None
    if op == "scan_bwd":
        s["dy"] = _normal(gen, b, case["seqlen"], d, dtype=DTYPES[case["dtype"]])
        s["dfin"] = _normal(gen, rows, d) if case["states"] else None
        s["y"] = _plain_scan(s)[0]   # what the forward pass left
    return s


# ------------------------------------------------------------------------------------ plain forms

def _plain_norm(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(-1) + EPS)
    o = h * rstd[:, None] * s["weight"]
    got = {}
    if s["out"] == "e4m3":
        got["out"], got["scales"] = _e4m3_rows(o)
    else:
        got["out"] = o.to(DTYPES[s["out"]])
    if s["res"] is not None:
        got["residual"] = h.to(s["res"].dtype)
    if s["train"]:
        got["rstd"] = rstd
    return got


def _plain_norm_bwd(s):
    xhat = s["h"].float() * s["rstd"][:, None]
    do = s["dout"].float()
    wd = do * s["weight"]
    dh = (wd - xhat * (wd * xhat).mean(-1, keepdim=True)) * s["rstd"][:, None]
    if s["dres"] is not None:
        dh = dh + s["dres"].float()
    return {"dx": dh.to(s["dout"].dtype), "dresidual": dh.to(s["h"].dtype), "dweight": (do * xhat).sum(0)}


def _act(v, kind):
    if kind == "silu":
        return v / (1.0 + torch.exp(-v))
    if kind == "gelu":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _act_slope(v, kind):
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-v))
        return p * (1.0 + v * (1.0 - p))
    u = math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)
    t = torch.tanh(u)
    return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * v * v)


def _plain_linear(s):
    v = s["x"].float() @ s["w"].float().t()
    if s["xs"] is not None:
        v = v * s["xs"][:, None] * s["ws"]
    if s["bias"] is not None:
        v = v + s["bias"]
    y = _act(v, s["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    got = {"y": y.to(torch.bfloat16)}
    if s["train"]:
        got["pre"] = v.to(torch.bfloat16)
    return got


def _plain_linear_bwd(s):
    d = s["dy"].float()
    if s["pre"] is not None:
        d = d * _act_slope(s["pre"].float(), s["act"])
    got = {"dx": (d @ s["w"].float()).to(torch.bfloat16), "dw": (d.t() @ s["x"].float()).to(torch.bfloat16)}
    if s["bias"]:
        got["dbias"] = d.sum(0)
    return got


def _compose(a, b):
    """Every h_t = a_t h_{t-1} + b_t from zero along axis 1, by doubling the stretch that each entry covers."""
    step = 1
    while step < a.shape[1]:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _plain_h(s):
    """The decays, the entering decays cut at row and document starts, and every state."""
    g, x = s["g"].float(), s["x"].float()
    a = 1.0 / (1.0 + torch.exp(-g))
    b = x / (1.0 + torch.exp(g))
    first = s["cu"][:-1].long() if s["cu"] is not None else torch.zeros(1, dtype=torch.long, device=g.device)
    cut = a.clone()
    cut[:, first] = 0
    if s["init"] is not None:
        b[:, first] += a[:, first] * (s["init"][None] if s["cu"] is not None else s["init"][:, None])
    return g, x, a, cut, first, _compose(cut, b)


def _plain_scan(s):
    h = _plain_h(s)[-1]
    if s["cu"] is not None:
        fin = h[0, s["cu"][1:].long() - 1]
    else:
        fin = h[:, -1]
    return h.to(s["x"].dtype), fin


def _plain_scan_bwd(s):
    g, x, a, cut, first, h = _plain_h(s)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    before[:, first] = 0
    if s["init"] is not None:
        before[:, first] = s["init"][None] if s["cu"] is not None else s["init"][:, None]
    d = s["dy"].float().clone()
    if s["dfin"] is not None:
        if s["cu"] is not None:
            d[0, s["cu"][1:].long() - 1] += s["dfin"]
        else:
            d[:, -1] += s["dfin"]
    later = torch.cat([cut[:, 1:], torch.zeros_like(cut[:, :1])], 1)
    lam = _compose(later.flip(1), d.flip(1)).flip(1)
    rest = 1.0 / (1.0 + torch.exp(g))
    got = {"dg": (lam * (before - x) * a * rest).to(s["g"].dtype), "dx": (lam * rest).to(s["x"].dtype)}
    if s["init"] is not None:
        got["dinit"] = (a * lam)[0, first] if s["cu"] is not None else (a * lam)[:, 0]
    return got


def _plain_step(s):
    g = s["g"].float()
    new = s["state"] / (1.0 + torch.exp(-g)) + s["x"].float() / (1.0 + torch.exp(g))
    s["state"].copy_(new)
    return {"y": new.to(s["x"].dtype), "state": s["state"]}


# -------------------------------------------------------------------------------------------- run

def run(state):
    s, op = state, state["op"]
    if not own:
        if op == "scan":
            y, fin = _plain_scan(s)
            return {"y": y, "final": fin} if s["states"] else {"y": y}
        return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "linear": _plain_linear, "linear_bwd": _plain_linear_bwd,
                "scan_bwd": _plain_scan_bwd, "step": _plain_step}[op](s)
    import mamba_ssd_chunked_scan_gb300 as ssd
    if op == "norm":
        r = ssd.add_norm(s["x"], s["weight"], s["res"], eps=EPS, out_dtype=DTYPES[s["out"]], return_rstd=s["train"])
        return {k: v for k, v in r.items() if v is not None}
    if op == "norm_bwd":
        return ssd.add_norm_bwd(s["dout"], s["h"], s["weight"], s["rstd"], s["dres"])
    if op == "linear":
        y = ssd.linear(s["x"], s["w"], s["bias"], s["res"], act=s["act"], x_scales=s["xs"], w_scales=s["ws"], return_pre=s["train"])
        return {"y": y[0], "pre": y[1]} if s["train"] else {"y": y}
    if op == "linear_bwd":
        r = ssd.linear_bwd(s["dy"], s["x"], s["w"], s["pre"], act=s["act"], want_dbias=s["bias"])
        return {k: v for k, v in r.items() if v is not None}
    if op == "scan":
        y = ssd.gate_scan(s["g"], s["x"], s["init"], s["cu"], return_final_states=s["states"])
        return {"y": y[0], "final": y[1]} if s["states"] else {"y": y}
    if op == "scan_bwd":
        r = ssd.gate_scan_bwd(s["g"], s["x"], s["y"], s["dy"], s["init"], s["dfin"], s["cu"], want_dinit=s["states"])
        return {k: v for k, v in r.items() if v is not None}
    return {"y": ssd.gate_scan_step(s["state"], s["g"], s["x"]), "state": s["state"]}


# ------------------------------------------------------------------------------------------- work

def work(case):
    op, c = case["op"], case
    if op in ("norm", "norm_bwd"):
        n, e, r = c["rows"] * c["width"], BYTES[c["dtype"]], BYTES[c["residual"]]
        if op == "norm":
            extra = 4 * c["rows"] * ((c["out"] == "e4m3") + c["train"]) + 4 * c["width"]
            return {"bytes": n * (e + 2 * r + BYTES[c["out"]]) + extra, "flops": 6 * n}
        # the incoming gradients and h are read; the gradient is written once in each of the two types
        moved = 2 * e + (3 * r - (e if r == e else 0) if r else e)
        return {"bytes": n * moved + 4 * c["rows"] + 8 * c["width"], "flops": 12 * n}
    if op == "linear":
        m, n, k, e = c["m"], c["n"], c["k"], BYTES[c["dtype"]]
        side = (4 * (m + n) if c["dtype"] == "e4m3" else 0) + (4 * n if c["bias"] else 0)
        return {"bytes": (m * k + n * k) * e + 2 * m * n * (1 + c["residual"] + c["train"]) + side, "flops": 2 * m * n * k}
    if op == "linear_bwd":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": 2 * (2 * m * k + 2 * n * k + m * n * (1 if c["act"] == "none" else 2)) + (4 * n if c["bias"] else 0), "flops": 4 * m * n * k}
    e, d = BYTES[c["dtype"]], c["width"]
    if op == "step":
        return {"bytes": c["batch"] * d * (3 * e + 8), "flops": 8 * c["batch"] * d}
    n = c["batch"] * c["seqlen"] * d
    rows = (c["docs"] or c["batch"]) * d * 4 if c["states"] else 0
    if op == "scan":
        return {"bytes": 3 * e * n + 2 * rows, "flops": 8 * n}
    return {"bytes": 5 * e * n + 3 * rows, "flops": 20 * n}


# ------------------------------------------------------------------------------------------ exact

def _walk(g, x, init, starts):
    """The recurrence token by token: all states, and the state before each token."""
    keep = torch.sigmoid(g)
    take = torch.sigmoid(-g)
    h, before, last = torch.empty_like(x), torch.empty_like(x), None
    for t in range(x.shape[1]):
        if t in starts:
            j = starts[t]
            last = torch.zeros_like(x[:, 0]) if init is None else (init if j is None else init[j][None])
        before[:, t] = last
        last = torch.addcmul(take[:, t] * x[:, t], keep[:, t], last)
        h[:, t] = last
    return keep, take, h, before


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    f = {k: (v.double() if torch.is_tensor(v) and v.is_floating_point() else v) for k, v in s.items()}
    if op == "norm":
        h = f["x"] if f["res"] is None else f["x"] + f["res"]
        rms = torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
        o = h / rms * f["weight"]
        got = {"out": o}
        if case["out"] == "e4m3":
            got["scales"] = o.abs().max(1).values.clamp(min=AMAX_MIN) / E4M3_MAX
            got["out"] = o / got["scales"][:, None]   # the values that the 8 bits stand for, before their rounding
        if f["res"] is not None:
            got["residual"] = h
        if case["train"]:
            got["rstd"] = 1 / rms[:, 0]
        return got
    if op == "norm_bwd":
        r = f["rstd"][:, None]
        n = case["width"]
        p = f["dout"] * f["weight"]
        dh = r * p - r ** 3 * f["h"] * (p * f["h"]).sum(1, keepdim=True) / n
        if f["dres"] is not None:
            dh = dh + f["dres"]
        return {"dx": dh, "dresidual": dh, "dweight": (f["dout"] * f["h"] * r).sum(0)}
    if op == "linear":
        v = torch.einsum("mk,nk->mn", f["x"], f["w"])
        if f["xs"] is not None:
            v = v * torch.outer(f["xs"], f["ws"])
        v = v if f["bias"] is None else v + f["bias"]
        y = {"none": lambda u: u, "silu": torch.nn.functional.silu, "gelu": lambda u: torch.nn.functional.gelu(u, approximate="tanh")}[case["act"]](v)
        got = {"y": y if f["res"] is None else y + f["res"]}
        if case["train"]:
            got["pre"] = v
        return got
    if op == "linear_bwd":
        d = f["dy"]
        if case["act"] != "none":
            v = f["pre"].requires_grad_(True)
            y = torch.nn.functional.silu(v) if case["act"] == "silu" else torch.nn.functional.gelu(v, approximate="tanh")
            d = torch.autograd.grad(y, v, d)[0]
        got = {"dx": torch.einsum("mn,nk->mk", d, f["w"]), "dw": torch.einsum("mn,mk->nk", d, f["x"])}
        if case["bias"]:
            got["dbias"] = d.sum(0)
        return got
    if op == "step":
        new = torch.sigmoid(f["g"]) * f["state"] + torch.sigmoid(-f["g"]) * f["x"]
        return {"y": new, "state": new}
    edges = s["cu"].tolist() if s["cu"] is not None else None
    starts = {0: None} if edges is None else {t: j for j, t in enumerate(edges[:-1])}
    keep, take, h, before = _walk(f["g"], f["x"], f["init"], starts)
    ends = [t - 1 for t in edges[1:]] if edges else None
    if op == "scan":
        if not case["states"]:
            return {"y": h}
        return {"y": h, "final": h[:, -1] if ends is None else h[0, ends]}
    del h
    lam, carry = f["dy"].clone(), None
    tail = {case["seqlen"] - 1: None} if ends is None else {t: j for j, t in enumerate(ends)}
    for t in range(case["seqlen"] - 1, -1, -1):
        if t in tail:
            j = tail[t]
            if f["dfin"] is not None:
                lam[:, t] += f["dfin"] if j is None else f["dfin"][j][None]
        else:
            lam[:, t] += carry
        carry = keep[:, t] * lam[:, t]
    got = {"dg": lam * keep * take * (before - f["x"]), "dx": lam * take}
    if f["init"] is not None:
        into = keep * lam
        got["dinit"] = into[:, 0] if edges is None else into[0, edges[:-1]]
    return got
