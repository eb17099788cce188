"""The norms around a block and their 8-bit checkpoints, as they are measured.

A layer's backward pass reads again what its forward pass read.  Kept as e4m3 rows, each with a power of
two as its scale, that is half of the bytes of bf16; the gate and norm after the scan, the norm after a block and the
projections take their gradients from such rows.  Cases: packing and unpacking rows; the gate and norm with its
checkpoint, and its gradient; the norm after a block with gate, residual scale and the next block's norm, and its
gradient; a projection's gradients from 8-bit rows.  Rows in 8 bits are returned as their e4m3 numbers, which are exact,
beside their scales.  Widths and lengths are those of the library's own workloads
(16,384 tokens of 5120 inner channels in layers of 2560, projections of 10,576 columns) or generic.
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
MIN_EXP = -108          # of a row's scale
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1, "none": 0}


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the gate branch of a training forward, kept in 8 bits from its columns of the input projection's rows
        dict(name="pack_gate_branch", op="pack", rows=16384, width=5120, groups=1, dtype="bf16", stride=10576),
        # a kept activation back in 32 bits, ragged in both directions
        dict(name="unpack_ragged", op="unpack", rows=4099, width=2557, groups=1, dtype="f32"),
        # gate and norm after the scan of a training forward, leaving y and z in 8 bits
        dict(name="gate_keep_train", op="gate", rows=16384, width=5120, groups=1, dtype="bf16", stride=10576),
        # the same in 32 bits over groups of 256 channels, a ragged number of tokens
        dict(name="gate_keep_groups", op="gate", rows=2049, width=2048, groups=8, dtype="f32", stride=0),
        # its gradient in a training step: z and its gradient in columns of the projection's rows
        dict(name="gate_bwd_train", op="gate_bwd", rows=16384, width=5120, groups=1, dtype="bf16", stride=10576, packed=False, out=False),
        # the gradient from the 8-bit checkpoint, with the forward's output again for the output projection's gradient
        dict(name="gate_bwd_kept", op="gate_bwd", rows=12289, width=5120, groups=1, dtype="bf16", stride=0, packed=True, out=True),
        # one decoding step of 8 sequences: the norm after a block, the residual, and the next block's norm as 8-bit rows
        dict(name="block_decode", op="block", rows=8, width=2560, dtype="bf16", residual="f32", gate=False, next=True, out="e4m3", keep=False, stride=0),
        # a training forward with a gate, the block's output and gate kept in 8 bits
        dict(name="block_train", op="block", rows=16384, width=2560, dtype="bf16", residual="f32", gate=True, next=True, out="bf16", keep=True, stride=0),
        # its gradient, from tensors as they were
        dict(name="block_bwd_train", op="block_bwd", rows=16384, width=2560, dtype="bf16", residual="f32", gate=True, next=True, packed=False, stride=0),
        # the gradient of a ragged batch of odd width, everything read again in 8 bits
        dict(name="block_bwd_kept", op="block_bwd", rows=9001, width=1533, dtype="bf16", residual="bf16", gate=True, next=True, packed=True, stride=0),
        # gradients of a projection with its activation, its input and the activation's argument kept in 8 bits
        dict(name="linear_bwd_kept_silu", op="linear_bwd", m=8192, n=5120, k=2560, act="silu", bias=True, scales="packed"),
        # gradients of an output projection over a ragged batch, from the e4m3 rows that the forward pass multiplied
        dict(name="linear_bwd_e4m3_rows", op="linear_bwd", m=4099, n=2560, k=5120, act="none", bias=False, scales="amax"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def _stride(rng, width):
    """Elements between rows that are columns of a wider matrix (0: rows of their own)."""
    return 0 if rng.random() < 0.6 else width + rng.choice((8, 80, 1, 33)) + rng.choice((0, width))


def draw(rng):
    op = rng.choice(("pack", "unpack", "gate", "gate_bwd", "gate_bwd", "block", "block", "block_bwd", "block_bwd", "linear_bwd"))
    if op == "linear_bwd":
        n = _log_int(rng, 33, 6000)
        k = _log_int(rng, 2, 320) * 16
        top = int(min(16384, 1.07e11 // (n * k), 42_000_000 // max(n, k)))
        act = rng.choice(("none", "silu", "gelu"))
        return dict(op=op, m=_log_int(rng, 1, top), n=n, k=k, act=act, bias=rng.random() < 0.5, scales=rng.choice(("packed", "amax")))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    width = _log_int(rng, 24, 8192)
    if rng.random() < 0.6:
        width = -(-width // 8) * 8
    rows = _log_int(rng, 1, min(20000, 40_000_000 // width))
    c = dict(op=op, rows=rows, width=width, dtype=dtype)
    if op in ("pack", "unpack", "gate", "gate_bwd"):
        c["groups"] = 1
        if rng.random() < 0.4:
            c["groups"] = rng.choice((2, 3, 8))
            size = max(8, -(-width // c["groups"]))
            if rng.random() < 0.6:
                size = -(-size // 8) * 8
            c["width"] = c["groups"] * size
            c["rows"] = min(rows, 40_000_000 // c["width"])
    if op == "unpack":
        return c
    c["stride"] = _stride(rng, c["width"])
    if op in ("block", "block_bwd"):
        c["residual"] = rng.choice(("f32", "bf16")) if dtype == "bf16" else "f32"
        c["gate"] = rng.random() < 0.5
        c["next"] = rng.random() < 0.8
        if not c["gate"]:
            c["stride"] = 0
    if op == "block":
        c["out"] = "none" if not c["next"] else rng.choice((dtype, dtype, "e4m3"))
        c["keep"] = rng.random() < 0.5
    if op in ("gate_bwd", "block_bwd"):
        c["packed"] = rng.random() < 0.5
        if c["packed"]:
            c["stride"] = 0
    if op == "gate_bwd":
        c["out"] = rng.random() < 0.5
    return c


# ----------------------------------------------------------------------------------------- inputs

def _normal(gen, *shape, scale=1.0, shift=0.0, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).add_(shift).to(dtype)


def _loud(gen, width):
    """A residual stream has a few channels far larger than the rest."""
    return 1.0 + 20.0 * (torch.rand(width, generator=gen, device="cuda") < 0.01)


def _columns(v, stride):
    """v as rows of its own (stride 0), or as columns of a wider matrix."""
    if not stride:
        return v
    wide = torch.zeros(v.shape[0], stride, dtype=v.dtype, device=v.device)
    wide[:, : v.shape[1]] = v
    return wide[:, : v.shape[1]]


def _pack(v, groups=1):
    """e4m3 codes of v's rows (or of each row's groups), and their scales: the smallest powers of two that fit."""
    rows, width = v.shape
    f = v.float().reshape(rows, groups, width // groups)
    size = torch.where(torch.isfinite(f), f.abs(), torch.zeros((), device=f.device))
    frac, exp = torch.frexp(size.amax(-1))
    exp = torch.where(frac > 0.875, exp - 8, exp - 9)
    scale = torch.ldexp(torch.ones_like(frac), torch.where(frac > 0, exp, torch.full_like(exp, MIN_EXP)).clamp(min=MIN_EXP))
    q = f / scale[..., None]
    q = torch.where(torch.isfinite(f), q, torch.full((), math.nan, device=f.device))
    return q.to(torch.float8_e4m3fn).reshape(rows, width), scale


def _pack_rows(v):
    """The same with one scale for each whole row: scales (rows)."""
    codes, scales = _pack(v)
    return codes, scales[:, 0].contiguous()


def _values(codes, scales):
    """What 8-bit rows stand for, in 32 bits; scales (rows, groups) or (rows)."""
    rows, width = codes.shape
    s = scales.reshape(rows, -1, 1)
    return (codes.float().reshape(rows, s.shape[1], -1) * s).reshape(rows, width)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 6007 + 29)
    op, s = case["op"], dict(case)
    if op == "linear_bwd":
        m, n, k = case["m"], case["n"], case["k"]
        x = _normal(gen, m, k)
        if case["scales"] == "packed":
            s["x"], s["xs"] = _pack_rows(x)
        else:   # as add_norm writes its e4m3 rows
            s["xs"] = x.abs().amax(-1) / E4M3_MAX
            s["x"] = (x / s["xs"][:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        del x
        s["w"] = _normal(gen, n, k, scale=1.0 / math.sqrt(k), dtype=torch.bfloat16)
        s["dy"] = _normal(gen, m, n, dtype=torch.bfloat16)
        s["pre"] = s["ps"] = None
        if case["act"] != "none":
            s["pre"], s["ps"] = _pack_rows(_normal(gen, m, n))
        return s
    rows, width, dt = case["rows"], case["width"], DTYPES[case["dtype"]]
    # padded tokens are rows of zeros
    live = (torch.arange(rows, device="cuda") % 97 != 96).float()[:, None]
    if op in ("pack", "unpack"):
        x = (_normal(gen, rows, width, scale=1.5) * _loud(gen, width) * live).to(dt)
        if op == "pack":
            s["x"] = _columns(x, case["stride"])
        else:
            s["q"], s["scales"] = _pack(x, case["groups"])
        return s
    weight = _normal(gen, width, scale=0.2, shift=1.0)
    if op in ("gate", "gate_bwd"):
        s["weight"] = weight
        s["y"] = (_normal(gen, rows, width, scale=0.7) * live).to(dt)
        s["z"] = _columns(_normal(gen, rows, width, scale=1.5, dtype=dt), case["stride"])
        if op == "gate":
            return s
        s["dout"] = _normal(gen, rows, width, dtype=dt)
        s["ys"] = s["zs"] = s["dz"] = None
        if case["packed"]:
            s["y"], s["ys"] = _pack(s["y"], case["groups"])
            s["z"], s["zs"] = _pack(s["z"], case["groups"])
        elif case["stride"]:   # the projection's gradient, whose columns the call writes
            s["dz"] = torch.zeros(rows, case["stride"], dtype=dt, device="cuda")[:, :width]
        return s
    s["weight"], s["scale"] = weight, 0.22
    s["next_weight"] = _normal(gen, width, scale=0.2, shift=1.0) if case["next"] else None
    s["x"] = (_normal(gen, rows, width, scale=2.0) * live).to(dt)
    s["gatev"] = _columns(_normal(gen, rows, width, scale=1.5, dtype=dt), case["stride"]) if case["gate"] else None
    rt = DTYPES[case["residual"]]
    res = (_normal(gen, rows, width, scale=3.0) * _loud(gen, width)).to(rt)
    if op == "block":
        s["res"] = res
        return s
    # the stream after the block, as the forward pass left it, and the gradients that come in
    s["h"] = res
    s["dout"] = _normal(gen, rows, width, dtype=dt) if case["next"] else None
    s["dres"] = _normal(gen, rows, width, dtype=rt)
    s["xs"] = s["gs"] = s["hs"] = s["dgate"] = None
    if case["packed"]:
        s["x"], s["xs"] = _pack_rows(s["x"])
        s["h"], s["hs"] = _pack_rows(s["h"])
        if case["gate"]:
            s["gatev"], s["gs"] = _pack_rows(s["gatev"])
    elif case["gate"] and case["stride"]:
        s["dgate"] = torch.zeros(rows, case["stride"], dtype=dt, device="cuda")[:, :width]
    return s


# ------------------------------------------------------------------------------------ plain forms

def _plain_pack(s):
    q, scales = _pack(s["x"], s["groups"])
    return {"codes": q, "scales": scales}


def _plain_unpack(s):
    return {"x": _values(s["q"], s["scales"]).to(DTYPES[s["dtype"]])}


def _grouped_mean(v, groups):
    rows, width = v.shape
    m = v.reshape(rows, groups, width // groups).mean(-1, keepdim=True)
    return m.expand(rows, groups, width // groups).reshape(rows, width)


def _plain_gate(s):
    z = s["z"].float()
    u = s["y"].float() * z / (1.0 + torch.exp(-z))
    out = u / torch.sqrt(_grouped_mean(u * u, s["groups"]) + EPS) * s["weight"]
    yq, ys = _pack(s["y"], s["groups"])
    zq, zs = _pack(s["z"], s["groups"])
    return {"out": out.to(s["y"].dtype), "y": yq, "y_scales": ys, "z": zq, "z_scales": zs}


def _plain_gate_bwd(s):
    dt = s["dout"].dtype
    y = s["y"].float() if s["ys"] is None else _values(s["y"], s["ys"])
    z = s["z"].float() if s["zs"] is None else _values(s["z"], s["zs"])
    sig = 1.0 / (1.0 + torch.exp(-z))
    a = z * sig
    u = y * a
    rstd = 1.0 / torch.sqrt(_grouped_mean(u * u, s["groups"]) + EPS)
    xhat = u * rstd
    do = s["dout"].float()
    p = do * s["weight"]
    du = (p - xhat * _grouped_mean(p * xhat, s["groups"])) * rstd
    got = {"dy": (du * a).to(dt), "dz": (du * y * sig * (1.0 + z * (1.0 - sig))).to(dt), "dweight": (do * xhat).sum(0)}
    if s["dz"] is not None:
        s["dz"].copy_(got["dz"])
        got["dz"] = s["dz"]
    if s["out"]:
        got["out"] = (xhat * s["weight"]).to(dt)
    return got


def _plain_block(s):
    u = s["x"].float()
    if s["gatev"] is not None:
        g = s["gatev"].float()
        u = u * g / (1.0 + torch.exp(-g))
    h = s["res"].float() + s["scale"] * (u / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS) * s["weight"])
    got = {"residual": h.to(s["res"].dtype)}
    if s["next_weight"] is not None:
        o = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * s["next_weight"]
        if s["out"] == "e4m3":
            got["out"], got["scales"] = _pack_rows(o)
        else:
            got["out"] = o.to(DTYPES[s["out"]])
    if s["keep"]:
        got["x"], got["x_scales"] = _pack_rows(s["x"])
        if s["gatev"] is not None:
            got["gate"], got["gate_scales"] = _pack_rows(s["gatev"])
    return got


def _plain_block_bwd(s):
    dt = DTYPES[s["dtype"]]
    x = s["x"].float() if s["xs"] is None else _values(s["x"], s["xs"])
    h = s["h"].float() if s["hs"] is None else _values(s["h"], s["hs"])
    dh = s["dres"].float()
    got = {}
    if s["dout"] is not None:
        hhat = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
        do = s["dout"].float()
        p = do * s["next_weight"]
        dh = dh + (p - hhat * (p * hhat).mean(-1, keepdim=True)) / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
        got["dnext_weight"] = (do * hhat).sum(0)
    got["dresidual"] = dh.to(s["dres"].dtype)
    u = x
    if s["gatev"] is not None:
        g = s["gatev"].float() if s["gs"] is None else _values(s["gatev"], s["gs"])
        sig = 1.0 / (1.0 + torch.exp(-g))
        u = x * g * sig
    rstd = 1.0 / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS)
    uhat = u * rstd
    dn = s["scale"] * dh
    p = dn * s["weight"]
    du = (p - uhat * (p * uhat).mean(-1, keepdim=True)) * rstd
    got["dweight"] = (dn * uhat).sum(0)
    if s["gatev"] is None:
        got["dx"] = du.to(dt)
        return got
    got["dx"] = (du * g * sig).to(dt)
    got["dgate"] = (du * x * sig * (1.0 + g * (1.0 - sig))).to(dt)
    if s["dgate"] is not None:
        s["dgate"].copy_(got["dgate"])
        got["dgate"] = s["dgate"]
    return got


def _act_slope(v, kind):
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-v))
        return p * (1.0 + v * (1.0 - p))
    u = math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)
    t = torch.tanh(u)
    return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * v * v)


def _plain_linear_bwd(s):
    d = s["dy"].float()
    if s["pre"] is not None:
        d = d * _act_slope(_values(s["pre"], s["ps"]), s["act"])
    got = {"dx": (d @ s["w"].float()).to(torch.bfloat16), "dw": (d.t() @ _values(s["x"], s["xs"])).to(torch.bfloat16)}
    if s["bias"]:
        got["dbias"] = d.sum(0)
    return got


# -------------------------------------------------------------------------------------------- run

def run(state):
    s, op = state, state["op"]
    if not own:
        return {"pack": _plain_pack, "unpack": _plain_unpack, "gate": _plain_gate, "gate_bwd": _plain_gate_bwd, "block": _plain_block,
                "block_bwd": _plain_block_bwd, "linear_bwd": _plain_linear_bwd}[op](s)
    import mamba_ssd_chunked_scan_gb300 as ssd
    size = s["width"] // s["groups"] if "groups" in s else 0
    if op == "pack":
        codes, scales = ssd.pack_rows(s["x"], size)
        return {"codes": codes, "scales": scales}
    if op == "unpack":
        return {"x": ssd.unpack_rows(s["q"], s["scales"], dtype=DTYPES[s["dtype"]])}
    if op == "gate":
        out, kept = ssd.gate_norm(s["y"], s["z"], s["weight"], size, EPS, pack=True)
        return {"out": out, **kept}
    if op == "gate_bwd":
        r = ssd.gate_norm_bwd(s["dout"], s["y"], s["z"], s["weight"], size, EPS, y_scales=s["ys"], z_scales=s["zs"], dz=s["dz"],
                              want_out=s["out"])
    elif op == "block":
        r = ssd.block_norm(s["x"], s["weight"], s["res"], s["gatev"], s["next_weight"], scale=s["scale"], eps=EPS,
                           out_dtype=None if s["out"] == "none" else DTYPES[s["out"]], pack=s["keep"])
    elif op == "block_bwd":
        r = ssd.block_norm_bwd(s["dout"], s["dres"], s["x"], s["h"], s["weight"], s["gatev"], s["next_weight"], scale=s["scale"], eps=EPS,
                               x_scales=s["xs"], h_scales=s["hs"], gate_scales=s["gs"], dgate=s["dgate"],
                               dtype=DTYPES[s["dtype"]])
    else:
        r = ssd.linear_bwd(s["dy"], s["x"], s["w"], s["pre"], act=s["act"], x_scales=s["xs"], pre_scales=s["ps"], want_dbias=s["bias"])
    return {k: v for k, v in r.items() if v is not None}


# ------------------------------------------------------------------------------------------- work

def work(case):
    op, c = case["op"], case
    if op == "linear_bwd":
        m, n, k = c["m"], c["n"], c["k"]
        moved = m * k * (1 + 2) + 2 * 2 * n * k + m * n * (2 if c["act"] == "none" else 3) + 4 * m * (1 if c["act"] == "none" else 2)
        return {"bytes": moved + (4 * n if c["bias"] else 0), "flops": 4 * m * n * k}
    n, e, w = c["rows"] * c["width"], BYTES[c["dtype"]], 4 * c["width"]
    units = c["rows"] * c.get("groups", 1)
    if op == "pack":
        return {"bytes": n * (e + 1) + 4 * units, "flops": 3 * n}
    if op == "unpack":
        return {"bytes": n * (e + 1) + 4 * units, "flops": n}
    if op == "gate":
        return {"bytes": n * (3 * e + 2) + 8 * units + w, "flops": 16 * n}
    if op == "gate_bwd":
        moved = e + (2 if c["packed"] else 2 * e) + 2 * e + (e if c["out"] else 0)
        return {"bytes": n * moved + (8 * units if c["packed"] else 0) + 2 * w, "flops": 25 * n}
    r, gate, nxt = BYTES[c["residual"]], int(c["gate"]), int(c["next"])
    if op == "block":
        kept = (1 + gate) * int(c["keep"])
        return {"bytes": n * (e * (1 + gate) + 2 * r + BYTES[c["out"]] + kept) + 4 * c["rows"] * (kept + (c["out"] == "e4m3")) + w * (1 + nxt),
                "flops": (12 + 6 * gate) * n}
    if c["packed"]:
        moved = (1 + gate) + nxt
    else:
        moved = e * (1 + gate) + r * nxt
    moved += e * nxt + 2 * r + e * (1 + gate)
    return {"bytes": n * moved + (4 * c["rows"] * (1 + gate + nxt) if c["packed"] else 0) + 2 * w * (1 + nxt), "flops": (25 + 12 * gate) * n}


# ------------------------------------------------------------------------------------------ exact

def _round_e4m3(v):
    """The nearest numbers of 3 fraction bits and exponents from -6 on, ties to even, of 64-bit numbers up to 448."""
    power = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -30)))
    power = torch.where(torch.exp2(power) > v.abs(), power - 1, power).clamp(min=-6)   # a logarithm next to a whole number
    power = torch.where(torch.exp2(power + 1) <= v.abs(), power + 1, power)
    step = torch.exp2(power - 3)
    return torch.round(v / step) * step


def _exact_rows(v, groups):
    """(codes, scales) of 8-bit rows of finite 64-bit numbers."""
    part = v.reshape(v.shape[0] * groups, -1)
    top = part.abs().max(1).values
    scale = torch.full_like(top, 2.0 ** MIN_EXP)
    least = torch.ceil(torch.log2(top.clamp(min=1e-300) / E4M3_MAX)).clamp(min=MIN_EXP)
    least = torch.where(torch.exp2(least) * E4M3_MAX < top, least + 1, least)   # a logarithm next to a whole number
    least = torch.where((torch.exp2(least - 1) * E4M3_MAX >= top) & (least > MIN_EXP), least - 1, least)
    scale = torch.where(top > 0, torch.exp2(least), scale)
    return _round_e4m3(part / scale[:, None]).reshape(v.shape), scale.reshape(v.shape[0], groups)


def _wide(codes, scales):
    """8-bit rows in 64 bits."""
    if scales is None:
        return codes.double()
    per = codes.shape[1] // (scales.numel() // codes.shape[0])
    return codes.double() * scales.double().reshape(codes.shape[0], -1).repeat_interleave(per, 1)


def _rms_norm(v, groups, weight):
    part = v.unflatten(1, (groups, -1))
    return (part * torch.rsqrt(part.square().mean(2, keepdim=True) + EPS)).flatten(1) * weight


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    silu = torch.nn.functional.silu
    if op == "pack":
        codes, scales = _exact_rows(s["x"].double(), case["groups"])
        return {"codes": codes, "scales": scales}
    if op == "unpack":
        return {"x": _wide(s["q"], s["scales"])}
    if op == "linear_bwd":
        d = s["dy"].double()
        if case["act"] != "none":
            v = _wide(s["pre"], s["ps"]).requires_grad_(True)
            y = silu(v) if case["act"] == "silu" else torch.nn.functional.gelu(v, approximate="tanh")
            d = torch.autograd.grad(y, v, d)[0]
        got = {"dx": torch.einsum("mn,nk->mk", d, s["w"].double()), "dw": torch.einsum("mn,mk->nk", d, _wide(s["x"], s["xs"]))}
        if case["bias"]:
            got["dbias"] = d.sum(0)
        return got
    weight = s["weight"].double()
    if op == "gate":
        got = {"out": _rms_norm(s["y"].double() * silu(s["z"].double()), case["groups"], weight)}
        got["y"], got["y_scales"] = _exact_rows(s["y"].double(), case["groups"])
        got["z"], got["z_scales"] = _exact_rows(s["z"].double(), case["groups"])
        return got
    if op == "gate_bwd":
        y, z = (_wide(s[k], s[k + "s"]).requires_grad_(True) for k in ("y", "z"))
        weight.requires_grad_(True)
        out = _rms_norm(y * silu(z), case["groups"], weight)
        dy, dz, dw = torch.autograd.grad(out, (y, z, weight), s["dout"].double())
        got = {"dy": dy, "dz": dz, "dweight": dw}
        if case["out"]:
            got["out"] = out.detach()
        return got
    after = None if s["next_weight"] is None else s["next_weight"].double()
    if op == "block":
        u = s["x"].double()
        if case["gate"]:
            u = u * silu(s["gatev"].double())
        h = s["res"].double() + s["scale"] * _rms_norm(u, 1, weight)
        got = {"residual": h}
        if case["next"]:
            got["out"] = _rms_norm(h, 1, after)
        keep = {"out": ("scales", got["out"])} if case["out"] == "e4m3" else {}
        if case["keep"]:
            keep["x"] = ("x_scales", s["x"].double())
            if case["gate"]:
                keep["gate"] = ("gate_scales", s["gatev"].double())
        for name, (scales, v) in keep.items():
            got[name], per = _exact_rows(v, 1)
            got[scales] = per[:, 0]
        return got
    # the gradients of <dout, out> + <dres, h>, with h as it was kept
    got, dh = {}, s["dres"].double()
    if case["next"]:
        h = _wide(s["h"], s["hs"]).requires_grad_(True)
        after.requires_grad_(True)
        into, got["dnext_weight"] = torch.autograd.grad(_rms_norm(h, 1, after), (h, after), s["dout"].double())
        dh = dh + into
    got["dresidual"] = dh
    x = _wide(s["x"], s["xs"]).requires_grad_(True)
    weight.requires_grad_(True)
    if case["gate"]:
        g = _wide(s["gatev"], s["gs"]).requires_grad_(True)
        grads = torch.autograd.grad(_rms_norm(x * silu(g), 1, weight), (x, weight, g), s["scale"] * dh)
        got["dgate"] = grads[2]
    else:
        grads = torch.autograd.grad(_rms_norm(x, 1, weight), (x, weight), s["scale"] * dh)
    got["dx"], got["dweight"] = grads[:2]
    return got
