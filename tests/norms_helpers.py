"""Shared by the tests of the norms around a block: the formulas in 64 bits, the sizes of their terms, and 8-bit
rows by table."""
import torch

BF, F4, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
# Half a step of an output's type relative to the value.
HALF = {F4: U, BF: 2.0 ** -8 * 1.01}
# Relative error of 1 / (1 + e^-z) for |z| <= 16: the exponent's rounding reaches e^-z as 1.5 |z| U, ex2.approx, rcp.approx (2^-22
# and 2^-23) and the sum add 7 U.
SIG = 32 * U
# Of a norm's result u rstd w: u's (the gate's, two products), half of that and of the sum's in rstd (16 products a thread, 5
# shuffles, 16 partials, 5 shuffles), the root and three products.
FP = SIG + (SIG + 48 * U) + 16 * U


def rows_by_table(x, groups=1):
    """(codes, scales) of 8-bit rows by the definition: the smallest power of two that fits, the nearest of all e4m3
    numbers, of two equally near ones the even code."""
    shape = x.shape
    v = x.double().cpu().reshape(-1, shape[-1] // groups)
    finite = v.isfinite()
    top = torch.where(finite, v.abs(), torch.zeros(())).amax(1)
    power = 2.0 ** torch.arange(-108, 121, dtype=torch.float64)
    scale = power[torch.searchsorted(448 * power, top)]
    number = torch.arange(127, dtype=torch.uint8).view(E4).double()   # 0 up to 448
    q = (v / scale[:, None]).abs().nan_to_num(nan=0.0, posinf=0.0)
    hi = torch.searchsorted(number, q).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    below, above = q - number[lo], number[hi] - q
    code = torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)
    code = torch.where(q == number[hi], hi, code)
    code = code + 128 * torch.signbit(v)
    code = torch.where(finite, code, torch.full((), 127)).to(torch.uint8)
    return code.view(E4).reshape(shape), scale.float().reshape(*shape[:-1], groups)


def same_codes(got, want):
    """Equal e4m3 numbers, NaNs in the same places (zeros of either sign are one number)."""
    a, b = got.cpu().float(), want.float()
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(nan=0.0), b.nan_to_num(nan=0.0))


def wide(codes, scales):
    """What an operand stands for, in 64 bits (scales None: itself)."""
    if scales is None:
        return codes.double()
    rows = codes.shape[:-1].numel()
    s = scales.double().reshape(rows, -1, 1)
    return (codes.double().reshape(rows, s.shape[1], -1) * s).reshape(codes.shape)


def mean(v, groups=1):
    g = v.unflatten(-1, (groups, -1))
    return g.mean(-1, keepdim=True).expand_as(g).flatten(-2)


def norm_bwd(g, u, weight, eps, groups=1):
    """du and sum g n of n = u / rms(u) weight from g = dn: values, and the sizes of their terms."""
    r = torch.rsqrt(mean(u * u, groups) + eps)
    n, p = u * r, g * weight
    du = r * (p - n * mean(p * n, groups))
    size = r * (p.abs() + 2 * n.abs() * mean((p * n).abs(), groups))
    return du, size, n, r


def gate(z):
    """silu(z), its slope, and the sizes of the slope's terms."""
    s = torch.sigmoid(z)
    b = z * s
    return b, s + b * (1 - s), s + b.abs()


def close(got, want, bound, what):
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got.double() - want).abs()
    worst = (off / bound).max().item() if off.numel() else 0.0
    assert worst <= 1, (what, worst)   # NaN fails too
