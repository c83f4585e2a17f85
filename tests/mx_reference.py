"""Microscaled rows and the experts on them, in 64 bits and from the definitions
(no test functions here): blocks of 32 columns share a scale 2^s; elements are
the nearest values of the format, ties to the even code."""
import torch

F64 = torch.float64
# mantissa bits, smallest and largest exponent, largest value, next scale from this significand on
FORMATS = {"mxfp4": (1, 0, 2, 6.0, 1.75), "mxfp8": (3, -6, 8, 448.0, 1.8125)}


def power(s):
    """2^s of whole s, from a table: a computed power may be rounded."""
    table = torch.tensor([2.0 ** i for i in range(-1000, 1001)], dtype=F64, device=s.device)
    return table[s.long() + 1000]


def grid(fmt, device="cpu"):
    """The values >= 0 of the format in order: place = code."""
    mant, lo, hi, top, _ = FORMATS[fmt]
    n = 1 << mant
    v = [i / n * 2.0 ** lo for i in range(n)] + [(1 + i / n) * 2.0 ** e for e in range(lo, hi + 1) for i in range(n)]
    return torch.tensor([x for x in v if x <= top], dtype=F64, device=device)


def blocks(x):
    """Rows [R, C] as [R, B, 32], zeros behind a short last block."""
    R, C = x.shape
    B = (C + 31) // 32
    full = torch.zeros((R, B * 32), dtype=F64, device=x.device)
    full[:, :C] = x
    return full.view(R, B, 32)


def quantize(x, fmt):
    """(codes [R, B, 32] with the sign in bit 7, exponents s [R, B]); s = 128 marks a block
    without values."""
    _, _, emax, _, bump = FORMATS[fmt]
    b = blocks(x.to(F64))
    bad = ~torch.isfinite(b).all(2)
    b = torch.where(bad[..., None], torch.zeros_like(b), b)
    a = b.abs().amax(2)
    p = torch.frexp(a)[1] - 1
    s = p - emax + (a >= bump * power(p)).long()
    s = torch.where(a > 0, s, torch.full_like(s, -127)).clamp(min=-127)
    y = b / power(s)[..., None]
    g = grid(fmt, x.device)
    mid = (g[1:] + g[:-1]) / 2
    code = torch.bucketize(y.abs().contiguous(), mid)  # middles below
    tie = (code < len(mid)) & (y.abs() == mid[code.clamp(max=len(mid) - 1)]) & (code % 2 == 1)
    code = code + tie.long() + 128 * torch.signbit(y).long()
    return torch.where(bad[..., None], torch.zeros_like(code), code), torch.where(bad, torch.full_like(s, 128), s)


def values(code, s, fmt, C):
    """The rows that codes and exponents stand for, [R, C] in 64 bits."""
    v = grid(fmt, code.device)[code & 127] * (1.0 - 2.0 * (code >> 7).to(F64))
    v = v * power(s.clamp(max=127))[..., None]
    v = torch.where((s == 128)[..., None], torch.full_like(v, float("nan")), v)
    return v.reshape(v.shape[0], -1)[:, :C]


def rounded(x, fmt):
    return values(*quantize(x, fmt), fmt, x.shape[1])


def held(mx):
    """The same of an MxRows (two-dimensional), decoded byte by byte."""
    v, s = mx.values.long(), mx.scales.long()
    if mx.format == "mxfp4":
        code = torch.stack([v & 15, v >> 4], -1).reshape(v.shape[0], -1)[:, :mx.cols]
        code = (code & 7) + 128 * (code >> 3)
    else:
        code = v
    pad = (-mx.cols) % 32
    code = torch.nn.functional.pad(code, (0, pad)).view(code.shape[0], -1, 32)
    return values(code, s - 127, mx.format, mx.cols)


def silu(g):
    return g * torch.sigmoid(g)


def experts4(x, gate, up, down, out_dtype):
    """4-bit experts on rows [n, H] of one expert (weights as held rows in 64 bits): the
    outputs, and how far FP32 sums may put each: an h that lies on a border within its own
    error may become either neighbour, and sums round once a 64-deep step."""
    eps = torch.finfo(out_dtype).eps / 2
    xq = rounded(x, "mxfp4")
    g, u = xq @ gate.t(), xq @ up.t()
    steps = x.shape[1] / 64 + 2
    dg = steps * 2.0 ** -22 * (xq.abs() @ gate.abs().t())
    du = steps * 2.0 ** -22 * (xq.abs() @ up.abs().t())
    h = silu(g) * u
    # |silu'| <= 1.1; the FP32 exponential, reciprocal and products: a few ulp, one more per unit of |g|
    dh = 1.1 * dg * u.abs() + silu(g).abs() * du + h.abs() * (8 + g.abs()) * 2.0 ** -22
    code, s = quantize(h, "mxfp4")
    hq = values(code, s, "mxfp4", h.shape[1])
    lo, hi = rounded_at(h - dh, s, "mxfp4"), rounded_at(h + dh, s, "mxfp4")
    slack = torch.maximum((lo - hq).abs(), (hi - hq).abs())
    # a block whose largest value is at a border of the scales may take either scale
    b, db = blocks(h).abs().amax(2), blocks(dh).amax(2)
    other = torch.zeros_like(s)
    for e in (b - db, b + db):
        p = torch.frexp(e.clamp(min=0))[1] - 1
        t = torch.where(e > 0, p - 2 + (e >= 1.75 * power(p)).long(), torch.full_like(s, -127)).clamp(min=-127)
        other = torch.where(t != s, t - s, other)
    moved = rounded_at(h, s + other, "mxfp4")
    n = h.shape[1]
    jumps = (other != 0)[..., None].expand(-1, -1, 32).reshape(len(h), -1)[:, :n]
    slack = torch.where(jumps, torch.maximum(slack, (moved - hq).abs() + 2 * slack), slack)
    out = hq @ down.t()
    tol = eps * out.abs() * 1.01 + slack @ down.abs().t() + (h.shape[1] / 64 + 2) * 2.0 ** -22 * (hq.abs() @ down.abs().t())
    return out, tol


def rounded_at(x, s, fmt):
    """Rows rounded at given scales (saturating)."""
    C = x.shape[1]
    y = blocks(x) / power(s)[..., None]
    g = grid(fmt, x.device)
    mid = (g[1:] + g[:-1]) / 2
    v = torch.copysign(g[torch.bucketize(y.abs().contiguous(), mid)], y) * power(s)[..., None]
    return v.reshape(x.shape[0], -1)[:, :C]
