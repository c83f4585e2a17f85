"""Cases of the experts' operators in microscaled form: rows held in 4 or 8 bits with a power-of-two
scale per 32 columns, SwiGLU experts whose operands are 4-bit, and the experts' training step with
its activations checkpointed in 8 bits.

Each case is one pass through one operator.  ``run`` computes it in plain torch operations, or, with
``own`` set, through this package's calls.  ``exact`` gives the same outputs from the definitions in
64 bits.

Shapes follow this repository's workloads (4 experts of 64 x 128 in FP32; 8 experts of 4096 x 14336;
64 of 2048 x 1408, top-6; 128 of 2048 x 768, top-8; 256 of 7168 x 2048, top-8) and ragged ones of the
same kinds.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_MAX_FLOPS = 3.4e12


def _case(name, op, T, H, dtype, E=1, k=1, I=0, skew=0.0):
    case = dict(op=op, T=T, H=H, dtype=dtype, E=E, k=k, I=I, skew=skew)
    return case if name is None else dict(name=name, **case)


def listed():
    return [
        # one small expert's weights to 4 bits and back: latency
        _case("round4_tiny_f32", "round4", 128, 64, "f32"),
        # gate weights of 64 experts to 4 bits, and read back in 16
        _case("round4_weights_bf16", "round4", 64 * 1408, 2048, "bf16"),
        # a ragged batch's tokens checkpointed in 8 bits and restored in dispatch order, odd row length
        _case("restore8_ragged_f16", "restore8", 4097, 1001, "f16", E=8, k=2),
        # the headline batch's tokens checkpointed and restored in dispatch order
        _case("restore8_headline_bf16", "restore8", 16384, 2048, "bf16", E=64, k=6),
        # one generated token through the whole layer, 4-bit experts
        _case("layer4_token_bf16", "layer4", 1, 2048, "bf16", E=64, k=6, I=1408),
        # a decode batch through the whole layer: the touched experts' weights are what there is to read
        _case("layer4_decode_bf16", "layer4", 32, 7168, "bf16", E=256, k=8, I=2048),
        # a prompt batch at the headline shape
        _case("experts4_headline_bf16", "experts4", 16384, 2048, "bf16", E=64, k=6, I=1408),
        # few wide experts
        _case("experts4_wide_bf16", "experts4", 4096, 4096, "bf16", E=8, k=2, I=14336),
        # a small training step that keeps its activations in 8 bits, ragged sizes
        _case("save8_small_f16", "save8", 509, 520, "f16", E=8, k=2, I=328),
        # the headline training step's expert forward
        _case("save8_headline_bf16", "save8", 16384, 2048, "bf16", E=64, k=6, I=1408),
        # the experts' backward from 8-bit checkpoints, skewed routing over many small experts
        _case("grad8_skewed_bf16", "grad8", 2048, 2048, "bf16", E=128, k=8, I=768, skew=1.0),
        # the headline training step's expert backward
        _case("grad8_headline_bf16", "grad8", 16384, 2048, "bf16", E=64, k=6, I=1408),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["round4", "restore8", "layer4", "layer4", "experts4", "experts4", "save8", "grad8"])
    if op == "round4":
        C = _log_uniform(rng, 32, 8192)
        C = C if rng.random() < 0.3 else (C + 31) // 32 * 32
        return _case(None, op, _log_uniform(rng, 1, (1 << 27) // C), C, rng.choice(["f32", "f16", "bf16"]))
    E = _log_uniform(rng, 2, 256)
    k = min(E, _log_uniform(rng, 1, 8))
    if op == "restore8":
        C = _log_uniform(rng, 32, 8192)
        C = C if rng.random() < 0.3 else (C + 31) // 32 * 32
        return _case(None, op, _log_uniform(rng, 1, (1 << 27) // (C * k)), C, rng.choice(["f32", "f16", "bf16"]),
                     E=E, k=k)
    step = 32 if op.endswith("4") else 8  # 4-bit rows are whole blocks, 16-bit rows whole 16-byte vectors
    H = max(64, _log_uniform(rng, 64, 7168) // step * step)
    I = max(64, _log_uniform(rng, 64, 8192) // step * step)
    E = max(k, min(E, (1 << 29) // (H * I)), 2)
    k = min(k, E)
    if op == "layer4":
        return _case(None, op, _log_uniform(rng, 1, 128), H, "bf16", E=E, k=k, I=I)
    most = _MAX_FLOPS / ((12 if op == "grad8" else 6) * k * H * I)
    return _case(None, op, _log_uniform(rng, 1, max(1, int(min(16384, most)))), H,
                 "bf16" if op == "experts4" else rng.choice(["f16", "bf16"]), E=E, k=k, I=I,
                 skew=rng.choice([0.0, 0.0, 1.0]))


# ---- the format, plain: q 2^s with q of 1 + mant bits of mantissa, s one per 32 columns ---------
# name: mantissa bits, largest exponent, smallest exponent, largest value, and from which
# significand on a block's largest value takes the next scale (half a step over the largest value)
_FORMAT = {"mxfp4": (1, 2, 0, 6.0, 1.75), "mxfp8": (3, 8, -6, 448.0, 1.8125)}


def _times2(x, s):
    """x 2^s, the power made of its bits: a rounded power would move values off the ties."""
    return x * ((s.long() + 1023) << 52).view(torch.float64).to(x.dtype)


def _quantize(x, fmt):
    """Elements [..., C/32, 32] (a short last block filled with zeros) and exponents [..., C/32, 1]."""
    mant, emax, emin, top, bump = _FORMAT[fmt]
    x = x.float()
    C = x.shape[-1]
    if C % 32:
        x = torch.nn.functional.pad(x, (0, 32 - C % 32))
    x = x.reshape(*x.shape[:-1], -1, 32)
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    s = e - 1 - emax + (2 * m >= bump).to(e.dtype)
    s = torch.where(m > 0, s, torch.full_like(s, -127)).clamp(-127, 127)
    y = _times2(x, -s)
    step = torch.frexp(y)[1]
    step = (step - 1).clamp(min=emin) - mant
    y = _times2(torch.round(_times2(y, -step)), step)
    return y.clamp(-top, top), s


def _values(q, s, C):
    v = _times2(q, s)
    return v.reshape(*v.shape[:-2], -1)[..., :C]


def _round(x, fmt):
    return _values(*_quantize(x, fmt), x.shape[-1])


def _pack4(q):
    """Two elements a byte, the first in the low half."""
    table = torch.zeros(13, dtype=torch.uint8, device=q.device)
    for code, twice in enumerate((0, 1, 2, 3, 4, 6, 8, 12)):
        table[twice] = code
    code = table[(2 * q.abs()).int()] + 8 * (q < 0).to(torch.uint8)
    code = code.reshape(*code.shape[:-2], -1, 2)
    return code[..., 0] + 16 * code[..., 1]


def _unpack4(packed, scales):
    """FP32 rows of packed elements and scale bytes."""
    half = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=packed.device)
    one = torch.cat([half, -half])
    byte = torch.arange(256, device=packed.device)
    pair = torch.stack([one[byte % 16], one[byte // 16]], 1)
    v = pair[packed.int()].reshape(*scales.shape, 32)
    v = _times2(v, scales.int()[..., None] - 127)
    return v.reshape(*scales.shape[:-1], -1)


# ---- inputs --------------------------------------------------------------------------------------
def _seed(case, seed):
    return (seed * 1000003 + case["T"] * 8191 + case["H"] * 131 + case["I"] * 17 + case["E"]) % (1 << 62)


def _chunks(E, per):
    step = max(1, (1 << 26) // per)
    return [(a, min(E, a + step)) for a in range(0, E, step)]


def _weights(gen, E, rows, cols, dt):
    w = torch.empty((E, rows, cols), dtype=dt, device="cuda")
    for a, b in _chunks(E, rows * cols):
        w[a:b] = torch.randn((b - a, rows, cols), generator=gen, device="cuda") / math.sqrt(cols)
    return w


def _weights4(gen, E, rows, cols):
    """Packed 4-bit weights [E, rows, cols/2] and scale bytes [E, rows, cols/32]."""
    values = torch.empty((E, rows, cols // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, rows, cols // 32), dtype=torch.uint8, device="cuda")
    for a, b in _chunks(E, rows * cols):
        w = torch.randn((b - a, rows, cols), generator=gen, device="cuda") / math.sqrt(cols)
        q, s = _quantize(w.to(torch.bfloat16), "mxfp4")
        values[a:b] = _pack4(q)
        scales[a:b] = (s[..., 0] + 127).to(torch.uint8)
    return values, scales


def prepare(case, seed):
    T, H, E, k, I = case["T"], case["H"], case["E"], case["k"], case["I"]
    dt, op = _DT[case["dtype"]], case["op"]
    N = T * k
    gen = torch.Generator(device="cuda").manual_seed(_seed(case, seed))
    st = {"case": case}

    # tokens behind a norm: unit normal, some channels larger than others
    def rows(n, c):
        return torch.randn((n, c), generator=gen, device="cuda") * torch.exp(
            0.5 * torch.randn((c,), generator=gen, device="cuda"))

    if op == "round4":  # weight rows
        st["x"] = (rows(T, H) / math.sqrt(H)).to(dt)
    elif op != "grad8":
        st["x"] = rows(T, H).to(dt)
    if op != "round4":
        logits = torch.randn((T, E), generator=gen, device="cuda")
        logits -= case["skew"] * torch.log(torch.arange(1, E + 1, device="cuda").float())
        if op == "layer4":
            st["logits"] = logits
        else:  # what dispatch hands on
            expert = torch.topk(logits, k, dim=1).indices.reshape(-1)
            counts = torch.bincount(expert, minlength=E)
            st["perm"] = torch.argsort(expert, stable=True).to(torch.int32)
            st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
            st["most"] = int(counts.max())
    if op in ("layer4", "experts4"):
        st["gate"], st["up"] = _weights4(gen, E, I, H), _weights4(gen, E, I, H)
        st["down"] = _weights4(gen, E, H, I)
    if op in ("save8", "grad8"):
        st["gate"], st["up"] = _weights(gen, E, I, H, dt), _weights(gen, E, I, H, dt)
        st["down"] = _weights(gen, E, H, I, dt)
    if op in ("experts4", "save8"):
        st["x_disp"] = st.pop("x")[st["perm"].long() // k]
    if op == "grad8":  # what the forward keeps: tokens and both projections in 8 bits
        for name, n, c in (("x8", T, H), ("g8", N, I), ("u8", N, I)):
            q, s = _quantize(rows(n, c), "mxfp8")
            st[name] = (q.reshape(n, -1)[:, :c].to(torch.float8_e4m3fn).view(torch.uint8).contiguous(),
                        (s[..., 0] + 127).to(torch.uint8))
        st["dout"] = (torch.randn((N, H), generator=gen, device="cuda") / math.sqrt(H)).to(dt)

    if own:
        import top_routing_grouped_fp32_gb300 as moe
        if op == "round4":
            st["mx"] = moe.MxRows.empty((T, H), "mxfp4", "cuda")
            st["out"] = torch.empty_like(st["x"])
        elif op == "restore8":
            st["mx"] = moe.MxRows.empty((T, H), "mxfp8", "cuda")
            st["out"] = torch.empty((N, H), dtype=dt, device="cuda")
        elif op in ("layer4", "experts4"):
            st["experts"] = moe.Mx4SwiGluExperts(*(moe.MxRows(*st[n], "mxfp4", c) for n, c in
                                                   (("gate", H), ("up", H), ("down", I))), dtype=dt)
            if op == "layer4":
                st["workspace"] = st["experts"].forward_workspace(T, k, torch.float32)
                st["out"] = torch.empty((T, H), dtype=dt, device="cuda")
            else:
                st["workspace"] = st["experts"].workspace(N)
                st["out"] = torch.empty((N, H), dtype=dt, device="cuda")
        else:
            st["experts"] = moe.SwiGluExperts(st["gate"], st["up"], st["down"])
            if op == "save8":
                st["checkpoint"] = moe.ExpertCheckpoint.empty(N, I, "cuda")
                st["workspace"] = st["experts"].checkpoint_workspace(N)
                st["out"] = torch.empty((N, H), dtype=dt, device="cuda")
                st["values"] = [torch.empty((N, I), dtype=dt, device="cuda") for _ in range(2)]
            else:
                st["x_mx"] = moe.MxRows(*st["x8"], "mxfp8", H)
                st["checkpoint"] = moe.ExpertCheckpoint(moe.MxRows(*st["g8"], "mxfp8", I),
                                                        moe.MxRows(*st["u8"], "mxfp8", I))
                st["workspace"] = st["experts"].backward_checkpoint_workspace(N)
                st["grads"] = (torch.empty_like(st["dout"]), torch.empty_like(st["gate"]),
                               torch.empty_like(st["up"]), torch.empty_like(st["down"]))
    return st


# ---- plain forms -----------------------------------------------------------------------------------
def _segments(st):
    """Rows by (expert, place): a gather into [E, most, .] with zeros behind each segment, and back."""
    off = st["offsets"].long()
    N, E = st["case"]["T"] * st["case"]["k"], st["case"]["E"]
    place = torch.arange(st["most"], device=off.device)
    row = off[:-1, None] + place
    inside = (row < off[1:, None])[..., None]
    row = row.clamp(max=N - 1)
    r = torch.arange(N, device=off.device)
    e = torch.bucketize(r, off[1:], right=True)
    return (lambda v: torch.where(inside, v.float()[row], torch.zeros((), device=off.device))), \
        (lambda v: v[e, r - off[e]])


def _silu(g):
    return g / (1 + torch.exp(-g))


def _plain_experts4(x, gate, up, down):
    """Batches of rows [B, n, H] by packed experts [B, ...]."""
    xq = _round(x, "mxfp4")
    g, u = (torch.bmm(xq, _unpack4(*w).transpose(1, 2)) for w in (gate, up))
    return torch.bmm(_round(_silu(g) * u, "mxfp4"), _unpack4(*down).transpose(1, 2))


def _layer4(st):
    case = st["case"]
    T, E, k = case["T"], case["E"], case["k"]
    p = torch.exp(st["logits"] - st["logits"].amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    v, i = torch.sort(st["logits"], dim=1, descending=True, stable=True)
    i = i[:, :k]
    w = torch.gather(p, 1, i)
    w = w / w.sum(1, keepdim=True)
    x = st["x"].float()
    if T * k <= E:  # each slot by its own expert
        sel = i.reshape(-1)
        part = [tuple(t[sel] for t in st[n]) for n in ("gate", "up", "down")]
        y = _plain_experts4(x[:, None].expand(T, k, -1).reshape(T * k, 1, -1), *part).view(T, k, -1)
    else:  # every token by every expert
        y = _plain_experts4(x[None].expand(E, -1, -1), st["gate"], st["up"], st["down"])
        y = y[i, torch.arange(T, device=x.device)[:, None]]
    return (w[..., None] * y).sum(1).to(st["x"].dtype)


def _save8(st):
    case = st["case"]
    spread, back = _segments(st)
    x = spread(st["x_disp"])
    g = torch.bmm(x, st["gate"].float().transpose(1, 2))
    u = torch.bmm(x, st["up"].float().transpose(1, 2))
    out = torch.bmm(_silu(g) * u, st["down"].float().transpose(1, 2))
    res = {"out": back(out).to(st["x_disp"].dtype)}
    for name, v in (("gate", g), ("up", u)):
        res[name] = _round(back(v), "mxfp8").to(res["out"].dtype)
    return res


def _unpack8(values, scales):
    v = values.view(torch.float8_e4m3fn).float()
    s = scales.int().repeat_interleave(32, dim=1)[:, :v.shape[1]] - 127
    return _times2(v, s)


def _grad8(st):
    k = st["case"]["k"]
    spread, back = _segments(st)
    x = spread(_unpack8(*st["x8"])[st["perm"].long() // k])
    g, u = spread(_unpack8(*st["g8"])), spread(_unpack8(*st["u8"]))
    dout = spread(st["dout"])
    da = torch.bmm(dout, st["down"].float())
    s = 1 / (1 + torch.exp(-g))
    dg = da * u * s * (1 + g * (1 - s))
    du = da * g * s
    a = g * s * u
    dx = torch.bmm(dg, st["gate"].float()) + torch.bmm(du, st["up"].float())
    dt = st["dout"].dtype
    return {"dinput": back(dx).to(dt), "dgate": torch.bmm(dg.transpose(1, 2), x).to(dt),
            "dup": torch.bmm(du.transpose(1, 2), x).to(dt), "ddown": torch.bmm(dout.transpose(1, 2), a).to(dt)}


def run(st):
    case = st["case"]
    op, k = case["op"], case["k"]
    if not own:
        if op == "round4":
            return _round(st["x"], "mxfp4").to(st["x"].dtype)
        if op == "restore8":
            return _round(st["x"], "mxfp8").to(st["x"].dtype)[st["perm"].long() // k]
        if op == "layer4":
            return _layer4(st)
        if op == "experts4":
            spread, back = _segments(st)
            return back(_plain_experts4(spread(st["x_disp"]), st["gate"], st["up"], st["down"])).to(
                st["x_disp"].dtype)
        return _save8(st) if op == "save8" else _grad8(st)
    import top_routing_grouped_fp32_gb300 as moe
    if op == "round4":
        mx = moe.moe_mx_quantize(st["x"], "mxfp4", out=st["mx"])
        return moe.moe_mx_dequantize(mx, st["x"].dtype, out=st["out"])
    if op == "restore8":
        mx = moe.moe_mx_quantize(st["x"], "mxfp8", out=st["mx"])
        return moe.moe_mx_dequantize(mx, st["x"].dtype, perm=st["perm"], top_k=k, out=st["out"])
    if op == "layer4":
        return st["experts"].forward(st["x"], st["logits"], k, True, y=st["out"], workspace=st["workspace"])
    if op == "experts4":
        return st["experts"].forward_dispatched(st["x_disp"], st["offsets"], out=st["out"],
                                                workspace=st["workspace"])
    if op == "save8":
        out, c = st["experts"].forward_checkpoint(st["x_disp"], st["offsets"], out=st["out"],
                                                  checkpoint=st["checkpoint"], workspace=st["workspace"])
        gate, up = (moe.moe_mx_dequantize(m, o.dtype, out=o) for m, o in zip((c.gate, c.up), st["values"]))
        return {"out": out, "gate": gate, "up": up}
    dinput, dgate, dup, ddown = st["experts"].backward_checkpoint(
        st["x_mx"], st["perm"], st["offsets"], st["checkpoint"], st["dout"], k, grads=st["grads"],
        workspace=st["workspace"])
    return {"dinput": dinput, "dgate": dgate, "dup": dup, "ddown": ddown}


def work(case):
    T, H, E, k, I = case["T"], case["H"], case["E"], case["k"], case["I"]
    size, op, N = _SIZE[case["dtype"]], case["op"], case["T"] * case["k"]
    if op == "round4":  # read, held, read back, written
        return {"bytes": T * H * (2 * size + 2 * 17 / 32), "flops": 4 * T * H}
    if op == "restore8":
        return {"bytes": T * H * (size + 2 * 33 / 32) + N * (H * size + 4), "flops": 3 * T * H + N * H}
    if op in ("layer4", "experts4"):
        touched = E * (1 - (1 - k / E) ** T)  # experts that an even routing meets
        rows = T * (2 * H * size + 4 * E) if op == "layer4" else N * 2 * H * size + 4 * E
        return {"bytes": touched * 3 * H * I * 17 / 32 + rows, "flops": 6 * N * H * I}
    weights = 3 * E * H * I * size
    blocks = I + (I + 31) // 32
    if op == "save8":  # the checkpoint is written, and read back
        return {"bytes": weights + N * (2 * H * size + 4 * blocks + 2 * I * size), "flops": 6 * N * H * I}
    return {"bytes": 2 * weights + N * (2 * H * size + 2 * blocks) + T * (H + (H + 31) // 32),
            "flops": 12 * N * H * I}


# ---- the definitions in 64 bits ----------------------------------------------------------------------
def _grid(fmt, dev):
    """The format's values >= 0 in order; a value's place is its code."""
    mant, emax, emin, top, _ = _FORMAT[fmt]
    v = [i * 2.0 ** (emin - mant) for i in range(1 << mant)]
    for e in range(emin, emax + 1):
        v += [(1 + i / (1 << mant)) * 2.0 ** e for i in range(1 << mant)]
    return torch.tensor([x for x in v if x <= top], dtype=torch.float64, device=dev)


def _power(p):
    """2^p in 64 bits, exactly, of whole p."""
    table = torch.tensor([2.0 ** i for i in range(-400, 401)], dtype=torch.float64, device=p.device)
    return table[p.long() + 400]


def _exact_blocks(x, fmt):
    """Elements [n, C] and scales [n, C/32] of rows x, FP64: the nearest value of the format, ties to the
    even code."""
    _, emax, _, top, bump = _FORMAT[fmt]
    n, C = x.shape
    B = (C + 31) // 32
    full = torch.zeros((n, B * 32), dtype=torch.float64, device=x.device)
    full[:, :C] = x
    full = full.view(n, B, 32)
    amax = full.abs().amax(2)
    p = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax))))
    p += (amax >= _power(p + 1)).double() - (amax < _power(p)).double()  # where the logarithm rounded
    s = p - emax + (amax >= bump * _power(p)).double()
    scale = _power(torch.where(amax > 0, s, torch.full_like(s, -127)).clamp(-127, 127))
    y = full / scale[..., None]
    grid = _grid(fmt, x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    code = torch.bucketize(y.abs().contiguous(), mid)  # number of middles below
    tie = (code < len(mid)) & (y.abs() == mid[code.clamp(max=len(mid) - 1)]) & (code % 2 == 1)
    q = torch.copysign(grid[code + tie.long()], y)
    return q.reshape(n, -1)[:, :C], scale


def _exact_round(x, fmt):
    q, scale = _exact_blocks(x, fmt)
    return q * scale.repeat_interleave(32, dim=1)[:, :x.shape[1]]


def _exact_weight4(values, scales):
    grid = _grid("mxfp4", values.device)
    code = torch.stack([values & 15, values >> 4], -1).reshape(values.shape[0], -1).long()
    v = grid[code & 7] * (1 - 2 * (code >> 3)).double()
    return v * _power(scales.int() - 127).repeat_interleave(32, dim=1)


def _exact_rows8(values, scales):
    v = values.view(torch.float8_e4m3fn).double()
    return v * _power(scales.int() - 127).repeat_interleave(32, dim=1)[:, :v.shape[1]]


def _exact_expert4(st, e, x):
    gate, up, down = (_exact_weight4(st[n][0][e], st[n][1][e]) for n in ("gate", "up", "down"))
    xq = _exact_round(x, "mxfp4")
    g, u = xq @ gate.t(), xq @ up.t()
    return _exact_round(g * torch.sigmoid(g) * u, "mxfp4") @ down.t()


def exact(case, seed):
    st = prepare(case, seed)
    T, H, E, k, I = case["T"], case["H"], case["E"], case["k"], case["I"]
    op, N, f64, dev = case["op"], case["T"] * case["k"], torch.float64, "cuda"
    if op in ("round4", "restore8"):
        fmt = "mxfp4" if op == "round4" else "mxfp8"
        step = max(1, (1 << 25) // H)
        v = torch.cat([_exact_round(st["x"][a:a + step].to(f64), fmt) for a in range(0, T, step)])
        return v if op == "round4" else v[st["perm"].long() // k]
    if op == "layer4":
        l = st["logits"].to(f64)
        order = torch.argsort(-l, dim=1, stable=True)[:, :k]
        w = torch.softmax(torch.gather(l, 1, order), 1)  # renormalised over the chosen
        y = torch.zeros((T, H), dtype=f64, device=dev)
        for e in order.unique().tolist():
            t, j = torch.nonzero(order == e, as_tuple=True)
            y.index_add_(0, t, w[t, j][:, None] * _exact_expert4(st, e, st["x"][t].to(f64)))
        return y
    off = st["offsets"].tolist()
    if op == "experts4":
        out = torch.zeros((N, H), dtype=f64, device=dev)
        for e in range(E):
            a, b = off[e], off[e + 1]
            if b > a:
                out[a:b] = _exact_expert4(st, e, st["x_disp"][a:b].to(f64))
        return out
    if op == "save8":
        out = torch.zeros((N, H), dtype=f64, device=dev)
        both = torch.zeros((2, N, I), dtype=f64, device=dev)
        for e in range(E):
            a, b = off[e], off[e + 1]
            x = st["x_disp"][a:b].to(f64)
            g, u = x @ st["gate"][e].to(f64).t(), x @ st["up"][e].to(f64).t()
            both[0, a:b], both[1, a:b] = g, u
            out[a:b] = (g * torch.sigmoid(g) * u) @ st["down"][e].to(f64).t()
        return {"out": out, "gate": _exact_round(both[0], "mxfp8"), "up": _exact_round(both[1], "mxfp8")}
    dx = torch.zeros((N, H), dtype=f64, device=dev)
    grads = {"dgate": torch.zeros((E, I, H), dtype=f64, device=dev),
             "dup": torch.zeros((E, I, H), dtype=f64, device=dev),
             "ddown": torch.zeros((E, H, I), dtype=f64, device=dev)}
    x8 = _exact_rows8(*st["x8"])
    for e in range(E):
        a, b = off[e], off[e + 1]
        x = x8[st["perm"][a:b].long() // k]
        g, u = (_exact_rows8(st[n][0][a:b], st[n][1][a:b]) for n in ("g8", "u8"))
        dout = st["dout"][a:b].to(f64)
        da = dout @ st["down"][e].to(f64)
        s = torch.sigmoid(g)
        dg, du = da * u * (s + g * s * (1 - s)), da * g * s
        dx[a:b] = dg @ st["gate"][e].to(f64) + du @ st["up"][e].to(f64)
        grads["dgate"][e], grads["dup"][e] = dg.t() @ x, du.t() @ x
        grads["ddown"][e] = dout.t() @ (g * s * u)
    return {"dinput": dx, **grads}
