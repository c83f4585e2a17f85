"""The experts' training step with activations in 8 bits, against the definition in
64 bits.  Tolerances: half a step of each 16-bit rounding (dg, du, a, the result),
FP32 sums once a 16-deep step, and half a step of e4m3 for what is held."""
import pytest
import torch

import mx_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
F64 = torch.float64


class Step:
    """A routed batch: x [T,H], its dispatch, experts and a gradient of their outputs."""

    def __init__(self, moe, T, E, k, H, I, dt, seed=0, skew=0.0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*s):
            return torch.randn(s, generator=g, device="cuda")
        self.moe, self.T, self.E, self.k, self.H, self.I, self.dt = moe, T, E, k, H, I, dt
        self.x = randn(T, H).to(dt)
        self.w = [(randn(E, a, b) / b ** 0.5).to(dt) for a, b in ((I, H), (I, H), (H, I))]
        logits = randn(T, E) - skew * torch.arange(E, device="cuda")
        self.idx, _ = moe.moe_route(logits, k, True)
        self.d = moe.moe_dispatch(self.idx, E, x=self.x)
        self.dout = (randn(T * k, H) / H ** 0.5).to(dt)
        self.ex = moe.SwiGluExperts(*self.w)
        self.x_mx = moe.moe_mx_quantize(self.x, "mxfp8")
        self.off = self.d.offsets.tolist()

    def forward(self, **kw):
        return self.ex.forward_checkpoint(self.d.x_disp, self.d.offsets, **kw)

    def backward(self, ck, **kw):
        return self.ex.backward_checkpoint(self.x_mx, self.d.perm, self.d.offsets, ck, kw.pop("dout", self.dout),
                                           self.k, **kw)


SIZES = [  # T, E, k, H, I, skew
    (1, 1, 1, 8, 8, 0.0), (5, 4, 2, 64, 40, 0.0), (64, 2, 1, 64, 64, 0.0), (129, 4, 2, 520, 328, 0.0),
    (300, 8, 3, 136, 272, 1.0), (256, 1, 1, 256, 256, 0.0), (700, 2, 2, 72, 520, 0.5), (40, 64, 2, 32, 32, 0.0),
]


@pytest.mark.parametrize("T,E,k,H,I,skew", SIZES)
@pytest.mark.parametrize("dt", sorted(DT))
def test_forward(cuda_lib, T, E, k, H, I, skew, dt):
    s = Step(cuda_lib, T, E, k, H, I, DT[dt], skew=skew)
    out, ck = s.forward()
    assert torch.equal(out, s.ex.forward_dispatched(s.d.x_disp, s.d.offsets))
    for name, mx, w in (("gate", ck.gate, s.w[0]), ("up", ck.up, s.w[1])):
        held = ref.held(mx)
        for e in range(E):
            a, b = s.off[e], s.off[e + 1]
            if a == b:
                continue
            x, we = s.d.x_disp[a:b].to(F64), w[e].to(F64)
            g = x @ we.t()
            slip = (H / 16 + 2) * 2.0 ** -23 * (x.abs() @ we.abs().t())
            # half a step of e4m3 at the value (of its subnormals: 2^-10 of the scale; the largest
            # value clips less than half its step), at the scale that the largest value asks for
            top = ref.blocks(g.abs() + slip).amax(2)
            scale = ref.power(torch.frexp(top)[1] - 8)[..., None].expand(-1, -1, 32).reshape(b - a, -1)[:, :I]
            tol = 2.0 ** -4 * g.abs() + 2.0 ** -10 * scale + 1.1 * slip
            assert ((held[a:b] - g).abs() <= tol).all(), (name, e)


def formulas(x, g, u, dout, gate, up, down):
    """The backward of one expert in 64 bits, and how far 16-bit operands may put it
    (in units of eps, to be multiplied by half a step)."""
    da = dout @ down
    s = torch.sigmoid(g)
    dg, du, a = da * u * s * (1 + g * (1 - s)), da * g * s, g * s * u
    res = [dg @ gate + du @ up, dg.t() @ x, du.t() @ x, dout.t() @ a]
    size = [dg.abs() @ gate.abs() + du.abs() @ up.abs(), dg.abs().t() @ x.abs(), du.abs().t() @ x.abs(),
            dout.abs().t() @ a.abs()]
    # da's own error: FP32 sums and the exponential's few ulp
    dda = (dout.shape[1] / 16 + 2) * 2.0 ** -23 * (dout.abs() @ down.abs()) + 64 * 2.0 ** -24 * da.abs()
    eg, eu = dda * (u * s * (1 + g * (1 - s))).abs(), dda * (g * s).abs()
    # cancelling 1 + g (1 - s): the slope is off by a few ulp of its terms
    eg = eg + (da * u).abs() * 16 * 2.0 ** -24 * (s + (g * s * (1 - s)).abs())
    slip = [eg @ gate.abs() + eu @ up.abs(), eg.t() @ x.abs(), eu.t() @ x.abs(),
            dout.abs().t() @ (a.abs() * 16 * 2.0 ** -24)]
    return res, size, slip


def check(s, ck, got, dout):
    eps = torch.finfo(s.dt).eps / 2
    least = torch.finfo(s.dt).smallest_normal * torch.finfo(s.dt).eps  # a step of the subnormals
    token = ref.held(s.x_mx)
    g, u = ref.held(ck.gate), ref.held(ck.up)
    perm = s.d.perm.long()
    for e in range(s.E):
        a, b = s.off[e], s.off[e + 1]
        args = (token[perm[a:b] // s.k].to(s.dt).to(F64), g[a:b], u[a:b], dout[a:b].to(F64), *(w[e].to(F64) for w in s.w))
        res, size, slip = formulas(*args)
        parts = (got[0][a:b], got[1][e], got[2][e], got[3][e])
        rows = max(b - a, s.I, 1)
        for name, o, r, z, p in zip(("dinput", "dgate", "dup", "ddown"), parts, res, size, slip):
            tol = (eps * (r.abs() + z) * 1.02 + p + (2 * rows / 16 + 2) * 2.0 ** -23 * z
                   + least * (1 + rows * (args[4].abs().max() + args[0].abs().max().nan_to_num() if b > a else 1)))
            assert ((o.to(F64) - r).abs() <= tol).all(), (name, e, ((o.to(F64) - r).abs() / tol).max())


@pytest.mark.parametrize("T,E,k,H,I,skew", SIZES)
@pytest.mark.parametrize("dt", sorted(DT))
def test_backward(cuda_lib, T, E, k, H, I, skew, dt):
    s = Step(cuda_lib, T, E, k, H, I, DT[dt], skew=skew)
    _, ck = s.forward()
    ws = s.ex.backward_checkpoint_workspace(T * k)
    ws.fill_(0xFF)
    got = s.backward(ck, workspace=ws)
    check(s, ck, got, s.dout)
    assert cuda_lib.moe_get_device_status(ws) == 0
    for a, b in zip(got, s.backward(ck)):
        assert torch.equal(a, b)
    for e in range(E):  # experts without rows
        if s.off[e] == s.off[e + 1]:
            assert not got[1][e].any() and not got[2][e].any() and not got[3][e].any()


def test_formulas_against_differences():
    """The reference's gradients are those of sum(dout * out) with g and u of x and the
    weights, by central differences in 64 bits."""
    gen = torch.Generator().manual_seed(0)
    x, dout = torch.randn((6, 8), generator=gen, dtype=F64), torch.randn((6, 8), generator=gen, dtype=F64)
    gate, up = (torch.randn((5, 8), generator=gen, dtype=F64) for _ in range(2))
    down = torch.randn((8, 5), generator=gen, dtype=F64)

    def loss():
        return (dout * ((ref.silu(x @ gate.t()) * (x @ up.t())) @ down.t())).sum()
    res, _, _ = formulas(x, x @ gate.t(), x @ up.t(), dout, gate, up, down)
    for t, grad in zip((x, gate, up, down), res):
        for i in range(0, t.numel(), 3):
            flat, h = t.view(-1), 1e-6
            keep = flat[i].item()
            flat[i] = keep + h
            hi = loss()
            flat[i] = keep - h
            lo = loss()
            flat[i] = keep
            assert abs((hi - lo) / (2 * h) - grad.reshape(-1)[i]) < 1e-7 * (1 + grad.abs().max())


@pytest.mark.parametrize("T,E,k,H,I,skew", [(1100, 1, 1, 72, 40, 0.0), (1300, 2, 2, 264, 40, 0.7), (900, 3, 1, 40, 296, 2.0)])
def test_few_tiles_over_many_rows(cuda_lib, T, E, k, H, I, skew):
    """Weight gradients of few tiles: the rows of an expert are cut into parts that are joined."""
    s = Step(cuda_lib, T, E, k, H, I, torch.bfloat16, skew=skew)
    _, ck = s.forward()
    ws = s.ex.backward_checkpoint_workspace(T * k)
    ws.fill_(0xFF)
    got = s.backward(ck, workspace=ws)
    check(s, ck, got, s.dout)
    assert all(torch.equal(a, b) for a, b in zip(got, s.backward(ck)))


@pytest.mark.parametrize("T,E,k,H,I,skew", [(3, 4, 2, 72, 1000, 0.0), (30, 6, 2, 296, 808, 3.0), (1, 1, 1, 8, 2056, 0.0),
                                            (300, 2, 1, 264, 1032, 0.5), (513, 1, 1, 40, 520, 0.0)])
@pytest.mark.parametrize("dt", sorted(DT))
def test_few_tiles_over_long_rows(cuda_lib, T, E, k, H, I, skew, dt):
    """dinput of few tiles: its sums over the intermediate size are cut into parts that are joined."""
    s = Step(cuda_lib, T, E, k, H, I, DT[dt], skew=skew)
    _, ck = s.forward()
    ws = s.ex.backward_checkpoint_workspace(T * k)
    ws.fill_(0xFF)
    got = s.backward(ck, workspace=ws)
    check(s, ck, got, s.dout)
    assert cuda_lib.moe_get_device_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, s.backward(ck)))


@pytest.mark.parametrize("I", [64, 1032])
def test_rows_behind_the_last_of_two_segments(cuda_lib, I):
    """An expert without rows, and rows behind the last segment, which no part of a sum may touch."""
    moe = cuda_lib
    s = Step(moe, 50, 2, 2, 64, I, torch.bfloat16)
    _, ck = s.forward()
    off = torch.tensor([0, 0, 33], dtype=torch.int32, device="cuda")
    grads = [torch.full(t, 3.0, dtype=torch.bfloat16, device="cuda") for t in
             ((100, 64), (2, I, 64), (2, I, 64), (2, 64, I))]
    dout = s.dout.clone()
    dout[33:] = float("nan")
    s.ex.backward_checkpoint(s.x_mx, s.d.perm, off, ck, dout, 2, grads=tuple(grads))
    assert (grads[0][33:] == 3).all() and torch.isfinite(grads[0][:33]).all()
    assert all(not g[0].any() and torch.isfinite(g[1]).all() and g[1].any() for g in grads[1:])


@pytest.mark.parametrize("T,E,k,I", [(40, 4, 2, 64), (500, 2, 1, 64)])
def test_what_is_not_finite_stays_in_its_expert(cuda_lib, T, E, k, I):
    """A NaN in a row of dout, next to a segment's end, reaches its own dinput row and its own
    expert's gradients; the other experts' are bit for bit what they were."""
    s = Step(cuda_lib, T, E, k, 64, I, torch.bfloat16)
    _, ck = s.forward()
    clean = s.backward(ck)
    for e in range(E):
        dout = s.dout.clone()
        row = s.off[e]  # the first row of e lies behind the last of e - 1
        dout[row] = float("nan")
        got = s.backward(ck, dout=dout)
        assert torch.isnan(got[0][row]).all() and torch.isnan(got[3][e]).any()
        others = [j for j in range(T * k) if j != row]
        assert torch.equal(got[0][others], clean[0][others])
        for o in range(E):
            if o != e:
                assert all(torch.equal(g[o], c[o]) for g, c in zip(got[1:], clean[1:]))


def test_rows_behind_the_segments(cuda_lib):
    """Offsets that end early: rows behind them are left as they were, and may hold NaN."""
    moe = cuda_lib
    s = Step(moe, 50, 2, 2, 64, 64, torch.bfloat16)
    off = torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda")
    ck = moe.ExpertCheckpoint.empty(100, 64)
    for m in (ck.gate, ck.up):
        m.values.fill_(9), m.scales.fill_(255)
    xd, dout = s.d.x_disp.clone(), s.dout.clone()
    xd[70:] = dout[70:] = float("nan")
    s.ex.forward_checkpoint(xd, off, checkpoint=ck)
    assert (ck.gate.values[70:] == 9).all() and (ck.up.scales[70:] == 255).all()
    assert (ck.gate.scales[:70] < 255).all()
    grads = [torch.full(t, 3.0, dtype=torch.bfloat16, device="cuda") for t in
             ((100, 64), (2, 64, 64), (2, 64, 64), (2, 64, 64))]
    perm = s.d.perm.clone()
    perm[70:] = -1
    s.ex.backward_checkpoint(s.x_mx, perm, off, ck, dout, 2, grads=tuple(grads))
    assert (grads[0][70:] == 3).all()
    assert all(torch.isfinite(g).all() for g in grads)


def test_offsets_that_are_wrong_and_no_rows(cuda_lib):
    moe = cuda_lib
    s = Step(moe, 20, 2, 2, 64, 64, torch.bfloat16)
    _, ck = s.forward()
    for bad in ([0, 50, 40], [0, 30, 20], [0, 10, 41]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        ws = s.ex.backward_checkpoint_workspace(40)
        s.ex.backward_checkpoint(s.x_mx, s.d.perm, off, ck, s.dout, 2, workspace=ws)
        assert moe.moe_get_device_status(ws) == 6
    none = moe.ExpertCheckpoint.empty(0, 64)
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    got = s.ex.backward_checkpoint(moe.MxRows.empty((0, 64), "mxfp8"), s.d.perm[:0], zero, none, s.dout[:0], 2)
    assert got[0].shape == (0, 64) and not any(g.any() for g in got[1:])


def test_a_training_step_and_its_graph(cuda_lib):
    """Forward and backward of the layer's experts as a step runs them, with the dispatch and
    combine around them; then the same captured, replayed on other tokens."""
    moe = cuda_lib
    s = Step(moe, 200, 4, 2, 136, 72, torch.bfloat16)
    x, weights = s.x.clone(), torch.rand((200, 2), device="cuda")
    dy = torch.randn_like(x)
    x_mx, ck = moe.MxRows.empty(x.shape, "mxfp8"), moe.ExpertCheckpoint.empty(400, 72)
    ws = (s.ex.checkpoint_workspace(400), s.ex.backward_checkpoint_workspace(400))
    grads = (torch.empty((400, 136), dtype=x.dtype, device="cuda"), *(torch.empty_like(w) for w in s.w))
    out = torch.empty_like(grads[0])

    def step():
        moe.moe_mx_quantize(x, "mxfp8", out=x_mx)
        x_disp = x[(s.d.perm // 2).long()]
        s.ex.forward_checkpoint(x_disp, s.d.offsets, out=out, checkpoint=ck, workspace=ws[0])
        dexpert, dweights = moe.moe_combine_backward(out, s.d.perm, weights, dy, 2)
        s.ex.backward_checkpoint(x_mx, s.d.perm, s.d.offsets, ck, dexpert, 2, grads=grads, workspace=ws[1])
        return moe.moe_dispatch_backward(grads[0], s.d.perm, 200, 2), dweights
    first = [t.clone() for t in (*step(), *grads)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    x.mul_(-0.5)
    graph.replay()
    replayed = [t.clone() for t in (*res, *grads)]
    x.mul_(-2.0)
    graph.replay()
    for a, b in zip(first, (*res, *grads)):
        assert torch.equal(a, b)
    x.mul_(-0.5)
    for a, b in zip(replayed, (*step(), *grads)):
        assert torch.equal(a, b)


def test_refusals(cuda_lib):
    moe = cuda_lib
    s = Step(moe, 10, 2, 2, 64, 64, torch.bfloat16)
    _, ck = s.forward()
    four = moe.moe_mx_quantize(s.x, "mxfp4")
    f32 = moe.SwiGluExperts(*[w.float() for w in s.w])
    odd = moe.SwiGluExperts(*[torch.zeros(t, dtype=torch.bfloat16, device="cuda") for t in ((2, 64, 60), (2, 64, 60), (2, 60, 64))])
    args = (s.x_mx, s.d.perm, s.d.offsets, ck, s.dout, 2)

    def with_(i, v):
        return tuple(v if j == i else a for j, a in enumerate(args))
    grads = s.ex.backward_checkpoint(*args)
    for call, status in (
            (lambda: s.ex.backward_checkpoint(*with_(0, four)), 3), (lambda: s.ex.backward_checkpoint(*with_(5, 3)), 2),
            (lambda: s.ex.backward_checkpoint(*with_(1, s.d.perm[:10].clone())), 2),
            (lambda: s.ex.backward_checkpoint(*with_(4, s.dout.half())), 3),
            (lambda: s.ex.backward_checkpoint(*with_(3, moe.ExpertCheckpoint(ck.gate, four))), 3),
            (lambda: s.ex.backward_checkpoint(*args, grads=(s.dout, *grads[1:])), 1),
            (lambda: s.ex.backward_checkpoint(*args, grads=(grads[0], grads[1], grads[1], grads[3])), 1),
            (lambda: s.ex.backward_checkpoint(*args, workspace=torch.empty(512, dtype=torch.uint8, device="cuda")), 1),
            (lambda: s.ex.forward_checkpoint(s.d.x_disp.half(), s.d.offsets), 3),
            (lambda: s.ex.forward_checkpoint(s.d.x_disp, s.d.offsets, checkpoint=moe.ExpertCheckpoint.empty(19, 64)), 2),
            (lambda: f32.forward_checkpoint(s.d.x_disp.float(), s.d.offsets), 4),
            (lambda: odd.forward_checkpoint(torch.zeros((20, 60), dtype=torch.bfloat16, device="cuda"), s.d.offsets), 4)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == status, e.value


def test_what_overlaps_is_refused(cuda_lib):
    """Gradients over what is still read, and a checkpoint over the forward's rows."""
    moe = cuda_lib
    s = Step(moe, 64, 2, 2, 64, 64, torch.bfloat16)
    out, ck = s.forward()
    grads = s.backward(ck)
    pool = torch.zeros(1 << 17, dtype=torch.uint8, device="cuda")  # [N, H] and [E, I, H] in 16 bits take 16 KiB each

    def at(i, n, shape, dtype):
        return pool[i:i + n].view(dtype).view(shape)
    dinput = at(16384, 16384, (128, 64), torch.bfloat16)
    x = moe.MxRows(at(16384 + 16368, 4096, (64, 64), torch.uint8), s.x_mx.scales, "mxfp8", 64)
    x_scales = moe.MxRows(s.x_mx.values, at(16384 - 127, 128, (64, 2), torch.uint8), "mxfp8", 64)
    perm = at(16384, 512, (128,), torch.int32)
    offsets = at(16384 + 16380, 12, (3,), torch.int32)
    gate = moe.MxRows(at(16384 - 8176, 8192, (128, 64), torch.uint8), ck.gate.scales, "mxfp8", 64)
    up = moe.MxRows(ck.up.values, at(32767, 256, (128, 2), torch.uint8), "mxfp8", 64)
    args = (s.x_mx, s.d.perm, s.d.offsets, ck, s.dout, 2)
    for i, v in ((0, x), (0, x_scales), (1, perm), (2, offsets), (3, moe.ExpertCheckpoint(gate, ck.up)),
                 (3, moe.ExpertCheckpoint(ck.gate, up))):
        with pytest.raises(moe.MoeError, match="overlap") as e:
            s.ex.backward_checkpoint(*(v if j == i else a for j, a in enumerate(args)), grads=(dinput, *grads[1:]))
        assert e.value.status == 1
    for kept in (moe.ExpertCheckpoint(gate, ck.up), moe.ExpertCheckpoint(ck.gate, up), moe.ExpertCheckpoint(ck.gate, ck.gate)):
        with pytest.raises(moe.MoeError, match="overlap"):
            s.ex.forward_checkpoint(s.d.x_disp, s.d.offsets, out=dinput, checkpoint=kept)
    assert not pool.any()
    # next to each other is not over each other
    x.values = at(32768, 4096, (64, 64), torch.uint8)
    x.values.copy_(s.x_mx.values)
    got = s.ex.backward_checkpoint(x, *args[1:], grads=(dinput, *(torch.empty_like(g) for g in grads[1:])))
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    assert torch.equal(s.ex.forward_checkpoint(s.d.x_disp, s.d.offsets, out=s.d.x_disp)[0], out)
