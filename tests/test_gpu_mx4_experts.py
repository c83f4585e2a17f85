"""Experts on 4-bit operands against the definition in 64 bits.  Tolerances count
the output's rounding, the FP32 sums' (once a 64-deep step) and the elements of h
that lie on a border of the format within their own error (mx_reference)."""
import pytest
import torch

import mx_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def make(moe, E, H, I, dt=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = [torch.randn((E, a, b), generator=g, device="cuda") / b ** 0.5 for a, b in ((I, H), (I, H), (H, I))]
    mx = [moe.moe_mx_quantize(t.to(torch.bfloat16), "mxfp4") for t in w]
    return moe.Mx4SwiGluExperts(*mx, dtype=dt), mx


def weights64(moe, mx, e):
    return [ref.held(moe.MxRows(m.values[e], m.scales[e], "mxfp4", m.cols)) for m in mx]


def rows(n, H, dt, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((n, H), generator=g, device="cuda") * torch.exp(0.5 * torch.randn(H, generator=g, device="cuda"))).to(dt)


def segments(counts, first=0):
    off = torch.tensor([first] + list(counts), dtype=torch.int64).cumsum(0)
    return off.to(torch.int32).cuda()


def check(moe, mx, x, off, out, dt):
    o = off.tolist()
    for e in range(len(o) - 1):
        a, b = o[e], o[e + 1]
        if a == b:
            continue
        want, tol = ref.experts4(x[a:b].double(), *weights64(moe, mx, e), dt)
        assert ((out[a:b].double() - want).abs() <= tol + 1e-30).all(), (
            e, ((out[a:b].double() - want).abs() / (tol + 1e-30)).max())


SIZES = [  # H, I, rows per expert
    (32, 32, [1]), (64, 96, [5, 0, 33]), (288, 544, [0, 0, 1, 32, 31, 0, 64]), (1056, 160, [129, 127]),
    (256, 256, [128]), (544, 1056, [257, 0, 300]), (512, 192, [1000]), (96, 3104, [3, 2]), (2048, 64, [40, 41, 42]),
    (64, 64, [255, 256, 1, 512]),
]


@pytest.mark.parametrize("H,I,counts", SIZES)
@pytest.mark.parametrize("dt", sorted(DT))
def test_dispatched_rows(cuda_lib, H, I, counts, dt):
    moe = cuda_lib
    ex, mx = make(moe, len(counts), H, I, DT[dt])
    n = sum(counts)
    x, off = rows(n, H, DT[dt]), segments(counts)
    ws = ex.workspace(n)
    ws.fill_(0xFF)  # scales of rows that no segment holds may be anything
    out = ex.forward_dispatched(x, off, workspace=ws)
    check(moe, mx, x, off, out, DT[dt])
    assert moe.moe_get_device_status(ws) == 0
    assert torch.equal(out, ex.forward_dispatched(x, off))


@pytest.mark.parametrize("H,I,counts", [
    (64, 2688, [9000, 0, 300, 12800]), (1056, 2720, [5121, 255, 16000, 600]), (2048, 2688, [11000, 11001]),
    (5376, 96, [9000, 0, 300, 12800]), (5408, 544, [1, 7000, 511, 14500]), (5408, 1568, [22001, 0, 0])])
def test_many_rows(cuda_lib, H, I, counts):
    """Weights' tiles kept for several of the rows' (three and four spans of 512 columns, cut and whole),
    and loaded again (one and two)."""
    moe = cuda_lib
    ex, mx = make(moe, len(counts), H, I)
    n = sum(counts)
    x, off = rows(n, H, torch.bfloat16), segments(counts)
    ws = ex.workspace(n)
    ws.fill_(0xFF)
    out = ex.forward_dispatched(x, off, workspace=ws)
    check(moe, mx, x, off, out, torch.bfloat16)
    assert moe.moe_get_device_status(ws) == 0
    assert torch.equal(out, ex.forward_dispatched(x, off))


@pytest.mark.parametrize("counts", [[3, 0, 20], [300, 0, 260]])
def test_rows_outside_the_segments_are_left(cuda_lib, counts):
    moe = cuda_lib
    ex, mx = make(moe, 3, 64, 96)
    n = sum(counts) + 12
    x, off = rows(n, 64, torch.bfloat16), segments(counts, first=5)
    x[:5] = x[n - 7:] = float("nan")
    out = torch.full((n, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ex.forward_dispatched(x, off, out=out)
    assert (out[:5] == 7).all() and (out[n - 7:] == 7).all()
    check(moe, mx, x, off, out, torch.bfloat16)


@pytest.mark.parametrize("counts", [[9, 4], [200, 190]])
def test_what_is_not_finite_stays_in_its_row(cuda_lib, counts):
    moe = cuda_lib
    ex, mx = make(moe, 2, 288, 96)
    n = sum(counts)
    x, off = rows(n, 288, torch.bfloat16), segments(counts)
    clean = ex.forward_dispatched(x, off)
    x[2, 287], x[n - 1, 0], x[5] = float("nan"), float("inf"), 0
    out = ex.forward_dispatched(x, off)
    assert torch.isnan(out[2]).all() and torch.isnan(out[n - 1]).all() and (out[5] == 0).all()
    keep = [i for i in range(n) if i not in (2, 5, n - 1)]
    assert torch.equal(out[keep], clean[keep])


def test_a_weight_block_without_values(cuda_lib):
    """Scale byte 255 in a row of down: that output column is NaN, for its expert only."""
    moe = cuda_lib
    _, mx = make(moe, 2, 64, 96)
    mx[2].scales[1, 7, 2] = 255
    ex = moe.Mx4SwiGluExperts(*mx)
    x, off = rows(40, 64, torch.bfloat16), segments([20, 20])
    out = ex.forward_dispatched(x, off)
    bad = torch.isnan(out)
    assert bad[20:, 7].all() and bad.sum() == 20


def test_offsets_that_are_wrong(cuda_lib):
    moe = cuda_lib
    ex, _ = make(moe, 4, 64, 64)
    x = rows(50, 64, torch.bfloat16)
    for bad in ([0, 10, 5, 40, 50], [0, 10, 20, 30, 60], [0, -1, 20, 30, 50]):
        ws = ex.workspace(50)
        ex.forward_dispatched(x, torch.tensor(bad, dtype=torch.int32, device="cuda"), workspace=ws)
        assert moe.moe_get_device_status(ws) == 6
    ws = ex.workspace(50)
    ex.forward_dispatched(x, segments([10, 10, 10, 20]), workspace=ws)
    assert moe.moe_get_device_status(ws) == 0


LAYERS = [(1, 5, 2, 64, 64), (3, 1, 1, 96, 32), (32, 256, 8, 256, 96), (7, 1024, 3, 64, 64), (128, 2, 2, 64, 64),
          (129, 2, 2, 64, 64), (40, 64, 40, 32, 32), (300, 3, 2, 288, 160)]


@pytest.mark.parametrize("T,E,k,H,I", LAYERS)
@pytest.mark.parametrize("ldt", ["f32", "bf16"])
def test_the_fused_forward_is_the_stages_together(cuda_lib, T, E, k, H, I, ldt):
    """route -> dispatch -> experts -> combine by the staged calls, the combine in 64 bits on
    the routing weights: the fused outputs are that, rounded once (its slots are FP32, the
    staged expert outputs 16-bit: half a step of each)."""
    moe = cuda_lib
    ex, mx = make(moe, E, H, I, seed=T)
    x = rows(T, H, torch.bfloat16)
    logits = torch.randn((T, E), device="cuda").to(torch.float32 if ldt == "f32" else torch.bfloat16)
    idx, w = moe.moe_route(logits, k, True)
    d = moe.moe_dispatch(idx, E, x=x)
    out = ex.forward_dispatched(d.x_disp, d.offsets)
    y = ex.forward(x, logits, k, True)
    slot = torch.empty((T * k, H), dtype=torch.float64, device="cuda")
    slot[d.perm.long()] = out.double()
    terms = w.double()[..., None] * slot.view(T, k, H)
    tol = 2.0 ** -8 * (terms.sum(1).abs() * 1.01 + terms.abs().sum(1) * 1.01) + k * 2.0 ** -23 * terms.abs().sum(1)
    assert ((y.double() - terms.sum(1)).abs() <= tol + 1e-30).all()
    assert torch.equal(y, ex.forward(x, logits, k, True))


def test_the_fused_forward_of_many_rows(cuda_lib):
    """Both products keep weights' tiles for several of the rows', the second into weighted slots."""
    test_the_fused_forward_is_the_stages_together(cuda_lib, 12288, 4, 2, 2048, 1056, "bf16")


def test_sigmoid_routing(cuda_lib):
    moe = cuda_lib
    T, E, k = 65, 32, 4
    ex, _ = make(moe, E, 64, 64)
    x, logits = rows(T, 64, torch.bfloat16), torch.randn((T, E), device="cuda")
    bias = 0.1 * torch.randn(E, device="cuda")
    args = (k, 4, 2, True, True, 2.5)
    idx, w = moe.moe_route_sigmoid_grouped(logits, *args, bias=bias)
    d = moe.moe_dispatch(idx, E, x=x)
    out = ex.forward_dispatched(d.x_disp, d.offsets)
    slot = torch.empty((T * k, 64), dtype=torch.float64, device="cuda")
    slot[d.perm.long()] = out.double()
    terms = w.double()[..., None] * slot.view(T, k, 64)
    y = ex.forward_sigmoid_grouped(x, logits, *args, bias=bias)
    tol = 2.0 ** -8 * (terms.sum(1).abs() + terms.abs().sum(1)) * 1.01 + k * 2.0 ** -23 * terms.abs().sum(1)
    assert ((y.double() - terms.sum(1)).abs() <= tol + 1e-30).all()


def test_poisoned_logits_and_no_tokens(cuda_lib):
    moe = cuda_lib
    ex, _ = make(moe, 8, 64, 64)
    x, logits = rows(20, 64, torch.bfloat16), torch.randn((20, 8), device="cuda")
    clean = ex.forward(x, logits, 2, False)
    logits[3, 1], logits[7] = float("nan"), float("-inf")
    y = ex.forward(x, logits, 2, False)
    assert torch.isnan(y[3]).all() and torch.isnan(y[7]).all()
    keep = [i for i in range(20) if i not in (3, 7)]
    assert torch.equal(y[keep], clean[keep])
    assert ex.forward(x[:0], logits[:0], 2, False).shape == (0, 64)
    assert ex.forward_dispatched(x[:0], segments([0] * 8)).shape == (0, 64)


@pytest.mark.parametrize("T", [9, 400])
def test_a_graph_and_two_streams(cuda_lib, T):
    """Captured and replayed on other inputs; two calls at once on streams and workspaces of
    their own; two graphs in turn that share a workspace."""
    moe = cuda_lib
    ex, _ = make(moe, 8, 288, 96)
    xs = [rows(T, 288, torch.bfloat16, s) for s in range(3)]
    ls = [torch.randn((T, 8), device="cuda") for _ in range(3)]
    want = [ex.forward(x, l, 2, True) for x, l in zip(xs, ls)]
    ws = [ex.forward_workspace(T, 2, torch.float32) for _ in range(2)]
    x, l = xs[0].clone(), ls[0].clone()
    ys = [torch.empty_like(x) for _ in range(2)]
    graphs = []
    for y in ys:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ex.forward(x, l, 2, True, y=y, workspace=ws[0])
        graphs.append(g)
    for i in (1, 2, 0):
        x.copy_(xs[i]), l.copy_(ls[i])
        graphs[i % 2].replay()
        assert torch.equal(ys[i % 2], want[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for r in range(20):
        for j, s in enumerate(streams):
            got[j] = ex.forward(xs[j], ls[j], 2, True, workspace=ws[j], stream=s)
    for s in streams:
        s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals(cuda_lib):
    moe = cuda_lib
    ex, mx = make(moe, 4, 64, 96)
    x, off = rows(10, 64, torch.bfloat16), segments([4, 2, 0, 4])
    logits = torch.zeros((10, 4), device="cuda")
    for call, status in (
            (lambda: ex.forward_dispatched(x.half(), off), 3), (lambda: ex.forward_dispatched(x[:, :32].contiguous(), off), 2),
            (lambda: ex.forward_dispatched(x, off[:4].clone()), 2), (lambda: ex.forward_dispatched(x, off.long()), 3),
            (lambda: ex.forward_dispatched(x, off, workspace=ex.workspace(9)[:1024].clone()), 1),
            (lambda: ex.forward(x, logits, 5, True), 1), (lambda: ex.forward(x, logits, 0, True), 1),
            (lambda: ex.forward(x, logits.double(), 2, True), 3), (lambda: ex.forward(x[0], logits, 2, True), 2),
            (lambda: ex.forward(x, logits[:, :3].contiguous(), 2, True), 2),
            (lambda: ex.forward_sigmoid_grouped(x, logits, 2, 3, 1, False, True), 1),
            (lambda: moe.Mx4SwiGluExperts(*mx, dtype=torch.float32), 3),
            (lambda: moe.Mx4SwiGluExperts(mx[0], mx[1], mx[0]), 2),
            (lambda: moe.Mx4SwiGluExperts(*[moe.moe_mx_quantize(torch.zeros(s, device="cuda"), "mxfp8")
                                            for s in ((4, 96, 64), (4, 96, 64), (4, 64, 96))]), 3),
            (lambda: moe.Mx4SwiGluExperts(*[moe.moe_mx_quantize(torch.zeros(s, device="cuda"), "mxfp4")
                                            for s in ((4, 96, 40), (4, 96, 40), (4, 40, 96))]), 4)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == status, e.value
    for call in (lambda: ex.forward_dispatched(x.t(), off), lambda: ex.forward_dispatched(x.cpu(), off),
                 lambda: ex.forward(x, logits.t().contiguous().t(), 2, True)):
        with pytest.raises((ValueError, moe.MoeError)):
            call()
