"""SwiGLU and its gradient where a product of finite values leaves FP32's range
on the way to a value that does not: silu(g) of a negative g is small or 0,
whatever u is.  All values are powers of two, so that sums are exact and what is
expected is the formula's value with the roundings that it goes through."""
import pytest
import torch

import mx_reference as ref

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
H, I = 32, 64


def weights(gate, up, down):
    """Experts of one kind of feature each for even and odd features (gate, up [2]); x = 1."""
    w = [torch.empty((1, I, H), device="cuda") for _ in range(2)] + [torch.full((1, H, I), down, device="cuda")]
    for t, pair in zip(w, (gate, up)):
        t[:, 0::2], t[:, 1::2] = pair[0], pair[1]
    return w


def h_of(g, u):
    g, u = torch.tensor(g, dtype=F64), torch.tensor(u, dtype=F64)
    return ref.silu(g) * u


# g and u of the even and of the odd features; |g u| of the even ones is 2^134 and 2^130, silu(g) u 0 and -1.5e32
FAR = [((-2.0 ** 67, 4.0), (2.0 ** 67, 4.0)), ((-16.0, -16.0), (2.0 ** 126, 2.0 ** 126))]


@pytest.mark.parametrize("n", [3, 300])
@pytest.mark.parametrize("g,u", FAR)
@pytest.mark.parametrize("dt", [torch.float16, BF16])
def test_experts4(cuda_lib, n, g, u, dt):
    moe = cuda_lib
    h = h_of(g, u).repeat(I // 2)[None]
    down = 2.0 ** -4 if h.abs().max() < 1e3 else 2.0 ** -120
    mx = [moe.moe_mx_quantize(t, "mxfp4") for t in weights([v / H for v in g], [v / H for v in u], down)]
    ex = moe.Mx4SwiGluExperts(*mx, dtype=dt)
    x = torch.ones((n, H), dtype=dt, device="cuda")
    out = ex.forward_dispatched(x, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    want = (ref.rounded(h, "mxfp4").sum() * down).item()
    assert abs(want) > 1e-7 and (out.double() == want).all(), (out.min(), out.max(), want)
    y = ex.forward(x, torch.zeros((n, 1), device="cuda"), 1, True)
    assert (y.double() == want).all()


@pytest.mark.parametrize("n", [3, 300])
@pytest.mark.parametrize("g,u", FAR)
def test_forward_of_16_bit_experts(cuda_lib, n, g, u):
    moe = cuda_lib
    h = h_of(g, u).repeat(I // 2)
    down = 2.0 ** -4 if h.abs().max() < 1e3 else 2.0 ** -120
    ex = moe.SwiGluExperts(*(t.to(BF16) for t in weights([v / H for v in g], [v / H for v in u], down)))
    x, off = torch.ones((n, H), dtype=BF16, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    want = h.sum().item() * down
    # all terms of a sum have one sign: half a step for h, half a step for the result, FP32 in between
    tol = abs(want) * (2 * 2.0 ** -8 + 2.0 ** -16)
    for out in (ex.forward_dispatched(x, off), ex.forward_checkpoint(x, off)[0],
                ex.forward(x, torch.zeros((n, 1), device="cuda"), 1, True)):
        assert ((out.double() - want).abs() <= tol).all(), (out.min(), out.max(), want)


@pytest.mark.parametrize("n", [3, 300])
@pytest.mark.parametrize("far", [-128.0, -16.0])
def test_backward_from_a_checkpoint(cuda_lib, n, far):
    """da u of the first block of features is 2^141; da u silu'(g) is 0 or -5e36."""
    moe = cuda_lib
    one = torch.ones((n, 32), device="cuda")
    g, u = torch.cat([far * one, one], 1), torch.cat([2.0 ** 66 * one, one], 1)
    w_down = torch.cat([torch.full((1, H, 32), v, device="cuda") for v in (2.0 ** 30, 2.0 ** -40)], 2)
    w = [torch.full((1, I, H), 2.0 ** -3, device="cuda")] * 2 + [w_down]
    ex = moe.SwiGluExperts(*(t.to(BF16) for t in w))
    ck = moe.ExpertCheckpoint(moe.moe_mx_quantize(g, "mxfp8"), moe.moe_mx_quantize(u, "mxfp8"))
    x = torch.full((n, H), 2.0 ** -10, dtype=BF16, device="cuda")
    dout = torch.full((n, H), 2.0 ** 40, dtype=BF16, device="cuda")
    perm, off = torch.arange(n, dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    got = ex.backward_checkpoint(moe.moe_mx_quantize(x, "mxfp8"), perm, off, ck, dout, 1)
    g, u, x, dout = (t.to(F64) for t in (g, u, x, dout))
    gate, up, down = (t[0].to(F64) for t in w)
    da, s = dout @ down, torch.sigmoid(g)
    dg, du, a = da * u * s * (1 + g * (1 - s)), da * g * s, g * s * u
    want = (dg @ gate + du @ up, dg.t() @ x, du.t() @ x, dout.t() @ a)
    # where a sum's terms differ in sign one of them outweighs the other by 2^60.  Half a step for each of the two
    # roundings; a sigmoid below 2^-126 may count as 0, which moves none of these by more than 1e-6
    for name, o, r in zip(("dinput", "dgate", "dup", "ddown"), got, want):
        o = o.to(F64).view(r.shape)
        assert ((o - r).abs() <= r.abs() * (2 * 2.0 ** -8 + 2.0 ** -15) + 1e-6).all(), (name, (o - r).abs().max())
