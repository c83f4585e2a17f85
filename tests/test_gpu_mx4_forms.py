"""The forms of the 4-bit kernels that F16 rows and large batches take, and rows whose
results do not depend on the batch around them."""
import pytest
import torch

from test_gpu_mx4_experts import check, make, rows, segments

pytestmark = pytest.mark.gpu
F16 = torch.float16


def layer(moe, ex, x, logits, k, dt, route, forward):
    """The staged calls with the combine in 64 bits against the fused one: its slots are FP32, the staged
    expert outputs carry half a step of their own, and the sum is rounded once."""
    T, E, H = x.shape[0], logits.shape[1], x.shape[1]
    idx, w = route(logits)
    d = moe.moe_dispatch(idx, E, x=x)
    out = ex.forward_dispatched(d.x_disp, d.offsets)
    y = forward(x, logits)
    slot = torch.empty((T * k, H), dtype=torch.float64, device="cuda")
    slot[d.perm.long()] = out.double()
    terms = w.double()[..., None] * slot.view(T, k, H)
    eps = torch.finfo(dt).eps / 2
    least = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps  # a step of the subnormals
    tol = eps * 1.01 * (terms.sum(1).abs() + terms.abs().sum(1)) + k * 2.0 ** -23 * terms.abs().sum(1) + (k + 1) * least
    assert ((y.double() - terms.sum(1)).abs() <= tol).all()
    assert torch.equal(y, forward(x, logits))


@pytest.mark.parametrize("T,E,k,H,I", [(1, 5, 2, 64, 64), (32, 256, 8, 256, 96), (128, 2, 2, 64, 64), (129, 2, 2, 64, 64),
                                       (300, 3, 2, 288, 160), (12288, 4, 2, 2048, 1056)])
@pytest.mark.parametrize("ldt", [torch.float32, F16])
def test_fused_forward_f16(cuda_lib, T, E, k, H, I, ldt):
    moe = cuda_lib
    ex, _ = make(moe, E, H, I, F16, seed=T)
    x, logits = rows(T, H, F16), torch.randn((T, E), device="cuda").to(ldt)
    layer(moe, ex, x, logits, k, F16, lambda l: moe.moe_route(l, k, True), lambda x, l: ex.forward(x, l, k, True))


@pytest.mark.parametrize("T", [65, 700])
@pytest.mark.parametrize("dt", [F16, torch.bfloat16])
def test_fused_sigmoid_forward(cuda_lib, T, dt):
    moe = cuda_lib
    E, k = 32, 4
    ex, _ = make(moe, E, 64, 64, dt)
    x, logits = rows(T, 64, dt), torch.randn((T, E), device="cuda")
    bias = 0.1 * torch.randn(E, device="cuda")
    args = (k, 4, 2, True, True, 2.5)
    layer(moe, ex, x, logits, k, dt, lambda l: moe.moe_route_sigmoid_grouped(l, *args, bias=bias),
          lambda x, l: ex.forward_sigmoid_grouped(x, l, *args, bias=bias))


@pytest.mark.parametrize("H,I,counts", [(2048, 2688, [11000, 11001]), (1056, 2720, [5121, 255, 16000, 600])])
def test_many_rows_f16(cuda_lib, H, I, counts):
    """Weights' tiles kept for several of the rows'."""
    moe = cuda_lib
    ex, mx = make(moe, len(counts), H, I, F16)
    n = sum(counts)
    x, off = rows(n, H, F16), segments(counts)
    ws = ex.workspace(n)
    ws.fill_(0xFF)
    out = ex.forward_dispatched(x, off, workspace=ws)
    check(moe, mx, x, off, out, F16)
    assert moe.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("T", [127, 128, 129, 1000])
def test_poisoned_logits_on_either_side_of_256_slots(cuda_lib, T):
    moe = cuda_lib
    ex, _ = make(moe, 8, 64, 64)
    x, logits = rows(T, 64, torch.bfloat16), torch.randn((T, 8), device="cuda")
    clean = ex.forward(x, logits, 2, False)
    bad = [3, 7, T - 1]
    logits[3, 1], logits[7], logits[T - 1] = float("nan"), float("-inf"), float("inf")
    y = ex.forward(x, logits, 2, False)
    assert torch.isnan(y[bad]).all()
    keep = [i for i in range(T) if i not in bad]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("H,I", [(64, 96), (2048, 1056), (1056, 2688)])
def test_rows_do_not_depend_on_the_batch_around_them(cuda_lib, H, I):
    """An expert's rows alone (single CTAs), in a batch of CTA pairs, and in one that keeps weights' tiles
    where rows are long enough: the same bits."""
    moe = cuda_lib
    ex, _ = make(moe, 2, H, I)
    x = rows(40 + 22000, H, torch.bfloat16)
    alone = ex.forward_dispatched(x[:40].contiguous(), segments([40, 0]))
    for n in (1, 300, 22000):
        out = ex.forward_dispatched(x[:40 + n].contiguous(), segments([40, n]))
        assert torch.equal(out[:40], alone)
    assert alone.any()
