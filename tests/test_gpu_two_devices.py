"""The experts' products on two devices in one process, neither of them the current
one at the time: what a device has to be asked for, it is asked for itself."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
@pytest.mark.parametrize("T", [20, 600])
def test_two_devices(cuda_lib, T):
    moe = cuda_lib
    E, H, I, k = 2, 264, 328, 2
    g = torch.Generator().manual_seed(T)
    w = [(torch.randn((E, a, b), generator=g) / b ** 0.5).to(torch.bfloat16) for a, b in ((I, H), (I, H), (H, I))]
    w4 = [(torch.randn((E, a, b), generator=g) / b ** 0.5).to(torch.bfloat16) for a, b in ((96, 64), (96, 64), (64, 96))]
    x, logits = torch.randn((T, H), generator=g).to(torch.bfloat16), torch.randn((T, E), generator=g)
    dout = torch.randn((T * k, H), generator=g).to(torch.bfloat16)
    results = []
    for i in (0, 1):
        dev = torch.device("cuda", i)
        with torch.cuda.device(dev):
            ex = moe.SwiGluExperts(*(t.to(dev) for t in w))
            idx, _ = moe.moe_route(logits.to(dev), k, True)
            d = moe.moe_dispatch(idx, E, x=x.to(dev))
            y = ex.forward(x.to(dev), logits.to(dev), k, True)
        with torch.cuda.device(1 - i):
            out, ck = ex.forward_checkpoint(d.x_disp, d.offsets)
            grads = ex.backward_checkpoint(moe.moe_mx_quantize(x.to(dev), "mxfp8"), d.perm, d.offsets, ck, dout.to(dev), k)
            ex4 = moe.Mx4SwiGluExperts(*(moe.moe_mx_quantize(t.to(dev), "mxfp4") for t in w4))
            y4 = ex4.forward(x[:, :64].contiguous().to(dev), logits.to(dev), k, True)
        results.append([t.cpu() for t in (y, out, *grads, y4)])
    assert all(torch.equal(a, b) for a, b in zip(*results))
