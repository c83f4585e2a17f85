"""The memory of 4-bit experts that go while a call on another stream waits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("created_on_side", [False, True])
@pytest.mark.parametrize("call", ["dispatched", "fused"])
def test_experts_that_go_before_their_call_ran(cuda_lib, created_on_side, call):
    moe = cuda_lib
    E, H, I, T = 4, 256, 288, 50
    g = torch.Generator(device="cuda").manual_seed(1)
    w = [torch.randn((E, a, b), generator=g, device="cuda") / b ** 0.5 for a, b in ((I, H), (I, H), (H, I))]
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn((T, E), generator=g, device="cuda")
    off = torch.tensor([0, 10, 25, 25, 50], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()

    def make():
        mx = [moe.moe_mx_quantize(t, "mxfp4") for t in w]
        side.wait_stream(torch.cuda.current_stream())
        ex = moe.Mx4SwiGluExperts(*mx, stream=side if created_on_side else None)
        side.wait_stream(torch.cuda.current_stream())
        return ex

    def run(ex, **kw):
        return ex.forward_dispatched(x, off, **kw) if call == "dispatched" else ex.forward(x, logits, 2, True, **kw)
    ex = make()
    torch.cuda.synchronize()
    want = run(ex)
    sizes = [t.numel() for t in ex._keep]
    ex = make()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # about 50 ms in front of the call
    out = run(ex, stream=side)
    del ex
    taken = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(8)]
    with torch.cuda.stream(side):
        taken += [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and len(taken) == 36
