"""A workspace serves every batch up to the one that it was made for."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def experts(moe, E, H, I):
    g = torch.Generator(device="cuda").manual_seed(E)
    return moe.SwiGluExperts(*((torch.randn((E, a, b), generator=g, device="cuda") / b ** 0.5).to(torch.bfloat16)
                               for a, b in ((I, H), (I, H), (H, I))))


def batch(moe, ex, T):
    E, H, I = ex.E, ex.H, ex.I
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    idx, _ = moe.moe_route(torch.randn((T, E), generator=g, device="cuda"), 1, True)
    d = moe.moe_dispatch(idx, E, x=x)
    _, ck = ex.forward_checkpoint(d.x_disp, d.offsets)
    dout = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    return moe.moe_mx_quantize(x, "mxfp8"), d.perm, d.offsets, ck, dout, 1


# the largest batch, then smaller ones: below a step of the rows' tiles, below the border of CTA pairs, a few rows
@pytest.mark.parametrize("E,H,I,sizes", [(2, 2048, 1408, (768, 767, 257, 255, 100, 3, 1)),
                                         (4, 1024, 1024, (1536, 1535, 512, 511, 4)), (1, 64, 520, (1700, 513, 128, 127))])
def test_a_smaller_batch_in_the_workspace_of_a_larger(cuda_lib, E, H, I, sizes):
    moe = cuda_lib
    ex = experts(moe, E, H, I)
    ws = ex.backward_checkpoint_workspace(sizes[0])
    for T in sizes:
        args = batch(moe, ex, T)
        want = ex.backward_checkpoint(*args)
        ws.fill_(0xFF)
        got = ex.backward_checkpoint(*args, workspace=ws)
        assert moe.moe_get_device_status(ws) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("E,H,I", [(2, 2048, 1408), (4, 1024, 1024), (1, 64, 520), (7, 512, 64)])
def test_sizes_do_not_fall(cuda_lib, E, H, I):
    moe = cuda_lib
    ex = experts(moe, E, H, I)
    ex4 = moe.Mx4SwiGluExperts(*(moe.moe_mx_quantize(torch.zeros(s, device="cuda"), "mxfp4")
                                 for s in ((E, 64, 96), (E, 64, 96), (E, 96, 64))))
    lib = ex._lib
    for size in (lambda n: lib.moe_experts_backward_checkpoint_workspace_size(ex.handle, n),
                 lambda n: lib.moe_experts_workspace_size(ex.handle, n),
                 lambda n: lib.moe_mx4_experts_workspace_size(ex4.handle, n),
                 lambda n: lib.moe_mx4_forward_workspace_size(ex4.handle, n, 1, 0)):
        sizes = [size(n) for n in range(1, 3000)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))
