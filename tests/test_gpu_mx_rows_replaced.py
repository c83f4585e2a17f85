"""Rows whose tensors are replaced: the old ones go at once, the new ones are what a
call reads, and what does not fit is refused as at first."""
import weakref

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_replaced_tensors(cuda_lib, fmt):
    moe = cuda_lib
    x = torch.randn((5, 70), device="cuda")
    mx, other = moe.moe_mx_quantize(x, fmt), moe.moe_mx_quantize(-2 * x, fmt)
    first = moe.moe_mx_dequantize(mx, torch.float32)
    old = weakref.ref(mx.values), weakref.ref(mx.scales)
    mx.values, mx.scales = other.values, other.scales
    assert old[0]() is None and old[1]() is None
    assert torch.equal(moe.moe_mx_dequantize(mx, torch.float32), -2 * first)
    for name, bad in (("values", other.values.to(torch.int8)), ("values", other.values[:4].clone()), ("scales", other.scales.cpu()),
                      ("scales", torch.cat([other.scales, other.scales], 1)[:, ::2]), ("cols", 71), ("cols", 32)):
        keep = getattr(mx, name)
        setattr(mx, name, bad)
        with pytest.raises((moe.MoeError, ValueError)):
            moe.moe_mx_dequantize(mx, torch.float32)
        setattr(mx, name, keep)
    assert torch.equal(moe.moe_mx_dequantize(mx, torch.float32), -2 * first)
