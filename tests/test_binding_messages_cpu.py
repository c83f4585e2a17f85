"""What a call says of a tensor or a stream on the wrong device: which one, where it is
and where it should be, without a word of tensors that the call may not have."""
import types

import pytest
import torch

from top_routing_grouped_fp32_gb300 import microscaling as mx
from top_routing_grouped_fp32_gb300 import router_losses as rl

DEVICE = torch.device("cuda", 0)


@pytest.mark.parametrize("module", [mx, rl])
def test_a_tensor_elsewhere(module):
    with pytest.raises(ValueError) as e:
        module._p(torch.zeros(2), "perm", (torch.float32,), (2,), DEVICE)
    assert all(word in str(e.value) for word in ("perm", "cpu", "cuda:0")) and "logits" not in str(e.value)


@pytest.mark.parametrize("module", [mx, rl])
def test_a_stream_elsewhere(module):
    stream = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError) as e:
        module._on(DEVICE, stream)
    assert all(word in str(e.value) for word in ("stream", "cuda:1", "cuda:0")) and "logits" not in str(e.value)
