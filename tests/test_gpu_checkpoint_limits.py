"""More rows than the padded row space of the checkpointed backward can count."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_too_many_rows(cuda_lib):
    moe = cuda_lib
    E, H, I = 2, 64, 64
    ex = moe.SwiGluExperts(*(torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((E, I, H), (E, I, H), (E, H, I))))
    lib, P = ex._lib, ctypes.c_void_p
    most = (1 << 31) - 1 - 63 * E - 1
    for N in (most + 1, (1 << 31) - 1):  # refused before any pointer is looked at
        assert lib.moe_experts_backward_checkpoint_workspace_size(ex.handle, N) == 0
        st = lib.moe_experts_backward_checkpoint(ex.handle, P(), P(), N, 1, *[P()] * 11, P(), 0, P())
        words = lib.moe_last_error().decode()
        assert st == 4 and str(N) in words and "F16" not in words, words
    assert lib.moe_experts_backward_checkpoint_workspace_size(ex.handle, most) > 0
