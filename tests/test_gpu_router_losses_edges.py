"""The router's training losses where they can go wrong beside the sizes and
masks of the main tests; tolerances as derived there."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_results_whose_memory_was_exchanged_are_refused(cuda_lib):
    """The Python object stays, what lies behind it is on the host, or half as large."""
    l, idx = torch.randn((8, 6), device="cuda"), torch.zeros((8, 2), dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    for exchange in (lambda t: t.cpu(), lambda t: t.half(), lambda t: t.t().contiguous()):
        bal = cuda_lib.moe_balance_loss(l, idx)
        cuda_lib.moe_balance_loss(l, idx, out=bal)
        bal.row_stats.data = exchange(bal.row_stats.data)
        with pytest.raises((cuda_lib.MoeError, ValueError)):
            cuda_lib.moe_balance_loss(l, idx, out=bal)
        with pytest.raises((cuda_lib.MoeError, ValueError)):
            cuda_lib.moe_balance_loss_backward(l, bal, 2, one)
    tg = cuda_lib.moe_distill_targets(l, 3)
    dis = cuda_lib.moe_distill_loss(l, tg)
    tg.idx.data = tg.idx.data.cpu()
    with pytest.raises(ValueError):
        cuda_lib.moe_distill_targets(l, 3, out=tg)
    with pytest.raises(ValueError):
        cuda_lib.moe_distill_loss(l, tg, out=dis)
    with pytest.raises(ValueError):
        cuda_lib.moe_distill_loss_backward(l, tg, dis, one)
