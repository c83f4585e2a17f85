"""The router's training losses where they can go wrong beside the sizes and
masks of the main tests; tolerances as derived there."""
import math

import pytest
import torch

import router_loss_reference as ref
from test_gpu_router_losses import DELTA, DT, F64, RT, _bits, _check, _check_grad, _close, _logits

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


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E,m", [(3000, 64, 6), (2000, 101, 40), (5000, 100, 7), (700, 999, 5)])
def test_gradient_in_place_is_the_one_beside_it(cuda_lib, T, E, m, dt):
    """A chain of gradients added in one buffer, launched back to back, against
    the same chain through buffers of its own: to the bit.  Rows of 400 bytes and
    odd ones share their lines with other warps' and blocks' rows."""
    g = torch.Generator().manual_seed(T + E)
    l = _logits(T, E, dt, g)
    far = torch.arange(0, T, 7)  # rows whose list holds all but exp(-200) of the student's mass
    teacher = l.clone()
    teacher[far, m:], l[far, m:] = -50.0, -200.0
    l, teacher = l.cuda(), teacher.cuda()
    idx, _ = cuda_lib.moe_route(l, min(m, 8), True)
    off = torch.tensor([0, T // 3, T // 3, T - 17], dtype=torch.int32, device="cuda")
    one = torch.linspace(0.5, 1.5, 3, device="cuda")
    bal = cuda_lib.moe_balance_loss(l, idx, seq_offsets=off, z_loss=True)
    tg = cuda_lib.moe_distill_targets(teacher, m)
    dis = cuda_lib.moe_distill_loss(l, tg, seq_offsets=off)
    base = (1e-3 * torch.randn((T, E), generator=g)).to(DT[dt]).cuda()
    there, kept = base.clone(), base.clone()
    for _ in range(4):
        out = cuda_lib.moe_balance_loss_backward(l, bal, min(m, 8), one, seq_offsets=off, dz_loss=one, base=kept)
        kept = cuda_lib.moe_distill_loss_backward(l, tg, dis, one, seq_offsets=off, base=out)
    for _ in range(4):
        cuda_lib.moe_balance_loss_backward(l, bal, min(m, 8), one, seq_offsets=off, dz_loss=one, base=there,
                                           dlogits=there)
        cuda_lib.moe_distill_loss_backward(l, tg, dis, one, seq_offsets=off, base=there, dlogits=there)
    assert torch.equal(_bits(there), _bits(kept))
    assert torch.equal(_bits(there[T - 17:]), _bits(base[T - 17:])) and torch.isfinite(there.float()).all()
    assert bool((dis.row_stats[4][far[far < T - 17].cuda()] < 0).all())  # they took the branch of their own


@pytest.mark.parametrize("tau", [1.0, 0.01])
@pytest.mark.parametrize("E", [16, 13])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_distill_rest_far_below_the_row(cuda_lib, dt, E, tau):
    """A student whose experts outside the list lie ever farther below the row,
    with a gradient scaled up: q_rest / p_rest alone is up to 1e30, its product
    with the scale leaves FP32, the gradient does not.  (Exponents up to 110 in
    base two: half a step of 2^-17 and log2(e)'s own, 2^-24, are 8e-6 relative in
    a score; the ratio carries as much again: RT = 2e-5 holds.)"""
    g = torch.Generator().manual_seed(E)
    levels = torch.tensor([-20.0, -30.0, -40.0, -44.0, -46.0, -50.0, -60.0, -68.0, -75.0, -150.0])
    T, m = len(levels), 4
    l = 0.5 * torch.randn((T, E), generator=g)
    l[:, m:] += levels[:, None]
    l = (tau * l).to(DT[dt])
    ti = torch.arange(m).expand(T, m).contiguous()
    tl = (0.5 * tau * torch.randn((T, m), generator=g)).to(DT[dt])
    tr = torch.zeros(T)
    dloss = torch.tensor([1e13])
    tg = cuda_lib.DistillTargets(ti.int().cuda(), tl.cuda(), tr.cuda())
    out = cuda_lib.moe_distill_loss(l.cuda(), tg, temperature=tau)
    _, tokens, row, diff = ref.distill(l.to(F64), ti, tl.to(F64), tr.to(F64), tau)
    _check(out.row_loss, row, RT * row + DELTA * diff + DELTA ** 2, "row_loss")
    d = cuda_lib.moe_distill_loss_backward(l.cuda(), tg, out, dloss.cuda(), temperature=tau)
    grad, size = ref.distill_grad(l.to(F64), ti, tl.to(F64), tr.to(F64), tau, tokens, dloss.to(F64))
    _check_grad(d, grad, size, dt, "dlogits")


@pytest.mark.parametrize("E,m", [(16, 4), (13, 4), (256, 40), (101, 40)])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_nan_rows_whose_rest_lies_far_below(cuda_lib, dt, E, m):
    """A row without a value has none at any expert, also where the experts outside
    its list lie so far below that their gradient is taken by itself."""
    g = torch.Generator().manual_seed(E)
    T = 9
    l = _logits(T, E, dt, g)
    l[:, m:] = -200.0
    ti = torch.arange(m).expand(T, m).clone()
    tl = torch.randn((T, m), generator=g).to(DT[dt])
    tr = torch.zeros(T)
    l[1, 1] = math.inf
    l[2, 0] = math.nan
    tl[3, 2] = math.nan
    tl[4, 0] = math.inf
    tr[5] = math.nan
    ti[6, 1] = E
    ti[7, 1] = ti[7, 2]
    tg = cuda_lib.DistillTargets(ti.int().cuda(), tl.cuda(), tr.cuda())
    off = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    out = cuda_lib.moe_distill_loss(l.cuda(), tg, seq_offsets=off)
    assert torch.isnan(out.row_loss).tolist() == [False] + 7 * [True] + [False]
    for base in (None, torch.ones((T, E), dtype=DT[dt], device="cuda")):
        d = cuda_lib.moe_distill_loss_backward(l.cuda(), tg, out, torch.ones(T, device="cuda"), seq_offsets=off,
                                               base=base)
        assert torch.isnan(d[1:8]).all()
        assert torch.isfinite(d[0].float()).all() and torch.isfinite(d[8].float()).all()


@pytest.mark.parametrize("E", [5, 8, 41, 64, 101, 256, 1000])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_sigmoid_scores_far_below_their_row(cuda_lib, dt, E):
    """Experts that every row puts at -45, -60 and -80: small scores, not none.
    (Exponents up to 117 in base two: half a step of 2^-17 and log2(e)'s own, 2^-24,
    are 8e-6 relative in a score, within RT.)"""
    g = torch.Generator().manual_seed(E)
    T, k = 75, 3
    level = torch.tensor([0.0, -45.0, -60.0, -80.0])[torch.arange(E) % 4]
    l = (0.3 * torch.randn((T, E), generator=g) + level).to(DT[dt])
    idx = torch.topk(l.float(), k, dim=1).indices
    out = cuda_lib.moe_balance_loss(l.cuda(), idx.int().cuda(), scoring="sigmoid")
    want = ref.balance(l.to(F64), idx, "sigmoid")
    _close(out.mean_scores, want["mean_scores"], what="mean_scores")
    _close(out.loss, want["loss"], what="loss")
    _close(out.row_stats, ref.balance_row_stats(l.to(F64), "sigmoid"), what="row_stats")
    assert bool((out.mean_scores > 0).all())
    dloss = torch.tensor([float(T * E)])
    grad, size = ref.balance_grad(l.to(F64), want["counts"], want["tokens"], k, "sigmoid", dloss.to(F64))
    d = cuda_lib.moe_balance_loss_backward(l.cuda(), out, k, dloss.cuda(), scoring="sigmoid")
    _check_grad(d, grad, size, dt, "dlogits")


def test_another_temperature_than_the_rest_s_or_the_forward_s_is_refused(cuda_lib):
    l = torch.randn((8, 6), device="cuda")
    one = torch.ones(1, device="cuda")
    tg = cuda_lib.moe_distill_targets(l, 3, temperature=2.0)
    assert tg.temperature == 2.0
    with pytest.raises(cuda_lib.MoeError):
        cuda_lib.moe_distill_loss(l, tg)
    dis = cuda_lib.moe_distill_loss(l, tg, temperature=2.0)
    with pytest.raises(cuda_lib.MoeError):
        cuda_lib.moe_distill_loss_backward(l, tg, dis, one)
    cuda_lib.moe_distill_loss_backward(l, tg, dis, one, temperature=2.0)
    # the results of a call follow the call
    cuda_lib.moe_distill_targets(l, 3, out=tg)
    cuda_lib.moe_distill_loss(l, tg, out=dis)
    cuda_lib.moe_distill_loss_backward(l, tg, dis, one)
    # a list alone serves every temperature
    tg.rest = None
    for tau in (0.5, 3.0):
        dis = cuda_lib.moe_distill_loss(l, tg, temperature=tau)
        cuda_lib.moe_distill_loss_backward(l, tg, dis, one, temperature=tau)
