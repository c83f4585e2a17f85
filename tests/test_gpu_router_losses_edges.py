"""The router's training losses where they can go wrong beside the sizes and
masks of the main tests; tolerances as derived there."""
import math

import pytest
import torch

import router_loss_reference as ref
from test_gpu_router_losses import (DELTA, DT, F64, RT, _bits, _check, _check_grad, _close, _dev, _lists, _logits,
                                    _rounded, _step_inputs)

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


def _shifted(t, by):
    """A copy that starts `by` elements behind a 16-byte boundary."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)[by:].view(t.shape)
    return buf.copy_(t)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("E,k", [(64, 6), (101, 9), (256, 40)])
@pytest.mark.parametrize("at,to", [(0, 1), (1, 0), (1, 1), (3, 2), (2, 3)])
def test_gradients_from_and_to_any_element(cuda_lib, at, to, E, k, dt):
    """Logits and gradient that start on different elements, each loss by itself."""
    T = 70
    g = torch.Generator().manual_seed(12 + E)
    l = _logits(T, E, dt, g)
    _, ti, tl, tr = _lists(l, k, 1.0, dt, g)
    idx = torch.topk(l.float(), k, dim=1).indices
    dl = _shifted(l.cuda(), at)
    tg = cuda_lib.DistillTargets(_shifted(ti.int().cuda(), 1), _shifted(tl.cuda(), 1), tr.cuda())
    bal = cuda_lib.moe_balance_loss(dl, _shifted(idx.int().cuda(), 1))
    dis = cuda_lib.moe_distill_loss(dl, tg)
    dloss = torch.tensor([float(T)])
    want = ref.balance(l.to(F64), idx, "softmax")
    _, tokens, _, _ = ref.distill(l.to(F64), ti, tl.to(F64), tr.to(F64), 1.0)
    base = torch.randn((T, E), generator=g).to(DT[dt])
    for grad, size, call in (
            (*ref.balance_grad(l.to(F64), want["counts"], want["tokens"], k, "softmax", dloss.to(F64)),
             lambda **kw: cuda_lib.moe_balance_loss_backward(dl, bal, k, dloss.cuda(), **kw)),
            (*ref.distill_grad(l.to(F64), ti, tl.to(F64), tr.to(F64), 1.0, tokens, dloss.to(F64)),
             lambda **kw: cuda_lib.moe_distill_loss_backward(dl, tg, dis, dloss.cuda(), **kw))):
        buf = torch.full((T * E + to + 9,), 7.0, dtype=DT[dt], device="cuda")
        out = buf[to:to + T * E].view(T, E)
        _check_grad(call(dlogits=out), grad, size, dt, "dlogits")
        assert bool((buf[:to] == 7).all()) and bool((buf[to + T * E:] == 7).all())
        # (the sum with base is rounded once in FP32 and once to its type)
        total, size = grad + base.to(F64), size + base.to(F64).abs() * 2.0 ** -24 / RT
        _check_grad(call(dlogits=out, base=_shifted(base.cuda(), at)), total, size, dt, "base + dlogits")
        buf = torch.full((T * E + to + 9,), 7.0, dtype=DT[dt], device="cuda")
        out = buf[to:to + T * E].view(T, E).copy_(base)
        _check_grad(call(dlogits=out, base=out), total, size, dt, "base + dlogits in place")
        assert bool((buf[:to] == 7).all()) and bool((buf[to + T * E:] == 7).all())


@pytest.mark.parametrize("T,E,k", [(64, 4, 2), (3000, 64, 6), (1500, 100, 8), (900, 257, 9)])
def test_what_each_loss_adds_to_a_step(cuda_lib, T, E, k):
    """Each gradient of a training step by what it adds to the one before it, with
    tolerances of its own size: the terms' RT and one rounding of the sum."""
    l, teacher, _ = _step_inputs(T, E, k, "f32", 4)
    idx, _ = cuda_lib.moe_route(l, k, True)
    half = torch.full((1,), 0.5, device="cuda")
    bal = cuda_lib.moe_balance_loss(l, idx, z_loss=True)
    tg = cuda_lib.moe_distill_targets(teacher, k)
    dis = cuda_lib.moe_distill_loss(l, tg)
    dw = torch.linspace(-1, 1, T * k, device="cuda").view(T, k)
    d = [cuda_lib.moe_router_backward(l, idx, dw, "softmax", True)]
    d.append(cuda_lib.moe_balance_loss_backward(l, bal, k, half, dz_loss=0.1 * half, base=d[0]))
    d.append(cuda_lib.moe_distill_loss_backward(l, tg, dis, half, base=d[1]))
    d = [x.cpu().to(F64) for x in d]
    x, ix = l.cpu().to(F64), idx.cpu().long()
    want = ref.balance(x, ix, "softmax")
    h = torch.tensor([0.5], dtype=F64)
    ti, tl, tr = ref.targets(teacher.cpu().to(F64), k, 1.0)
    # (a rest in FP32, as the loss takes it)
    parts = (ref.balance_grad(x, want["counts"], want["tokens"], k, "softmax", h, 0.1 * h),
             ref.distill_grad(x, ti, tl, tr.float().to(F64), 1.0, torch.tensor([T]), h))
    for (grad, size), before, after in zip(parts, d, d[1:]):
        tol = RT * size + after.abs() * 2.0 ** -24 + 2.0 ** -126
        _check(after - before, grad, tol, "what was added")
        assert float((grad.abs() > 10 * tol).double().mean()) > 0.9  # a gradient that is left out shows
    p = torch.softmax(x, 1)
    w = p.gather(1, ix)
    total = w.sum(1, keepdim=True)
    w, gw = w / total, dw.cpu().to(F64)
    mean = (w * gw).sum(1, keepdim=True)
    task = torch.zeros_like(x).scatter_(1, ix, w * (gw - mean))
    # the selected experts' terms, and p times their sum for every expert
    terms = gw.abs() + (w * gw.abs()).sum(1, keepdim=True)
    size = torch.zeros_like(x).scatter_(1, ix, w * terms) + p * (w * terms).sum(1, keepdim=True)
    _check(d[0], task, RT * size + 2.0 ** -126, "the routing weights' gradient")


ODD = [(40, "f16"), (41, "f32"), (41, "f16"), (41, "bf16"), (257, "f32"), (257, "f16"), (257, "bf16"), (7, "bf16")]


@pytest.mark.parametrize("E,dt", ODD)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_balance_rows_at_the_edge_of_other_layouts(cuda_lib, scoring, E, dt):
    """Masked experts, far rows, poisoned rows and poison in rows that do not count,
    beside each other in rows that are no whole vectors."""
    T, k = 40, 4
    g = torch.Generator().manual_seed(5 + E)
    l = _logits(T, E, dt, g)
    low = torch.finfo(DT[dt]).min
    l[0, 3:] = -math.inf
    l[1, ::2] = low
    l[2, :] = low
    l[3, :] = -1000.0
    l[4] = l[4] - 300.0
    l[5] = l[5] + 300.0
    l[6, E // 2] = 500.0
    off = [0, 8, 9, 10, 11, 36]
    l[8, 3] = math.nan
    l[9, 3] = math.inf
    l[10] = -math.inf
    mask = torch.ones(T, dtype=torch.bool)
    for i, t in enumerate(range(12, 34, 3)):  # poison on both sides of rows that count
        l[t], mask[t] = (math.nan, math.inf, -math.inf, low)[i % 4], False
    l[36:] = math.nan  # behind the last sequence
    idx = torch.randint(0, E, (T, k), generator=g)
    idx[12], idx[37] = -1, 2 ** 31 - 1  # not read: their rows do not count
    z = scoring == "softmax"
    dl, doff = l.cuda(), _dev(off, torch.int32)
    out = cuda_lib.moe_balance_loss(dl, idx.int().cuda(), scoring=scoring, token_mask=mask.cuda(), seq_offsets=doff,
                                    z_loss=z)
    want = ref.balance(l.to(F64), idx, scoring, mask, off)
    assert cuda_lib.moe_get_device_status(out.workspace) == 0
    assert torch.equal(out.counts.cpu().long(), want["counts"])
    assert torch.equal(out.tokens.cpu().long(), want["tokens"])
    _close(out.loss, want["loss"], what="loss")
    _close(out.mean_scores, want["mean_scores"], at=1e-30, what="mean_scores")
    if z:  # the last sequence's rows are within the bound that `at` stands for; squares of `low` leave FP32
        _close(out.z_loss[4:], want["z_loss"][4:], at=32 * 2.0 ** -20, what="z_loss")
        assert torch.isnan(out.z_loss[1:4]).all()
    dloss = torch.ones(5)
    grad, size = ref.balance_grad(l.to(F64), want["counts"], want["tokens"], k, scoring, dloss.to(F64), None, mask,
                                  off)
    gone = torch.tensor([t for t in range(T) if not mask[t] or t >= 36])
    base = torch.randn((T, E), generator=g).to(DT[dt])
    for b in (None, base):
        d = cuda_lib.moe_balance_loss_backward(dl, out, k, dloss.cuda(), scoring=scoring, seq_offsets=doff,
                                               base=_dev(b)).cpu()
        w, s = (grad, size) if b is None else (grad + b.to(F64), size + b.to(F64).abs() * 2.0 ** -24 / RT)
        _check(d, w, _rounded(torch.nan_to_num(s), torch.nan_to_num(w), dt), "dlogits")
        assert torch.equal(d[gone], torch.zeros_like(d[gone]) if b is None else b[gone])


@pytest.mark.parametrize("m", [5, 40])
@pytest.mark.parametrize("E,dt", [(48, "f32"), (48, "f16")] + ODD[1:-1])
def test_distill_rows_at_the_edge_of_other_layouts(cuda_lib, E, dt, m):
    """The same for the distillation, with lists longer than a row's lanes keep, and
    rows whose rest lies far below them added to a gradient that is there."""
    T = 32
    g = torch.Generator().manual_seed(9 + E + m)
    l = _logits(T, E, dt, g)
    _, ti, tl, tr = _lists(l, m, 1.0, dt, g)
    low = torch.finfo(DT[dt]).min
    outside = [torch.ones(E, dtype=torch.bool).index_fill(0, ti[t], False).nonzero()[:, 0] for t in range(T)]
    tl[0] = -math.inf                      # only a rest
    tr[1] = -math.inf                      # only a list
    tl[2], tr[2] = -math.inf, -math.inf    # no target
    l[3, int(ti[3, 0])] = -math.inf        # the teacher gives mass to it: +inf
    for t in (4, 11):                      # the student's rest underflows
        l[t, outside[t]] = (-200.0 - torch.arange(len(outside[t])) % 4).to(DT[dt])
    tl[11, m - 1] = -math.inf              # and an absent entry belongs to the rest
    l[11, int(ti[11, m - 1])] = -190.0
    l[5, outside[5][1:]] = -math.inf       # a part of the row only
    l[6] = low
    l[7, E // 2:] = low
    tl[8] = low
    l[9] = l[9] + 300
    off = [0, 13, 14, 15, 16, 17, 18, 19, 30]
    l[13, 3] = math.nan
    l[14, 3] = math.inf
    l[15] = -math.inf
    tl[16, 2] = math.nan
    tr[17] = math.inf
    ti[18, 1] = E
    mask = torch.ones(T, dtype=torch.bool)
    for i, t in enumerate((10, 20, 23, 26, 29)):
        l[t], tl[t], ti[t], mask[t] = (math.nan, math.inf, -math.inf)[i % 3], math.nan, -1, False
    l[30:], tl[30:], tr[30:] = math.nan, math.inf, math.nan
    tg = cuda_lib.DistillTargets(ti.int().cuda(), tl.cuda(), tr.cuda())
    doff = _dev(off, torch.int32)
    out = cuda_lib.moe_distill_loss(l.cuda(), tg, token_mask=mask.cuda(), seq_offsets=doff)
    row = out.row_loss.cpu()
    tokens = [11, 1, 1, 1, 1, 1, 1, 7]
    assert out.tokens.tolist() == tokens
    assert torch.isnan(row[13:19]).all() and torch.isnan(out.loss[1:7]).all()
    gone = [t for t in range(T) if t == 2 or not mask[t] or t >= 30]
    assert not row[gone].any() and not out.row_stats[:, gone].any()
    assert row[3] == math.inf and out.loss[0] == math.inf
    assert cuda_lib.moe_get_device_status(out.workspace) == 6  # row 18
    dloss = torch.ones(8)
    base = torch.randn((T, E), generator=g).to(DT[dt])
    for fine, s in (([0, 1, 4, 5, 6, 7, 8, 9, 11, 12], 0), ([19, 21, 22, 24, 25, 27, 28], 7)):
        x, i, a, r = l.to(F64)[fine], ti[fine], tl.to(F64)[fine], tr.to(F64)[fine]
        _, _, want, diff = ref.distill(x, i, a, r, 1.0)
        _check(row[fine], want, RT * want + DELTA * diff + DELTA ** 2, "row_loss")
        grad, size = ref.distill_grad(x, i, a, r, 1.0, torch.tensor([tokens[s]]), dloss.to(F64))
        for b in (None, base):
            d = cuda_lib.moe_distill_loss_backward(l.cuda(), tg, out, dloss.cuda(), seq_offsets=doff,
                                                   base=_dev(b)).cpu()
            assert torch.isnan(d[13:19]).all() and torch.isfinite(d[3].float()).all()
            assert torch.equal(d[gone], torch.zeros_like(d[gone]) if b is None else b[gone])
            w, sz = (grad, size) if b is None else (grad + b.to(F64)[fine], size + b.to(F64)[fine].abs() * 2.0 ** -24 / RT)
            _check(d[fine], w, _rounded(sz, w, dt), "dlogits")


@pytest.mark.parametrize("tau", [1e-3, 1e3])
@pytest.mark.parametrize("E,m", [(64, 6), (101, 40)])
def test_temperatures_at_their_limits(cuda_lib, E, m, tau):
    """Logits of the temperature's size: what is exponentiated is as at 1, and so
    are its errors (the rest carries tau times its logarithm's)."""
    T = 200
    g = torch.Generator().manual_seed(E)
    l = tau * _logits(T, E, "f32", g)
    teacher = l + tau * 0.7 * torch.randn((T, E), generator=g)
    tg = cuda_lib.moe_distill_targets(teacher.cuda(), m, temperature=tau)
    ti, tl, tr = ref.targets(teacher.to(F64), m, tau)
    assert torch.equal(tg.idx.cpu().long(), ti)
    _close(tg.rest, tr, at=tau * DELTA, what="rest")
    tr = tg.rest.cpu().to(F64)
    out = cuda_lib.moe_distill_loss(l.cuda(), tg, temperature=tau)
    loss, tokens, row, diff = ref.distill(l.to(F64), ti, tl, tr, tau)
    _check(out.row_loss, row, RT * row + DELTA * diff + DELTA ** 2, "row_loss")
    dloss = torch.tensor([float(T)])
    grad, size = ref.distill_grad(l.to(F64), ti, tl, tr, tau, tokens, dloss.to(F64))
    d = cuda_lib.moe_distill_loss_backward(l.cuda(), tg, out, dloss.cuda(), temperature=tau)
    _check_grad(d, grad, size, "f32", "dlogits")


@pytest.mark.parametrize("T,E,k", [(50, 8, 2), (3, 100, 7)])
def test_more_sequences_than_rows(cuda_lib, T, E, k):
    """70000 sequences, nearly all of them empty, before, between and behind the rows."""
    g = torch.Generator().manual_seed(T)
    l = _logits(T, E, "f32", g)
    idx = torch.topk(l, k, dim=1).indices
    _, ti, tl, tr = _lists(l, k, 1.0, "f32", g)
    S = 70000
    off = torch.cat([torch.zeros(S // 3, dtype=torch.int64), torch.randint(0, T + 1, (S // 3,), generator=g)])
    off = torch.cat([off, torch.full((S + 1 - len(off),), T)]).sort().values
    doff, dl = off.int().cuda(), l.cuda()
    rows = off[1:] - off[:-1]
    some = rows.nonzero()[:, 0]
    where = torch.cat([off[some], off[-1:]]).tolist()  # the sequences that hold rows
    bal = cuda_lib.moe_balance_loss(dl, idx.int().cuda(), seq_offsets=doff, z_loss=True)
    tg = cuda_lib.DistillTargets(ti.int().cuda(), tl.cuda(), tr.cuda())
    dis = cuda_lib.moe_distill_loss(dl, tg, seq_offsets=doff)
    assert torch.equal(bal.tokens.cpu().long(), rows) and torch.equal(dis.tokens.cpu().long(), rows)
    empty = (rows == 0).cuda()
    for t in (bal.loss, bal.z_loss, bal.mean_scores, bal.counts, dis.loss):
        assert not t[empty].any()
    want = ref.balance(l.to(F64), idx, "softmax", None, where)
    _close(bal.loss[some.cuda()], want["loss"], what="loss")
    loss, tokens, _, diff = ref.distill(l.to(F64), ti, tl.to(F64), tr.to(F64), 1.0, None, where)
    _check(dis.loss[some.cuda()], loss, RT * loss + DELTA * diff.max() + DELTA ** 2, "distillation loss")
    dloss = torch.linspace(0.5, 1.5, S)
    grad, size = ref.balance_grad(l.to(F64), want["counts"], want["tokens"], k, "softmax", dloss[some].to(F64), None,
                                  None, where)
    d = cuda_lib.moe_balance_loss_backward(dl, bal, k, dloss.cuda(), seq_offsets=doff)
    _check_grad(d, grad, size, "f32", "dlogits")
    grad, size = ref.distill_grad(l.to(F64), ti, tl.to(F64), tr.to(F64), 1.0, tokens, dloss[some].to(F64), None, where)
    d = cuda_lib.moe_distill_loss_backward(dl, tg, dis, dloss.cuda(), seq_offsets=doff)
    _check_grad(d, grad, size, "f32", "dlogits")


@pytest.mark.parametrize("m", [4, 12, 40])
@pytest.mark.parametrize("E", [48, 41, 256, 257, 1000])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_targets_at_the_edge_of_other_layouts(cuda_lib, dt, E, m):
    """Ties, masked rows and rows that are none, between others; results that start
    on any element."""
    T = 37
    g = torch.Generator().manual_seed(E + m)
    l = (2 * _logits(T, E, "f32", g)).round().div(2).to(DT[dt])  # many ties
    low = torch.finfo(DT[dt]).min
    l[0] = -math.inf
    l[1, 2:] = -math.inf
    l[2] = low
    l[3, 1:] = low
    l[4] = 3.0
    l[5, ::2] = -math.inf
    l[6] = l[6] - 300.0
    l[7, : E // 2], l[7, E // 2:] = 0.0, -0.0
    broken = [9, 12, 15, 20]
    l[9, E // 2] = math.nan
    l[12, E - 1] = math.inf
    l[15, 0] = math.copysign(math.nan, -1.0)
    l[20] = math.inf
    fine = torch.tensor([t for t in range(T) if t not in broken])
    ti, tl, tr = ref.targets(l.to(F64)[fine], m, 1.0)
    for by in (0, 1):
        out = cuda_lib.DistillTargets(_shifted(torch.empty((T, m), dtype=torch.int32, device="cuda"), by),
                                      _shifted(torch.empty((T, m), dtype=DT[dt], device="cuda"), by),
                                      _shifted(torch.empty(T, device="cuda"), by))
        cuda_lib.moe_distill_targets(_shifted(l.cuda(), by), m, out=out)
        assert torch.equal(out.idx.cpu().long()[fine], ti)
        assert torch.equal(out.logits.cpu().to(F64)[fine], tl)
        _close(out.rest.cpu()[fine], tr, at=DELTA, what="rest")
        for t in broken:
            assert out.idx[t].tolist() == list(range(m))
            assert torch.isnan(out.logits[t]).all() and torch.isnan(out.rest[t])


def test_two_graphs_that_share_a_workspace(cuda_lib):
    """Replayed in turn, each gives its own results, and each call its own status."""
    T, E, k = 3000, 64, 6
    bal_ws, dis_ws = cuda_lib.moe_balance_loss_workspace(T, E), cuda_lib.moe_distill_loss_workspace(T)
    graphs, results, wants, inputs = [], [], [], []
    for seed in (1, 2):
        l, teacher, _ = _step_inputs(T, E, k, "bf16", seed)
        idx, _ = cuda_lib.moe_route(l, k, True)
        if seed == 2:
            idx[5, 1] = E  # reported by this one alone
        tg = cuda_lib.moe_distill_targets(teacher, k)
        call = lambda: (cuda_lib.moe_balance_loss(l, idx, z_loss=True, workspace=bal_ws),
                        cuda_lib.moe_distill_loss(l, tg, workspace=dis_ws))
        wants.append([x.clone() for r in call() for x in (r.loss, r.row_stats)])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b, d = call()
        inputs.append((l, idx, tg))  # what a graph reads has to live
        graphs.append(graph)
        results.append([b.loss, b.row_stats, d.loss, d.row_stats])
    for _ in range(3):
        for graph, result, want, status in zip(graphs, results, wants, (0, 6)):
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(result, want):
                assert torch.equal(_bits(a), _bits(b))
            assert cuda_lib.moe_get_device_status(bal_ws) == status
            assert cuda_lib.moe_get_device_status(dis_ws) == 0
