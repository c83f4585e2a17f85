"""The router's training losses on the GPU against their definitions in 64 bits.

Tolerances.  A score p = exp(x) / s carries: two roundings of x (|x| <= 40 here,
so 2 * 40 * 2^-24 relative in exp(x)), 2 ulp of the exponential, and the sum's
and the division's few roundings: below 100 * 2^-24 = 6e-6 relative.  Sums of
scores are of one sign, so they keep the relative error and add one rounding per
addition of the longest chain (rows of a lane, 8 warps, partials of a lane):
below 100 more here.  RT = 2e-5 covers both.  Gradients are held against the
size of the terms that they are summed from (the reference gives it) with the
same RT, and end in one rounding to their type: half a step, eps / 2 of the
value, or half the smallest subnormal.  z: log s and the maximum each carry an
absolute error below 2^-21 (|lse| <= 16), so z is within 2 |lse| 2^-20 + RT z.
KL is a sum of terms q h(d) >= 0, d = log(q / p): d's absolute error is below
DELTA = 8e-6 (as x above, and two logs), which moves the sum by sum |q - p| DELTA.
The reference's own KL sums fewer than 100 terms of size <= 10 in 64 bits and is
off by up to 100 * 10 * 2^-53 = 1.1e-13 (REF) where the kernel's is exactly 0.
"""
import math

import pytest
import torch

import router_loss_reference as ref

pytestmark = pytest.mark.gpu
F64 = torch.float64
RT = 2e-5
DELTA = 8e-6
REF = 1.2e-13
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}  # f32/bf16: kernels flush subnormals

# T, E, k: one row, one expert, odd and ragged sizes, each lane layout, the limits
SIZES = [(1, 1, 1), (1, 2, 1), (3, 7, 2), (64, 4, 2), (37, 16, 16), (100, 60, 4), (129, 64, 6), (257, 101, 8),
         (300, 128, 8), (77, 256, 8), (50, 257, 9), (41, 320, 5), (40, 512, 3), (33, 1000, 64), (21, 1023, 7),
         (20, 1024, 64), (5000, 8, 2)]


def _offsets(T, kind, g):
    """None, or offsets with empty sequences, sequences of one row and rows behind the last."""
    if kind == "one":
        return None
    n = 5 if kind == "ragged" else max(1, T // 2)
    cuts = torch.sort(torch.randint(0, T + 1, (n,), generator=g)).values.tolist()
    return [0, 0] + cuts + [max(cuts[-1], T - T // 9)]


def _dev(x, dtype=None):
    return None if x is None else torch.as_tensor(x, dtype=dtype).cuda()


def _mask(T, g, masked):
    return (torch.rand(T, generator=g) < 0.75) if masked else None


def _logits(T, E, dt, g, spread=1.5):
    return (spread * torch.randn((T, E), generator=g)).to(DT[dt])


def _check(got, want, tol, what):
    got, want = got.detach().cpu().to(F64), want.to(F64)
    assert got.shape == want.shape, what
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN positions differ"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    ok = ~(nan | inf)
    over = ((got - want).abs() - tol)[ok] if torch.is_tensor(tol) and tol.shape == want.shape else None
    if over is None:
        over = (got - want).abs()[ok] - tol
    assert over.numel() == 0 or float(over.max()) <= 0.0, \
        f"{what}: off by {float((got - want).abs()[ok].max()):.3e}, {float(over.max()):.3e} over"


def _check_grad(got, want, size, dt, what):
    """A gradient within _rounded of `want`.  A value that lies beyond the type's
    largest by half a step or more (65520 in FP16) rounds to infinity, so an
    infinity is right exactly where the value, within its error, does."""
    tol = _rounded(size, want, dt)
    top = torch.finfo(DT[dt]).max
    edge = top * (1 + torch.finfo(DT[dt]).eps / 4)
    g = got.detach().cpu().to(F64)
    over = torch.isinf(g) & (want.abs() + tol >= edge) & (torch.sign(g) == torch.sign(want))
    _check(torch.where(over, torch.zeros_like(g), g), torch.where(over, torch.zeros_like(g), want), tol, what)


def _rounded(size, want, dt):
    """Error allowed to a gradient: RT of its terms and one rounding to dt."""
    return RT * size + (want.abs() + RT * size) * torch.finfo(DT[dt]).eps / 2 + TINY[dt]


def _close(got, want, rt=RT, at=0.0, what=""):
    _check(got, want, rt * torch.nan_to_num(want.to(F64)).abs() + at, what)


# ---- balance ---------------------------------------------------------------------
def _balance_case(T, E, k, dt, scoring, seqs, masked, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * T + E)
    l = _logits(T, E, dt, g)
    idx = torch.topk(l.float(), k, dim=1).indices
    return l, idx, _mask(T, g, masked), _offsets(T, seqs, g), g


CASES = [(s, "f32", "softmax", "one", False) for s in SIZES] + \
        [(s, "bf16", "softmax", "ragged", True) for s in SIZES] + \
        [(s, "f16", "sigmoid", "ragged", True) for s in SIZES] + \
        [(s, "bf16", "sigmoid", "one", True) for s in SIZES[3:9]] + \
        [(s, "f32", "sigmoid", "short", True) for s in SIZES[2:10]] + \
        [(s, "f16", "softmax", "short", False) for s in SIZES[2:10]]


@pytest.mark.parametrize("size,dt,scoring,seqs,masked", CASES)
def test_balance_forward_and_backward(cuda_lib, size, dt, scoring, seqs, masked):
    T, E, k = size
    l, idx, mask, off, g = _balance_case(T, E, k, dt, scoring, seqs, masked)
    z = scoring == "softmax"
    dl, doff, dmask = l.cuda(), _dev(off, torch.int32), _dev(mask)
    out = cuda_lib.moe_balance_loss(dl, idx.int().cuda(), scoring=scoring, token_mask=dmask, seq_offsets=doff,
                                    z_loss=z)
    want = ref.balance(l.to(F64), idx, scoring, mask, off)
    assert torch.equal(out.counts.cpu().long(), want["counts"])
    assert torch.equal(out.tokens.cpu().long(), want["tokens"])
    _close(out.mean_scores, want["mean_scores"], what="mean_scores")
    _close(out.loss, want["loss"], what="loss")
    if z:
        _close(out.z_loss, want["z_loss"], at=32 * 2.0 ** -20, what="z_loss")
    _close(out.row_stats, ref.balance_row_stats(l.to(F64), scoring, mask, off), what="row_stats")
    assert cuda_lib.moe_get_device_status(out.workspace) == 0

    S = len(want["tokens"])
    scale = float(T * E) if dt == "f16" else 1.0
    dloss, dz = scale * torch.randn(S, generator=g), scale * torch.randn(S, generator=g) if z else None
    grad, size_ = ref.balance_grad(l.to(F64), want["counts"], want["tokens"], k, scoring, dloss.to(F64),
                                   dz.to(F64) if z else None, mask, off)
    d = cuda_lib.moe_balance_loss_backward(dl, out, k, dloss.cuda(), scoring=scoring, seq_offsets=doff,
                                           dz_loss=_dev(dz))
    assert d.dtype == DT[dt]
    _check_grad(d, grad, size_, dt, "dlogits")
    # added to a gradient that is there, in its own buffer
    base = torch.randn((T, E), generator=g).to(DT[dt])
    buf = base.cuda()
    cuda_lib.moe_balance_loss_backward(dl, out, k, dloss.cuda(), scoring=scoring, seq_offsets=doff, dz_loss=_dev(dz),
                                       base=buf, dlogits=buf)
    total = grad + base.to(F64)
    _check_grad(buf, total, size_ + base.to(F64).abs() * 2.0 ** -24 / RT, dt, "base + dlogits")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_balance_rows_at_the_edge(cuda_lib, dt, scoring):
    """Experts masked with -inf or the type's lowest value, rows with nothing but
    the lowest value, far-below and far-above logits, poisoned rows (in a sequence
    of their own) and poison in rows that do not count."""
    T, E, k = 24, 40, 4
    g = torch.Generator().manual_seed(5)
    l = _logits(T, E, dt, g)
    low = torch.finfo(DT[dt]).min
    l[0, 5:] = -math.inf
    l[1, ::2] = low
    l[2, :] = low
    l[3, :] = -1000.0
    l[4] = l[4] - 300.0
    l[5] = l[5] + 300.0
    l[6, 7] = 500.0
    off = [0, 8, 9, 10, 11, 20]
    l[8, 3] = math.nan
    l[9, 3] = math.inf
    l[10] = -math.inf
    mask = torch.ones(T, dtype=torch.bool)
    l[12], mask[12] = math.nan, False
    l[13], mask[13] = math.inf, False
    l[14, 0], mask[14] = -math.inf, False
    l[20:] = math.nan  # behind the last sequence
    idx = torch.randint(0, E, (T, k), generator=g)
    idx[12], idx[21] = -1, 2 ** 31 - 1  # not read: their rows do not count
    dl, doff = l.cuda(), _dev(off, torch.int32)
    out = cuda_lib.moe_balance_loss(dl, idx.int().cuda(), scoring=scoring, token_mask=mask.cuda(), seq_offsets=doff)
    want = ref.balance(l.to(F64), idx, scoring, mask, off)
    assert cuda_lib.moe_get_device_status(out.workspace) == 0
    assert torch.equal(out.counts.cpu().long(), want["counts"])
    assert torch.equal(out.tokens.cpu().long(), want["tokens"])
    _close(out.loss, want["loss"], what="loss")
    _close(out.mean_scores, want["mean_scores"], at=1e-30, what="mean_scores")
    dloss = torch.ones(5)
    grad, size = ref.balance_grad(l.to(F64), want["counts"], want["tokens"], k, scoring, dloss.to(F64), None, mask,
                                  off)
    d = cuda_lib.moe_balance_loss_backward(dl, out, k, dloss.cuda(), scoring=scoring, seq_offsets=doff)
    # a +inf logit: its sigmoid is one and its slope zero; softmax has no value there
    _check(d, grad, _rounded(torch.nan_to_num(size), torch.nan_to_num(grad), dt), "dlogits")
    for t in (12, 13, 14, 20, 23):
        assert not d[t].any(), "a row that does not count has a gradient"


def test_balance_indices(cuda_lib):
    """The same expert twice in a row counts twice; an index that is none is
    counted nowhere and reported; the status word is reset by the next call."""
    l = torch.randn(50, 6)
    idx = torch.randint(0, 6, (50, 3))
    idx[7] = 2
    a = cuda_lib.moe_balance_loss(l.cuda(), idx.int().cuda())
    assert torch.equal(a.counts.cpu().long()[0], torch.bincount(idx.flatten(), minlength=6))
    bad = idx.clone()
    bad[9, 1], bad[10, 0] = 6, -1
    b = cuda_lib.moe_balance_loss(l.cuda(), bad.int().cuda(), workspace=a.workspace)
    keep = bad.flatten()[(bad.flatten() >= 0) & (bad.flatten() < 6)]
    assert torch.equal(b.counts.cpu().long()[0], torch.bincount(keep, minlength=6))
    assert cuda_lib.moe_get_device_status(a.workspace) == 6
    cuda_lib.moe_balance_loss(l.cuda(), idx.int().cuda(), workspace=a.workspace)
    assert cuda_lib.moe_get_device_status(a.workspace) == 0


# ---- distillation ------------------------------------------------------------------
def _lists(l, m, tau, dt, g, noise=0.7):
    teacher = (l.float() + noise * torch.randn(l.shape, generator=g)).to(DT[dt])
    ti, tl, tr = ref.targets(teacher.to(F64), m, tau)
    return teacher, ti, tl.to(DT[dt]), tr.float()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", SIZES)
def test_targets(cuda_lib, size, dt):
    T, E, m = size
    g = torch.Generator().manual_seed(T + E)
    l = _logits(T, E, dt, g)
    if dt != "f32":
        l = (l.float() * 2).round().div(2).to(DT[dt])  # many ties
    l[0, : E // 2] = 0.0
    l[0, : E // 4] = -0.0
    for tau in (1.0, 2.5):
        out = cuda_lib.moe_distill_targets(l.cuda(), m, temperature=tau)
        ti, tl, tr = ref.targets(l.to(F64), m, tau)
        assert torch.equal(out.idx.cpu().long(), ti)
        assert torch.equal(out.logits.cpu().to(F64), tl)
        # tau log s + maximum: |x| roundings as for a score, and two logs of a sum
        _close(out.rest, tr, at=tau * DELTA, what="rest")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_targets_at_the_edge(cuda_lib, dt):
    l = torch.randn(9, 33).to(DT[dt])
    low = torch.finfo(DT[dt]).min
    l[0] = -math.inf
    l[1, 2:] = -math.inf
    l[2] = low
    l[3, 1:] = low
    l[4, 7] = math.nan
    l[5, 30] = math.inf
    l[6] = 3.0
    l[8, 0] = math.copysign(math.nan, -1.0)
    m = 4
    out = cuda_lib.moe_distill_targets(l.cuda(), m)
    ti, tl, tr = ref.targets(l.to(F64), m, 1.0)
    for t in (0, 1, 2, 3, 6, 7):
        assert torch.equal(out.idx[t].cpu().long(), ti[t]), t
        assert torch.equal(out.logits[t].cpu().to(F64), tl[t]), t
    keep = torch.tensor([0, 1, 2, 3, 6, 7])
    _close(out.rest[keep.cuda()], tr[keep], at=DELTA, what="rest")
    for t in (4, 5, 8):
        assert out.idx[t].tolist() == list(range(m))
        assert torch.isnan(out.logits[t]).all() and torch.isnan(out.rest[t])


DCASES = [(s, "f32", "f32", True, "one", False, 1.0) for s in SIZES] + \
         [(s, "bf16", "bf16", True, "ragged", True, 2.0) for s in SIZES] + \
         [(s, "f16", "f32", False, "ragged", True, 1.0) for s in SIZES] + \
         [(s, "f32", "bf16", False, "short", False, 0.5) for s in SIZES[2:10]]


@pytest.mark.parametrize("size,dt,tdt,rest,seqs,masked,tau", DCASES)
def test_distill_forward_and_backward(cuda_lib, size, dt, tdt, rest, seqs, masked, tau):
    T, E, m = size
    if T > 1000:
        T = 700
    g = torch.Generator().manual_seed(3 * T + E)
    l = _logits(T, E, dt, g)
    _, ti, tl, tr = _lists(l, m, tau, tdt, g)
    if m > 1:
        tl[::3, m - 1] = -math.inf   # absent, whatever its index
        ti[::3, m - 1] = -1
    if T > 4 and not rest:
        tl[4] = -math.inf            # no target
    mask, off = _mask(T, g, masked), _offsets(T, seqs, g)
    perm = torch.randperm(m, generator=g)  # lists in any order
    ti, tl = ti[:, perm].contiguous(), tl[:, perm].contiguous()
    tg = cuda_lib.DistillTargets(ti.int().cuda(), tl.cuda(), tr.cuda() if rest else None)
    dl, doff, dmask = l.cuda(), _dev(off, torch.int32), _dev(mask)
    out = cuda_lib.moe_distill_loss(dl, tg, temperature=tau, token_mask=dmask, seq_offsets=doff)
    r64 = tr.to(F64) if rest else None
    loss, tokens, row, diff = ref.distill(l.to(F64), ti, tl.to(F64), r64, tau, mask, off)
    assert torch.equal(out.tokens.cpu().long(), tokens)
    assert cuda_lib.moe_get_device_status(out.workspace) == 0
    _check(out.row_loss, row, RT * torch.nan_to_num(row, posinf=0.0) + DELTA / min(tau, 1.0) * diff + REF, "row_loss")
    mean_diff = torch.stack([diff[r].sum() / max(int(n), 1) for r, n in zip(ref.counted(T, mask, off), tokens)])
    _check(out.loss, loss, RT * loss + DELTA / min(tau, 1.0) * mean_diff + REF, "loss")

    dloss = torch.randn(len(tokens), generator=g) * (float(T) if dt == "f16" else 1.0)
    grad, size_ = ref.distill_grad(l.to(F64), ti, tl.to(F64), r64, tau, tokens, dloss.to(F64), mask, off)
    d = cuda_lib.moe_distill_loss_backward(dl, tg, out, dloss.cuda(), temperature=tau, seq_offsets=doff)
    assert d.dtype == DT[dt]
    _check_grad(d, grad, size_ / min(tau, 1.0), dt, "dlogits")
    base = torch.randn((T, E), generator=g).to(DT[dt])
    buf = base.cuda()
    cuda_lib.moe_distill_loss_backward(dl, tg, out, dloss.cuda(), temperature=tau, seq_offsets=doff, base=buf,
                                       dlogits=buf)
    total = grad + base.to(F64)
    _check_grad(buf, total, size_ / min(tau, 1.0) + base.to(F64).abs() * 2.0 ** -24 / RT, dt, "base + dlogits")


def test_distill_near_teacher_keeps_its_digits(cuda_lib):
    """A student within 1e-3 of its teacher: KL ~ 1e-7, far below FP32's step at
    the size of log p."""
    g = torch.Generator().manual_seed(1)
    teacher = torch.randn((64, 32), generator=g)
    student = teacher + 1e-3 * torch.randn((64, 32), generator=g)
    for m, rest in ((8, True), (8, False), (32, True), (32, False)):
        ti, tl, tr = ref.targets(teacher.to(F64), m, 1.0)
        tl, tr = tl.float(), tr.float()
        tg = cuda_lib.DistillTargets(ti.int().cuda(), tl.cuda(), tr.cuda() if rest else None)
        out = cuda_lib.moe_distill_loss(student.cuda(), tg)
        _, _, row, diff = ref.distill(student.to(F64), ti, tl.to(F64), tr.to(F64) if rest else None, 1.0)
        _check(out.row_loss, row, RT * row + DELTA * diff + DELTA ** 2, "row_loss")
        assert (out.row_loss >= 0).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_distill_rows_at_the_edge(cuda_lib, dt):
    T, E, m = 20, 48, 5
    g = torch.Generator().manual_seed(9)
    l = _logits(T, E, dt, g)
    _, ti, tl, tr = _lists(l, m, 1.0, dt, g)
    low = torch.finfo(DT[dt]).min
    tl[0] = -math.inf                      # only a rest
    tr[1] = -math.inf                      # only a list
    tl[2], tr[2] = -math.inf, -math.inf    # no target
    l[3, int(ti[3, 0])] = -math.inf        # the teacher gives mass to it: +inf
    out3 = torch.ones(E, dtype=torch.bool)
    out3[ti[4]] = False
    l[4, out3] = (-200.0 - torch.arange(int(out3.sum())) % 4).to(DT[dt])  # the student's rest underflows
    l[5, out3] = -math.inf                 # some of the row only
    l[6] = low
    l[7, E // 2:] = low
    tl[8] = low
    l[9] = l[9] + 300
    off = [0, 12, 13, 14, 15, 16, 17, 18]
    l[12, 3] = math.nan
    l[13, 3] = math.inf
    l[14] = -math.inf
    tl[15, 2] = math.nan
    tr[16] = math.inf
    ti[17, 1] = E
    mask = torch.ones(T, dtype=torch.bool)
    l[10], tl[10], ti[10], mask[10] = math.nan, math.nan, -1, False
    l[18:], tl[18:], tr[18:] = math.nan, math.inf, math.nan
    tg = cuda_lib.DistillTargets(ti.int().cuda(), tl.cuda(), tr.cuda())
    doff = _dev(off, torch.int32)
    out = cuda_lib.moe_distill_loss(l.cuda(), tg, token_mask=mask.cuda(), seq_offsets=doff)
    row = out.row_loss.cpu()
    assert out.tokens.tolist() == [10, 1, 1, 1, 1, 1, 1]
    assert torch.isnan(row[12:18]).all() and torch.isnan(out.loss[1:]).all()
    assert row[2] == 0 and row[10] == 0 and not row[18:].any()
    assert row[3] == math.inf and out.loss[0] == math.inf
    assert cuda_lib.moe_get_device_status(out.workspace) == 6  # row 17
    fine = [0, 1, 4, 5, 6, 7, 8, 9, 11]
    _, _, want, diff = ref.distill(l.to(F64)[fine], ti[fine], tl.to(F64)[fine], tr.to(F64)[fine], 1.0)
    _check(row[fine], want, RT * want + DELTA * diff + REF, "row_loss")
    dloss = torch.ones(7)
    d = cuda_lib.moe_distill_loss_backward(l.cuda(), tg, out, dloss.cuda(), seq_offsets=doff).cpu()
    assert torch.isnan(d[12:18]).all()
    for t in (2, 10, 18, 19):
        assert not d[t].any()
    grad, size = ref.distill_grad(l.to(F64)[fine], ti[fine], tl.to(F64)[fine], tr.to(F64)[fine], 1.0,
                                  torch.tensor([10]), dloss.to(F64))
    _check(d[fine], grad, _rounded(size, grad, dt), "dlogits")
    assert torch.isfinite(d[3].float()).all()


def test_distill_listed_twice(cuda_lib):
    l = torch.randn(6, 70)
    ti, tl, tr = ref.targets(torch.randn(6, 70, dtype=F64), 40, 1.0)
    ti[2, 39] = ti[2, 0]
    ti[4, 3] = ti[4, 1]
    tl[4, 3] = -math.inf  # absent: not twice
    tg = cuda_lib.DistillTargets(ti.int().cuda(), tl.float().cuda(), tr.float().cuda())
    out = cuda_lib.moe_distill_loss(l.cuda(), tg)
    assert torch.isnan(out.row_loss).tolist() == [False, False, True, False, False, False]
    assert cuda_lib.moe_get_device_status(out.workspace) == 6


# ---- batches -----------------------------------------------------------------------
def _all_calls(moe, l, idx, teacher, k, off=None, mask=None, stream=None):
    """A router's training step: both losses, their gradients added to the routing weights'."""
    T, E = l.shape
    S = 1 if off is None else off.shape[0] - 1
    one = torch.linspace(0.5, 1.5, S, device=l.device)
    bal = moe.moe_balance_loss(l, idx, token_mask=mask, seq_offsets=off, z_loss=True, stream=stream)
    tg = moe.moe_distill_targets(teacher, k, stream=stream)
    dis = moe.moe_distill_loss(l, tg, token_mask=mask, seq_offsets=off, stream=stream)
    dw = torch.linspace(-1, 1, T * k, device=l.device).view(T, k)
    d = moe.moe_router_backward(l, idx, dw, "softmax", True, stream=stream)
    moe.moe_balance_loss_backward(l, bal, k, one, seq_offsets=off, dz_loss=0.1 * one, base=d, dlogits=d,
                                  stream=stream)
    moe.moe_distill_loss_backward(l, tg, dis, one, seq_offsets=off, base=d, dlogits=d, stream=stream)
    return [bal.loss, bal.z_loss, bal.mean_scores, bal.counts, bal.tokens, bal.row_stats, tg.idx, tg.logits, tg.rest,
            dis.loss, dis.tokens, dis.row_loss, dis.row_stats, d]


def _step_inputs(T, E, k, dt, seed, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    l = _logits(T, E, dt, g)
    teacher = (l.float() + 0.5 * torch.randn((T, E), generator=g)).to(DT[dt])
    return l.to(device), teacher.to(device), g


def _bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("T,E,k", [(64, 4, 2), (3000, 64, 6), (1500, 100, 8)])
def test_training_step(cuda_lib, T, E, k):
    """The losses together, as a training step makes them, against one total in 64 bits."""
    l, teacher, _ = _step_inputs(T, E, k, "f32", 4)
    idx, _ = cuda_lib.moe_route(l, k, True)
    outs = _all_calls(cuda_lib, l, idx, teacher, k)
    x = l.cpu().to(F64).requires_grad_(True)
    ix = idx.cpu().long()
    p = torch.softmax(x, 1).gather(1, ix)
    w = p / p.sum(1, keepdim=True)
    task = (w * torch.linspace(-1, 1, T * k).view(T, k).to(F64)).sum()
    b = ref.balance(x, ix, "softmax")
    lp = torch.log_softmax(x, 1)
    ti, tl, tr = ref.targets(teacher.cpu().to(F64), k, 1.0)
    logq = torch.log_softmax(torch.cat([tl, tr[:, None]], 1), 1)
    out = lp.scatter(1, ti, -math.inf)
    kl = (logq.exp() * (logq - torch.cat([lp.gather(1, ti), torch.logsumexp(out, 1)[:, None]], 1))).sum(1)
    one = 0.5
    total = task + one * b["loss"].sum() + 0.1 * one * b["z_loss"].sum() + one * kl.mean()
    total.backward()
    # three FP32 gradients, each of terms below 2 in size, added with two roundings
    _check(outs[-1], x.grad, torch.full_like(x.grad, 3 * 2 * RT), "step gradient")


def test_results_are_reproducible_and_other_streams_agree(cuda_lib):
    T, E, k = 40000, 96, 6
    l, teacher, g = _step_inputs(T, E, k, "bf16", 6)
    idx, _ = cuda_lib.moe_route(l, k, True)
    off = torch.tensor([0, 5, 10000, 10000, 39000], dtype=torch.int32, device="cuda")
    mask = (torch.rand(T, generator=g) < 0.9).cuda()
    first = _all_calls(cuda_lib, l, idx, teacher, k, off, mask)
    for _ in range(3):
        for a, b in zip(first, _all_calls(cuda_lib, l, idx, teacher, k, off, mask)):
            assert torch.equal(_bits(a), _bits(b))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    # two steps at once, each with its own buffers
    other = _all_calls(cuda_lib, l, idx, teacher, k, off, mask, stream=side)
    here = _all_calls(cuda_lib, l, idx, teacher, k, off, mask)
    torch.cuda.synchronize()
    for a, b, c in zip(first, other, here):
        assert torch.equal(_bits(a), _bits(b)) and torch.equal(_bits(a), _bits(c))


def test_graph_replay_follows_its_inputs(cuda_lib):
    T, E, k = 2000, 64, 6
    l, teacher, g = _step_inputs(T, E, k, "bf16", 8)
    idx, _ = cuda_lib.moe_route(l, k, True)
    _all_calls(cuda_lib, l, idx, teacher, k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _all_calls(cuda_lib, l, idx, teacher, k)
    l2, t2, _ = _step_inputs(T, E, k, "bf16", 9)
    idx2, _ = cuda_lib.moe_route(l2, k, True)
    want = _all_calls(cuda_lib, l2, idx2, t2, k)
    l.copy_(l2), teacher.copy_(t2), idx.copy_(idx2)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(_bits(a), _bits(b))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_any_element_alignment(cuda_lib, dt):
    """Buffers that start on any element give the aligned buffers' results (up to
    the order of a row's sum)."""
    T, E, k = 70, 64, 6
    l, teacher, _ = _step_inputs(T, E, k, dt, 12)
    idx, _ = cuda_lib.moe_route(l, k, True)

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        return buf.copy_(t)
    a = _all_calls(cuda_lib, l, idx, teacher, k)
    b = _all_calls(cuda_lib, shifted(l), shifted(idx), shifted(teacher), k)
    for x, y in zip(a, b):
        if not x.is_floating_point():
            assert torch.equal(x, y)
        else:
            tol = 3 * RT * (1 + y.abs().double()) + torch.finfo(x.dtype).eps * y.abs().double() * (x is a[-1]) \
                + 3 * 2.0 ** -11 * (x is a[-1])
            _check(x, y.cpu().to(F64), tol.cpu(), "shifted")


@pytest.mark.parametrize("bad", [[5, 3, 9, 100], [0, 2 ** 31 - 1, 50, 100], [0, -1, -1, -1], [90, 10, 20, 5],
                                 [0, 200, 300, 400]])
def test_malformed_offsets_stay_inside_and_are_reported(cuda_lib, bad):
    T, E, k = 100, 24, 3
    l, teacher, _ = _step_inputs(T, E, k, "f32", 13)
    idx, _ = cuda_lib.moe_route(l, k, True)
    off = torch.tensor(bad, dtype=torch.int64).to(torch.int32).cuda()
    bal = cuda_lib.moe_balance_loss(l, idx, seq_offsets=off)
    assert cuda_lib.moe_get_device_status(bal.workspace) == 6
    tg = cuda_lib.moe_distill_targets(teacher, k)
    dis = cuda_lib.moe_distill_loss(l, tg, seq_offsets=off)
    assert cuda_lib.moe_get_device_status(dis.workspace) == 6
    one = torch.ones(3, device="cuda")
    cuda_lib.moe_balance_loss_backward(l, bal, k, one, seq_offsets=off)
    cuda_lib.moe_distill_loss_backward(l, tg, dis, one, seq_offsets=off)
    torch.cuda.synchronize()
    good = cuda_lib.moe_balance_loss(l, idx, workspace=bal.workspace)
    assert cuda_lib.moe_get_device_status(bal.workspace) == 0 and int(good.tokens[0]) == T


@pytest.mark.parametrize("T,E,k,dt", [(90000, 24, 3, "bf16"), (70000, 64, 6, "f32"), (60000, 96, 8, "f16"),
                                      (50000, 131, 5, "bf16"), (40000, 200, 9, "f32"), (50000, 257, 20, "f16"),
                                      (50000, 256, 40, "bf16"), (20000, 1000, 12, "bf16"), (15000, 999, 7, "f32")])
def test_long_batches_match_their_parts(cuda_lib, T, E, k, dt):
    """Batches long enough that every warp goes round its ring of rows several
    times: a row's results do not depend on the batch around it, and the sums are
    those of the rows (in 64 bits)."""
    l, teacher, g = _step_inputs(T, E, k, dt, 20)
    idx, _ = cuda_lib.moe_route(l, k, False)
    mask = (torch.rand(T, generator=g) < 0.9).cuda()
    off = torch.tensor([3, 1000, T // 2 + 1, T // 2 + 1, T - 5], dtype=torch.int32, device="cuda")
    one = torch.linspace(0.5, 1.5, 4, device="cuda")
    bal = cuda_lib.moe_balance_loss(l, idx, token_mask=mask, seq_offsets=off, z_loss=True)
    tg = cuda_lib.moe_distill_targets(teacher, k)
    dis = cuda_lib.moe_distill_loss(l, tg, token_mask=mask, seq_offsets=off)
    db = cuda_lib.moe_balance_loss_backward(l, bal, k, one, seq_offsets=off, dz_loss=one)
    dd = cuda_lib.moe_distill_loss_backward(l, tg, dis, one, seq_offsets=off)
    assert cuda_lib.moe_get_device_status(bal.workspace) == 0
    for s, (a, b) in enumerate(zip([3, 1000, T // 2 + 1, T // 2 + 1], [1000, T // 2 + 1, T // 2 + 1, T - 5])):
        rows = torch.arange(a, b, device="cuda")[mask[a:b]]
        n = len(rows)
        assert int(bal.tokens[s]) == n and int(dis.tokens[s]) == n
        if n == 0:
            continue
        assert torch.equal(bal.counts[s].long(), torch.bincount(idx[rows].long().flatten(), minlength=E))
        p = torch.softmax(l[rows].double(), 1).mean(0)
        _close(bal.mean_scores[s], p.cpu(), what="mean_scores")
        _close(dis.loss[s], dis.row_loss[rows].double().mean().cpu(), what="distillation loss")
        z = (torch.logsumexp(l[rows].double(), 1) ** 2).mean()
        _close(bal.z_loss[s], z.cpu(), at=32 * 2.0 ** -20, what="z_loss")
        for c in (a, (a + b) // 2, b - 200):  # the same rows alone
            part = slice(c, c + 200)
            m = mask[part].contiguous()
            pl, pi = l[part].clone(), idx[part].clone()
            pb = cuda_lib.moe_balance_loss(pl, pi, token_mask=m)
            assert torch.equal(_bits(pb.row_stats), _bits(bal.row_stats[part]))
            pt = cuda_lib.moe_distill_targets(teacher[part].clone(), k)
            for x, y in ((pt.idx, tg.idx), (pt.logits, tg.logits), (pt.rest, tg.rest)):
                assert torch.equal(_bits(x), _bits(y[part]))
            pd = cuda_lib.moe_distill_loss(pl, pt, token_mask=m)
            assert torch.equal(_bits(pd.row_loss), _bits(dis.row_loss[part]))
            assert torch.equal(_bits(pd.row_stats), _bits(dis.row_stats[:, part]))
            pb.counts, pb.tokens, pd.tokens = bal.counts[s:s + 1], bal.tokens[s:s + 1], dis.tokens[s:s + 1]
            w = one[s:s + 1].contiguous()
            assert torch.equal(_bits(cuda_lib.moe_balance_loss_backward(pl, pb, k, w, dz_loss=w)), _bits(db[part]))
            assert torch.equal(_bits(cuda_lib.moe_distill_loss_backward(pl, pt, pd, w)), _bits(dd[part]))
    for out in (bal.row_stats, db, dd):  # rows outside every sequence
        assert not out[:3].any() and not out[T - 5:].any()


def test_results_that_are_replaced_are_checked_again(cuda_lib):
    l, idx = torch.randn((8, 6), device="cuda"), torch.zeros((8, 2), dtype=torch.int32, device="cuda")
    bal = cuda_lib.moe_balance_loss(l, idx)
    one = torch.ones(1, device="cuda")
    bal.counts = bal.counts.long()
    with pytest.raises(cuda_lib.MoeError):
        cuda_lib.moe_balance_loss_backward(l, bal, 2, one)
    bal.counts = torch.zeros((1, 5), dtype=torch.int32, device="cuda")
    with pytest.raises(cuda_lib.MoeError):
        cuda_lib.moe_balance_loss_backward(l, bal, 2, one)
    bal = cuda_lib.moe_balance_loss(l, idx)
    cuda_lib.moe_balance_loss(l, idx, out=bal)
    bal.row_stats.resize_(4, 2)
    with pytest.raises(cuda_lib.MoeError):
        cuda_lib.moe_balance_loss(l, idx, out=bal)
    with pytest.raises(cuda_lib.MoeError):
        cuda_lib.moe_balance_loss(l[:4].contiguous(), idx[:4].contiguous(), out=bal, z_loss=True)


def test_no_rows(cuda_lib):
    """T = 0, and sequences that hold nothing."""
    l, idx = torch.empty((0, 8), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda")
    for off in (None, torch.zeros(4, dtype=torch.int32, device="cuda")):
        bal = cuda_lib.moe_balance_loss(l, idx, seq_offsets=off, z_loss=True)
        tg = cuda_lib.moe_distill_targets(l, 2)
        dis = cuda_lib.moe_distill_loss(l, tg, seq_offsets=off)
        for t in (bal.loss, bal.z_loss, bal.mean_scores, bal.counts, bal.tokens, dis.loss, dis.tokens):
            assert not t.any() and t.shape[0] == (1 if off is None else 3)
        one = torch.ones(1 if off is None else 3, device="cuda")
        assert cuda_lib.moe_balance_loss_backward(l, bal, 2, one, seq_offsets=off).shape == (0, 8)
        assert cuda_lib.moe_distill_loss_backward(l, tg, dis, one, seq_offsets=off).shape == (0, 8)
    l = torch.randn((5, 8), device="cuda")
    idx = torch.zeros((5, 2), dtype=torch.int32, device="cuda")
    none = torch.zeros(5, dtype=torch.bool, device="cuda")
    bal = cuda_lib.moe_balance_loss(l, idx, token_mask=none)
    d = cuda_lib.moe_balance_loss_backward(l, bal, 2, torch.ones(1, device="cuda"))
    assert not bal.loss.any() and not bal.counts.any() and not d.any()


def test_parts_of_a_larger_batch(cuda_lib):
    """Counts and tokens added up over the parts of a batch before the backward
    give the gradient of the whole batch's loss."""
    T, E, k = 600, 32, 4
    l, _, _ = _step_inputs(T, E, k, "f32", 14)
    idx, _ = cuda_lib.moe_route(l, k, True)
    one = torch.ones(1, device="cuda")
    whole = cuda_lib.moe_balance_loss(l, idx)
    want = cuda_lib.moe_balance_loss_backward(l, whole, k, one)
    parts = [cuda_lib.moe_balance_loss(l[a:a + 200].contiguous(), idx[a:a + 200].contiguous()) for a in (0, 200, 400)]
    counts, tokens = sum(p.counts for p in parts), sum(p.tokens for p in parts)
    assert torch.equal(counts, whole.counts)
    for a, p in zip((0, 200, 400), parts):
        p.counts, p.tokens = counts, tokens
        got = cuda_lib.moe_balance_loss_backward(l[a:a + 200].contiguous(), p, k, one)
        assert torch.equal(got, want[a:a + 200])


def test_binding_checks(cuda_lib):
    l, idx = torch.randn((8, 6), device="cuda"), torch.zeros((8, 2), dtype=torch.int32, device="cuda")
    bal = cuda_lib.moe_balance_loss(l, idx)
    one = torch.ones(1, device="cuda")
    E = cuda_lib.MoeError
    for kind, call in (
            (E, lambda: cuda_lib.moe_balance_loss(l, idx.long())),
            (E, lambda: cuda_lib.moe_balance_loss(l, idx[:7])),
            (E, lambda: cuda_lib.moe_balance_loss(l.double(), idx)),
            (E, lambda: cuda_lib.moe_balance_loss(l, idx, token_mask=torch.ones(8, device="cuda"))),
            (E, lambda: cuda_lib.moe_balance_loss(l, idx, token_mask=torch.ones(7, dtype=torch.bool, device="cuda"))),
            (E, lambda: cuda_lib.moe_balance_loss(l, idx, seq_offsets=torch.zeros(1, dtype=torch.int32,
                                                                                   device="cuda"))),
            (E, lambda: cuda_lib.moe_balance_loss(l, idx, scoring="sigmoid", z_loss=True)),
            (E, lambda: cuda_lib.moe_balance_loss(l, idx, z_loss=True, out=bal)),
            (E, lambda: cuda_lib.moe_balance_loss(l, idx, workspace=torch.empty(256, dtype=torch.uint8,
                                                                                device="cuda"))),
            (ValueError, lambda: cuda_lib.moe_balance_loss(l.t().contiguous().t(), idx)),
            (ValueError, lambda: cuda_lib.moe_balance_loss(l, idx.cpu())),
            (E, lambda: cuda_lib.moe_balance_loss_backward(l, bal, 0, one)),
            (E, lambda: cuda_lib.moe_balance_loss_backward(l, bal, 2, one.half())),
            (E, lambda: cuda_lib.moe_balance_loss_backward(l, bal, 2, one, base=l.half())),
            (E, lambda: cuda_lib.moe_balance_loss_backward(l[:4].contiguous(), bal, 2, one)),
            (E, lambda: cuda_lib.moe_distill_targets(l, 7)),
            (E, lambda: cuda_lib.moe_distill_targets(l, 0)),
            (E, lambda: cuda_lib.moe_distill_targets(l, 2, temperature=0.0))):
        with pytest.raises(kind):
            call()


def test_past_two_to_the_31_elements(cuda_lib):
    """Rows whose offsets pass 2^31 elements: the tail of a long batch against
    the same rows alone."""
    E, k, tail = 1024, 4, 1000
    T = (1 << 31) // E + 30000
    g = torch.Generator(device="cuda").manual_seed(2)
    l = torch.empty((T, E), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    idx = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    idx[-tail:] = torch.randint(0, E, (tail, k), generator=g, device="cuda").int()
    off = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    part, pidx = l[-tail:].clone(), idx[-tail:].clone()
    two, one = torch.ones(2, device="cuda"), torch.ones(1, device="cuda")
    bal, pbal = cuda_lib.moe_balance_loss(l, idx, seq_offsets=off), cuda_lib.moe_balance_loss(part, pidx)
    assert torch.equal(bal.counts[1:], pbal.counts) and bal.tokens.tolist() == [T - tail, tail]
    assert int(bal.counts[0, 0]) == (T - tail) * k
    assert torch.equal(bal.row_stats[-tail:], pbal.row_stats)
    _close(bal.loss[1:], pbal.loss.cpu().double(), what="loss")
    d = cuda_lib.moe_balance_loss_backward(l, bal, k, two, seq_offsets=off)
    pd = cuda_lib.moe_balance_loss_backward(part, pbal, k, one)
    assert torch.equal(d[-tail:], pd)
    tg, ptg = cuda_lib.moe_distill_targets(l, 8), cuda_lib.moe_distill_targets(part, 8)
    assert torch.equal(tg.idx[-tail:], ptg.idx) and torch.equal(tg.rest[-tail:], ptg.rest)
    dis, pdis = cuda_lib.moe_distill_loss(l, tg, seq_offsets=off), cuda_lib.moe_distill_loss(part, ptg)
    assert torch.equal(dis.row_loss[-tail:], pdis.row_loss)
    del d
    d = cuda_lib.moe_distill_loss_backward(l, tg, dis, two, seq_offsets=off)
    assert torch.equal(d[-tail:], cuda_lib.moe_distill_loss_backward(part, ptg, pdis, one))
