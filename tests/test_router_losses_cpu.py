"""The router's training losses without a GPU: the reference's closed-form
gradients against differences and against autograd of its losses, and the
refusals of the C ABI and of the Python binding."""
import ctypes

import pytest
import torch

import router_loss_reference as ref

F64 = torch.float64
OK, INVALID_ARG, SHAPE, DTYPE, UNSUPPORTED = 0, 1, 2, 3, 4
F32, F16, BF16 = 0, 1, 2
FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call below fails its checks first
ODD = ctypes.c_void_p(0x10001)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from top_routing_grouped_fp32_gb300 import build as native_build
    from top_routing_grouped_fp32_gb300 import _lib
    native_build.build()
    return _lib.load()


def _batch(T, E, k, seed):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((T, E), generator=g, dtype=F64)
    idx = torch.topk(logits, k, dim=1).indices
    mask = torch.rand(T, generator=g) < 0.8
    return logits, idx, mask, g


def _differences(f, x, rows, cols, h=1e-5):
    """Central differences of f at x[t, e] for the given entries (error h^2 f'''/6 + 1e-16/h)."""
    out = []
    for t, e in zip(rows, cols):
        a, b = x.clone(), x.clone()
        a[t, e] += h
        b[t, e] -= h
        out.append((f(a) - f(b)) / (2 * h))
    return torch.stack(out)


@pytest.mark.parametrize("scoring,z", [("softmax", False), ("softmax", True), ("sigmoid", False)])
def test_balance_gradient_formula(scoring, z):
    T, E, k = 23, 7, 3
    logits, idx, mask, g = _batch(T, E, k, 1)
    off = [0, 9, 9, 20]
    dloss = torch.randn(3, generator=g, dtype=F64)
    dz = torch.randn(3, generator=g, dtype=F64) if z else None

    def value(l):
        r = ref.balance(l, idx, scoring, mask, off)
        return (dloss * r["loss"]).sum() + ((dz * r["z_loss"]).sum() if z else 0.0)

    r = ref.balance(logits, idx, scoring, mask, off)
    d, _ = ref.balance_grad(logits, r["counts"], r["tokens"], k, scoring, dloss, dz, mask, off)
    x = logits.clone().requires_grad_(True)
    value(x).backward()
    # both are FP64 sums of < 100 terms of size <= 1: 100 * 2^-53 is far below 1e-12
    assert torch.allclose(d, x.grad, rtol=0, atol=1e-12)
    rows, cols = [0, 3, 10, 15, 19, 22], [1, 0, 6, 2, 5, 3]
    num = _differences(value, logits, rows, cols)
    # h^2 / 6 times a third derivative of at most a few units: below 1e-9
    assert torch.allclose(d[rows, cols], num, rtol=0, atol=1e-9)


@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_distill_gradient_formula(rest, tau):
    T, E, m = 17, 9, 4
    logits, _, mask, g = _batch(T, E, m, 2)
    off = [0, 5, 5, 14]
    teacher = logits + 0.5 * torch.randn((T, E), generator=g, dtype=F64)
    ti, tl, tr = ref.targets(teacher, m, tau)
    tl[2, 1] = -float("inf")           # an absent entry
    tl[6] = -float("inf")              # no list, only a rest (no target at all without one)
    trest = tr if rest else None
    dloss = torch.randn(3, generator=g, dtype=F64)

    def value(l):
        return (dloss * ref.distill(l, ti, tl, trest, tau, mask, off)[0]).sum()

    _, tokens, _, _ = ref.distill(logits, ti, tl, trest, tau, mask, off)
    d, _ = ref.distill_grad(logits, ti, tl, trest, tau, tokens, dloss, mask, off)
    x = logits.clone().requires_grad_(True)
    value(x).backward()
    assert torch.allclose(d, x.grad, rtol=0, atol=1e-12)
    rows, cols = [0, 2, 4, 7, 12, 13], [1, 0, 6, 2, 5, 3]
    assert torch.allclose(d[rows, cols], _differences(value, logits, rows, cols), rtol=0, atol=1e-9)


def test_full_rest_is_the_full_divergence():
    """With its rest a list loses nothing where the student agrees outside the
    list up to a factor: KL over the buckets is at most the full KL, and equal to
    it when the list is the whole row."""
    logits, _, _, g = _batch(11, 8, 3, 3)
    teacher = logits + torch.randn((11, 8), generator=g, dtype=F64)
    full = (torch.softmax(teacher, 1) * (torch.log_softmax(teacher, 1) - torch.log_softmax(logits, 1))).sum(1)
    for m in (1, 3, 8):
        ti, tl, tr = ref.targets(teacher, m, 1.0)
        row = ref.distill(logits, ti, tl, tr, 1.0)[2]
        assert (row <= full + 1e-12).all() and (row >= -1e-12).all()
    assert torch.allclose(row, full, rtol=0, atol=1e-12)


# ---- refusals of the C ABI ---------------------------------------------------------
def _balance(lib, logits=FAKE, dt=BF16, idx=FAKE, mask=None, off=None, T=8, E=8, k=2, S=1, scoring=0, loss=FAKE,
             z=None, mean=None, counts=FAKE, tokens=FAKE, stats=FAKE, ws=FAKE, nbytes=BIG):
    return lib.moe_balance_loss(logits, dt, idx, mask, off, T, E, k, S, scoring, loss, z, mean, counts, tokens,
                                stats, ws, nbytes, None)


def _balance_bwd(lib, logits=FAKE, dt=BF16, stats=FAKE, counts=FAKE, tokens=FAKE, off=None, T=8, E=8, k=2, S=1,
                 scoring=0, dloss=FAKE, dz=None, base=None, out=FAKE):
    return lib.moe_balance_loss_backward(logits, dt, stats, counts, tokens, off, T, E, k, S, scoring, dloss, dz,
                                         base, out, None)


def _targets(lib, logits=FAKE, dt=BF16, T=8, E=8, m=2, tau=1.0, idx=FAKE, top=FAKE, rest=FAKE):
    return lib.moe_distill_targets(logits, dt, T, E, m, tau, idx, top, rest, None)


def _distill(lib, logits=FAKE, dt=BF16, idx=FAKE, tl=FAKE, tdt=BF16, rest=None, mask=None, off=None, T=8, E=8, m=2,
             S=1, tau=1.0, loss=FAKE, tokens=FAKE, row=FAKE, stats=FAKE, ws=FAKE, nbytes=BIG):
    return lib.moe_distill_loss(logits, dt, idx, tl, tdt, rest, mask, off, T, E, m, S, tau, loss, tokens, row, stats,
                                ws, nbytes, None)


def _distill_bwd(lib, logits=FAKE, dt=BF16, idx=FAKE, tl=FAKE, tdt=BF16, stats=FAKE, tokens=FAKE, off=None, T=8, E=8,
                 m=2, S=1, tau=1.0, dloss=FAKE, base=None, out=FAKE):
    return lib.moe_distill_loss_backward(logits, dt, idx, tl, tdt, stats, tokens, off, T, E, m, S, tau, dloss, base,
                                         out, None)


SHAPES = [(dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), UNSUPPORTED), (dict(T=2 ** 31), UNSUPPORTED),
          (dict(dt=7), DTYPE), (dict(dt=-1), DTYPE), (dict(logits=None), INVALID_ARG)]
SEQS = [(dict(S=0), SHAPE), (dict(S=2), INVALID_ARG), (dict(S=2 ** 20 + 1, off=FAKE), UNSUPPORTED),
        (dict(off=ODD), INVALID_ARG)]
LISTS = [(dict(m=0), INVALID_ARG), (dict(m=9), INVALID_ARG), (dict(m=65, E=128), UNSUPPORTED),
         (dict(tau=0.0), INVALID_ARG), (dict(tau=-1.0), INVALID_ARG), (dict(tau=float("nan")), INVALID_ARG),
         (dict(tau=float("inf")), INVALID_ARG), (dict(tau=1e-4), INVALID_ARG)]
TOPK = [(dict(k=0), INVALID_ARG), (dict(k=9), INVALID_ARG), (dict(k=65, E=128), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", SHAPES + SEQS + TOPK + [
    (dict(scoring=2), INVALID_ARG), (dict(scoring=1, z=FAKE), UNSUPPORTED), (dict(idx=None), INVALID_ARG),
    (dict(loss=None), INVALID_ARG), (dict(counts=None), INVALID_ARG), (dict(tokens=None), INVALID_ARG),
    (dict(stats=None), INVALID_ARG), (dict(stats=ctypes.c_void_p(0x10004)), INVALID_ARG),
    (dict(logits=ODD), INVALID_ARG), (dict(idx=ODD), INVALID_ARG), (dict(mean=ODD), INVALID_ARG),
    (dict(ws=None), INVALID_ARG), (dict(ws=ctypes.c_void_p(0x10080)), INVALID_ARG), (dict(nbytes=256), INVALID_ARG)])
def test_balance_loss_refusals(lib, kw, want):
    assert _balance(lib, **kw) == want, lib.moe_last_error().decode()
    assert lib.moe_last_error()


@pytest.mark.parametrize("kw,want", SHAPES + SEQS + TOPK + [
    (dict(scoring=-1), INVALID_ARG), (dict(scoring=1, dz=FAKE), UNSUPPORTED), (dict(stats=None), INVALID_ARG),
    (dict(counts=None), INVALID_ARG), (dict(tokens=None), INVALID_ARG), (dict(dloss=None), INVALID_ARG),
    (dict(out=None), INVALID_ARG), (dict(out=ODD), INVALID_ARG), (dict(base=ODD), INVALID_ARG),
    (dict(stats=ctypes.c_void_p(0x10004)), INVALID_ARG)])
def test_balance_loss_backward_refusals(lib, kw, want):
    assert _balance_bwd(lib, **kw) == want, lib.moe_last_error().decode()


@pytest.mark.parametrize("kw,want", SHAPES + LISTS + [
    (dict(idx=None), INVALID_ARG), (dict(top=None), INVALID_ARG), (dict(rest=None), INVALID_ARG),
    (dict(top=ODD), INVALID_ARG), (dict(rest=ODD), INVALID_ARG)])
def test_distill_targets_refusals(lib, kw, want):
    assert _targets(lib, **kw) == want, lib.moe_last_error().decode()


@pytest.mark.parametrize("kw,want", SHAPES + SEQS + LISTS + [
    (dict(tdt=3), DTYPE), (dict(idx=None), INVALID_ARG), (dict(tl=None), INVALID_ARG), (dict(loss=None), INVALID_ARG),
    (dict(tokens=None), INVALID_ARG), (dict(row=None), INVALID_ARG), (dict(stats=None), INVALID_ARG),
    (dict(rest=ODD), INVALID_ARG), (dict(tl=ODD), INVALID_ARG), (dict(ws=None), INVALID_ARG),
    (dict(ws=ctypes.c_void_p(0x10080)), INVALID_ARG), (dict(nbytes=256), INVALID_ARG)])
def test_distill_loss_refusals(lib, kw, want):
    assert _distill(lib, **kw) == want, lib.moe_last_error().decode()


@pytest.mark.parametrize("kw,want", SHAPES + SEQS + LISTS + [
    (dict(tdt=3), DTYPE), (dict(idx=None), INVALID_ARG), (dict(tl=None), INVALID_ARG), (dict(stats=None), INVALID_ARG),
    (dict(tokens=None), INVALID_ARG), (dict(dloss=None), INVALID_ARG), (dict(out=None), INVALID_ARG),
    (dict(out=ODD), INVALID_ARG), (dict(base=ODD), INVALID_ARG)])
def test_distill_loss_backward_refusals(lib, kw, want):
    assert _distill_bwd(lib, **kw) == want, lib.moe_last_error().decode()


FAR = ctypes.c_void_p(0x40000)  # 8 x 8 BF16 elements are 128 bytes


@pytest.mark.parametrize("kw", [
    dict(out=FAKE), dict(out=ctypes.c_void_p(FAKE.value + 126)), dict(out=ctypes.c_void_p(FAKE.value - 126)),
    dict(out=FAR, base=ctypes.c_void_p(FAR.value + 16)), dict(out=FAR, base=ctypes.c_void_p(FAR.value - 126))])
def test_backward_refuses_overlapping_gradients(lib, kw):
    for call in (_balance_bwd, _distill_bwd):
        assert call(lib, **kw) == INVALID_ARG
        assert b"overlap" in lib.moe_last_error()


def test_empty_backward_and_targets_are_noops(lib):
    assert _balance_bwd(lib, logits=None, stats=None, counts=None, tokens=None, dloss=None, out=None, T=0) == OK
    assert _distill_bwd(lib, logits=None, idx=None, tl=None, stats=None, tokens=None, dloss=None, out=None, T=0) == OK
    assert _targets(lib, logits=None, idx=None, top=None, rest=None, T=0) == OK


def test_workspace_sizes(lib):
    assert lib.moe_balance_loss_workspace_size(16384, 64, 1) > 256
    assert lib.moe_balance_loss_workspace_size(1, 1, 1) > 256
    assert lib.moe_balance_loss_workspace_size(16384, 64, 100) > lib.moe_balance_loss_workspace_size(16384, 64, 1)
    for bad in ((-1, 8, 1), (8, 0, 1), (8, 1025, 1), (8, 8, 0), (8, 8, 2 ** 20 + 1)):
        assert lib.moe_balance_loss_workspace_size(*bad) == 0
    assert lib.moe_distill_loss_workspace_size(1, 1) > 256
    assert lib.moe_distill_loss_workspace_size(-1, 1) == 0 and lib.moe_distill_loss_workspace_size(1, 0) == 0


# ---- refusals of the binding -------------------------------------------------------
def test_binding_refuses_host_tensors_and_bad_names(lib):
    import top_routing_grouped_fp32_gb300 as moe
    logits, idx = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32)
    tg = moe.DistillTargets(idx, torch.zeros((4, 2)), None)
    with pytest.raises(ValueError):
        moe.moe_balance_loss(logits, idx)
    with pytest.raises(ValueError):
        moe.moe_distill_targets(logits, 2)
    with pytest.raises(ValueError):
        moe.moe_distill_loss(logits, tg)
    with pytest.raises(moe.MoeError) as e:
        moe.moe_balance_loss(torch.zeros(8), idx)
    assert e.value.status == SHAPE
    for bad in ("tanh", None, 0):
        with pytest.raises(moe.MoeError):
            moe.router_losses._scoring(bad)
