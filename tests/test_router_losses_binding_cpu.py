"""What the binding of the router's losses remembers of a result's tensors, on
host tensors: each call sees what lies in them now."""
import pytest
import torch

from top_routing_grouped_fp32_gb300 import router_losses as rl

CPU = torch.device("cpu")
T, E, S, M = 6, 8, 2, 3


def _swap(t, new):
    """Exchanges what lies behind the Python object `t`."""
    torch.utils.swap_tensors(t, new)


# what a program can do to a tensor without replacing the attribute that holds it
EXCHANGES = {
    "half the bytes": lambda t: setattr(t, "data", t.data.to(torch.int16)),
    "another type of the size": lambda t: setattr(
        t, "data", t.data.view(torch.int32 if t.dtype == torch.float32 else torch.float32)),
    "transposed": lambda t: t.t_(),
    "strided": lambda t: t.set_(torch.zeros(t.shape + (2,), dtype=t.dtype)[..., 0]),
    "another shape": lambda t: t.resize_(t.numel(), 1),
    "swapped": lambda t: _swap(t, torch.zeros(t.shape, dtype=torch.float64)),
}


@pytest.mark.parametrize("what", sorted(EXCHANGES))
@pytest.mark.parametrize("kind,name", [("balance", "row_stats"), ("balance", "counts"), ("distill", "row_stats"),
                                       ("targets", "idx")])
def test_exchanged_memory_is_seen(kind, name, what):
    make = {"balance": lambda: (rl.BalanceLoss.empty(T, E, S, CPU), (T, E, S)),
            "distill": lambda: (rl.DistillLoss.empty(T, S, CPU), (T, S)),
            "targets": lambda: (rl.DistillTargets.empty(T, M, torch.bfloat16, CPU), (T, M))}
    out, sizes = make[kind]()
    names = [n for n, _, _ in out._tensors(*sizes)]
    first = out._pointers(CPU, *sizes)
    assert first[names.index(name)] == getattr(out, name).data_ptr()
    EXCHANGES[what](getattr(out, name))
    with pytest.raises((rl.MoeError, ValueError)):
        out._pointers(CPU, *sizes)
    with pytest.raises((rl.MoeError, ValueError)):  # a refusal is not remembered as a check
        out._pointers(CPU, *sizes)


def test_pointers_follow_their_tensors():
    """The same metadata in other memory is what a program may do: the new address is handed on."""
    out = rl.BalanceLoss.empty(T, E, S, CPU)
    a = out._pointers(CPU, T, E, S)
    assert a == out._pointers(CPU, T, E, S) and a[1] is None  # no z-loss
    out.row_stats.data = torch.zeros((T, 2))
    b = out._pointers(CPU, T, E, S)
    assert b[5] == out.row_stats.data_ptr() and b[:5] == a[:5]
    # a teacher's list may change its type: it is handed on with its own code
    tg = rl.DistillTargets.empty(T, M, torch.bfloat16, CPU)
    assert rl._list_args(tg, T, CPU)[1][2] == 2
    tg.logits.data = tg.logits.data.half()
    assert rl._list_args(tg, T, CPU)[1][1:] == (tg.logits.data_ptr(), 1)


def test_a_rest_knows_its_temperature():
    tg = rl.DistillTargets.empty(T, M, torch.bfloat16, CPU)
    assert tg.temperature is None
    assert rl.DistillTargets(tg.idx, tg.logits, tg.rest, 2.0).temperature == 2.0
    tg.temperature = 2.0
    tg.logits = tg.logits.clone()
    assert tg.temperature == 2.0
    tg.rest = tg.rest.clone()
    assert tg.temperature is None
    dis = rl.DistillLoss.empty(T, S, CPU)
    dis.temperature = 0.5
    dis.tokens = dis.tokens.clone()
    assert dis.temperature == 0.5
    dis.row_stats = dis.row_stats.clone()
    assert dis.temperature is None


def test_other_temperatures_are_refused():
    for kept, given in ((None, 2.0), (1, 1.0), (2.0, 2.0), (0.1, float(torch.tensor(0.1)))):  # the same in FP32
        rl._same_temperature(kept, given, "the forward")
    for kept, given in ((2.0, 1.0), (1.0, 1.0 + 2.0 ** -22), (1.0, float("nan"))):
        with pytest.raises(rl.MoeError) as e:
            rl._same_temperature(kept, given, "the forward")
        assert e.value.status == 1 and "temperature" in str(e.value)
