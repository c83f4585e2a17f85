"""Each refusal of the router's losses by itself: the call is right but for one
argument, and the message names it.  Every buffer has an address of its own."""
import ctypes

import pytest

OK, INVALID_ARG, SHAPE, DTYPE, UNSUPPORTED = 0, 1, 2, 3, 4
BF16 = 2
T, E, K, S = 8, 128, 2, 3


def _at(n, off=0):
    """The n-th buffer: none is dereferenced, since every call below is refused."""
    return ctypes.c_void_p(0x10000000 + (n << 20) + off)


@pytest.fixture(scope="module")
def lib():
    from top_routing_grouped_fp32_gb300 import build as native_build
    from top_routing_grouped_fp32_gb300 import _lib
    native_build.build()
    return _lib.load()


# argument names in the order of the C ABI, with a valid value each
BALANCE = dict(logits=_at(0), dt=BF16, idx=_at(1), mask=_at(2), off=_at(3), T=T, E=E, k=K, S=S, scoring=0,
               loss=_at(4), z=_at(5), mean=_at(6), counts=_at(7), tokens=_at(8), stats=_at(9), ws=_at(10),
               nbytes=1 << 30, stream=None)
BALANCE_BWD = dict(logits=_at(0), dt=BF16, stats=_at(9), counts=_at(7), tokens=_at(8), off=_at(3), T=T, E=E, k=K,
                   S=S, scoring=0, dloss=_at(4), dz=_at(5), base=_at(11), out=_at(12), stream=None)
TARGETS = dict(logits=_at(0), dt=BF16, T=T, E=E, m=K, tau=1.0, idx=_at(1), top=_at(2), rest=_at(3), stream=None)
DISTILL = dict(logits=_at(0), dt=BF16, idx=_at(1), top=_at(2), tdt=BF16, rest=_at(3), mask=_at(4), off=_at(5), T=T,
               E=E, m=K, S=S, tau=1.0, loss=_at(6), tokens=_at(7), row=_at(8), stats=_at(9), ws=_at(10),
               nbytes=1 << 30, stream=None)
DISTILL_BWD = dict(logits=_at(0), dt=BF16, idx=_at(1), top=_at(2), tdt=BF16, stats=_at(9), tokens=_at(7),
                   off=_at(5), T=T, E=E, m=K, S=S, tau=1.0, dloss=_at(6), base=_at(11), out=_at(12), stream=None)
CALLS = {"moe_balance_loss": BALANCE, "moe_balance_loss_backward": BALANCE_BWD, "moe_distill_targets": TARGETS,
         "moe_distill_loss": DISTILL, "moe_distill_loss_backward": DISTILL_BWD}
# buffers that may be NULL, and the alignment of each in bytes (1: bytes, nothing to refuse)
MAY_BE_NULL = {"mask", "z", "mean", "dz", "base"}
ALIGN = dict(logits=2, idx=4, mask=1, off=4, loss=4, z=4, mean=4, counts=4, tokens=4, dloss=4, dz=4, base=2, out=2,
             top=2, rest=4, row=4)


def _cases():
    for name, args in CALLS.items():
        what = "teacher logits" if name == "moe_distill_targets" else "logits"
        cases = [(dict(dt=7), DTYPE, f"{what} dtype"), (dict(dt=-1), DTYPE, f"{what} dtype"),
                 (dict(T=-1), SHAPE, "T must be"), (dict(E=0), SHAPE, "E must be"),
                 (dict(E=1025), UNSUPPORTED, "E=1025"), (dict(T=2 ** 31), UNSUPPORTED, "exceeds")]
        if "k" in args:
            cases += [(dict(k=0), INVALID_ARG, "top_k"), (dict(k=E + 1), INVALID_ARG, "top_k"),
                      (dict(k=65), UNSUPPORTED, "top_k=65"), (dict(scoring=2), INVALID_ARG, "scoring must be"),
                      (dict(scoring=-1), INVALID_ARG, "scoring must be"), (dict(scoring=1), UNSUPPORTED, "z-loss")]
        else:
            cases += [(dict(m=0), INVALID_ARG, "top_m"), (dict(m=E + 1), INVALID_ARG, "top_m"),
                      (dict(m=65), UNSUPPORTED, "top_m=65")]
            cases += [(dict(tau=x), INVALID_ARG, "temperature")
                      for x in (0.0, -1.0, float("nan"), float("inf"), 1e-4, 1001.0)]
        if "tdt" in args:
            cases += [(dict(tdt=3), DTYPE, "teacher logits dtype")]
        if "S" in args:
            cases += [(dict(S=0), SHAPE, "num_seqs must be"), (dict(S=2 ** 20 + 1), UNSUPPORTED, "exceeds 2^20"),
                      (dict(off=None), INVALID_ARG, "needs seq_offsets"),
                      (dict(off=_at(3, 2)), INVALID_ARG, "seq_offsets must be 4-byte aligned")]
        if "ws" in args:
            cases += [(dict(ws=None), INVALID_ARG, "workspace"), (dict(ws=_at(10, 128)), INVALID_ARG, "workspace"),
                      (dict(nbytes=256), INVALID_ARG, "workspace")]
        for a, value in args.items():
            if not isinstance(value, ctypes.c_void_p) or a in ("ws", "off"):
                continue
            if a not in MAY_BE_NULL and not (a == "rest" and name == "moe_distill_loss"):
                cases.append(({a: None}, INVALID_ARG, "must be non-NULL"))
            step = 4 if a == "stats" and "m" in args else 8 if a == "stats" else ALIGN[a]
            if step > 1:
                cases.append(({a: ctypes.c_void_p(value.value + step // 2)}, INVALID_ARG, "misaligned"))
        if "out" in args:
            n = T * E * 2  # bytes
            for other in ("logits", "base"):
                p = args[other].value
                cases += [(dict(out=ctypes.c_void_p(p + d)), INVALID_ARG,
                           f"{'dlogits must not overlap logits' if other == 'logits' else 'base must be dlogits'}")
                          for d in (16, -16, n - 2, 2 - n)]
            cases.append((dict(out=args["logits"]), INVALID_ARG, "dlogits must not overlap logits"))
        for change, status, words in cases:
            yield pytest.param(name, change, status, words, id=f"{name}-{'-'.join(change)}-{words}")


@pytest.mark.parametrize("name,change,status,words", list(_cases()))
def test_refusal(lib, name, change, status, words):
    args = {**CALLS[name], **change}
    got = getattr(lib, name)(*args.values())
    message = lib.moe_last_error().decode()
    assert got == status, message
    assert words in message


@pytest.mark.parametrize("name", ["moe_balance_loss_backward", "moe_distill_targets", "moe_distill_loss_backward"])
def test_the_unchanged_call_is_right(lib, name):
    """With no rows the same arguments pass: nothing else in them is refused."""
    assert getattr(lib, name)(*{**CALLS[name], "T": 0}.values()) == OK
