"""moe_mx_quantize and moe_mx_dequantize against the definition in 64 bits: every
bit of values and scales is determined by the input, so they are equal."""
import pytest
import torch

import mx_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _rows(R, C, dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((R, C), generator=g, device="cuda") * torch.exp(2 * torch.randn((R, 1), generator=g, device="cuda"))
    return x.to(dt)


def _check(moe, x, fmt, out=None):
    mx = moe.moe_mx_quantize(x, fmt, out=out)
    code, s = ref.quantize(x.double(), fmt)
    assert torch.equal(mx.scales.long(), s + 127)
    want = ref.values(code, s, fmt, x.shape[1])
    got = ref.held(mx)
    assert torch.equal(torch.nan_to_num(got, 7e77), torch.nan_to_num(want, 7e77))
    for dt in DT.values():
        back = moe.moe_mx_dequantize(mx, dt)
        assert torch.equal(torch.nan_to_num(back.float(), 7e33), torch.nan_to_num(want.to(dt).float(), 7e33))
    return mx


@pytest.mark.parametrize("dt", sorted(DT))
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 32), (3, 31), (5, 33), (2, 64), (7, 1001), (33, 512), (9, 513),
                                 (257, 96), (64, 2048)])
def test_rows(cuda_lib, dt, fmt, R, C):
    _check(cuda_lib, _rows(R, C, DT[dt], R + C), fmt)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("C", [32, 33])
def test_every_border(cuda_lib, fmt, C):
    """Ties, the largest values and the significands from which the next scale is taken, at
    every scale from the smallest on, both signs; neighbours of each on either side."""
    _, _, emax, top, bump = ref.FORMATS[fmt]
    g = ref.grid(fmt)
    points = torch.cat([g, (g[1:] + g[:-1]) / 2, torch.tensor([top, bump * 2.0 ** emax, 2.0 ** (emax + 1)], dtype=ref.F64)])
    points = points.to(torch.float32)
    near = torch.cat([points, torch.nextafter(points, torch.tensor(torch.inf)),
                      torch.nextafter(points, torch.tensor(-torch.inf)).clamp(min=0)])
    rows = []
    for e in (-149, -140, -130, -127, -126, -100, -2, 0, 1, 60, 118):
        for lead in (top, bump * 2.0 ** emax, 2.0 ** emax):  # what sets the scale
            for part in near.split(31):
                r = torch.zeros(C, dtype=ref.F64)
                r[0], r[1:1 + len(part)] = lead, part.double()
                rows.append((r * 2.0 ** e).float())
    x = torch.stack(rows).cuda()
    x[1::2] *= -1
    _check(cuda_lib, x, fmt)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("C", [96, 97])
@pytest.mark.parametrize("dt", sorted(DT))
def test_special_values(cuda_lib, fmt, C, dt):
    """Zeros, subnormals, the largest value of the type, and NaN and infinities, which take
    their own block and no other."""
    x = _rows(8, C, DT[dt], 3)
    x[0] = 0
    x[1] = -0.0
    x[2, 5], x[3, 40], x[4, C - 1] = float("nan"), float("inf"), float("-inf")
    x[5] = torch.finfo(DT[dt]).max
    x[6] = torch.finfo(DT[dt]).smallest_normal / 4
    mx = _check(cuda_lib, x, fmt)
    s = mx.scales.long()
    assert (s[0] == 0).all() and (s[1] == 0).all()
    assert s[2, 0] == s[3, 1] == s[4, (C - 1) // 32] == 255
    assert (s == 255).sum() == 3
    back = cuda_lib.moe_mx_dequantize(mx, torch.float32)
    assert torch.isnan(back).sum() == 32 + 32 + ((C - 1) % 32 + 1)


def test_odd_rows_end_in_a_zero_half(cuda_lib):
    mx = cuda_lib.moe_mx_quantize(_rows(50, 33, torch.float32), "mxfp4")
    assert ((mx.values[:, -1] >> 4) == 0).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("shift", [1, 3, 8])
def test_unaligned(cuda_lib, fmt, shift):
    """Rows that begin anywhere, and values at any byte."""
    moe = cuda_lib
    flat = _rows(1, 4 * 64 + shift, torch.bfloat16)[0]
    x = flat[shift:].view(4, 64)
    aligned = moe.moe_mx_quantize(x.clone(), fmt)
    n = aligned.values.numel()
    room = torch.zeros(n + shift, dtype=torch.uint8, device="cuda")
    out = moe.MxRows(room[shift:].view(aligned.values.shape), torch.empty_like(aligned.scales), fmt, 64)
    got = moe.moe_mx_quantize(x, fmt, out=out)
    assert got is out and torch.equal(out.values, aligned.values) and torch.equal(out.scales, aligned.scales)
    wide = torch.zeros(4 * 64 + shift, dtype=torch.bfloat16, device="cuda")
    o = wide[shift:].view(4, 64)
    assert moe.moe_mx_dequantize(out, torch.bfloat16, out=o) is o
    assert torch.equal(o, moe.moe_mx_dequantize(aligned, torch.bfloat16)) and (wide[:shift] == 0).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("C", [64, 65, 544])
@pytest.mark.parametrize("k", [1, 3])
def test_through_a_dispatch_map(cuda_lib, fmt, C, k):
    """Row r is token perm[r] / k; an entry that names no token gives zeros; repeated entries
    are fine."""
    moe = cuda_lib
    T = 11
    x = _rows(T, C, torch.float16)
    x[4, 3] = float("nan")
    mx = moe.moe_mx_quantize(x, fmt)
    perm = torch.randint(0, T * k, (40,), device="cuda", dtype=torch.int32)
    perm[3], perm[7], perm[8] = -1, T * k, T * k + 5
    for dt in DT.values():
        plain = moe.moe_mx_dequantize(mx, dt).float()
        want = torch.zeros((40, C), device="cuda")
        ok = (perm >= 0) & (perm < T * k)
        want[ok] = plain[perm[ok].long() // k]
        got = moe.moe_mx_dequantize(mx, dt, perm=perm, top_k=k).float()
        assert torch.equal(torch.nan_to_num(got, 7e33), torch.nan_to_num(want, 7e33))
    empty = moe.moe_mx_dequantize(mx, torch.float32, perm=perm[:0], top_k=k)
    assert empty.shape == (0, C)


def test_more_dimensions_and_no_rows(cuda_lib):
    moe = cuda_lib
    x = _rows(24, 64, torch.bfloat16)
    flat, deep = moe.moe_mx_quantize(x, "mxfp4"), moe.moe_mx_quantize(x.view(2, 3, 4, 64), "mxfp4")
    assert deep.shape == (2, 3, 4, 64) and torch.equal(deep.values.view(24, 32), flat.values)
    assert moe.moe_mx_dequantize(deep, torch.float32).shape == (2, 3, 4, 64)
    none = moe.moe_mx_quantize(x[:0], "mxfp8")
    assert none.shape == (0, 64) and moe.moe_mx_dequantize(none, torch.float32).shape == (0, 64)
    perm = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert (moe.moe_mx_dequantize(none, torch.float32, perm=perm) == 0).all()


def test_past_32_bits(cuda_lib):
    """More than 2^32 values: the last rows are what they are alone."""
    moe = cuda_lib
    C, R = 4096, (1 << 20) + 5
    x = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    x[-4:] = _rows(4, C, torch.bfloat16)
    mx, alone = moe.moe_mx_quantize(x, "mxfp8"), moe.moe_mx_quantize(x[-4:].clone(), "mxfp8")
    assert torch.equal(mx.values[-4:], alone.values) and torch.equal(mx.scales[-4:], alone.scales)
    assert not mx.values[:-4].any() and not mx.scales[:-4].any()
    back = moe.moe_mx_dequantize(mx, torch.bfloat16, out=x)
    assert torch.equal(back[-4:], moe.moe_mx_dequantize(alone, torch.bfloat16)) and not back[:-4].any()


def test_streams_and_graphs(cuda_lib):
    moe = cuda_lib
    x = _rows(300, 1024, torch.bfloat16)
    want = moe.moe_mx_quantize(x, "mxfp4")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = moe.moe_mx_quantize(x, "mxfp4", stream=s)
    s.synchronize()
    assert torch.equal(other.values, want.values) and torch.equal(other.scales, want.scales)
    out, back = moe.MxRows.empty(x.shape, "mxfp4"), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_mx_quantize(x, "mxfp4", out=out)
        moe.moe_mx_dequantize(out, x.dtype, out=back)
    x.copy_(_rows(300, 1024, torch.bfloat16, 9))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(back.double(), ref.rounded(x.double(), "mxfp4"))


def test_exchanged_tensors_are_seen(cuda_lib):
    """What an MxRows holds is looked at in every call."""
    moe = cuda_lib
    x = _rows(4, 64, torch.float32)
    mx = moe.moe_mx_quantize(x, "mxfp8")
    moe.moe_mx_quantize(x, "mxfp8", out=mx)
    mx.scales = mx.scales[:, :1].clone()
    with pytest.raises(moe.MoeError):
        moe.moe_mx_dequantize(mx, torch.float32)
    mx = moe.moe_mx_quantize(x, "mxfp8")
    mx.values.t_()
    with pytest.raises((moe.MoeError, ValueError)):
        moe.moe_mx_quantize(x, "mxfp8", out=mx)
    mx = moe.moe_mx_quantize(x, "mxfp8")
    mx.values = mx.values.cpu()
    with pytest.raises(ValueError):
        moe.moe_mx_dequantize(mx, torch.float32)
    with pytest.raises(moe.MoeError):
        moe.moe_mx_quantize(_rows(4, 32, torch.float32), "mxfp8", out=moe.MxRows.empty((4, 64), "mxfp8"))
    with pytest.raises(ValueError):
        moe.moe_mx_quantize(_rows(4, 64, torch.float32).t(), "mxfp8")
