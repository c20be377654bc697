"""Activations packed into 8 bits: the packed bytes and restored values equal the
definition's bit for bit; the weight gradient formed from them lies within the
bound of a 32-bit sum."""
from __future__ import annotations

import math

import pytest
import torch

from tests import ops_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def dp():
    import zero_mixed_precision_gb300 as mod
    return mod


def _rand(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * scale


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _padded(rows, cols, ld, dtype, offset=0):
    """A rows x cols view with row stride ld, its first element `offset` past an aligned
    address, over a buffer of a recognisable value."""
    buf = torch.full((offset + max(rows, 1) * ld + 32,), 77, dtype=dtype, device="cuda")
    return buf, buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]


def _check_pack(dp, x):
    rows, cols = x.shape
    codes, exps = dp.act8_empty(rows, cols)
    dp.act8_pack(x, codes, exps)
    back = torch.empty(rows, cols, dtype=x.dtype, device="cuda")
    dp.act8_unpack(codes, exps, back)
    dp.stream_status()
    want_c, want_e = ref.pack(x)
    assert torch.equal(codes.cpu(), want_c)
    assert torch.equal(exps.cpu(), want_e)
    value = ref.unpack(want_c, want_e)
    got = back.cpu().double()
    assert torch.equal(got.nan_to_num(nan=1e300), value.nan_to_num(nan=1e300))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 31), (5, 33), (7, 64), (1, 8200),
                                       (33, 1001), (130, 768), (257, 2048), (4099, 40)])
def test_pack_equals_the_definition(dp, rows, cols, dtype):
    g = _gen(rows * 1000 + cols)
    x = _rand(g, rows, cols) * torch.exp(_rand(g, cols, scale=2.0))
    _check_pack(dp, x.to(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
def test_pack_edge_values(dp, dtype):
    info = torch.finfo(dtype)
    sub = 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -133 if dtype == torch.bfloat16 \
        else 2.0 ** -149
    rows = [
        [0.0] * 40, [-0.0] * 40, [info.max] * 40, [info.min] + [1.0] * 39, [sub] * 40,
        [sub, -3 * sub, 5 * sub] + [0.0] * 37, [info.tiny] * 20 + [-info.tiny / 4] * 20,
        [127.5, 127.0, 126.5, -127.5, 0.5, 1.5, 2.5, -0.5] * 5,      # ties to even, the clamp
        [64.0, 63.75, 32.5, -33.5, 1.0, 0.25, 0.5, 0.75] * 5,
        [1.0] * 10 + [math.inf] + [1.0] * 29, [1.0] * 33 + [-math.inf] + [2.0] * 6,
        [math.nan] + [1.0] * 39, [1.0] * 31 + [math.nan] + [3.0] * 8,
    ]
    _check_pack(dp, torch.tensor(rows, dtype=torch.float64).to(dtype).cuda())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols,ld,off,ldc,offc", [(64, 72, 0, 64, 0), (61, 63, 1, 67, 3),
                                                  (96, 96, 3, 96, 0), (96, 97, 0, 104, 8),
                                                  (40, 48, 8, 41, 0)])
def test_pack_strides_and_alignment(dp, cols, ld, off, ldc, offc, dtype):
    rows = 19
    bufx, x = _padded(rows, cols, ld, dtype, off)
    x.copy_(_rand(_gen(5), rows, cols))
    bufc, codes = _padded(rows, cols, ldc, torch.int8, offc)
    bufe, exps = _padded(rows, -(-cols // 32), -(-cols // 32) + 3, torch.uint8, 1)
    dp.act8_pack(x, codes, exps)
    want_c, want_e = ref.pack(x)
    assert torch.equal(codes.cpu(), want_c) and torch.equal(exps.cpu(), want_e)
    bufb, back = _padded(rows, cols, ld, dtype, off)
    dp.act8_unpack(codes, exps, back)
    dp.stream_status()
    assert torch.equal(back.cpu().double(), ref.unpack(want_c, want_e))
    # nothing outside the matrices was written
    for buf, view, w in ((bufc, codes, ldc), (bufb, back, ld), (bufe, exps, exps.shape[1] + 3)):
        keep = torch.ones_like(buf, dtype=torch.bool)
        o = view.storage_offset()
        keep[o:o + rows * w].view(rows, w)[:, :view.shape[1]] = False
        assert bool((buf[keep] == 77).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [1, 9, 255, 257, 515, 1031])
@pytest.mark.parametrize("pad,off,padc,offc", [(0, 0, 0, 0), (1, 1, 0, 3), (3, 7, 5, 1),
                                               (6, 2, 2, 6), (8, 5, 8, 7)])
def test_pack_rows_at_any_alignment(dp, cols, pad, off, padc, offc, dtype):
    """Rows of several units that start anywhere, between neighbours that are NaN: those
    neither enter a block nor are written."""
    rows = 6
    bufx, x = _padded(rows, cols, cols + pad, dtype, off)
    bufx.fill_(math.nan)
    x.copy_(_rand(_gen(cols + pad), rows, cols))
    bufc, codes = _padded(rows, cols, cols + padc, torch.int8, offc)
    _, exps = dp.act8_empty(rows, cols)
    dp.act8_pack(x, codes, exps)
    want_c, want_e = ref.pack(x)
    assert torch.equal(codes.cpu(), want_c) and torch.equal(exps.cpu(), want_e)
    bufb, back = _padded(rows, cols, cols + pad, dtype, off)
    dp.act8_unpack(codes, exps, back)
    dp.stream_status()
    assert torch.equal(back.cpu().double(), ref.unpack(want_c, want_e))
    for buf, view, w in ((bufc, codes, cols + padc), (bufb, back, cols + pad)):
        keep = torch.ones_like(buf, dtype=torch.bool)
        o = view.storage_offset()
        keep[o:o + rows * w].view(rows, w)[:, :cols] = False
        assert bool((buf[keep] == 77).all())


def test_pack_error_bound_and_exact_restore(dp):
    """|value - x| <= step / 2 (<= step above 127.5 steps), and the restored value is exact in
    the source type: packing it again changes nothing."""
    for dtype in DTYPES:
        x = (_rand(_gen(8), 50, 640) * 10).to(dtype)
        codes, exps = dp.act8_empty(50, 640)
        dp.act8_pack(x, codes, exps)
        back = torch.empty_like(x)
        dp.act8_unpack(codes, exps, back)
        step = torch.pow(2.0, exps.double() - 127).repeat_interleave(32, 1)
        err = (back.double() - x.double()).abs()
        lim = torch.where(x.double().abs() > 127.5 * step, step, step / 2)
        assert bool((err <= lim).all())
        c2, e2 = dp.act8_empty(50, 640)
        dp.act8_pack(back, c2, e2)
        again = torch.empty_like(x)
        dp.act8_unpack(c2, e2, again)
        assert torch.equal(again, back)


def test_empty_matrices(dp):
    for rows, cols in ((0, 64), (5, 0), (0, 0)):
        x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        codes, exps = dp.act8_empty(rows, cols)
        dp.act8_pack(x, codes, exps)
        dp.act8_unpack(codes, exps, x)
    dp.stream_status()


# ---------------------------------------------------------------------------
# weight gradient
# ---------------------------------------------------------------------------

def _wgrad(dp, tokens, n, k, dtype, out, add=False, pad=0, off=0, seed=0, inplace=False):
    g = _gen(seed + tokens + n * 7 + k)
    x = (_rand(g, tokens, k) * torch.exp(_rand(g, k, scale=0.5))).to(dtype)
    codes, exps = dp.act8_empty(tokens, k)
    dp.act8_pack(x, codes, exps)
    _, dy = _padded(tokens, n, n + pad, dtype, off)
    dy.copy_(_rand(g, tokens, n, scale=0.05))
    dw = torch.full((n, k), math.nan, dtype=out, device="cuda")
    addend = _rand(g, n, k).to(out) if add else None
    if inplace:
        dw.copy_(addend)
    scratch = torch.empty(dp.act8_wgrad_scratch_bytes(tokens, n, k), dtype=torch.uint8,
                          device="cuda")
    dp.act8_wgrad(dy, codes, exps, dw, scratch, addend=dw if inplace else addend)
    dp.stream_status()
    v = ref.unpack(codes, exps).cuda()
    d = dy.double()
    want, mag = d.t() @ v, d.t().abs() @ v.abs()
    if add:
        want, mag = want + addend.double(), mag + addend.double().abs()
    # the operands are exact; a product of two of them is exact in fp32.  A sum of
    # `tokens` products in 32 bits, each addition off by at most one unit in the last
    # place of the larger of its parts (the tensor cores cut off rather than round):
    bound = (tokens + 8) * 2 * ref.EPS * mag
    ref.within(dw, want, ref.stored(bound, want, out), f"dw {tokens}x{n}x{k}")
    return dw, (dy, codes, exps, scratch, addend)


@pytest.mark.parametrize("dtype", DTYPES[:2])
@pytest.mark.parametrize("tokens,n,k", [(1, 1, 1), (1, 64, 64), (16, 128, 256), (17, 129, 257),
                                        (63, 128, 128), (64, 200, 96), (65, 31, 1000),
                                        (200, 384, 512), (257, 768, 768), (513, 100, 1547),
                                        (2100, 264, 320), (5000, 130, 72)])
def test_wgrad(dp, tokens, n, k, dtype):
    _wgrad(dp, tokens, n, k, dtype, dtype)


@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("add", [False, True])
def test_wgrad_output_types_and_addend(dp, out, add):
    for dtype in DTYPES[:2]:
        _wgrad(dp, 300, 256, 384, dtype, out, add)
        _wgrad(dp, 77, 131, 203, dtype, out, add)


@pytest.mark.parametrize("pad,off", [(8, 0), (24, 0), (1, 0), (8, 1), (13, 5)])
def test_wgrad_strides_and_alignment(dp, pad, off):
    _wgrad(dp, 150, 256, 320, torch.bfloat16, torch.float32, pad=pad, off=off)


@pytest.mark.parametrize("n,k,pad,off", [(515, 321, 0, 0), (301, 777, 4, 3), (8, 257, 1, 7)])
def test_wgrad_odd_rows(dp, n, k, pad, off):
    for dtype in DTYPES[:2]:
        _wgrad(dp, 90, n, k, dtype, torch.float32, pad=pad, off=off)


def test_wgrad_adds_in_place(dp):
    for out in DTYPES:
        _wgrad(dp, 130, 140, 260, torch.bfloat16, out, add=True, inplace=True)


def test_wgrad_without_tokens(dp):
    for add in (None, torch.ones(40, 72, device="cuda")):
        dy = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
        codes, exps = dp.act8_empty(0, 72)
        dw = torch.full((40, 72), 5.0, device="cuda")
        scratch = torch.empty(max(1, dp.act8_wgrad_scratch_bytes(0, 40, 72)), dtype=torch.uint8,
                              device="cuda")
        dp.act8_wgrad(dy, codes, exps, dw, scratch, addend=add)
        dp.stream_status()
        assert bool((dw == (0.0 if add is None else 1.0)).all())


def test_wgrad_is_reproducible_and_carries_non_finite_values(dp):
    a, args = _wgrad(dp, 4000, 256, 256, torch.bfloat16, torch.float32)
    dy, codes, exps, scratch, _ = args
    scratch.fill_(255)  # what the scratch held before does not matter
    b = torch.empty_like(a)
    dp.act8_wgrad(dy, codes, exps, b, scratch)
    assert torch.equal(a, b)
    exps[2000, 3] = 255  # an overflowed block of columns 96..127
    dp.act8_wgrad(dy, codes, exps, b, scratch)
    dp.stream_status()
    bad = torch.isnan(b)
    assert bool(bad[:, 96:128].all()) and not bool(bad[:, :96].any() or bad[:, 128:].any())
    dy[17, 5] = math.inf
    exps[2000, 3] = 120
    dp.act8_wgrad(dy, codes, exps, b, scratch)
    dp.stream_status()
    odd = ~torch.isfinite(b)
    assert bool(odd[5].all()) and not bool(odd[:5].any() or odd[6:].any())


def test_wgrad_against_differences(dp):
    """The weight gradient against central differences of sum(dy * (x W^T)) in 64 bits."""
    tokens, n, k = 40, 24, 48
    dw, (dy, codes, exps, _, _) = _wgrad(dp, tokens, n, k, torch.bfloat16, torch.float32)
    x, d = ref.unpack(codes, exps), dy.double().cpu()
    g = torch.Generator().manual_seed(3)
    w = torch.randn(n, k, generator=g, dtype=torch.float64)
    for _ in range(4):
        v = torch.randn(n, k, generator=g, dtype=torch.float64)
        h = 1e-4
        fd = ((d * (x @ (w + h * v).t())).sum() - (d * (x @ (w - h * v).t())).sum()) / (2 * h)
        got = (dw.double().cpu() * v).sum()
        mag = ((d.abs().t() @ x.abs()) * v.abs()).sum()
        assert abs(got - fd) <= (tokens + 16) * 2 * ref.EPS * mag + 1e-9 * abs(fd)


def test_side_stream_and_graph(dp):
    """Calls run on the stream given, and in a captured graph."""
    x = _rand(_gen(4), 512, 768).bfloat16()
    dy = _rand(_gen(6), 512, 256).bfloat16()
    codes, exps = dp.act8_empty(512, 768)
    dw = torch.empty(256, 768, device="cuda")
    scratch = torch.empty(dp.act8_wgrad_scratch_bytes(512, 256, 768), dtype=torch.uint8,
                          device="cuda")
    dp.act8_pack(x, codes, exps)
    dp.act8_wgrad(dy, codes, exps, dw, scratch)
    want = dw.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dw.zero_()
    codes.zero_()
    side.wait_stream(torch.cuda.current_stream())
    dp.act8_pack(x, codes, exps, stream=side)
    dp.act8_wgrad(dy, codes, exps, dw, scratch, stream=side)
    dp.stream_status(side)
    assert torch.equal(dw, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dp.act8_pack(x, codes, exps)
        dp.act8_wgrad(dy, codes, exps, dw, scratch)
    dw.zero_()
    graph.replay()
    dp.stream_status()
    assert torch.equal(dw, want)
