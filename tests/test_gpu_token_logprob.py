"""Log probabilities of given tokens, entropy, top alternatives and the gradient
against the formulas in 64 bits."""
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


def _logits(rows, vocab, dtype, seed=0, scale=2.5, pad=0, off=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 31 + rows * 7 + vocab)
    buf = torch.zeros(off + rows * (vocab + pad) + 8, dtype=dtype, device="cuda")
    x = buf[off:off + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]
    x.copy_(torch.randn(rows, vocab, generator=g, device="cuda") * scale)
    return x, g


def _tokens(g, rows, n, vocab, none=0.2):
    t = torch.randint(0, vocab, (rows, n), generator=g, device="cuda")
    t[torch.rand(rows, n, generator=g, device="cuda") < none] = -1
    return t


def _forward(dp, x, tok, inv_temp=1.0, top=0, entropy=True):
    rows, vocab = x.shape
    o = dict(logprob=torch.full(tok.shape, 9.0, device="cuda"),
             stats=torch.full((rows, 2), 9.0, device="cuda"))
    if entropy:
        o["entropy"] = torch.full((rows,), 9.0, device="cuda")
    if top:
        o["top_logprob"] = torch.full((rows, top), 9.0, device="cuda")
        o["top_index"] = torch.full((rows, top), -9, dtype=torch.int64, device="cuda")
    scratch = torch.full((max(1, dp.token_logprob_scratch_bytes(rows, vocab, top)),), 255,
                         dtype=torch.uint8, device="cuda")
    dp.token_logprob(x, tok, o["logprob"], o["stats"], scratch, entropy=o.get("entropy"),
                     top_logprob=o.get("top_logprob"), top_index=o.get("top_index"),
                     inv_temperature=inv_temp)
    dp.stream_status()
    return o


def _check_forward(dp, x, tok, inv_temp=1.0, top=0, entropy=True):
    o = _forward(dp, x, tok, inv_temp, top, entropy)
    want = ref.logprob(x, tok, inv_temp, top)
    for name, t in o.items():
        if name == "top_index":
            assert torch.equal(t.cpu(), want[name])
        else:
            value, bound = want[name]
            ref.within(t.cpu(), value, ref.stored(bound, value, torch.float32), name)
    return o


def _check_backward(dp, x, tok, o, inv_temp=1.0, entropy=True, scale=None, inplace=False, out=None):
    rows = x.shape[0]
    g = torch.Generator(device="cuda").manual_seed(5)
    dlp = torch.randn(tok.shape, generator=g, device="cuda")
    dent = torch.randn(rows, generator=g, device="cuda") if entropy else None
    ent = o["entropy"] if entropy else None
    state = None
    if scale is not None:
        state = torch.zeros(4, dtype=torch.int64, device="cuda")
        dp.loss_scale_init(state, init_scale=scale)
    src = x.clone() if inplace else x
    d = src if inplace else torch.full_like(x, 9.0) if out is None else out
    dp.token_logprob_backward(src, tok, o["stats"], d, dlogprob=dlp, entropy=ent, dentropy=dent,
                              inv_temperature=inv_temp, loss_scale=state)
    dp.stream_status()
    value, bound = ref.logprob_grad(x, tok, o["stats"], dlp, ent, dent, inv_temp, scale or 1.0)
    ref.within(d.cpu(), value, ref.stored(bound, value, x.dtype), "dlogits")
    return d


SHAPES = [(1, 1), (3, 2), (1, 31), (5, 33), (2, 1000), (1, 4097), (7, 8192), (3, 32001), (2, 50257),
          (40, 5003), (1, 131072), (300, 517)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_forward_and_gradient(dp, rows, vocab, dtype):
    x, g = _logits(rows, vocab, dtype)
    tok = _tokens(g, rows, 1, vocab)
    o = _check_forward(dp, x, tok, top=min(8, vocab))
    _check_backward(dp, x, tok, o)


@pytest.mark.parametrize("n", [0, 1, 2, 5, 33, 64])
@pytest.mark.parametrize("top", [0, 1, 3, 20, 32])
def test_given_tokens_and_alternatives(dp, n, top):
    for rows, vocab in ((4, 700), (2, 40001)):
        x, g = _logits(rows, vocab, torch.bfloat16, seed=n)
        tok = _tokens(g, rows, n, vocab)
        if n > 2:
            tok[:, 2] = tok[:, 0]  # one token given twice
            tok[:, 1] = vocab - 1
        for entropy in (False, True):
            o = _check_forward(dp, x, tok, top=top, entropy=entropy)
            if n:
                _check_backward(dp, x, tok, o, entropy=entropy)


@pytest.mark.parametrize("vocab", [32, 255, 256, 257, 640, 1024, 1025, 1500, 2048])
def test_alternatives_of_short_rows(dp, vocab):
    """Rows that do not reach every thread: most or all of their logits are candidates."""
    for dtype in DTYPES:
        x, g = _logits(6, vocab, dtype, seed=vocab)
        x[1] = x[1].round()       # few distinct logits
        x[2, 5:] = -math.inf      # fewer than are asked for
        tok = _tokens(g, 6, 1, vocab)
        for top in (17, 32):
            _check_forward(dp, x, tok, top=top)


@pytest.mark.parametrize("inv_temp", [0.5, 1.25, 3.0])
@pytest.mark.parametrize("scale", [None, 1.0, 1024.0])
def test_temperature_and_loss_scale(dp, inv_temp, scale):
    x, g = _logits(6, 3000, torch.float32)
    tok = _tokens(g, 6, 2, 3000)
    o = _check_forward(dp, x, tok, inv_temp, top=4)
    _check_backward(dp, x, tok, o, inv_temp, scale=scale)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,off", [(8, 0), (1, 0), (3, 1), (16, 8), (0, 5)])
def test_strides_alignment_and_in_place(dp, pad, off, dtype):
    x, g = _logits(9, 1001, dtype, pad=pad, off=off)
    tok = _tokens(g, 9, 2, 1001)
    o = _check_forward(dp, x, tok, top=5)
    a = _check_backward(dp, x, tok, o)
    b = _check_backward(dp, x, tok, o, inplace=True)
    assert torch.equal(a, b)
    # an output of another alignment than the logits', nothing written outside it
    buf = torch.full((9 * 1013 + 11,), 77.0, dtype=dtype, device="cuda")
    out = buf[3:3 + 9 * 1013].view(9, 1013)[:, :1001]
    c = _check_backward(dp, x, tok, o, out=out)
    assert torch.equal(a, c)
    assert bool((buf[3:3 + 9 * 1013].view(9, 1013)[:, 1001:] == 77).all()) and \
        bool((buf[:3] == 77).all() and (buf[3 + 9 * 1013:] == 77).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_masks(dp, dtype):
    """Masked entries (-Inf and the type's lowest value), rows masked but for one entry and
    rows masked entirely."""
    low = torch.finfo(dtype).min
    for vocab in (130, 5000, 40000):
        x, g = _logits(9, vocab, dtype)
        x[0, vocab // 2:] = -math.inf
        x[1, : vocab - 1] = -math.inf
        x[2] = -math.inf
        x[3, ::2] = low
        x[4] = low
        x[5, 1:] = low
        x[6] = torch.finfo(dtype).max
        x[7, ::3] = -math.inf
        x[7, 1::3] = low
        tok = _tokens(g, 9, 3, vocab, none=0.0)
        tok[:, 0] = vocab - 1
        o = _check_forward(dp, x, tok, top=7)
        _check_backward(dp, x, tok, o)
        assert bool((o["logprob"][2] == -math.inf).all()) and float(o["entropy"][2]) == 0.0
        assert o["top_index"][2].tolist() == list(range(7))
        o = _check_forward(dp, x, tok, 2.0, top=7)
        _check_backward(dp, x, tok, o, 2.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_ties_go_to_the_lowest_index(dp, dtype):
    for vocab in (64, 3001, 50257):
        x = torch.zeros(4, vocab, dtype=dtype, device="cuda")
        x[0, vocab // 3] = 1
        x[1, vocab - 1] = x[1, 7] = 2
        x[2, ::2] = -0.0
        x[3] = (torch.arange(vocab, device="cuda") % 5).to(dtype)
        tok = torch.zeros(4, 1, dtype=torch.int64, device="cuda")
        _check_forward(dp, x, tok, top=32)


@pytest.mark.parametrize("order", ["up", "down"])
def test_sorted_rows(dp, order):
    """The worst orders for a running list of the largest."""
    vocab = 20000
    x = torch.linspace(-8, 8, vocab, device="cuda").repeat(2, 1)
    if order == "down":
        x = x.flip(1).contiguous()
    _check_forward(dp, x, torch.zeros(2, 1, dtype=torch.int64, device="cuda"), top=32)
    _check_forward(dp, x.bfloat16(), torch.zeros(2, 1, dtype=torch.int64, device="cuda"), top=32)


@pytest.mark.parametrize("vocab", [200, 40000])
def test_non_finite_logits(dp, vocab):
    x, g = _logits(5, vocab, torch.bfloat16)
    x[0, 17] = math.nan
    x[1, 5] = math.inf
    x[2, 9], x[2, 3] = math.inf, math.nan
    x[3, vocab - 1], x[3, 100] = math.nan, math.nan
    tok = torch.full((5, 1), 2, dtype=torch.int64, device="cuda")
    o = _forward(dp, x, tok, top=3)
    for r in range(4):
        assert math.isnan(float(o["stats"][r, 1])) and math.isnan(float(o["entropy"][r]))
        assert math.isnan(float(o["logprob"][r, 0]))
    assert int(o["top_index"][0, 0]) == 17 and int(o["top_index"][1, 0]) == 5
    assert o["top_index"][2, :2].tolist() == [3, 9]
    assert o["top_index"][3, :2].tolist() == [100, vocab - 1]
    assert math.isfinite(float(o["logprob"][4, 0]))
    d = torch.empty_like(x)
    dp.token_logprob_backward(x, tok, o["stats"], d, dlogprob=torch.ones(5, 1, device="cuda"))
    dp.stream_status()
    assert bool(torch.isnan(d[:4]).any(1).all()) and bool(torch.isfinite(d[4]).all())


def test_tokens_out_of_range(dp):
    x, _ = _logits(3, 500, torch.float32)
    tok = torch.tensor([[499], [500], [1 << 40]], device="cuda")
    o = _forward(dp, x, tok)
    assert math.isfinite(float(o["logprob"][0, 0])) and bool(torch.isnan(o["logprob"][1:]).all())
    d = torch.empty_like(x)
    dp.token_logprob_backward(x, tok, o["stats"], d, dlogprob=torch.ones(3, 1, device="cuda"))
    dp.stream_status()
    assert bool(torch.isfinite(d[0]).all()) and bool(torch.isnan(d[1:]).all())


def test_rows_without_tokens_get_zeros(dp):
    x, _ = _logits(3, 4000, torch.float16)
    tok = torch.full((3, 2), -1, dtype=torch.int64, device="cuda")
    o = _check_forward(dp, x, tok)
    assert bool((o["logprob"] == 0).all())
    d = torch.full_like(x, 9.0)
    dp.token_logprob_backward(x, tok, o["stats"], d, dlogprob=torch.ones(3, 2, device="cuda"))
    dp.stream_status()
    assert bool((d == 0).all())


def test_no_rows(dp):
    x = torch.empty(0, 50, dtype=torch.bfloat16, device="cuda")
    tok = torch.empty(0, 1, dtype=torch.int64, device="cuda")
    o = _forward(dp, x, tok, top=2)
    dp.token_logprob_backward(x, tok, o["stats"], x, dlogprob=torch.empty(0, 1, device="cuda"))
    dp.stream_status()


def test_gradient_against_differences(dp):
    x, g = _logits(4, 300, torch.float32)
    x[1, 200:] = -math.inf
    tok = _tokens(g, 4, 2, 200)
    o = _forward(dp, x, tok, 1.25)
    gen = torch.Generator().manual_seed(1)
    dlp = torch.randn(4, 2, generator=gen)
    dent = torch.randn(4, generator=gen)
    d = torch.empty_like(x)
    dp.token_logprob_backward(x, tok, o["stats"], d, dlogprob=dlp.cuda(), entropy=o["entropy"],
                              dentropy=dent.cuda(), inv_temperature=1.25)
    dp.stream_status()
    xd, d = x.double().cpu(), d.double().cpu()

    def loss(z):
        r = ref.logprob(z, tok, 1.25, 0)
        return float((dlp.double() * r["logprob"][0]).sum() + (dent.double() * r["entropy"][0]).sum())

    for _ in range(4):
        v = torch.randn(4, 300, generator=gen, dtype=torch.float64)
        step = 1e-5
        fd = (loss(xd + step * v) - loss(xd - step * v)) / (2 * step)
        assert abs(float((d * v).sum()) - fd) <= 1e-7 + 300 * ref.EPS * float((d.abs() * v.abs()).sum())


def test_repeated_runs_give_the_same_bits(dp):
    for rows, vocab in ((1, 131072), (5, 50257), (700, 1003)):
        x, g = _logits(rows, vocab, torch.bfloat16)
        tok = _tokens(g, rows, 1, vocab)
        a, b = _forward(dp, x, tok, top=8), _forward(dp, x, tok, top=8)
        for n in a:
            assert torch.equal(a[n], b[n]), n


def test_offsets_pass_32_bits(dp):
    """Rows that start past 2^31 elements."""
    ld, vocab = 1_100_000_000, 3001
    buf = torch.empty(2 * ld + vocab, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (3, vocab), (ld, 1))
    y, g = _logits(3, vocab, torch.bfloat16)
    x.copy_(y)
    tok = _tokens(g, 3, 1, vocab)
    a, b = _forward(dp, x, tok, top=4), _forward(dp, y, tok, top=4)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    dlp = torch.ones(3, 1, device="cuda")
    d = torch.empty_like(y)
    dp.token_logprob_backward(y, tok, b["stats"], d, dlogprob=dlp)
    dp.token_logprob_backward(x, tok, b["stats"], x, dlogprob=dlp)
    dp.stream_status()
    assert torch.equal(x, d)
