"""The block join and its gradient against the formulas in 64 bits."""
from __future__ import annotations

import itertools

import pytest
import torch

from tests import ops_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
SHAPES = [(1, 1), (1, 768), (2, 7), (3, 64), (5, 100), (33, 256), (4, 513), (7, 1547), (64, 2048),
          (3, 2056), (5, 4096), (2, 8192), (3, 9000), (1, 16384)]


@pytest.fixture(scope="module")
def dp():
    import zero_mixed_precision_gb300 as mod
    return mod


class Case:
    """The inputs of one join."""

    def __init__(self, rows, cols, dtype, *, post=True, pre=True, weights=True, gate_rows=0,
                 gate=True, param=None, pad=0, off=0, res=1.0, branch=0.5, seed=0, zero_row=None):
        g = torch.Generator(device="cuda").manual_seed(seed * 7919 + rows * 31 + cols)
        param = param or dtype

        def rn(*s, scale=1.0):
            return torch.randn(*s, generator=g, device="cuda") * scale

        def mat(scale):
            buf = torch.zeros(off + rows * (cols + pad) + 8, dtype=dtype, device="cuda")
            m = buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
            m.copy_(rn(rows, cols, scale=scale))
            return m

        self.rows, self.cols, self.dtype, self.pad, self.off = rows, cols, dtype, pad, off
        self.h, self.y = mat(1.0), mat(0.4)
        if zero_row is not None:
            self.h[zero_row] = 0
            self.y[zero_row] = 0
        self.dh_out, self.du = mat(0.1), mat(0.1)
        self.w_post = (1 + rn(cols, scale=0.2)).to(param) if weights and post else None
        self.w_pre = (1 + rn(cols, scale=0.2)).to(param) if weights and pre else None
        ng = 1 if gate_rows == 0 else -(-rows // gate_rows)
        self.gate = rn(ng, cols).to(param) if gate else None
        self.param, self.post, self.pre, self.gate_rows = param, post, pre, gate_rows
        self.res, self.branch, self.eps = res, branch, 1e-5

    def new(self, dtype=None):
        t = torch.full((self.off + self.rows * (self.cols + self.pad) + 8,), 9.0,
                       dtype=dtype or self.dtype, device="cuda")
        return t[self.off:self.off + self.rows * (self.cols + self.pad)].view(
            self.rows, self.cols + self.pad)[:, :self.cols]

    def forward(self, dp, keep8=False, inplace=False):
        o = {"h_out": self.h.clone() if inplace else self.new()}
        h = o["h_out"] if inplace else self.h
        if self.post:
            o["rstd_post"] = torch.empty(self.rows, device="cuda")
        if self.pre:
            o["u"], o["rstd_pre"] = self.new(), torch.empty(self.rows, device="cuda")
        packs = {}
        if keep8:
            packs = {n: dp.act8_empty(self.rows, self.cols) for n in
                     ("y8", "h8", *(["u8"] if self.pre else []))}
        dp.block_join(h, self.y, o["h_out"], eps=self.eps, rstd_post=o.get("rstd_post"),
                      w_post=self.w_post, gate=self.gate, gate_rows=self.gate_rows,
                      res_scale=self.res, branch_scale=self.branch, u=o.get("u"),
                      rstd_pre=o.get("rstd_pre"), w_pre=self.w_pre, **packs)
        dp.stream_status()
        return o, packs

    def want(self):
        return ref.join(self.h, self.y, eps=self.eps, post=self.post, w_post=self.w_post,
                        gate=self.gate, gate_rows=self.gate_rows, res_scale=self.res,
                        branch_scale=self.branch, pre=self.pre, w_pre=self.w_pre)

    def check_forward(self, dp, **kw):
        o, packs = self.forward(dp, **kw)
        want = self.want()
        assert set(want) == set(o)
        for name, (value, bound) in want.items():
            dt = torch.float32 if name.startswith("rstd") else self.dtype
            ref.within(o[name].cpu(), value, ref.stored(bound, value, dt), name)
        return o, packs

    def backward(self, dp, y, h, r1, r2, inplace=False):
        o = {"dy": self.new(), "dh": self.dh_out.clone() if inplace else self.new()}
        kw = {}
        nan = float("nan")
        if self.post:
            o["dw_post"] = torch.full((self.cols,), nan, dtype=self.param, device="cuda")
            kw.update(rstd_post=r2, w_post=self.w_post, dw_post=o["dw_post"])
        if self.pre:
            o["dw_pre"] = torch.full((self.cols,), nan, dtype=self.param, device="cuda")
            kw.update(du=self.du, h_out=h, rstd_pre=r1, w_pre=self.w_pre, dw_pre=o["dw_pre"])
        if self.gate is not None:
            o["dgate"] = torch.full_like(self.gate, nan)
            kw.update(gate=self.gate, gate_rows=self.gate_rows, dgate=o["dgate"])
        scratch = torch.full((dp.block_join_scratch_bytes(self.rows, self.cols, self.gate_rows),),
                             255, dtype=torch.uint8, device="cuda")
        dp.block_join_backward(o["dh"] if inplace else self.dh_out, y, o["dy"], o["dh"], scratch,
                               res_scale=self.res, branch_scale=self.branch, **kw)
        dp.stream_status()
        return o

    def check_backward(self, dp, y, h, r1, r2, yv=None, hv=None, **kw):
        """y, h: what the call gets; yv, hv: the values they stand for."""
        o = self.backward(dp, y, h, r1, r2, **kw)
        want = ref.join_grad(self.dh_out, self.du if self.pre else None, y if yv is None else yv,
                             (h if hv is None else hv) if self.pre else None, r1=r1, r2=r2,
                             w_post=self.w_post, w_pre=self.w_pre, gate=self.gate,
                             gate_rows=self.gate_rows, res_scale=self.res,
                             branch_scale=self.branch)
        for name, t in o.items():
            value, bound = want[name]
            ref.within(t.cpu(), value, ref.stored(bound, value, t.dtype), name)
        return o

    def check_both(self, dp):
        o, _ = self.check_forward(dp)
        self.check_backward(dp, self.y, o["h_out"], o.get("rstd_pre"), o.get("rstd_post"))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_join_and_gradient(dp, rows, cols, dtype):
    Case(rows, cols, dtype).check_both(dp)


@pytest.mark.parametrize("post,pre,weights,gate", list(itertools.product([False, True], repeat=4)))
def test_parts_left_out(dp, post, pre, weights, gate):
    for cols in (264, 131):
        Case(9, cols, torch.bfloat16, post=post, pre=pre, weights=weights, gate=gate).check_both(dp)


@pytest.mark.parametrize("gate_rows", [0, 1, 2, 3, 7, 100, 350, 699, 700, 5000])
@pytest.mark.parametrize("cols", [96, 301])
def test_gate_rows(dp, gate_rows, cols):
    """Gate rows that lie inside a run of rows, that cross its border, and that span many."""
    Case(700, cols, torch.float32, gate_rows=gate_rows).check_both(dp)


@pytest.mark.parametrize("rows", [303, 304, 305, 608, 609, 1000])
def test_row_counts_around_the_parts(dp, rows):
    Case(rows, 72, torch.bfloat16, gate_rows=50, param=torch.float32).check_both(dp)


@pytest.mark.parametrize("param", DTYPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_parameter_types(dp, dtype, param):
    Case(20, 512, dtype, param=param, gate_rows=1).check_both(dp)
    Case(20, 77, dtype, param=param).check_both(dp)


@pytest.mark.parametrize("pad,off", [(8, 0), (1, 0), (0, 1), (8, 3), (13, 8)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_alignment(dp, dtype, pad, off):
    c = Case(11, 256, dtype, pad=pad, off=off)
    c.check_both(dp)
    c.check_forward(dp, keep8=True)


@pytest.mark.parametrize("res,branch", [(0.0, 1.0), (1.0, 0.0), (0.7071, -2.0)])
def test_scales(dp, res, branch):
    Case(6, 320, torch.float32, res=res, branch=branch).check_both(dp)


def test_rows_of_zeros(dp):
    """A zero row: rstd = 1 / sqrt(eps), finite everything."""
    Case(5, 192, torch.float32, zero_row=2).check_both(dp)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 768), (9, 100), (40, 2048), (3, 1547), (2, 8192),
                                       (2, 10000)])
def test_kept_checkpoints_are_the_packed_outputs(dp, rows, cols, dtype):
    """y8, h8 and u8 are bit for bit what packing y, h_out and u gives."""
    c = Case(rows, cols, dtype)
    o, packs = c.check_forward(dp, keep8=True)
    for name, src in (("y8", c.y), ("h8", o["h_out"]), ("u8", o["u"])):
        codes, exps = dp.act8_empty(rows, cols)
        dp.act8_pack(src, codes, exps)
        assert torch.equal(packs[name][0], codes) and torch.equal(packs[name][1], exps), name


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,gate_rows", [(1, 64, 0), (40, 2048, 0), (9, 1547, 4),
                                                 (320, 104, 50), (3, 8192, 1)])
def test_gradient_from_checkpoints(dp, rows, cols, gate_rows, dtype):
    c = Case(rows, cols, dtype, gate_rows=gate_rows)
    o, packs = c.forward(dp, keep8=True)
    yv, hv = (ref.unpack(*packs[n]) for n in ("y8", "h8"))
    r1, r2 = o["rstd_pre"], o["rstd_post"]
    c.check_backward(dp, packs["y8"], packs["h8"], r1, r2, yv, hv)
    c.check_backward(dp, packs["y8"], o["h_out"], r1, r2, yv, None)
    c.check_backward(dp, c.y, packs["h8"], r1, r2, None, hv)


@pytest.mark.parametrize("cols", [256, 131])
def test_in_place(dp, cols):
    c = Case(12, cols, torch.bfloat16)
    a, _ = c.forward(dp)
    b, _ = c.forward(dp, inplace=True)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    x = c.backward(dp, c.y, a["h_out"], a["rstd_pre"], a["rstd_post"])
    z = c.backward(dp, c.y, a["h_out"], a["rstd_pre"], a["rstd_post"], inplace=True)
    for n in x:
        assert torch.equal(x[n], z[n]), n


def test_dh_and_parameter_gradients_may_be_left_out(dp):
    c = Case(30, 200, torch.bfloat16)
    o, _ = c.forward(dp)
    full = c.backward(dp, c.y, o["h_out"], o["rstd_pre"], o["rstd_post"])
    dy = c.new()
    scratch = torch.empty(dp.block_join_scratch_bytes(30, 200, 0), dtype=torch.uint8, device="cuda")
    dp.block_join_backward(c.dh_out, c.y, dy, None, scratch, rstd_post=o["rstd_post"],
                           w_post=c.w_post, gate=c.gate, branch_scale=c.branch, du=c.du,
                           h_out=o["h_out"], rstd_pre=o["rstd_pre"], w_pre=c.w_pre)
    dp.stream_status()
    assert torch.equal(dy, full["dy"])


def test_no_rows(dp):
    c = Case(0, 64, torch.bfloat16)
    c.forward(dp)
    o = c.backward(dp, c.y, c.h, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"))
    for n in ("dw_post", "dw_pre", "dgate"):
        assert bool((o[n] == 0).all()), n


def test_non_finite_rows_stay_in_their_rows(dp):
    c = Case(8, 256, torch.bfloat16)
    c.y[3, 17] = float("inf")
    c.h[5, 2] = float("nan")
    o, packs = c.forward(dp, keep8=True)
    for n in ("h_out", "u"):
        ok = torch.isfinite(o[n]).all(1).cpu()
        assert ok.tolist() == [True, True, True, False, True, False, True, True]
    assert int(packs["y8"][1][3, 0]) == 255 and int(packs["h8"][1][5, 0]) == 255
    g = c.backward(dp, packs["y8"], packs["h8"], o["rstd_pre"], o["rstd_post"])
    assert not bool(torch.isfinite(g["dy"][3]).all() or torch.isfinite(g["dh"][5]).all())
    assert not bool(torch.isfinite(g["dw_post"]).all())
    assert bool(torch.isfinite(g["dy"][[0, 1, 2, 4, 6, 7]]).all())


def test_repeated_runs_give_the_same_bits(dp):
    c = Case(1000, 384, torch.bfloat16, gate_rows=130, param=torch.float32)
    o, _ = c.forward(dp)
    args = (c.y, o["h_out"], o["rstd_pre"], o["rstd_post"])
    a, b = c.backward(dp, *args), c.backward(dp, *args)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_gradient_against_differences(dp):
    """fp32 gradients against central differences of the join in 64 bits, along random
    directions of every input and parameter."""
    rows, cols = 6, 40
    c = Case(rows, cols, torch.float32, gate_rows=4)
    o, _ = c.forward(dp)
    g = c.backward(dp, c.y, o["h_out"], o["rstd_pre"], o["rstd_post"])
    base = {n: getattr(c, n).double().cpu() for n in ("h", "y", "w_post", "w_pre", "gate")}
    name = {"h": "dh", "y": "dy", "w_post": "dw_post", "w_pre": "dw_pre", "gate": "dgate"}
    dho, du = c.dh_out.double().cpu(), c.du.double().cpu()

    def loss(p):
        r = ref.join(p["h"], p["y"], eps=c.eps, post=True, w_post=p["w_post"], gate=p["gate"],
                     gate_rows=4, res_scale=c.res, branch_scale=c.branch, pre=True,
                     w_pre=p["w_pre"])
        return float((dho * r["h_out"][0]).sum() + (du * r["u"][0]).sum())

    gen = torch.Generator().manual_seed(2)
    for key in base:
        v = torch.randn(base[key].shape, generator=gen, dtype=torch.float64)
        step = 1e-5
        fd = (loss({**base, key: base[key] + step * v}) -
              loss({**base, key: base[key] - step * v})) / (2 * step)
        t = g[name[key]].double().cpu()
        # the difference quotient's own error is of order step^2 and 1e-16 / step; the
        # gradient is off by at most a few hundred fp32 roundings of its terms
        assert abs(float((t * v).sum()) - fd) <= 1e-7 + 300 * ref.EPS * float((t.abs() * v.abs()).sum())


def test_long_strides_pass_32_bits(dp):
    """Element offsets past 2^31: three rows 1.2e9 elements apart."""
    ld, cols = 1_200_000_000, 512
    buf = torch.empty(2 * ld + cols, dtype=torch.bfloat16, device="cuda")
    h = torch.as_strided(buf, (3, cols), (ld, 1))
    c = Case(3, cols, torch.bfloat16)
    h.copy_(c.h)
    o, _ = c.forward(dp)
    out = {n: torch.empty_like(o["h_out"]) for n in ("h_out", "u")}
    rs = [torch.empty(3, device="cuda") for _ in range(2)]
    dp.block_join(h, c.y, out["h_out"], eps=c.eps, rstd_post=rs[0], w_post=c.w_post, gate=c.gate,
                  res_scale=c.res, branch_scale=c.branch, u=out["u"], rstd_pre=rs[1],
                  w_pre=c.w_pre)
    dp.stream_status()
    assert torch.equal(out["h_out"], o["h_out"]) and torch.equal(out["u"], o["u"])
    codes, exps = dp.act8_empty(3, cols)
    c2, e2 = dp.act8_empty(3, cols)
    dp.act8_pack(h, codes, exps)
    dp.act8_pack(c.h, c2, e2)
    dp.stream_status()
    assert torch.equal(codes, c2) and torch.equal(exps, e2)
