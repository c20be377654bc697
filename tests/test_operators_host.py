"""The training-side operators on the host (no GPU): argument blocks laid out as the
header declares them, scratch sizes, refusals before any launch, and the
definitions used as the oracle checked against torch."""
from __future__ import annotations

import ctypes
import math
import os
import subprocess

import pytest
import torch

from tests import ops_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dpopt.h")


@pytest.fixture(scope="module")
def dp():
    import __graft_entry__
    __graft_entry__.build_module().build()
    import zero_mixed_precision_gb300 as mod
    return mod


def test_argument_blocks_match_the_header(dp, tmp_path):
    blocks = {"dpopt_matrix": dp.binding.Matrix, "dpopt_act8": dp.binding.Act8,
              "dpopt_block_join_args": dp.binding.BlockJoinArgs,
              "dpopt_block_join_grad_args": dp.binding.BlockJoinGradArgs}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "dpopt.h"', "int main(void){"]
    for c, py in blocks.items():
        lines.append(f'printf("{c} size %zu\\n", sizeof({c}));')
        lines += [f'printf("{c} {n} %zu\\n", offsetof({c}, {n}));' for n, _ in py._fields_]
    lines.append("return 0;}")
    src, exe = tmp_path / "t.c", tmp_path / "t"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), str(src), "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    for line in out.splitlines():
        c, field, value = line.split()
        py = blocks[c]
        assert int(value) == (ctypes.sizeof(py) if field == "size" else getattr(py, field).offset)


def test_packed_argument_layouts_match_the_blocks(dp):
    """The wrappers pack the argument blocks with struct formats: the same sizes and, field
    by field, the same bytes as the ctypes structures."""
    for fmt, py in ((dp.operators._JOIN, dp.binding.BlockJoinArgs),
                    (dp.operators._JOIN_GRAD, dp.binding.BlockJoinGradArgs)):
        assert fmt.size == ctypes.sizeof(py)
        values = []

        def leaves(kind):
            for _, t in kind._fields_:
                if hasattr(t, "_fields_"):
                    leaves(t)
                else:
                    v = len(values) + 1
                    values.append(float(v) if t is ctypes.c_float else v)

        leaves(py)
        raw = fmt.pack(*values)
        obj, it = py.from_buffer_copy(raw), iter(values)

        def check(o):
            for n, t in o._fields_:
                x = getattr(o, n)
                if hasattr(t, "_fields_"):
                    check(x)
                else:
                    assert x == next(it), n

        check(obj)


# fake, never-dereferenced device addresses
A = [0x10_0000_0000 + i * 0x1_0000_0000 for i in range(32)]


def test_scratch_sizes(dp):
    for fn, ok, bad in (
            (dp.dpopt_act8_wgrad_scratch_bytes, (100, 64, 64), [(-1, 2, 2), (2, -1, 2), (2, 2, -1)]),
            (dp.dpopt_block_join_scratch_bytes, (100, 64, 0), [(-1, 2, 0), (2, -1, 0), (2, 2, -1)]),
            (dp.dpopt_token_logprob_scratch_bytes, (10, 1000, 8),
             [(-1, 10, 0), (1, 0, 0), (1, 10, 11), (1, 10, -1), (1, 100, 33)])):
        rc, nbytes = fn(*ok)
        assert rc == 0 and nbytes >= 0
        for b in bad:
            assert fn(*b)[0] == dp.DPOPT_ERR_INVALID_ARG, (fn, b)
    assert dp.dpopt_block_join_scratch_bytes(5, 16385, 0)[0] == dp.DPOPT_ERR_UNSUPPORTED
    with pytest.raises(dp.DpoptError):
        dp.block_join_scratch_bytes(-1, 4)


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), 1), (dict(cols=-1), 1), (dict(dtype=9), 1), (dict(x=0), 1), (dict(codes=0), 1),
    (dict(exps=0), 1), (dict(x=A[0] + 1), 1), (dict(ldx=63), 1), (dict(ld_codes=63), 1),
    (dict(ld_exps=1), 1), (dict(codes=A[0] + 64), 1), (dict(exps=A[1] + 5), 1),
    (dict(ldx=1 << 62), 1),
])
def test_pack_refuses(dp, over, code):
    a = dict(x=A[0], dtype=0, rows=8, cols=64, ldx=64, codes=A[1], ld_codes=64, exps=A[2],
             ld_exps=2)
    a.update(over)
    assert dp.dpopt_act8_pack(*a.values(), 0) == code
    assert dp.dpopt_last_error() != ""
    if "exps" in over and over["exps"]:
        return  # two arrays that unpacking only reads may overlap
    assert dp.dpopt_act8_unpack(a["codes"], a["ld_codes"], a["exps"], a["ld_exps"], a["rows"],
                                a["cols"], a["x"], a["dtype"], a["ldx"], 0) == code


@pytest.mark.parametrize("over,code", [
    (dict(tokens=-1), 1), (dict(n=-1), 1), (dict(k=-1), 1), (dict(dtype=7), 1),
    (dict(dtype=1, ), 2), (dict(out_dtype=7), 1), (dict(dy=0), 1), (dict(codes=0), 1),
    (dict(exps=0), 1), (dict(dw=0), 1), (dict(dy=A[0] + 1), 1), (dict(dw=A[3] + 1), 1),
    (dict(ld_dy=63), 1), (dict(ld_codes=95), 1), (dict(ld_exps=2), 1), (dict(ld_dw=95), 1),
    (dict(addend=A[4] + 1), 1), (dict(addend=A[4], ld_addend=3), 1),
    (dict(addend=A[3] + 4, ld_addend=96), 1), (dict(dw=A[0]), 1), (dict(dw=A[1]), 1),
    (dict(tokens=1 << 31), 2),
    (dict(tokens=(1 << 31) - 1, k=(1 << 31) - 1, ld_codes=(1 << 31) - 1, ld_exps=1 << 26,
          ld_dw=(1 << 31) - 1), 2),
])
def test_wgrad_refuses(dp, over, code):
    a = dict(dy=A[0], dtype=0, ld_dy=64, codes=A[1], ld_codes=96, exps=A[2], ld_exps=3, tokens=70,
             n=64, k=96, dw=A[3], out_dtype=0, ld_dw=96, addend=0, ld_addend=0, scratch=A[5],
             scratch_bytes=1 << 40)
    a.update(over)
    assert dp.dpopt_act8_wgrad(*a.values(), 0) == code
    assert dp.dpopt_last_error() != ""


def test_wgrad_refuses_a_small_or_misaligned_scratch(dp):
    a = [A[0], 0, 8192, A[1], 8192, A[2], 256, 16384, 8192, 8192, A[3], 0, 8192, 0, 0]
    need = dp.act8_wgrad_scratch_bytes(16384, 8192, 8192)
    if need:
        for scratch, size in ((0, need), (A[5], need - 1), (A[5] + 16, need), (A[3], need)):
            assert dp.dpopt_act8_wgrad(*a, scratch, size, 0) == dp.DPOPT_ERR_INVALID_ARG


def _join_args(dp, **over):
    M, E = dp.binding.Matrix, dp.binding.Act8
    a = dp.binding.BlockJoinArgs(
        rows=10, cols=64, dtype=0, param_dtype=0, eps=1e-5, res_scale=1, branch_scale=1,
        gate_rows=0, h=M(A[0], 64), y=M(A[1], 64), gate=M(A[2], 64), h_out=M(A[3], 64),
        u=M(A[4], 64), w_post=A[5], w_pre=A[6], rstd_post=A[7], rstd_pre=A[8],
        y8=E(A[9], 64, A[10], 2))
    for k, v in over.items():
        setattr(a, k, v)
    return a


def test_join_refuses(dp):
    M, E = dp.binding.Matrix, dp.binding.Act8
    bad = [dict(rows=-1), dict(cols=-1), dict(dtype=5), dict(param_dtype=5), dict(gate_rows=-1),
           dict(eps=-1.0), dict(eps=math.nan), dict(res_scale=math.inf),
           dict(branch_scale=math.nan), dict(h=M(0, 64)), dict(y=M(0, 64)), dict(h_out=M(0, 64)),
           dict(h=M(A[0], 63)), dict(u=M(A[4] + 1, 64)), dict(h_out=M(A[0], 65)),
           dict(h_out=M(A[1], 64)), dict(u=M(A[3], 64)), dict(rstd_pre=0), dict(rstd_post=0),
           dict(rstd_pre=A[8] + 2), dict(w_post=A[5] + 1), dict(u=M(0, 0)),
           dict(y8=E(A[9], 64, 0, 2)), dict(y8=E(A[9], 60, A[10], 2)),
           dict(y8=E(A[9], 64, A[10], 1)), dict(y8=E(A[0], 64, A[10], 2)),
           dict(gate_rows=3, gate=M(A[2], 8)), dict(w_pre=A[4] + 16)]
    for over in bad:
        assert dp.dpopt_block_join(_join_args(dp, **over)) == dp.DPOPT_ERR_INVALID_ARG, over
    assert dp.dpopt_block_join(None) == dp.DPOPT_ERR_INVALID_ARG
    big = _join_args(dp, cols=16385)
    assert dp.dpopt_block_join(big) == dp.DPOPT_ERR_UNSUPPORTED


def _grad_args(dp, **over):
    M = dp.binding.Matrix
    a = dp.binding.BlockJoinGradArgs(
        rows=10, cols=64, dtype=0, param_dtype=0, res_scale=1, branch_scale=1, gate_rows=0,
        dh_out=M(A[0], 64), du=M(A[1], 64), y=M(A[2], 64), h_out=M(A[3], 64), gate=M(A[4], 64),
        dh=M(A[5], 64), dy=M(A[6], 64), dgate=M(A[7], 64), w_post=A[8], w_pre=A[9],
        rstd_post=A[10], rstd_pre=A[11], dw_post=A[12], dw_pre=A[13], scratch=A[14],
        scratch_bytes=1 << 30)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def test_join_gradient_refuses(dp):
    M, E = dp.binding.Matrix, dp.binding.Act8
    need = dp.block_join_scratch_bytes(10, 64, 0)
    eight = E(A[20], 64, A[21], 2)
    bad = [dict(rows=-1), dict(dtype=5), dict(param_dtype=5), dict(gate_rows=-2),
           dict(res_scale=math.nan), dict(dh_out=M(0, 64)), dict(dy=M(0, 64)), dict(y=M(0, 64)),
           dict(y8=eight), dict(h8=eight), dict(h_out=M(0, 64)), dict(du=M(0, 64)),
           dict(rstd_pre=0), dict(rstd_post=0), dict(gate=M(0, 64)), dict(dh=M(A[0], 65)),
           dict(dy=M(A[0], 64)), dict(dy=M(A[2], 64)), dict(dw_post=A[8]), dict(dw_pre=A[12] + 2),
           dict(dgate=M(A[4], 64)), dict(scratch=0), dict(scratch=A[14] + 64),
           dict(scratch_bytes=need - 1), dict(scratch=A[3]), dict(dy=M(A[6], 20))]
    for over in bad:
        assert dp.dpopt_block_join_backward(_grad_args(dp, **over)) == dp.DPOPT_ERR_INVALID_ARG, over
    assert dp.dpopt_block_join_backward(None) == dp.DPOPT_ERR_INVALID_ARG
    assert dp.dpopt_block_join_backward(_grad_args(dp, cols=20000)) == dp.DPOPT_ERR_UNSUPPORTED


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), 1), (dict(vocab=0), 1), (dict(vocab=1 << 31, ld=1 << 31), 2), (dict(dtype=4), 1),
    (dict(ld=99), 1), (dict(n=65), 1), (dict(n=-1), 1), (dict(it=0.0), 1), (dict(it=math.inf), 1),
    (dict(it=-1.0), 1), (dict(logits=0), 1), (dict(logits=A[0] + 1), 1), (dict(tokens=0), 1),
    (dict(tokens=A[1] + 4), 1), (dict(logprob=0), 1), (dict(stats=0), 1), (dict(stats=A[3] + 2), 1),
    (dict(entropy=A[3]), 1), (dict(top=33), 1), (dict(top=-1), 1), (dict(top_logprob=0), 1),
    (dict(top_index=0), 1), (dict(top_index=A[6] + 4), 1), (dict(logprob=A[0] + 64), 1),
])
def test_logprob_refuses(dp, over, code):
    a = dict(logits=A[0], dtype=0, rows=4, vocab=100, ld=100, tokens=A[1], n=2, it=1.0,
             logprob=A[2], stats=A[3], entropy=A[4], top=5, top_logprob=A[5], top_index=A[6],
             scratch=A[7], scratch_bytes=1 << 40)
    a.update(over)
    assert dp.dpopt_token_logprob(*a.values(), 0) == code
    assert dp.dpopt_last_error() != ""


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), 1), (dict(vocab=0), 1), (dict(dtype=4), 1), (dict(ld=99), 1), (dict(n=65), 1),
    (dict(it=math.nan), 1), (dict(logits=0), 1), (dict(tokens=0), 1), (dict(stats=0), 1),
    (dict(dlogprob=0), 1), (dict(entropy=0), 1), (dict(dentropy=0), 1), (dict(scale=A[6] + 4), 1),
    (dict(dlogits=0), 1), (dict(dlogits=A[7] + 1), 1), (dict(ldd=99), 1), (dict(dlogits=A[2]), 1),
    (dict(dlogits=A[0], ldd=101), 1), (dict(dlogits=A[0] + 2), 1), (dict(scale=A[7] + 8), 1),
])
def test_logprob_gradient_refuses(dp, over, code):
    a = dict(logits=A[0], dtype=0, rows=4, vocab=100, ld=100, tokens=A[1], n=2, it=1.0, stats=A[2],
             dlogprob=A[3], entropy=A[4], dentropy=A[5], scale=A[6], dlogits=A[7], ldd=100)
    a.update(over)
    assert dp.dpopt_token_logprob_backward(*a.values(), 0) == code
    assert dp.dpopt_last_error() != ""


def test_wrappers_refuse_wrong_shapes_types_and_memory(dp):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    codes, exps = dp.act8_empty(4, 64, "cpu")
    with pytest.raises(ValueError, match="pageable"):
        dp.act8_pack(x, codes, exps, stream=0)
    with pytest.raises(ValueError, match="device memory"):
        dp.act8_wgrad(x, codes, exps, torch.zeros(64, 64), stream=0)
    with pytest.raises(ValueError, match="dimensions"):
        dp.act8_pack(x[0], codes, exps, stream=0)
    with pytest.raises(ValueError, match="adjacent"):
        dp.act8_pack(torch.zeros(64, 4, dtype=torch.bfloat16).t(), codes, exps, stream=0)
    empty = torch.empty(0, 64, dtype=torch.bfloat16)
    c0, e0 = dp.act8_empty(0, 64, "cpu")
    dp.act8_pack(empty, c0, e0, stream=0)  # nothing to do, nothing launched
    with pytest.raises(ValueError, match="shape"):
        dp.act8_pack(empty[:, :32], c0, e0, stream=0)
    with pytest.raises(TypeError):
        dp.act8_pack(torch.empty(0, 64, dtype=torch.float64), c0, e0, stream=0)
    with pytest.raises(TypeError):
        dp.act8_pack(empty, c0.to(torch.int16), e0, stream=0)
    with pytest.raises(ValueError, match="shape"):
        dp.block_join(empty, empty[:, :3], empty, eps=1e-5, stream=0)
    with pytest.raises(TypeError, match="share one type"):
        dp.block_join(empty, empty, empty, eps=1e-5, w_post=torch.zeros(64),
                      gate=torch.zeros(1, 64, dtype=torch.float16), stream=0)
    with pytest.raises(ValueError, match="together"):
        dp.token_logprob(empty, torch.empty(0, 1, dtype=torch.int64), torch.empty(0, 1),
                         torch.empty(0, 2), top_logprob=torch.empty(0, 3), stream=0)


# ---------------------------------------------------------------------------
# the oracle itself
# ---------------------------------------------------------------------------

def test_oracle_join_gradient_is_the_formula_s_derivative():
    """join_grad against torch's automatic differentiation of join, in 64 bits."""
    torch.manual_seed(0)
    rows, cols, R = 7, 24, 3
    p = {"h": torch.randn(rows, cols), "y": torch.randn(rows, cols), "w_post": torch.randn(cols),
         "w_pre": torch.randn(cols), "gate": torch.randn(3, cols)}
    p = {k: v.double().requires_grad_() for k, v in p.items()}
    dho, du = torch.randn(rows, cols).double(), torch.randn(rows, cols).double()
    o = ref.join(p["h"], p["y"], eps=1e-3, post=True, w_post=p["w_post"], gate=p["gate"],
                 gate_rows=R, res_scale=0.9, branch_scale=0.3, pre=True, w_pre=p["w_pre"])
    ((dho * o["h_out"][0]).sum() + (du * o["u"][0]).sum()).backward()
    d = {k: v.detach() for k, v in p.items()}
    g = ref.join_grad(dho, du, d["y"], o["h_out"][0].detach(), r1=o["rstd_pre"][0].detach(),
                      r2=o["rstd_post"][0].detach(), w_post=d["w_post"], w_pre=d["w_pre"],
                      gate=d["gate"], gate_rows=R, res_scale=0.9, branch_scale=0.3)
    for k, n in (("h", "dh"), ("y", "dy"), ("w_post", "dw_post"), ("w_pre", "dw_pre"),
                 ("gate", "dgate")):
        assert torch.allclose(g[n][0], p[k].grad, rtol=1e-10, atol=1e-12), n


def test_oracle_logprob_is_torch_s():
    torch.manual_seed(0)
    x = torch.randn(5, 60, dtype=torch.float64, requires_grad=True)
    tok = torch.randint(0, 60, (5, 2))
    tok[1, 0] = -1
    o = ref.logprob(x.detach(), tok, 1.5, 4)
    dist = torch.distributions.Categorical(logits=x * 1.5)
    lp = torch.log_softmax(x * 1.5, 1)
    given = torch.where(tok < 0, 0.0, lp.gather(1, tok.clamp_min(0)))
    assert torch.allclose(o["logprob"][0], given.detach())
    assert torch.allclose(o["entropy"][0], dist.entropy().detach())
    top = torch.topk(x.detach(), 4)
    assert torch.equal(o["top_index"], top.indices)
    dlp, dent = torch.randn(5, 2).double(), torch.randn(5).double()
    ((dlp * given).sum() + (dent * dist.entropy()).sum()).backward()
    stats, ent = o["stats"][0], o["entropy"][0]
    g, _ = ref.logprob_grad(x.detach(), tok, stats, dlp, ent, dent, 1.5, 8.0)
    assert torch.allclose(g, 8.0 * x.grad, rtol=1e-10, atol=1e-12)


def test_oracle_pack_by_hand():
    """Blocks worked out by hand: amax 100 -> step 1; amax 1 -> step 1/64; 127.9 clamps."""
    x = torch.zeros(3, 34)
    x[0, :4] = torch.tensor([100.0, -99.5, 0.5, 1.5])
    x[1, 0], x[1, 33] = 1.0, -0.3
    x[2, 0], x[2, 1] = 127.9, -127.4
    codes, byte = ref.pack(x)
    assert codes[0, :4].tolist() == [100, -100, 0, 2] and int(byte[0, 0]) == 127
    assert int(codes[1, 0]) == 64 and int(byte[1, 0]) == 121
    assert int(codes[1, 33]) == -77 and int(byte[1, 1]) == 119   # 0.3 * 256 = 76.8
    assert codes[2, :2].tolist() == [127, -127] and int(byte[0, 1]) == 1
    v = ref.unpack(codes, byte)
    assert float(v[1, 0]) == 1.0 and float(v[1, 33]) == -77 / 256
