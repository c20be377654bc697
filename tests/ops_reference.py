"""The training-side operators from their definitions, in 64 bits (test
infrastructure; nothing here calls the library), with bounds on what rounding
to 32 bits may add.

Bounds.  eps = 2^-24 is the unit roundoff of fp32.  A sum of n terms taken in
chains of at most `chain` additions differs from the exact one by at most
(chain + 2) eps times the sum of the terms' magnitudes (each term itself
rounded twice).  A kernel may split a row of C columns over as few as 32
threads, so a chain is at most C / 32 + 16 long.  Elementwise expressions of k
roundings add k eps times the sum of their parts' magnitudes; storing adds half
a unit in the last place of the stored type (and half its smallest step).
"""
from __future__ import annotations

import torch

EPS = 2.0 ** -24
# half a unit in the last place, relative: bf16 keeps 8 significant bits, fp16 11, fp32 24
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SMALLEST = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
BLOCK = 32


def stored(bound, value, dtype):
    """The bound of a value after it is stored in dtype."""
    return bound + UNIT[dtype] * (value.abs() + bound) + SMALLEST[dtype]


def within(got, want, bound, what):
    """got against want, element by element; NaN and Inf must stand in the same places."""
    got = got.double()
    odd = ~torch.isfinite(want)
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    assert bool(same[odd].all()), f"{what}: non-finite values differ"
    err = (got - want).abs()[~odd]
    lim = (bound if torch.is_tensor(bound) else torch.full_like(want, bound)).expand_as(want)[~odd]
    bad = ~(err <= lim)
    if bool(bad.any()):
        i = int(torch.argmax(torch.where(bad, err / lim, torch.zeros_like(err))))
        raise AssertionError(f"{what}: {int(bad.sum())} of {err.numel()} off, worst "
                             f"{float(err[i]):.3e} against a bound of {float(lim[i]):.3e}")


# ---------------------------------------------------------------------------
# 8-bit blocks
# ---------------------------------------------------------------------------

def pack(x):
    """(codes, bytes) of x, by the definition."""
    low = -24 if x.dtype == torch.float16 else -126
    rows, cols = x.shape
    codes = torch.zeros(rows, cols, dtype=torch.int8)
    byte = torch.zeros(rows, -(-cols // BLOCK), dtype=torch.uint8)
    xd = x.double().cpu()
    for b in range(byte.shape[1]):
        v = xd[:, b * BLOCK:(b + 1) * BLOCK]
        finite = torch.isfinite(v).all(1)
        amax = torch.where(finite, v.abs().amax(1), torch.zeros(rows, dtype=torch.float64))
        e = torch.frexp(amax).exponent - 7  # floor(log2) - 6
        e = torch.where(amax > 0, e, torch.full_like(e, low)).clamp_min(low)
        c = torch.round(torch.ldexp(v, -e[:, None])).clamp(-127, 127)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = torch.where(finite[:, None], c,
                                                          torch.zeros_like(c)).to(torch.int8)
        byte[:, b] = torch.where(finite, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return codes, byte


def unpack(codes, byte):
    e = byte.cpu().double() - 127
    scale = torch.where(byte.cpu() == 255, torch.full_like(e, float("nan")),
                        torch.pow(torch.tensor(2.0, dtype=torch.float64), e))
    return codes.cpu().double() * scale.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


# ---------------------------------------------------------------------------
# block join
# ---------------------------------------------------------------------------

def chain_eps(cols):
    return (cols / 32 + 18) * EPS


def gates(gate, gate_rows, rows, cols):
    if gate is None:
        return torch.ones(rows, cols, dtype=torch.float64)
    g = gate.double().cpu()
    return g[torch.zeros(rows, dtype=torch.int64) if gate_rows == 0
             else torch.arange(rows) // gate_rows]


def vec(w, cols):
    return torch.ones(cols, dtype=torch.float64) if w is None else w.double().cpu()


def rstd(x, eps):
    return 1.0 / torch.sqrt((x * x).mean(1) + eps)


def join(h, y, *, eps, post, w_post, gate, gate_rows, res_scale, branch_scale, pre, w_pre):
    """{name: (value, bound before storing)} of the join's outputs."""
    h, y = h.double().cpu(), y.double().cpu()
    rows, cols = h.shape
    g, wp, w = gates(gate, gate_rows, rows, cols), vec(w_post, cols), vec(w_pre, cols)
    out = {}
    r2 = rstd(y, eps) if post else torch.ones(rows, dtype=torch.float64)
    er = chain_eps(cols) + 4 * EPS if post else 0.0
    if post:
        out["rstd_post"] = (r2, er * r2)
    branch = branch_scale * g * y * r2[:, None] * wp
    new = res_scale * h + branch
    dnew = (er + 6 * EPS) * branch.abs() + 4 * EPS * (res_scale * h).abs()
    out["h_out"] = (new, dnew)
    if pre:
        r1 = rstd(new, eps)
        rel = chain_eps(cols) + 4 * EPS + \
            dnew.norm(dim=1) / (new.norm(dim=1) + 1e-300) * (new.norm(dim=1) > 0)
        out["rstd_pre"] = (r1, rel * r1)
        u = new * r1[:, None] * w
        out["u"] = (u, u.abs() * (rel[:, None] + 4 * EPS) + dnew * (r1[:, None] * w).abs())
    return out


def join_grad(dh_out, du, y, h, *, r1, r2, w_post, w_pre, gate, gate_rows, res_scale,
              branch_scale):
    """{name: (value, bound)} of the join's gradients; du, h None: no norm before the next
    block; r2 None: none after this one."""
    d0, y = dh_out.double().cpu(), y.double().cpu()
    rows, cols = d0.shape
    g, wp, w = gates(gate, gate_rows, rows, cols), vec(w_post, cols), vec(w_pre, cols)
    ce = chain_eps(cols)
    zero = torch.zeros(rows, dtype=torch.float64)
    if du is not None:
        t, h, r1 = du.double().cpu(), h.double().cpu(), r1.double().cpu()
        wt = w * t
        s = (wt * h).sum(1)
        k1 = r1 ** 3 * s / cols
        ek1 = r1 ** 3 / cols * (ce * (wt * h).abs().sum(1)) + 6 * EPS * k1.abs()
        lin = r1[:, None] * wt
        d = d0 + lin - k1[:, None] * h
        size = d0.abs() + lin.abs() + (k1[:, None] * h).abs()
        ed = 6 * EPS * size + ek1[:, None] * h.abs()
    else:
        h = t = torch.zeros_like(d0)
        r1, k1, ek1, lin, d = zero, zero, zero, torch.zeros_like(d0), d0
        size, ed = d0.abs(), torch.zeros_like(d0)
    dz, edz = branch_scale * g * d, (branch_scale * g).abs() * (ed + 3 * EPS * d.abs())
    out = {"dh": (res_scale * d, abs(res_scale) * (ed + 2 * EPS * d.abs()))}
    r = torch.ones(rows, dtype=torch.float64) if r2 is None else r2.double().cpu()
    if r2 is None:
        out["dy"] = (dz, edz)
    else:
        q = wp * g * y
        dot = (q * d).sum(1)  # <w_post dz, y> / branch
        mags = (q.abs() * (d0.abs() + lin.abs())).sum(1)
        hq = (q * h).abs().sum(1)
        edot = (ce + 6 * EPS) * (mags + k1.abs() * hq) + ek1 * hq
        k2 = r ** 3 * branch_scale * dot / cols
        ek2 = (r ** 3 * branch_scale / cols).abs() * edot + 8 * EPS * k2.abs()
        a = r[:, None] * wp * dz
        dy = a - k2[:, None] * y
        out["dy"] = (dy, (r[:, None] * wp).abs() * edz + ek2[:, None] * y.abs() +
                     6 * EPS * (a.abs() + (k2[:, None] * y).abs()))
    # sums over rows: chains of at most `rows` additions
    rc = (rows + 16) * EPS

    def total(term, eterm):
        return term.sum(0), eterm.sum(0) + rc * (term.abs() + eterm).sum(0)

    a = t * h * r1[:, None]
    out["dw_pre"] = total(a, 4 * EPS * a.abs())
    z = y * r[:, None]
    out["dw_post"] = total(dz * z, edz * z.abs() + 4 * EPS * (dz * z).abs())
    term = branch_scale * d * z * wp
    eterm = (branch_scale * z * wp).abs() * ed + 6 * EPS * term.abs()
    if gate_rows == 0:
        v, e = total(term, eterm)
        out["dgate"] = (v[None], e[None])
    else:
        parts = [total(term[i:i + gate_rows], eterm[i:i + gate_rows])
                 for i in range(0, rows, gate_rows)]
        out["dgate"] = (torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])) \
            if parts else (torch.zeros(0, cols), torch.zeros(0, cols))
    return out


# ---------------------------------------------------------------------------
# token log probabilities
# ---------------------------------------------------------------------------

def in_range_f32(v):
    """What lies beyond fp32's range is stored as an infinity."""
    big = v.abs() > torch.finfo(torch.float32).max
    return torch.where(big, torch.copysign(torch.full_like(v, float("inf")), v), v)


def logprob(logits, tokens, inv_temp, top):
    """{name: (value, bound)}, with top_index as plain integers."""
    x = logits.double().cpu()
    tok = tokens.cpu()
    rows, vocab = x.shape
    m = x.amax(1)
    empty = m == float("-inf")
    s = (x - m[:, None]) * inv_temp
    s[empty] = float("-inf")
    e = torch.exp(s)
    total = e.sum(1)
    L = torch.where(empty, torch.zeros_like(total), total.log())
    lp = s - L[:, None]
    p = torch.exp(lp)
    masked = s == float("-inf")  # keeps NaN entries
    sf = torch.where(masked, torch.zeros_like(s), s)
    ps = torch.where(masked, torch.zeros_like(s), p * s).sum(1)
    ent = torch.where(empty, torch.zeros_like(L), L - ps)
    # exp's argument is off by a few roundings of |s|; its own error is a few units
    chain = (vocab / 128 + 64) * EPS
    rel = chain + 4 * EPS * (p * sf.abs()).nan_to_num(0).sum(1) + 8 * EPS
    eL = rel + 4 * EPS * L.abs()
    out = {"stats": (torch.stack([m, L], 1), torch.stack([torch.zeros_like(eL), eL], 1))}
    clip = tok.clamp(0, vocab - 1)
    given = torch.where(tok < 0, torch.zeros_like(clip, dtype=torch.float64), lp.gather(1, clip))
    given[tok >= vocab] = float("nan")
    out["logprob"] = (in_range_f32(given), eL[:, None] + 4 * EPS * (sf.gather(1, clip).abs() + given.abs()))
    out["entropy"] = (ent, eL + (3 * rel + 4 * EPS) * (p * sf.abs()).nan_to_num(0).sum(1) +
                      4 * EPS * ((p * sf * sf).nan_to_num(0).sum(1) + ent.abs()))
    if top:
        # NaN first, then by value, among equals by index
        key = torch.where(torch.isnan(x), torch.full_like(x, float("inf")), x)
        order = torch.sort(key, dim=1, descending=True, stable=True).indices
        isn = torch.isnan(x).gather(1, order)
        order = order.gather(1, torch.sort(isn.to(torch.int8), dim=1, descending=True,
                                           stable=True).indices)
        idx = order[:, :top]
        out["top_index"] = idx
        tl = lp.gather(1, idx)
        out["top_logprob"] = (in_range_f32(tl), eL[:, None] + 4 * EPS * (sf.gather(1, idx).abs() + tl.abs()))
    return out


def logprob_grad(logits, tokens, stats, dlogprob, entropy, dentropy, inv_temp, scale):
    """(value, bound) of dlogits, from the statistics given."""
    x, tok = logits.double().cpu(), tokens.cpu()
    vocab = x.shape[1]
    m, L = stats.double().cpu().unbind(1)
    empty = m == float("-inf")
    lp = (x - m[:, None]) * inv_temp - L[:, None]
    p = torch.exp(lp)
    masked = (lp == float("-inf")) | empty[:, None]
    a = torch.where(tok < 0, torch.zeros_like(tok, dtype=torch.float64), dlogprob.double().cpu())
    a[tok >= vocab] = float("nan")
    own = torch.zeros_like(x)
    own.scatter_add_(1, tok.clamp(0, vocab - 1), a.nan_to_num(0) * (tok >= 0))
    asum, amag = a.sum(1, keepdim=True), a.abs().sum(1, keepdim=True)
    lpf = torch.where(masked, torch.zeros_like(lp), lp)
    dh = torch.zeros_like(m) if dentropy is None else dentropy.double().cpu()
    h = torch.zeros_like(m) if entropy is None else entropy.double().cpu()
    inner = asum + dh[:, None] * (lpf + h[:, None])
    g = own - p * inner
    # |s| + |L| rounded in the exponent, exp, the factors
    erel = EPS * (4 * (lpf.abs() + 2 * L.abs()[:, None]) + 8)
    emag = amag + (dh[:, None] * (lpf.abs() + 2 * L.abs()[:, None] + h[:, None].abs())).abs()
    ntok = tok.shape[1]
    bound = p * emag * (erel + (ntok + 6) * EPS) + \
        (ntok + 4) * EPS * (own.abs() + torch.zeros_like(own).scatter_add_(
            1, tok.clamp(0, vocab - 1), a.abs().nan_to_num(0)))
    k = inv_temp * scale
    value = torch.where(masked, torch.zeros_like(g), g * k)
    return value, torch.where(masked, torch.zeros_like(g), bound * k + 3 * EPS * value.abs())
