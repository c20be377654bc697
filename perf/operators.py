"""Measured cases of the training-side operators: the fused block join (norms
before and after a block, its gate and residual scale), activation checkpoints
in 8 bits with their weight-gradient product, and log probabilities of given
tokens with entropy and top alternatives.

run(state) makes one pass through one operator: with own = False in its plain
form (elementary torch operations in 32 bits, rounded once at the end), with
own = True through the library's entry points.  exact(case, seed) evaluates
the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = 32  # columns that share one exponent byte in a packed activation


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the join between two blocks for a handful of positions (evaluation or
        # sampling beside training): launch latency is everything
        dict(name="join_8x768", op="join", rows=8, cols=768, dtype="bf16", gate_rows=0,
             packed=False),
        # the join of an ordinary training micro-batch, keeping the block's
        # output as an 8-bit checkpoint for the backward pass
        dict(name="join_8192x2048_keep8", op="join", rows=8192, cols=2048, dtype="bf16",
             gate_rows=0, packed=True),
        # the join's gradient at a large model's width, both activations read
        # back from their 8-bit checkpoints
        dict(name="join_bwd_16384x8192_from8", op="join_bwd", rows=16384, cols=8192, dtype="bf16",
             gate_rows=0, packed=True),
        # fp16 with an odd width and one gate row per sequence of 500
        # positions, the last sequence short; 16-bit activations
        dict(name="join_bwd_3001x1547_fp16", op="join_bwd", rows=3001, cols=1547, dtype="fp16",
             gate_rows=500, packed=False),
        # a layer input packed into its checkpoint and restored
        dict(name="pack_8192x8192", op="pack", rows=8192, cols=8192, pad=0, dtype="bf16"),
        # a small fp32 activation, ragged last block, rows inside a wider array
        dict(name="pack_333x1001_fp32", op="pack", rows=333, cols=1001, pad=23, dtype="fp32"),
        # weight gradient of a layer of a small model from one short sequence
        dict(name="wgrad_257x768x768", op="wgrad", tokens=257, n=768, k=768, pad=0, dtype="bf16",
             out="bf16", add=False),
        # odd sizes, fp16, added to an fp32 gradient accumulated over micro-batches
        dict(name="wgrad_2011x1000x1547_fp16_add", op="wgrad", tokens=2011, n=1000, k=1547, pad=24,
             dtype="fp16", out="fp32", add=True),
        # weight gradient of a wide layer over a large micro-batch
        dict(name="wgrad_16384x8192x8192", op="wgrad", tokens=16384, n=8192, k=8192, pad=0,
             dtype="bf16", out="bf16", add=False),
        # one position, a large vocabulary, eight alternatives
        dict(name="logprob_1x131072", op="logprob", rows=1, vocab=131072, given=1, top=8,
             dtype="bf16", entropy=True, masked=0,
             inv_temperature=1.0),
        # a training or scoring batch: vocabulary of odd size
        dict(name="logprob_8192x50257", op="logprob", rows=8192, vocab=50257, given=1, top=8,
             dtype="bf16", entropy=True, masked=0,
             inv_temperature=1.0),
        # the loss's gradient with loss scaling, padded vocabulary columns masked
        dict(name="logprob_bwd_8192x50304_fp16", op="logprob_bwd", rows=8192, vocab=50304, given=1,
             top=0, dtype="fp16", entropy=True, masked=47,
             inv_temperature=1.0),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: a multiple of 64, or any number."""
    w = _log_uniform(rng, lo, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.6 else w


def draw(rng):
    op = rng.choice(["join", "join_bwd", "pack", "wgrad", "logprob", "logprob_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("join", "join_bwd"):
        cols = _width(rng, 64, 8192)
        rows = _log_uniform(rng, 1, min(16384, (1 << 26) // cols))
        return dict(op=op, rows=rows, cols=cols, dtype=dtype,
                    gate_rows=rng.choice([0, 0, 1, max(1, rows // rng.randint(1, 9))]),
                    packed=rng.random() < 0.5)
    if op == "pack":
        cols = _width(rng, 64, 8192)
        return dict(op=op, rows=_log_uniform(rng, 1, min(16384, (1 << 26) // cols)), cols=cols,
                    pad=rng.choice([0, 0, 8, 13]), dtype=dtype)
    if op == "wgrad":
        dtype = rng.choice(["bf16", "fp16"])
        return dict(op=op, tokens=_log_uniform(rng, 1, 8192), n=_width(rng, 64, 4096),
                    k=_width(rng, 64, 4096), pad=rng.choice([0, 0, 8, 13]), dtype=dtype,
                    out=rng.choice([dtype, dtype, "fp32"]), add=rng.random() < 0.4)
    vocab = _width(rng, 1000, 131072)
    rows = _log_uniform(rng, 1, min(8192, (1 << 28) // vocab))
    return dict(op=op, rows=rows, vocab=vocab, given=rng.choice([1, 1, 1, 5, 16]),
                top=0 if op == "logprob_bwd" else rng.choice([0, 1, 5, 8, 20]), dtype=dtype,
                entropy=rng.random() < 0.6, masked=rng.choice([0, 0, 17, vocab // 3]),
                inv_temperature=rng.choice([1.0, 1.0, 1.25]))


def work(case):
    op = case["op"]
    if op in ("join", "join_bwd"):
        r, c, e = case["rows"], case["cols"], SIZE[case["dtype"]]
        eight = c + -(-c // BLOCK)
        gates = 1 if case["gate_rows"] == 0 else -(-r // case["gate_rows"])
        if op == "join":  # h, y read; h_out, u written; two weights, the gates, two statistics
            b = r * c * 4 * e + (2 + gates) * c * e + 8 * r
            if case["packed"]:  # the checkpoint written, and restored for the comparison
                b += r * (2 * eight + c * e)
            return {"bytes": b, "flops": 14 * r * c}
        act = r * (eight if case["packed"] else c * e)
        return {"bytes": 4 * r * c * e + 2 * act + (2 + gates) * c * 2 * e + 8 * r,
                "flops": 30 * r * c}
    if op == "pack":
        r, c, e = case["rows"], case["cols"], SIZE[case["dtype"]]
        return {"bytes": 2 * r * (c * e + c + -(-c // BLOCK)), "flops": 4 * r * c}
    if op == "wgrad":
        t, n, k = case["tokens"], case["n"], case["k"]
        b = t * n * SIZE[case["dtype"]] + t * (k + -(-k // BLOCK))
        return {"bytes": b + n * k * SIZE[case["out"]] * (2 if case["add"] else 1),
                "flops": 2 * t * n * k}
    r, v, g = case["rows"], case["vocab"], case["given"]
    e = SIZE[case["dtype"]]
    if op == "logprob":
        small = r * (12 * g + 8 + 4 * case["entropy"] + 12 * case["top"])
        return {"bytes": r * v * e + small, "flops": 6 * r * v}
    return {"bytes": 2 * r * v * e + r * (12 * g + 8 + 8 * case["entropy"]), "flops": 8 * r * v}


# ---------------------------------------------------------------------------
# plain forms of the pieces
# ---------------------------------------------------------------------------

def _lowest_exponent(dtype):
    return -24 if dtype == torch.float16 else -126


def _power_of_two(e):
    """2^e in fp32 for -126 <= e <= 127, from its bit pattern."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_pack(x):
    """codes (int8) and exponent bytes of x: blocks of 32 columns, the exponent
    that puts the block's largest magnitude in [64, 128)."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    f = torch.zeros(rows, nb * BLOCK, device=x.device)
    f[:, :cols] = x
    f = f.view(rows, nb, BLOCK)
    amax = f.abs().amax(2, keepdim=True)
    e = (torch.frexp(amax).exponent - 7).clamp_min(_lowest_exponent(x.dtype))
    e = torch.where(amax == 0, torch.full_like(e, _lowest_exponent(x.dtype)), e)
    codes = (f * _power_of_two(-e)).round().clamp(-127, 127).to(torch.int8)
    return codes.view(rows, -1)[:, :cols].contiguous(), (e + 127).to(torch.uint8).view(rows, nb)


def _plain_unpack(codes, exps):
    scale = _power_of_two(exps.to(torch.int32) - 127)
    return codes.float() * scale.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _gates(gate, gate_rows, rows):
    """The gate of every row: one row for all, or one for each run of gate_rows."""
    if gate_rows == 0:
        return gate.float()
    return gate.float().repeat_interleave(gate_rows, 0)[:rows]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * scale

    st = dict(case=case, op=case["op"])
    dt = DT[case["dtype"]]
    if case["op"] in ("join", "join_bwd"):
        r, c = case["rows"], case["cols"]
        ng = 1 if case["gate_rows"] == 0 else -(-r // case["gate_rows"])
        # a residual stream with a few large channels, a block output of its own scale
        wide = 1.0 + 7.0 * (torch.rand(c, generator=g, device=DEV) < 0.01)
        st.update(eps=1e-5, res_scale=1.0, branch_scale=0.5,
                  w_post=(1 + randn(c, scale=0.1)).to(dt), w_pre=(1 + randn(c, scale=0.1)).to(dt),
                  gate=(0.5 + randn(ng, c, scale=0.2)).to(dt))
        h, y = (randn(r, c) * wide).to(dt), randn(r, c, scale=0.3).to(dt)
        if case["op"] == "join":
            st.update(h=h, y=y)
        else:
            st.update(rstd_post=torch.rsqrt(y.float().square().mean(1) + st["eps"]),
                      rstd_pre=torch.rsqrt(h.float().square().mean(1) + st["eps"]),
                      h_out=_plain_pack(h) if case["packed"] else h,
                      y=_plain_pack(y) if case["packed"] else y,
                      dh_out=randn(r, c, scale=0.01).to(dt), du=randn(r, c, scale=0.01).to(dt))
        if own:
            import zero_mixed_precision_gb300 as dp
            if case["op"] == "join_bwd":
                st["scratch"] = torch.empty(
                    dp.block_join_scratch_bytes(r, c, case["gate_rows"]), dtype=torch.uint8,
                    device=DEV)
    elif case["op"] == "pack":
        r, c = case["rows"], case["cols"]
        x = randn(r, c + case["pad"])
        x *= torch.exp(randn(c + case["pad"], scale=0.5))
        st["x"] = x.to(dt)[:, :c]
    elif case["op"] == "wgrad":
        t, n, k = case["tokens"], case["n"], case["k"]
        x = randn(t, k) * torch.exp(randn(k, scale=0.5))
        st["codes"], st["exps"] = _plain_pack(x.to(dt))
        del x
        st["dy"] = randn(t, n + case["pad"], scale=0.01).to(dt)[:, :n]
        st["add"] = randn(n, k, scale=0.01 * math.sqrt(t)).to(DT[case["out"]]) \
            if case["add"] else None
        if own:
            import zero_mixed_precision_gb300 as dp
            st["scratch"] = torch.empty(dp.act8_wgrad_scratch_bytes(t, n, k), dtype=torch.uint8,
                                        device=DEV)
    else:
        r, v, m = case["rows"], case["vocab"], case["given"]
        x = randn(r, v, scale=2.5)
        if case["masked"]:
            x[:, v - case["masked"]:] = -math.inf
        st["logits"] = x.to(dt)
        del x
        tok = torch.randint(0, v - case["masked"], (r, m), generator=g, device=DEV)
        # one position in ten carries no token (a prompt or padding): -1
        tok[torch.rand(r, m, generator=g, device=DEV) < 0.1] = -1
        st.update(tokens=tok, inv_temperature=case["inv_temperature"])
        if case["op"] == "logprob_bwd":
            mx, logsum, ent = [], [], []
            for part in st["logits"].split(1024):
                x = part.float()
                top = x.amax(1, keepdim=True)
                d = (x - top) * st["inv_temperature"]
                e = d.exp()
                s = e.sum(1)
                mx.append(top[:, 0])
                logsum.append(s.log())
                ent.append(s.log() - torch.where(e > 0, e * d, 0.0).sum(1) / s)
            st["stats"] = torch.stack([torch.cat(mx), torch.cat(logsum)], 1).contiguous()
            st["entropy"] = torch.cat(ent) if case["entropy"] else None
            st["dlogprob"] = randn(r, m) / max(r, 256)
            st["dentropy"] = randn(r, scale=0.1) / max(r, 256) if case["entropy"] else None
            # the device-resident state of dynamic loss scaling; its first word is the scale
            st["loss_scale"] = torch.zeros(4, dtype=torch.int64, device=DEV)
            st["loss_scale"].view(torch.float32)[0] = 65536.0
        elif own:
            import zero_mixed_precision_gb300 as dp
            st["scratch"] = torch.empty(
                max(1, dp.token_logprob_scratch_bytes(r, v, case["top"])), dtype=torch.uint8,
                device=DEV)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _plain_join(s):
    dt = s["h"].dtype
    r = s["h"].shape[0]
    y = s["y"].float()
    rstd_post = torch.rsqrt(y.square().mean(1) + s["eps"])
    z = y * rstd_post[:, None] * s["w_post"].float()
    h = s["res_scale"] * s["h"].float() + \
        s["branch_scale"] * _gates(s["gate"], s["case"]["gate_rows"], r) * z
    rstd_pre = torch.rsqrt(h.square().mean(1) + s["eps"])
    u = h * rstd_pre[:, None] * s["w_pre"].float()
    out = dict(h=h.to(dt), u=u.to(dt), rstd_post=rstd_post, rstd_pre=rstd_pre)
    if s["case"]["packed"]:
        out["y8"] = _plain_unpack(*_plain_pack(s["y"])).to(dt)
    return out


def _own_join(s):
    import zero_mixed_precision_gb300 as dp
    h, y, c = s["h"], s["y"], s["case"]
    r, cols = h.shape
    out = dict(h=torch.empty_like(h), u=torch.empty_like(h),
               rstd_post=torch.empty(r, device=DEV), rstd_pre=torch.empty(r, device=DEV))
    y8 = dp.act8_empty(r, cols, DEV) if c["packed"] else None
    dp.block_join(h, y, out["h"], eps=s["eps"], rstd_post=out["rstd_post"], w_post=s["w_post"],
                  gate=s["gate"], gate_rows=c["gate_rows"], res_scale=s["res_scale"],
                  branch_scale=s["branch_scale"], u=out["u"], rstd_pre=out["rstd_pre"],
                  w_pre=s["w_pre"], y8=y8)
    if c["packed"]:
        out["y8"] = torch.empty_like(y)
        dp.act8_unpack(*y8, out["y8"])
    return out


def _plain_norm_bwd(dz, x, rstd, w):
    xhat = x * rstd[:, None]
    p = dz * w
    return rstd[:, None] * (p - xhat * (p * xhat).mean(1, keepdim=True)), (dz * xhat).sum(0)


def _plain_join_bwd(s):
    dt, c = s["dh_out"].dtype, s["case"]
    r = c["rows"]
    h = _plain_unpack(*s["h_out"]) if c["packed"] else s["h_out"].float()
    y = _plain_unpack(*s["y"]) if c["packed"] else s["y"].float()
    dh, dw_pre = _plain_norm_bwd(s["du"].float(), h, s["rstd_pre"], s["w_pre"].float())
    dh = dh + s["dh_out"].float()
    gate = _gates(s["gate"], c["gate_rows"], r)
    wp = s["w_post"].float()
    dgate = s["branch_scale"] * dh * (y * s["rstd_post"][:, None] * wp)
    if c["gate_rows"] == 0:
        dgate = dgate.sum(0, keepdim=True)
    else:
        dgate = torch.zeros(s["gate"].shape, device=DEV).index_add_(
            0, torch.arange(r, device=DEV) // c["gate_rows"], dgate)
    dy, dw_post = _plain_norm_bwd(s["branch_scale"] * gate * dh, y, s["rstd_post"], wp)
    return dict(dh=(s["res_scale"] * dh).to(dt), dy=dy.to(dt), dw_pre=dw_pre.to(dt),
                dw_post=dw_post.to(dt), dgate=dgate.to(dt))


def _own_join_bwd(s):
    import zero_mixed_precision_gb300 as dp
    out = dict(dh=torch.empty_like(s["dh_out"]), dy=torch.empty_like(s["dh_out"]),
               dw_pre=torch.empty_like(s["w_pre"]), dw_post=torch.empty_like(s["w_post"]),
               dgate=torch.empty_like(s["gate"]))
    dp.block_join_backward(s["dh_out"], s["y"], out["dy"], out["dh"], s["scratch"],
                           rstd_post=s["rstd_post"], w_post=s["w_post"], dw_post=out["dw_post"],
                           gate=s["gate"], gate_rows=s["case"]["gate_rows"], dgate=out["dgate"],
                           res_scale=s["res_scale"], branch_scale=s["branch_scale"], du=s["du"],
                           h_out=s["h_out"], rstd_pre=s["rstd_pre"], w_pre=s["w_pre"],
                           dw_pre=out["dw_pre"])
    return out


def _plain_pack_restore(s):
    return _plain_unpack(*_plain_pack(s["x"])).to(s["x"].dtype)


def _own_pack_restore(s):
    import zero_mixed_precision_gb300 as dp
    x = s["x"]
    packed = dp.act8_empty(*x.shape, DEV)
    dp.act8_pack(x, *packed)
    back = torch.empty(x.shape, dtype=x.dtype, device=DEV)
    dp.act8_unpack(*packed, back)
    return back


def _plain_wgrad(s):
    dw = s["dy"].float().t() @ _plain_unpack(s["codes"], s["exps"])
    if s["add"] is not None:
        dw += s["add"].float()
    return dw.to(DT[s["case"]["out"]])


def _own_wgrad(s):
    import zero_mixed_precision_gb300 as dp
    c = s["case"]
    dw = torch.empty(c["n"], c["k"], dtype=DT[c["out"]], device=DEV)
    dp.act8_wgrad(s["dy"], s["codes"], s["exps"], dw, s["scratch"], addend=s["add"])
    return dw


def _plain_logprob(s):
    x, c, tok = s["logits"].float(), s["case"], s["tokens"]
    mx = x.amax(1, keepdim=True)
    x = (x - mx) * s["inv_temperature"]
    e = x.exp()
    total = e.sum(1, keepdim=True)
    logsum = total.log()
    lp = x.gather(1, tok.clamp_min(0)) - logsum
    out = dict(logprob=torch.where(tok < 0, 0.0, lp),
               stats=torch.cat([mx, logsum], 1))
    if c["entropy"]:
        e *= torch.where(e > 0, x, 0.0)
        out["entropy"] = (logsum - e.sum(1, keepdim=True) / total)[:, 0]
    del e
    if c["top"]:
        # the largest, again and again; among equals the lowest index
        cols = torch.arange(c["vocab"], device=DEV)
        vals, idx = [], []
        for _ in range(c["top"]):
            best = x.amax(1, keepdim=True)
            at = torch.where(x == best, cols, c["vocab"]).amin(1, keepdim=True)
            vals.append(best - logsum)
            idx.append(at)
            x.scatter_(1, at, -math.inf)
        out.update(top_logprob=torch.cat(vals, 1), top_index=torch.cat(idx, 1))
    return out


def _own_logprob(s):
    import zero_mixed_precision_gb300 as dp
    c = s["case"]
    r = c["rows"]
    out = dict(logprob=torch.empty(r, c["given"], device=DEV), stats=torch.empty(r, 2, device=DEV))
    if c["entropy"]:
        out["entropy"] = torch.empty(r, device=DEV)
    if c["top"]:
        out["top_logprob"] = torch.empty(r, c["top"], device=DEV)
        out["top_index"] = torch.empty(r, c["top"], dtype=torch.int64, device=DEV)
    dp.token_logprob(s["logits"], s["tokens"], out["logprob"], out["stats"], s["scratch"],
                     entropy=out.get("entropy"), top_logprob=out.get("top_logprob"),
                     top_index=out.get("top_index"), inv_temperature=s["inv_temperature"])
    return out


def _plain_logprob_bwd(s):
    tok, c = s["tokens"], s["case"]
    x = s["logits"].float()
    x -= s["stats"][:, :1]
    x = x * s["inv_temperature"] - s["stats"][:, 1:]  # log probabilities
    p = x.exp()
    given = torch.where(tok < 0, 0.0, s["dlogprob"])
    grad = -p * given.sum(1, keepdim=True)
    grad.scatter_add_(1, tok.clamp_min(0), given)
    if c["entropy"]:
        x = torch.where(p > 0, x, 0.0)
        grad -= s["dentropy"][:, None] * p * (x + s["entropy"][:, None])
    grad *= s["inv_temperature"] * s["loss_scale"].view(torch.float32)[0]
    return grad.to(s["logits"].dtype)


def _own_logprob_bwd(s):
    import zero_mixed_precision_gb300 as dp
    d = torch.empty_like(s["logits"])
    dp.token_logprob_backward(s["logits"], s["tokens"], s["stats"], d, dlogprob=s["dlogprob"],
                              entropy=s["entropy"], dentropy=s["dentropy"],
                              inv_temperature=s["inv_temperature"], loss_scale=s["loss_scale"])
    return d


_PLAIN = dict(join=_plain_join, join_bwd=_plain_join_bwd, pack=_plain_pack_restore,
              wgrad=_plain_wgrad, logprob=_plain_logprob, logprob_bwd=_plain_logprob_bwd)
_OWN = dict(join=_own_join, join_bwd=_own_join_bwd, pack=_own_pack_restore, wgrad=_own_wgrad,
            logprob=_own_logprob, logprob_bwd=_own_logprob_bwd)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written on their own (row by row blocks)
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s, case)


def _restore64(codes, exps):
    """value = code * 2^(byte - 127), element by element."""
    col = torch.arange(codes.shape[1], device=codes.device) // BLOCK
    return codes.double() * torch.pow(2.0, exps.double() - 127.0)[:, col]


def _quantised64(x):
    low = -24.0 if x.dtype == torch.float16 else -126.0
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for j in range(0, x.shape[1], BLOCK):
        b = x[:, j:j + BLOCK].double()
        # the 1e-9 is far below the gap of any input's logarithm under a whole number
        e = torch.floor(torch.log2(b.abs().amax(1, keepdim=True)) + 1e-9) - 6.0
        step = torch.pow(2.0, torch.clamp(e, min=low))
        out[:, j:j + BLOCK] = torch.clamp(torch.round(b / step), -127, 127) * step
    return out


def _gate_of(s, case, lo, hi):
    if case["gate_rows"] == 0:
        return s["gate"].double()
    return s["gate"].double()[torch.arange(lo, hi, device=DEV) // case["gate_rows"]]


def _row_parts(rows, cols):
    step = max(1, (1 << 24) // cols)
    return [(lo, min(rows, lo + step)) for lo in range(0, rows, step)]


def _exact_join(s, case):
    parts = []
    for lo, hi in _row_parts(case["rows"], case["cols"]):
        y, h = s["y"][lo:hi].double(), s["h"][lo:hi].double()
        ry = 1.0 / torch.sqrt(torch.linalg.vecdot(y, y) / case["cols"] + s["eps"])
        new = s["res_scale"] * h + s["branch_scale"] * torch.einsum(
            "r,rc,c,rc->rc", ry, y, s["w_post"].double(),
            _gate_of(s, case, lo, hi).expand(hi - lo, -1))
        rh = 1.0 / torch.sqrt(torch.linalg.vecdot(new, new) / case["cols"] + s["eps"])
        parts.append((new, torch.einsum("r,rc,c->rc", rh, new, s["w_pre"].double()), ry, rh))
    out = {k: torch.cat([p[i] for p in parts])
           for i, k in enumerate(("h", "u", "rstd_post", "rstd_pre"))}
    if case["packed"]:
        out["y8"] = _quantised64(s["y"])
    return out


def _exact_join_bwd(s, case):
    c = case["cols"]
    wpre, wpost = s["w_pre"].double(), s["w_post"].double()
    zero = torch.zeros(c, dtype=torch.float64, device=DEV)
    dw_pre, dw_post = zero.clone(), zero.clone()
    dgate = torch.zeros(s["gate"].shape, dtype=torch.float64, device=DEV)
    dhs, dys = [], []

    def part_of(t, lo, hi):
        return _restore64(t[0][lo:hi], t[1][lo:hi]) if case["packed"] else t[lo:hi].double()

    for lo, hi in _row_parts(case["rows"], c):
        h, y = part_of(s["h_out"], lo, hi), part_of(s["y"], lo, hi)
        r1, r2 = s["rstd_pre"][lo:hi].double(), s["rstd_post"][lo:hi].double()
        du = s["du"][lo:hi].double()
        # u_j = w_j h_j r(h):  du/dh = r (w du - r^2 h <w du, h> / c)
        dot = torch.einsum("rc,c,rc->r", du, wpre, h)
        total = s["dh_out"][lo:hi].double() + r1[:, None] * (
            du * wpre - h * (r1 * r1 * dot / c)[:, None])
        dw_pre += torch.einsum("rc,rc,r->c", du, h, r1)
        b = s["branch_scale"]
        gate = _gate_of(s, case, lo, hi).expand(hi - lo, -1)
        dg = b * torch.einsum("rc,rc,r,c->rc", total, y, r2, wpost)
        group = torch.zeros(hi - lo, dtype=torch.int64, device=DEV) if case["gate_rows"] == 0 \
            else torch.arange(lo, hi, device=DEV) // case["gate_rows"]
        dgate.index_add_(0, group, dg)
        dz = b * gate * total
        dot = torch.einsum("rc,c,rc->r", dz, wpost, y)
        dys.append(r2[:, None] * (dz * wpost - y * (r2 * r2 * dot / c)[:, None]))
        dw_post += torch.einsum("rc,rc,r->c", dz, y, r2)
        dhs.append(s["res_scale"] * total)
    return dict(dh=torch.cat(dhs), dy=torch.cat(dys), dw_pre=dw_pre, dw_post=dw_post, dgate=dgate)


def _exact_pack(s, case):
    return _quantised64(s["x"])


def _exact_wgrad(s, case):
    # 64-bit products run near 1 TFLOP/s here
    if 2 * case["tokens"] * case["n"] * case["k"] > 8e12:
        return None
    total = torch.zeros(case["n"], case["k"], dtype=torch.float64, device=DEV)
    for lo in range(0, case["tokens"], 2048):
        x = _restore64(s["codes"][lo:lo + 2048], s["exps"][lo:lo + 2048])
        total += torch.einsum("tn,tk->nk", s["dy"][lo:lo + 2048].double(), x)
    return total if s["add"] is None else total + s["add"].double()


def _exact_logprob(s, case):
    keys = ["logprob", "stats"] + ["entropy"] * case["entropy"] + \
        ["top_logprob", "top_index"] * (case["top"] > 0)
    out = {k: [] for k in keys}
    for lo, hi in _row_parts(case["rows"], case["vocab"]):
        x = s["logits"][lo:hi].double()
        t = x * s["inv_temperature"]
        lse = torch.logsumexp(t, 1, keepdim=True)
        lp = t - lse
        tok = s["tokens"][lo:hi]
        out["logprob"].append(torch.where(tok < 0, 0.0, lp.gather(1, tok.clamp_min(0))))
        top = x.amax(1, keepdim=True)
        out["stats"].append(torch.cat([top, lse - top * s["inv_temperature"]], 1))
        if case["entropy"]:
            out["entropy"].append(torch.special.entr(lp.exp()).sum(1))
        if case["top"]:
            idx = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["top"]]
            out["top_index"].append(idx)
            out["top_logprob"].append(lp.gather(1, idx))
    return {k: torch.cat(v) for k, v in out.items()}


def _exact_logprob_bwd(s, case):
    """d/dx of sum(dlogprob * logprob) + sum(dentropy * entropy), times the loss scale."""
    parts = []
    for lo, hi in _row_parts(case["rows"], case["vocab"]):
        p = torch.softmax(s["logits"][lo:hi].double() * s["inv_temperature"], 1)
        tok = s["tokens"][lo:hi]
        a = torch.where(tok < 0, 0.0, s["dlogprob"][lo:hi].double())
        g = torch.zeros_like(p).scatter_add_(1, tok.clamp_min(0), a) - p * a.sum(1, keepdim=True)
        if case["entropy"]:
            plogp = torch.special.xlogy(p, p)
            g -= s["dentropy"][lo:hi, None].double() * (plogp - p * plogp.sum(1, keepdim=True))
        parts.append(g * (s["inv_temperature"] * 65536.0))
    return torch.cat(parts)


_EXACT = dict(join=_exact_join, join_bwd=_exact_join_bwd, pack=_exact_pack, wgrad=_exact_wgrad,
              logprob=_exact_logprob, logprob_bwd=_exact_logprob_bwd)
