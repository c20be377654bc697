"""A battery of the training-side operators' calls that walks their index paths: vector
and element forms, ragged widths, gate rows crossing the runs of rows, split rows and
tokens, both forms of the weight gradient's product, in-place calls.

run() returns every output and the stream status after each call;
tests/test_gpu_operators_bounds.py compares the release library (in the test process)
with the bounds-checked build (this file run as a script in a child process)."""
from __future__ import annotations

import sys

import numpy as np
import torch


def _host(t):
    t = t.contiguous()
    return (t.view(torch.int16) if t.dtype in (torch.bfloat16, torch.float16) else t).cpu().numpy()


def run():
    import zero_mixed_precision_gb300 as dp
    gen = torch.Generator(device="cuda").manual_seed(99)
    out, status = {}, []

    def rand(*s, dt=torch.float32, scale=1.0):
        return (torch.randn(*s, generator=gen, device="cuda") * scale).to(dt)

    def keep(name, *tensors):
        torch.cuda.synchronize()
        status.append((name, dp.dpopt_stream_status(0)))
        for i, t in enumerate(tensors):
            out[f"{name}/{i}"] = _host(t)

    def scratch(n):
        return torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda")

    for rows, cols, dt in ((5, 1, torch.bfloat16), (37, 1000, torch.float16),
                           (300, 2056, torch.bfloat16), (9, 1547, torch.float32)):
        x = rand(rows, cols, dt=dt)
        pair = dp.act8_empty(rows, cols)
        dp.act8_pack(x, *pair)
        back = torch.empty_like(x)
        dp.act8_unpack(*pair, back)
        keep(f"pack_{rows}x{cols}", *pair, back)

    for rows, cols, gate_rows, dt in ((7, 96, 0, torch.bfloat16), (701, 264, 100, torch.float16),
                                      (700, 131, 0, torch.float32), (3, 8192, 1, torch.bfloat16),
                                      (4, 9001, 3, torch.bfloat16)):
        h, y, dho, du = (rand(rows, cols, dt=dt) for _ in range(4))
        w, wp = rand(cols, dt=dt), rand(cols, dt=dt)
        gate = rand(1 if gate_rows == 0 else -(-rows // gate_rows), cols, dt=dt)
        ho, u = torch.empty_like(h), torch.empty_like(h)
        r1, r2 = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        eight = [dp.act8_empty(rows, cols) for _ in range(3)]
        dp.block_join(h, y, ho, eps=1e-5, rstd_post=r2, w_post=wp, gate=gate, gate_rows=gate_rows,
                      u=u, rstd_pre=r1, w_pre=w, y8=eight[0], h8=eight[1], u8=eight[2])
        keep(f"join_{rows}x{cols}", ho, u, r1, r2, *(t for p in eight for t in p))
        for name, yy, hh in (("16", y, ho), ("8", eight[0], eight[1])):
            dy, dh = torch.empty_like(h), torch.empty_like(h)
            dw, dwp, dg = torch.empty_like(w), torch.empty_like(w), torch.empty_like(gate)
            dp.block_join_backward(dho, yy, dy, dh,
                                   scratch(dp.block_join_scratch_bytes(rows, cols, gate_rows)),
                                   rstd_post=r2, w_post=wp, dw_post=dwp, gate=gate,
                                   gate_rows=gate_rows, dgate=dg, du=du, h_out=hh, rstd_pre=r1,
                                   w_pre=w, dw_pre=dw)
            keep(f"join_grad_{rows}x{cols}_{name}", dy, dh, dw, dwp, dg)

    for t, n, k, dt, od, add in ((1, 1, 1, torch.bfloat16, torch.bfloat16, False),
                                 (130, 200, 333, torch.float16, torch.float32, True),
                                 (4100, 128, 128, torch.bfloat16, torch.bfloat16, True),
                                 (700, 2600, 2100, torch.bfloat16, torch.float32, False)):
        pair = dp.act8_empty(t, k)
        dp.act8_pack(rand(t, k, dt=dt), *pair)
        dw = torch.empty(n, k, dtype=od, device="cuda")
        dp.act8_wgrad(rand(t, n, dt=dt), *pair, dw, scratch(dp.act8_wgrad_scratch_bytes(t, n, k)),
                      addend=rand(n, k, dt=od) if add else None)
        keep(f"wgrad_{t}x{n}x{k}", dw)

    for rows, vocab, n, top, dt in ((1, 1, 1, 1, torch.float32), (3, 50257, 1, 8, torch.bfloat16),
                                    (600, 777, 5, 3, torch.float16), (2, 131072, 64, 32,
                                                                     torch.bfloat16)):
        x = rand(rows, vocab, dt=dt, scale=2.0)
        tok = torch.randint(-1, vocab, (rows, n), generator=gen, device="cuda")
        lp, st = torch.empty(rows, n, device="cuda"), torch.empty(rows, 2, device="cuda")
        ent = torch.empty(rows, device="cuda")
        tl = torch.empty(rows, top, device="cuda")
        ti = torch.empty(rows, top, dtype=torch.int64, device="cuda")
        dp.token_logprob(x, tok, lp, st, scratch(dp.token_logprob_scratch_bytes(rows, vocab, top)),
                         entropy=ent, top_logprob=tl, top_index=ti)
        keep(f"logprob_{rows}x{vocab}", lp, st, ent, tl, ti)
        dp.token_logprob_backward(x, tok, st, x, dlogprob=rand(rows, n), entropy=ent,
                                  dentropy=rand(rows))
        keep(f"logprob_grad_{rows}x{vocab}", x)
    return out, status


def main(path):
    import zero_mixed_precision_gb300 as dp
    out, status = run()
    np.savez(path, __version__=np.array(dp.dpopt_version()),
             __names__=np.array([n for n, _ in status]),
             __status__=np.array([s for _, s in status], dtype=np.int64), **out)


if __name__ == "__main__":
    main(sys.argv[1])
