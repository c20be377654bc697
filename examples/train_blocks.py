"""A training step end to end on one GPU: residual blocks whose activations are kept in 8
bits, a token loss whose gradient carries the device loss scale, and the loss-scaled
AdamW step over the replicas' gradients.

The model is a stack of position-wise blocks on a residual stream h (tokens x width):

    u   = norm(h) w_pre                    the join's norm before the block
    y   = W2 relu(W1 u)^2                  two linear layers (library products)
    h  <- h + gate * norm(y) w_post        the join, one gate value per channel
    logits = E norm(h)                     after the last block

Per block the backward pass keeps three packed matrices -- u, relu(W1 u) and the
block's output y -- and one of the residual stream, each 8.25 bits per element, and
two floats per token; the weight gradients are formed from the packed inputs and
land in flat gradient buffers, one per micro-batch, which are the step's replicas.

    python examples/train_blocks.py [--steps 60]

prints the loss of a synthetic next-token task and the bytes kept per token.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_mixed_precision_gb300 as dp  # noqa: E402

BF16 = torch.bfloat16


class BlockStack:
    """Parameters in one flat fp32 master vector with a bf16 working copy, and one flat bf16
    gradient buffer per micro-batch (replica)."""

    def __init__(self, vocab=2048, width=256, inner=512, blocks=2, replicas=2, seed=0,
                 device="cuda"):
        self.vocab, self.width, self.inner, self.blocks = vocab, width, inner, blocks
        self.device, self.eps = device, 1e-5
        shapes = [("embed", (vocab, width))]
        for i in range(blocks):
            shapes += [(f"w_pre{i}", (width,)), (f"w1_{i}", (inner, width)),
                       (f"w2_{i}", (width, inner)), (f"w_post{i}", (width,)),
                       (f"gate{i}", (1, width))]
        shapes += [("w_last", (width,))]
        self.where, n = {}, 0
        for name, shape in shapes:
            self.where[name] = (n, shape)
            n += math.prod(shape)
        self.numel = -(-n // 64) * 64
        g = torch.Generator(device=device).manual_seed(seed)
        self.master = torch.zeros(self.numel, device=device)
        for name, (_, shape) in self.where.items():
            p = self.view(self.master, name)
            if name.startswith("w_"):
                p.fill_(1.0)
            elif name.startswith("gate"):
                p.fill_(0.5)
            else:
                p.copy_(torch.randn(*shape, generator=g, device=device) /
                        math.sqrt(shape[1]))
        self.work = self.master.to(BF16)
        self.m, self.v = torch.zeros_like(self.master), torch.zeros_like(self.master)
        self.grads = [torch.zeros(self.numel, dtype=BF16, device=device) for _ in range(replicas)]
        self.average = torch.zeros(self.numel, device=device)
        self.scale_state = torch.zeros(4, dtype=torch.int64, device=device)
        self.scale_cfg = dp.loss_scale_init(self.scale_state, init_scale=1024.0, window=1000)
        self.sqnorm = torch.zeros(1, dtype=torch.float64, device=device)
        self.sqnorms = torch.zeros(replicas, dtype=torch.float64, device=device)
        self.norm_scratch = torch.empty(8 * (self.numel // replicas // 4096 + 2), dtype=torch.uint8,
                                        device=device)
        self.scratch = None

    def view(self, flat, name):
        at, shape = self.where[name]
        return flat[at:at + math.prod(shape)].view(shape)

    def p(self, name):
        return self.view(self.work, name)

    def _scratch(self, tokens):
        if self.scratch is None or self.scratch[0] < tokens:
            sizes = [dp.act8_wgrad_scratch_bytes(tokens, n, k) for n, k in
                     ((self.vocab, self.width), (self.inner, self.width),
                      (self.width, self.inner))]
            sizes += [dp.block_join_scratch_bytes(tokens, self.width, 0),
                      dp.token_logprob_scratch_bytes(tokens, self.vocab, 0)]
            self.scratch = (tokens, torch.empty(max(sizes), dtype=torch.uint8,
                                                device=self.device))
        return self.scratch[1]

    def forward(self, inputs, targets):
        """Log probabilities of the targets, and what the backward pass needs."""
        T, C, dev = inputs.numel(), self.width, self.device
        scratch = self._scratch(T)
        h = self.p("embed")[inputs]
        kept = {"inputs": inputs, "targets": targets.view(T, 1), "blocks": []}
        kept["bytes"] = 0

        def keep(cols):
            pair = dp.act8_empty(T, cols, dev)
            kept["bytes"] += pair[0].numel() + pair[1].numel()
            return pair

        def new():
            return torch.empty(T, C, dtype=BF16, device=dev)

        # the first norm: a join of the embedding with nothing (branch scale 0)
        u, r_pre, u8, h8 = new(), torch.empty(T, device=dev), keep(C), keep(C)
        dp.block_join(h, torch.zeros_like(h), h, eps=self.eps, branch_scale=0.0, u=u, rstd_pre=r_pre,
                      w_pre=self.p("w_pre0" if self.blocks else "w_last"), h8=h8, u8=u8)
        for i in range(self.blocks):
            a = u @ self.p(f"w1_{i}").t()
            a.relu_()
            a8 = keep(self.inner)
            dp.act8_pack(a, *a8)
            y = a.square_() @ self.p(f"w2_{i}").t()
            last = i + 1 == self.blocks
            h_next, u_next, r_post, r_next = new(), new(), r_pre.new_empty(T), r_pre.new_empty(T)
            y8, h8_next, u8_next = keep(C), keep(C), keep(C)
            dp.block_join(h, y, h_next, eps=self.eps, rstd_post=r_post,
                          w_post=self.p(f"w_post{i}"), gate=self.p(f"gate{i}"), u=u_next,
                          rstd_pre=r_next, w_pre=self.p("w_last" if last else f"w_pre{i + 1}"),
                          y8=y8, h8=h8_next, u8=u8_next)
            kept["blocks"].append(dict(u8=u8, a8=a8, y8=y8, r_post=r_post, h8=h8_next,
                                       r_pre=r_next))
            h, u, u8 = h_next, u_next, u8_next
        kept.update(first_h8=h8, first_r=r_pre, u8=u8)
        logits = u @ self.p("embed").t()
        kept["logits"] = logits
        kept["logprob"] = torch.empty(T, 1, device=dev)
        kept["stats"] = torch.empty(T, 2, device=dev)
        dp.token_logprob(logits, kept["targets"], kept["logprob"], kept["stats"], scratch)
        return kept

    def backward(self, kept, grad):
        """Gradients of -mean(logprob), times the loss scale, into the flat buffer `grad`."""
        T, C, dev = kept["inputs"].numel(), self.width, self.device
        scratch = self._scratch(T)

        def g(name):
            return self.view(grad, name)

        dlogits = kept["logits"]  # in place
        dp.token_logprob_backward(dlogits, kept["targets"], kept["stats"], dlogits,
                                  dlogprob=torch.full((T, 1), -1.0 / T, device=dev),
                                  loss_scale=self.scale_state)
        du = dlogits @ self.p("embed")
        dp.act8_wgrad(dlogits, *kept["u8"], g("embed"), scratch)
        dh = torch.zeros(T, C, dtype=BF16, device=dev)
        for i in reversed(range(self.blocks)):
            b = kept["blocks"][i]
            name = "w_last" if i + 1 == self.blocks else f"w_pre{i + 1}"
            dy = torch.empty(T, C, dtype=BF16, device=dev)
            dp.block_join_backward(dh, b["y8"], dy, dh, scratch, rstd_post=b["r_post"],
                                   w_post=self.p(f"w_post{i}"), dw_post=g(f"w_post{i}"),
                                   gate=self.p(f"gate{i}"), dgate=g(f"gate{i}"), du=du,
                                   h_out=b["h8"], rstd_pre=b["r_pre"], w_pre=self.p(name),
                                   dw_pre=g(name))
            # from the restored relu(z): d relu(z)^2 / dz = 2 relu(z), and the square
            # that W2 multiplied, packed for its weight gradient
            a = torch.empty(T, self.inner, dtype=BF16, device=dev)
            dp.act8_unpack(*b["a8"], a)
            da = (dy @ self.p(f"w2_{i}")) * (2 * a)
            dp.act8_pack(a.square_(), *b["a8"])
            dp.act8_wgrad(dy, *b["a8"], g(f"w2_{i}"), scratch)
            dp.act8_wgrad(da, *b["u8"], g(f"w1_{i}"), scratch)
            du = da @ self.p(f"w1_{i}")
        # the first norm's gradient: its "block output" is the stream itself, unused
        spare = torch.empty(T, C, dtype=BF16, device=dev)
        first = "w_pre0" if self.blocks else "w_last"
        dp.block_join_backward(dh, kept["first_h8"], spare, dh, scratch, branch_scale=0.0, du=du,
                               h_out=kept["first_h8"], rstd_pre=kept["first_r"],
                               w_pre=self.p(first), dw_pre=g(first))
        # the embedding's two roles share one gradient
        rows = torch.zeros(self.vocab, C, device=dev).index_add_(0, kept["inputs"], dh.float())
        g("embed").add_(rows)

    def update(self, lr=3e-3):
        """One loss-scaled AdamW step over the replicas' gradients: every rank's shard is
        averaged into the reduced gradient (and its squared norm taken), then one step
        reads it -- or is skipped where the global norm is not finite."""
        n = len(self.grads)
        shard = self.numel // n
        for r in range(n):
            dp.amp_average_sqnorm(self.grads, r, self.scale_state,
                                  self.average[r * shard:(r + 1) * shard], self.sqnorms[r:r + 1],
                                  self.norm_scratch)
        torch.sum(self.sqnorms, dim=0, keepdim=True, out=self.sqnorm)
        dp.amp_step([self.average], 0, self.numel, self.master, self.m, self.v, self.work, lr=lr,
                    beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, max_grad_norm=1.0,
                    global_sqnorm=self.sqnorm, state=self.scale_state, cfg=self.scale_cfg)


def batch(model, tokens, generator):
    """A synthetic task: the next token is a fixed permutation of the present one."""
    x = torch.randint(0, model.vocab, (tokens,), generator=generator, device=model.device)
    return x, (x * 5 + 17) % model.vocab


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=1024, help="tokens of a micro-batch")
    args = ap.parse_args(argv)
    model = BlockStack()
    g = torch.Generator(device=model.device).manual_seed(1)
    losses = []
    for step in range(args.steps):
        loss = 0.0
        for grad in model.grads:
            kept = model.forward(*batch(model, args.tokens, g))
            loss = loss - kept["logprob"].mean()
            model.backward(kept, grad)
        model.update()
        losses.append(loss / len(model.grads))
        if step % 10 == 0 or step + 1 == args.steps:
            print(f"step {step:4d}  loss {float(losses[-1]):.4f}")
    dp.stream_status()
    s = dp.read_loss_scale(model.scale_state)
    print(f"kept for the backward pass: {kept['bytes'] / args.tokens:.0f} bytes per token in 8 "
          f"bits; steps {s.step}, skipped {s.skipped}, loss scale {s.scale:g}")
    return [float(x) for x in losses]


if __name__ == "__main__":
    main()
