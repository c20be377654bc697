"""Tensor wrappers of the training-side operators (include/dpopt.h): the block
join and its gradient, activations packed into 8 bits and the weight gradient
formed from them, log probabilities of given tokens and their gradient.

Marshalling and shape checks only; the work runs in the CUDA library.  A matrix
is a 2-D tensor whose columns are adjacent (any row stride).  A packed matrix is
the pair (codes, exps) that act8_empty() makes: int8 rows x cols, uint8 rows x
ceil(cols / 32).  Nothing is allocated by a call; outputs and scratch are the
caller's.  Calls enqueue on `stream` (default: the current one), to which the
tensors must belong like those of any kernel launched there.
"""
from __future__ import annotations

from .binding import (
    Act8, BlockJoinArgs, BlockJoinGradArgs, Matrix, _check, _grad_dtype, _operand, _stream_handle,
    dpopt_act8_pack, dpopt_act8_unpack, dpopt_act8_wgrad, dpopt_act8_wgrad_scratch_bytes,
    dpopt_block_join, dpopt_block_join_backward, dpopt_block_join_scratch_bytes,
    dpopt_token_logprob, dpopt_token_logprob_backward, dpopt_token_logprob_scratch_bytes,
)

ACT8_BLOCK = 32


def _want(t, name: str, shape, dtype=None) -> None:
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: {t.dtype}, expected {dtype}")


def _address(t) -> int:
    return _operand(t) if t.numel() else 0


def _matrix(t, name: str, shape, dtype=None) -> tuple[int, int]:
    """Address and row stride of a 2-D tensor with adjacent columns."""
    _want(t, name, shape, dtype)
    if t.numel() and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: columns must be adjacent (column stride {t.stride(1)})")
    return _address(t), t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _flat(t, name: str, shape, dtype) -> int:
    """Address of a contiguous tensor."""
    _want(t, name, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return _address(t)


def _packed(pair, name: str, rows: int, cols: int) -> tuple[int, int, int, int]:
    import torch
    codes, exps = pair
    return (*_matrix(codes, f"{name} codes", (rows, cols), torch.int8),
            *_matrix(exps, f"{name} exps", (rows, -(-cols // ACT8_BLOCK)), torch.uint8))


def _scratch(t) -> tuple[int, int]:
    if t is None:
        return 0, 0
    if not t.is_contiguous():
        raise ValueError("scratch: must be contiguous")
    return _address(t), t.numel() * t.element_size()


def _rows_cols(t, name: str) -> tuple[int, int]:
    if t.dim() != 2:
        raise ValueError(f"{name}: expected 2 dimensions, got {t.dim()}")
    return t.shape[0], t.shape[1]


def act8_empty(rows: int, cols: int, device="cuda"):
    """Storage for a packed rows x cols matrix: (codes, exps), uninitialised."""
    import torch
    return (torch.empty(rows, cols, dtype=torch.int8, device=device),
            torch.empty(rows, -(-cols // ACT8_BLOCK), dtype=torch.uint8, device=device))


def act8_pack(x, codes, exps, stream=None) -> None:
    """Pack x (bf16, fp16 or fp32) into 8-bit codes and one exponent byte per 32 columns."""
    rows, cols = _rows_cols(x, "x")
    px, ldx = _matrix(x, "x", (rows, cols))
    c, ldc, e, lde = _packed((codes, exps), "packed", rows, cols)
    _check(dpopt_act8_pack(px, _grad_dtype(x), rows, cols, ldx, c, ldc, e, lde,
                           _stream_handle(stream)), "dpopt_act8_pack")


def act8_unpack(codes, exps, x, stream=None) -> None:
    """Write the packed matrix's values to x."""
    rows, cols = _rows_cols(x, "x")
    px, ldx = _matrix(x, "x", (rows, cols))
    c, ldc, e, lde = _packed((codes, exps), "packed", rows, cols)
    _check(dpopt_act8_unpack(c, ldc, e, lde, rows, cols, px, _grad_dtype(x), ldx,
                             _stream_handle(stream)), "dpopt_act8_unpack")


def act8_wgrad_scratch_bytes(tokens: int, n: int, k: int) -> int:
    rc, nbytes = dpopt_act8_wgrad_scratch_bytes(tokens, n, k)
    _check(rc, "dpopt_act8_wgrad_scratch_bytes")
    return nbytes


def act8_wgrad(dy, codes, exps, dw, scratch=None, *, addend=None, stream=None) -> None:
    """dw (n x k) = dy^T X (+ addend): the weight gradient of y = x W^T from dy (tokens x n,
    bf16 or fp16) and the packed x (tokens x k).  addend: a matrix like dw, or dw itself.
    scratch: a device tensor of act8_wgrad_scratch_bytes(tokens, n, k) bytes."""
    tokens, n = _rows_cols(dy, "dy")
    k = _rows_cols(codes, "codes")[1]
    pdy, lddy = _matrix(dy, "dy", (tokens, n))
    c, ldc, e, lde = _packed((codes, exps), "packed", tokens, k)
    pdw, lddw = _matrix(dw, "dw", (n, k))
    pa, lda = (0, 0) if addend is None else _matrix(addend, "addend", (n, k), dw.dtype)
    _check(dpopt_act8_wgrad(pdy, _grad_dtype(dy), lddy, c, ldc, e, lde, tokens, n, k, pdw,
                            _grad_dtype(dw), lddw, pa, lda, *_scratch(scratch),
                            _stream_handle(stream)), "dpopt_act8_wgrad")


def block_join_scratch_bytes(rows: int, cols: int, gate_rows: int = 0) -> int:
    rc, nbytes = dpopt_block_join_scratch_bytes(rows, cols, gate_rows)
    _check(rc, "dpopt_block_join_scratch_bytes")
    return nbytes


def _param_dtype(tensors, default) -> int:
    """The one type of the weights and gates given."""
    kinds = {t.dtype for t in tensors if t is not None}
    if len(kinds) > 1:
        raise TypeError(f"weights, gates and their gradients must share one type, got {kinds}")
    return _grad_dtype(next(t for t in tensors if t is not None)) if kinds else default


def _gate_shape(rows: int, cols: int, gate_rows: int) -> tuple[int, int]:
    if gate_rows < 0:
        raise ValueError("gate_rows must be >= 0")
    return (1 if gate_rows == 0 else -(-rows // gate_rows), cols)


def block_join(h, y, h_out, *, eps: float, rstd_post=None, w_post=None, gate=None,
               gate_rows: int = 0, res_scale: float = 1.0, branch_scale: float = 1.0, u=None,
               rstd_pre=None, w_pre=None, y8=None, h8=None, u8=None, stream=None) -> None:
    """h_out = res_scale * h + branch_scale * gate * norm(y) * w_post and u = norm(h_out) * w_pre.

    h, y, h_out, u: rows x cols of one type (h_out may be h).  rstd_post, rstd_pre: float32
    rows, written (rstd_post None: no norm after the block; u None: none before the next).
    gate: one row for all rows (gate_rows 0) or one for each run of gate_rows rows.  y8,
    h8, u8: packed matrices that receive the 8-bit checkpoints of y, h_out and u."""
    import torch
    rows, cols = _rows_cols(h, "h")
    dt = h.dtype
    a = BlockJoinArgs(rows=rows, cols=cols, dtype=_grad_dtype(h),
                      param_dtype=_param_dtype((w_post, w_pre, gate), _grad_dtype(h)), eps=eps,
                      res_scale=res_scale, branch_scale=branch_scale, gate_rows=gate_rows)
    a.h = Matrix(*_matrix(h, "h", (rows, cols)))
    a.y = Matrix(*_matrix(y, "y", (rows, cols), dt))
    a.h_out = Matrix(*_matrix(h_out, "h_out", (rows, cols), dt))
    if u is not None:
        a.u = Matrix(*_matrix(u, "u", (rows, cols), dt))
    if gate is not None:
        a.gate = Matrix(*_matrix(gate, "gate", _gate_shape(rows, cols, gate_rows)))
    for name, t in (("w_post", w_post), ("w_pre", w_pre)):
        if t is not None:
            setattr(a, name, _flat(t, name, (cols,), t.dtype))
    for name, t in (("rstd_post", rstd_post), ("rstd_pre", rstd_pre)):
        if t is not None:
            setattr(a, name, _flat(t, name, (rows,), torch.float32))
    for name, pair in (("y8", y8), ("h8", h8), ("u8", u8)):
        if pair is not None:
            setattr(a, name, Act8(*_packed(pair, name, rows, cols)))
    _check(dpopt_block_join(a, _stream_handle(stream)), "dpopt_block_join")


def block_join_backward(dh_out, y, dy, dh, scratch, *, rstd_post=None, w_post=None, dw_post=None,
                        gate=None, gate_rows: int = 0, dgate=None, res_scale: float = 1.0,
                        branch_scale: float = 1.0, du=None, h_out=None, rstd_pre=None, w_pre=None,
                        dw_pre=None, stream=None) -> None:
    """Gradients of block_join: dy and dh (None: not wanted; may be dh_out), and dw_post, dw_pre,
    dgate where given.  y and h_out are the forward call's tensors or their packed
    checkpoints (codes, exps); rstd_post and rstd_pre are those it stored.  du None: the
    join had no norm before the next block.  scratch: a device tensor of
    block_join_scratch_bytes(rows, cols, gate_rows) bytes."""
    import torch
    rows, cols = _rows_cols(dh_out, "dh_out")
    dt = dh_out.dtype
    a = BlockJoinGradArgs(
        rows=rows, cols=cols, dtype=_grad_dtype(dh_out),
        param_dtype=_param_dtype((w_post, w_pre, gate, dw_post, dw_pre, dgate),
                                 _grad_dtype(dh_out)),
        res_scale=res_scale, branch_scale=branch_scale, gate_rows=gate_rows)
    a.dh_out = Matrix(*_matrix(dh_out, "dh_out", (rows, cols)))
    a.dy = Matrix(*_matrix(dy, "dy", (rows, cols), dt))
    for name, t in (("dh", dh), ("du", du)):
        if t is not None:
            setattr(a, name, Matrix(*_matrix(t, name, (rows, cols), dt)))
    for name, eight, t in (("y", "y8", y), ("h_out", "h8", h_out)):
        if isinstance(t, (tuple, list)):
            setattr(a, eight, Act8(*_packed(t, name, rows, cols)))
        elif t is not None:
            setattr(a, name, Matrix(*_matrix(t, name, (rows, cols), dt)))
    for name, t in (("gate", gate), ("dgate", dgate)):
        if t is not None:
            setattr(a, name, Matrix(*_matrix(t, name, _gate_shape(rows, cols, gate_rows))))
    for name, t in (("w_post", w_post), ("w_pre", w_pre), ("dw_post", dw_post),
                    ("dw_pre", dw_pre)):
        if t is not None:
            setattr(a, name, _flat(t, name, (cols,), t.dtype))
    for name, t in (("rstd_post", rstd_post), ("rstd_pre", rstd_pre)):
        if t is not None:
            setattr(a, name, _flat(t, name, (rows,), torch.float32))
    a.scratch, a.scratch_bytes = _scratch(scratch)
    _check(dpopt_block_join_backward(a, _stream_handle(stream)), "dpopt_block_join_backward")


def token_logprob_scratch_bytes(rows: int, vocab: int, top: int = 0) -> int:
    rc, nbytes = dpopt_token_logprob_scratch_bytes(rows, vocab, top)
    _check(rc, "dpopt_token_logprob_scratch_bytes")
    return nbytes


def token_logprob(logits, tokens, logprob, stats, scratch=None, *, entropy=None,
                  top_logprob=None, top_index=None, inv_temperature: float = 1.0,
                  stream=None) -> None:
    """Log probabilities of `tokens` (int64, rows x n; negative: none) under softmax(logits *
    inv_temperature): logprob (float32, rows x n) and stats (float32, rows x 2, for the
    gradient); optionally entropy (float32 rows) and the largest alternatives, top_logprob
    (float32) and top_index (int64), rows x top.  scratch: a device tensor of
    token_logprob_scratch_bytes(rows, vocab, top) bytes."""
    import torch
    rows, vocab = _rows_cols(logits, "logits")
    n = _rows_cols(tokens, "tokens")[1]
    px, ld = _matrix(logits, "logits", (rows, vocab))
    if (top_logprob is None) != (top_index is None):
        raise ValueError("top_logprob and top_index must be given together")
    top = 0 if top_index is None else _rows_cols(top_index, "top_index")[1]
    f32 = torch.float32
    _check(dpopt_token_logprob(
        px, _grad_dtype(logits), rows, vocab, ld, _flat(tokens, "tokens", (rows, n), torch.int64),
        n, inv_temperature, _flat(logprob, "logprob", (rows, n), f32),
        _flat(stats, "stats", (rows, 2), f32),
        0 if entropy is None else _flat(entropy, "entropy", (rows,), f32), top,
        0 if top == 0 else _flat(top_logprob, "top_logprob", (rows, top), f32),
        0 if top == 0 else _flat(top_index, "top_index", (rows, top), torch.int64),
        *_scratch(scratch), _stream_handle(stream)), "dpopt_token_logprob")


def token_logprob_backward(logits, tokens, stats, dlogits, *, dlogprob, entropy=None,
                           dentropy=None, inv_temperature: float = 1.0, loss_scale=None,
                           stream=None) -> None:
    """dlogits (may be logits) = the gradient of sum(dlogprob * logprob) + sum(dentropy *
    entropy), times the current scale of `loss_scale` (the device state of
    loss_scale_init(); None: 1).  stats and entropy are those token_logprob stored."""
    import torch
    rows, vocab = _rows_cols(logits, "logits")
    n = _rows_cols(tokens, "tokens")[1]
    px, ld = _matrix(logits, "logits", (rows, vocab))
    pd, ldd = _matrix(dlogits, "dlogits", (rows, vocab), logits.dtype)
    f32 = torch.float32
    if loss_scale is not None and loss_scale.numel() * loss_scale.element_size() < 32:
        raise ValueError("loss_scale: the state is 32 bytes")
    _check(dpopt_token_logprob_backward(
        px, _grad_dtype(logits), rows, vocab, ld, _flat(tokens, "tokens", (rows, n), torch.int64),
        n, inv_temperature, _flat(stats, "stats", (rows, 2), f32),
        _flat(dlogprob, "dlogprob", (rows, n), f32),
        0 if entropy is None else _flat(entropy, "entropy", (rows,), f32),
        0 if dentropy is None else _flat(dentropy, "dentropy", (rows,), f32),
        0 if loss_scale is None else _operand(loss_scale), pd, ldd, _stream_handle(stream)),
        "dpopt_token_logprob_backward")
