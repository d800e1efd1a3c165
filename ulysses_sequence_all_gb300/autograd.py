"""Differentiable forms of the library calls for PyTorch callers.

The pages' collective is differentiable and its backward uses the plan saved by its forward
(fast-ulysses 0.2.1, README, "Quick start" and "Limits"; FastVideo, "Ulysses performance on
GB200"). Here each call is a ``torch.autograd.Function`` over the C entry points, keeping the
plan for the backward:

* ``a2a_4d(plan, xs, mode)``: the relayout; its backward is the relayout in the other mode on
  the same plan (the relayout is a permutation, so its adjoint is its inverse).
* ``qk_fused(plan, q, k, rms_w, eps, rope_theta)``: the fused mode-0 call; its backward is
  ``ulysses_a2a_4d_qk_fused_backward`` (dq, dk and the gradient of ``rms_w``), with a workspace
  allocated by torch.
* ``qkv_fused(plan, qkv, rms_w, eps, rope_theta)``: the interleaved packed-QKV call; its backward
  is ``ulysses_a2a_4d_qkv_fused_backward`` (packed dqkv and the gradient of ``rms_w``).
* ``packed_fused(plan, packed, planes, q_plane, k_plane, rms_w, eps, rope_theta)``: the call on
  any packing of C planes per token (QKVG, ...); its backward is
  ``ulysses_a2a_4d_packed_fused_backward``; a token's columns beyond its planes get zero gradient.
* ``attention(q_plan, kv_plan, q, k, v, scale, causal, kv_lens, q_start)``: attention of every
  rank's heads over the whole sequence; its backward is ``ulysses_attention_backward``, from the
  output and the log-sum-exp that the forward keeps.

Inputs and outputs are lists of W tensors (one per virtual rank) on the current CUDA device;
the outputs are new tensors the caller owns. The relayout can be differentiated again, the others
once: a gradient of theirs raises where it is differentiated. Nothing here computes: every step runs in the
library's kernels, on the current stream.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding as B


def _shapes(plan: B.Plan, mode: int):
    """Output shapes of a call in `mode`: rank r's (b, S, n_r, d) for mode 0, rank q's
    (b, s_q, N, d) for mode 1."""
    S, N = sum(plan.seq_splits), sum(plan.head_splits)
    if mode == 0:
        return [(plan.b, S, n, plan.d) for n in plan.head_splits]
    return [(plan.b, s, N, plan.d) for s in plan.seq_splits]


def _empty(plan: B.Plan, mode: int, like: torch.Tensor):
    return [torch.empty(sh, dtype=like.dtype, device=like.device) for sh in _shapes(plan, mode)]


def _grads(grads, plan: B.Plan, mode: int, like: torch.Tensor):
    """Contiguous gradients of a call's outputs (mode: the call's), zeros where autograd passes
    None; `like` gives dtype and device."""
    out = []
    for g, sh in zip(grads, _shapes(plan, mode)):
        if g is None:
            g = torch.zeros(sh, dtype=like.dtype, device=like.device)
        out.append(g.contiguous())
    return out


class _A2A4D(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, mode, *xs):
        xs = [x.contiguous() for x in xs]
        outs = _empty(plan, mode, xs[0])
        B.ulysses_a2a_4d(plan, mode, xs, outs)
        ctx.plan, ctx.mode = plan, mode
        ctx.like = torch.empty(0, dtype=xs[0].dtype, device=xs[0].device)
        return tuple(outs)

    @staticmethod
    def backward(ctx, *grads):  # a relayout itself, and as differentiable
        gs = _grads(grads, ctx.plan, ctx.mode, ctx.like)
        return (None, None, *_A2A4D.apply(ctx.plan, 1 - ctx.mode, *gs))


def a2a_4d(plan: B.Plan, xs, mode: int = 0):
    """The relayout of W tensors, differentiable (backward: the other mode, same plan)."""
    if mode not in (0, 1):
        raise ValueError("mode must be 0 or 1")
    return list(_A2A4D.apply(plan, mode, *xs))


def _rope_plan(ctx):
    """The forward's plan, which rotates as it did then: the gradient of other positions or pairs would be
    another function's."""
    if ctx.plan.rope != ctx.rope:
        raise RuntimeError(f"the plan's RoPE settings changed between forward {ctx.rope} and backward "
                           f"{ctx.plan.rope}")
    return ctx.plan


class _QKFused(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, eps, rope_theta, rms_w, *qk):
        W = len(qk) // 2
        q = [x.contiguous() for x in qk[:W]]
        k = [x.contiguous() for x in qk[W:]]
        rms_w = rms_w.contiguous()
        qo, ko = _empty(plan, 0, q[0]), _empty(plan, 0, q[0])
        B.ulysses_a2a_4d_qk_fused(plan, q, k, qo, ko, rms_w, eps, rope_theta)
        ctx.rope = plan.rope
        ctx.plan, ctx.eps, ctx.theta, ctx.W = plan, eps, rope_theta, W
        ctx.save_for_backward(rms_w, *q, *k)
        return tuple(qo + ko)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        plan, W = _rope_plan(ctx), ctx.W
        rms_w, *qk = ctx.saved_tensors
        q, k = qk[:W], qk[W:]
        like = q[0]
        gq = _grads(grads[:W], plan, 0, like)
        gk = _grads(grads[W:], plan, 0, like)
        dq, dk = _empty(plan, 1, like), _empty(plan, 1, like)
        dw = torch.empty_like(rms_w, dtype=torch.float32)
        ws = torch.empty(B.ulysses_qk_fused_backward_workspace(plan), dtype=torch.uint8,
                         device=like.device)
        B.ulysses_a2a_4d_qk_fused_backward(plan, dq, dk, q, k, gq, gk, rms_w, dw, ctx.eps,
                                           ctx.theta, ws)
        return (None, None, None, dw, *dq, *dk)


class _QKVFused(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, eps, rope_theta, rms_w, *qkv):
        qkv = [x.contiguous() for x in qkv]
        rms_w = rms_w.contiguous()
        like = qkv[0]
        qo, ko, vo = _empty(plan, 0, like), _empty(plan, 0, like), _empty(plan, 0, like)
        B.ulysses_a2a_4d_qkv_fused(plan, qkv, qo, ko, vo, rms_w, eps, rope_theta)
        ctx.rope = plan.rope
        ctx.plan, ctx.eps, ctx.theta, ctx.W = plan, eps, rope_theta, len(qkv)
        ctx.save_for_backward(rms_w, *qkv)
        return tuple(qo + ko + vo)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        plan, W = _rope_plan(ctx), ctx.W
        rms_w, *qkv = ctx.saved_tensors
        like = qkv[0]
        gq = _grads(grads[:W], plan, 0, like)
        gk = _grads(grads[W:2 * W], plan, 0, like)
        gv = _grads(grads[2 * W:], plan, 0, like)
        dqkv = [torch.empty_like(x) for x in qkv]
        dw = torch.empty_like(rms_w, dtype=torch.float32)
        ws = torch.empty(B.ulysses_qk_fused_backward_workspace(plan), dtype=torch.uint8,
                         device=like.device)
        B.ulysses_a2a_4d_qkv_fused_backward(plan, dqkv, qkv, gq, gk, gv, rms_w, dw, ctx.eps,
                                            ctx.theta, ws)
        return (None, None, None, dw, *dqkv)


def qkv_fused(plan: B.Plan, qkv, rms_w: torch.Tensor, eps: float, rope_theta: float):
    """The interleaved call on packed (b, s_q, 3, N, d) inputs, differentiable in qkv and rms_w.
    Returns (q_out, k_out, v_out), lists of W tensors."""
    out = _QKVFused.apply(plan, eps, rope_theta, rms_w, *qkv)
    W = len(qkv)
    return list(out[:W]), list(out[W:2 * W]), list(out[2 * W:])


def qk_fused(plan: B.Plan, q, k, rms_w: torch.Tensor, eps: float, rope_theta: float):
    """The fused mode-0 call (QK RMSNorm + RoPE in the scatter), differentiable in q, k and
    rms_w ((2, d) fp32). Returns (q_out, k_out), lists of W tensors."""
    out = _QKFused.apply(plan, eps, rope_theta, rms_w, *q, *k)
    W = len(q)
    return list(out[:W]), list(out[W:])


class _PackedFused(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, planes, q_plane, k_plane, eps, rope_theta, rms_w, *packed):
        packed = [x.contiguous() for x in packed]
        rms_w = rms_w.contiguous()
        like = packed[0]
        pitch = like[0, 0].numel() * like.element_size() if like.dim() > 2 else like.element_size()
        outs = [_empty(plan, 0, like) for _ in range(planes)]
        B.ulysses_a2a_4d_packed_fused(plan, planes, q_plane, k_plane, pitch, packed, outs, rms_w,
                                      eps, rope_theta)
        ctx.rope = plan.rope
        ctx.plan, ctx.eps, ctx.theta, ctx.W = plan, eps, rope_theta, len(packed)
        ctx.planes, ctx.q_plane, ctx.k_plane, ctx.pitch = planes, q_plane, k_plane, pitch
        ctx.save_for_backward(rms_w, *packed)
        return tuple(t for plane in outs for t in plane)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        plan, W = _rope_plan(ctx), ctx.W
        rms_w, *packed = ctx.saved_tensors
        like = packed[0]
        gs = [_grads(grads[c * W:(c + 1) * W], plan, 0, like) for c in range(ctx.planes)]
        dpacked = [torch.zeros_like(x) for x in packed]  # columns beyond the planes: zero
        dw = torch.empty_like(rms_w, dtype=torch.float32)
        ws = torch.empty(B.ulysses_qk_fused_backward_workspace(plan), dtype=torch.uint8,
                         device=like.device)
        B.ulysses_a2a_4d_packed_fused_backward(plan, ctx.planes, ctx.q_plane, ctx.k_plane,
                                               ctx.pitch, dpacked, packed, gs, rms_w, dw, ctx.eps,
                                               ctx.theta, ws)
        return (None, None, None, None, None, None, dw, *dpacked)


def packed_fused(plan: B.Plan, packed, planes: int, q_plane: int, k_plane: int,
                 rms_w: torch.Tensor, eps: float, rope_theta: float):
    """The fused call on packed inputs (rank q's tensor: (b, s_q, ...) with `planes` planes of
    N * d elements at the start of each token, the token pitch being the product of the trailing
    dimensions), differentiable in packed and rms_w. Returns one list of W tensors per plane."""
    out = _PackedFused.apply(plan, planes, q_plane, k_plane, eps, rope_theta, rms_w, *packed)
    W = len(packed)
    return [list(out[c * W:(c + 1) * W]) for c in range(planes)]


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q_plan, kv_plan, scale, causal, kv_lens, q_start, *qkv):
        W = len(qkv) // 3
        qkv = [x.contiguous() for x in qkv]
        q, k, v = qkv[:W], qkv[W:2 * W], qkv[2 * W:]
        kv_lens = _counts(kv_lens, q_plan.b, q[0].device, "kv_lens")
        q_start = _counts(q_start, q_plan.b, q[0].device, "q_start")
        out = [torch.empty_like(x) for x in q]
        lse = [torch.empty((x.shape[0], x.shape[2], x.shape[1]), dtype=torch.float32,
                           device=x.device) for x in q]
        need = B.ulysses_attention_workspace(q_plan, kv_plan)
        ws = torch.empty(need, dtype=torch.uint8, device=q[0].device) if need else None
        B.ulysses_attention(q_plan, kv_plan, q, k, v, out, lse, scale, causal, kv_lens, q_start, ws)
        ctx.plans, ctx.scale, ctx.causal, ctx.W = (q_plan, kv_plan), scale, causal, W
        ctx.save_for_backward(kv_lens, q_start, *qkv, *out, *lse)
        return tuple(out)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        W = ctx.W
        kv_lens, q_start, *saved = ctx.saved_tensors
        q, k, v, out, lse = (saved[i * W:(i + 1) * W] for i in range(5))
        go = _grads(grads, ctx.plans[0], 0, q[0])
        dq, dk, dv = ([torch.empty_like(x) for x in t] for t in (q, k, v))
        ws = torch.empty(B.ulysses_attention_backward_workspace(*ctx.plans), dtype=torch.uint8,
                         device=q[0].device)
        B.ulysses_attention_backward(*ctx.plans, dq, dk, dv, q, k, v, out, lse, go, ctx.scale,
                                     ctx.causal, kv_lens, q_start, ws)
        return (None,) * 6 + (*dq, *dk, *dv)


def _counts(x, b, device, what):
    """A mask's counts as the library takes them: b int32 on the device (None stays None); wider ones
    that do not fit are beyond every key either way."""
    if x is None:
        return None
    x = torch.as_tensor(x)
    if x.numel() != b or x.is_floating_point() or x.is_complex():
        raise ValueError(f"{what}: {b} whole numbers, one per batch element, not {x.dtype} "
                         f"{tuple(x.shape)}")
    if x.dtype == torch.int64:
        x = x.clamp(-2 ** 31, 2 ** 31 - 1)
    return x.to(device=device, dtype=torch.int32).contiguous()


def _check_heads(plan, xs, what):
    """W device tensors shaped as mode 0's outputs with this plan, in its type: the kernels read as
    many elements as the plan says."""
    shapes = _shapes(plan, 0)
    if len(xs) != len(shapes):
        raise ValueError(f"{what}: {len(shapes)} tensors, one per rank, not {len(xs)}")
    for r, (x, sh) in enumerate(zip(xs, shapes)):
        if tuple(x.shape) != sh or not x.is_cuda or B.DTYPE_CODES.get(str(x.dtype)[6:]) != plan.code:
            raise ValueError(f"{what}[{r}]: {plan.dtype} {sh} on the device, not {x.dtype} "
                             f"{tuple(x.shape)} on {x.device}")


def attention(q_plan: B.Plan, kv_plan: B.Plan, q, k, v, scale: float | None = None,
              causal: bool = False, kv_lens=None, q_start=None):
    """Attention of every rank's heads over the whole sequence, on the head-side tensors that mode
    0 returns (lists of W: q (b, Sq, n_r, d), k and v (b, Skv, m_r, d)), differentiable in q, k and
    v; `scale` defaults to d ** -0.5. kv_lens and q_start: b whole numbers, a tensor on any device or
    a list. Returns a list of W tensors shaped as q."""
    for plan, xs, what in ((q_plan, q, "q"), (kv_plan, k, "k"), (kv_plan, v, "v")):
        _check_heads(plan, xs, what)
    scale = q_plan.d ** -0.5 if scale is None else scale
    return list(_Attention.apply(q_plan, kv_plan, scale, causal, kv_lens, q_start, *q, *k, *v))
