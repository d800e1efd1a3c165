"""The attention of a sequence-parallel transformer block on W virtual ranks, every step in the
library: the packed QKV projection's output of each sequence shard goes through QK RMSNorm and
rotary positions into head shards (one launch), attends over the whole sequence, and comes back to
sequence shards (fast-ulysses 0.2.1, README, "Quick start": the block around the two all-to-alls).

    python -m ulysses_sequence_all_gb300.attention_block [--backward]

runs it on the video shape of the benchmark (21 x 45 x 80 tokens; a quarter of its heads by
default) with positions of time, height and width, and prints the time of each step.
"""
from __future__ import annotations

import argparse

import torch

from . import autograd as A
from . import binding as B


def axis_pairs(d: int, axes: int) -> list[int]:
    """RoPE pairs of a head of d columns shared out over the axes of a video (time, height, width)
    or an image (rows, columns): equal shares of d // (2 * axes), the first axis with the rest."""
    share = d // (2 * axes)
    return [d // 2 - share * (axes - 1)] + [share] * (axes - 1)


def attention_block(plan: B.Plan, qkv, rms_w, eps: float = 1e-6, rope_theta: float = 1e4,
                    scale: float | None = None, causal: bool = False, kv_lens=None):
    """Attention of packed shards: qkv is W tensors (b, s_q, 3, N, d), rms_w (2, d) fp32 the norm
    weights of q and k. The plan's RoPE settings hold (ulysses_plan_set_rope_grid gives positions
    of several axes). kv_lens: b key counts where the batch is padded at its end. Differentiable
    in qkv and rms_w. Returns W tensors (b, s_q, N, d)."""
    q, k, v = A.qkv_fused(plan, qkv, rms_w, eps, rope_theta)
    o = A.attention(plan, plan, q, k, v, scale, causal, kv_lens)
    return A.a2a_4d(plan, o, mode=1)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--grid", type=int, nargs="+", default=[21, 45, 80],
                    help="tokens along each position axis, the last fastest")
    ap.add_argument("--heads", type=int, default=8, help="a multiple of the ranks")
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--d", type=int, default=128)
    ap.add_argument("--backward", action="store_true")
    args = ap.parse_args(argv)
    W, d, N = args.ranks, args.d, args.heads
    if N % W:
        ap.error("--heads must be a multiple of --ranks")
    S = 1
    for n in args.grid:
        S *= n
    seq = [S // W + (r < S % W) for r in range(W)]
    plan = B.ulysses_plan(W, 1, seq, [N // W] * W, d, "bfloat16")
    B.ulysses_plan_set_rope_grid(plan, args.grid, axis_pairs(d, len(args.grid)))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    qkv = [torch.randn((1, s, 3, N, d), generator=gen, device="cuda").bfloat16()
           .requires_grad_(args.backward) for s in seq]
    rms_w = torch.ones(2, d, device="cuda", requires_grad=args.backward)

    def timed(what, fn, reps=3):
        fn()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(reps):
            out = fn()
        end.record()
        end.synchronize()
        print(f"{what:28s} {start.elapsed_time(end) / reps:9.3f} ms")
        return out

    q, k, v = timed("norm, rotation, to heads", lambda: A.qkv_fused(plan, qkv, rms_w, 1e-6, 1e4))
    o = timed("attention", lambda: A.attention(plan, plan, q, k, v))
    timed("back to the sequence", lambda: A.a2a_4d(plan, o, mode=1))
    if args.backward:
        def step():
            out = attention_block(plan, qkv, rms_w)
            torch.autograd.backward(out, [torch.ones_like(x) for x in out])
        timed("block, forward and backward", step)
    if B.ulysses_device_status():
        raise SystemExit("a kernel recorded a wait timeout")


if __name__ == "__main__":
    main()
