"""A stack of MLP blocks with 4-bit weights, each between its norms:

    f = relu(h · W_upᵀ),   o = f · W_downᵀ,
    x ← x + scale · gate ⊙ rms(o)·post,   h ← rms(x)·pre of the next block

Three calls per block: gemm_w4 (with the ReLU), gemm_w4, and norm_residual, which is
the post-norm, the gate, the residual sum and the next block's pre-norm in one pass.

run():     the rows of a prompt.
Token:     one row at a time, the whole stack captured as one CUDA graph.
tune():    a gradient step on the last block's post, gate and pre, through
           norm_residual_backward (the 4-bit weights stay as they are).

    python examples/mlp_block.py [--dim 4096] [--hidden 16384] [--blocks 4]
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_fp16_gemm_gb300 as tg  # noqa: E402


def quantise(w, group, dtype):
    """4-bit codes, scales and zero points of w [out][in]: each group of `group`
    inputs of a row spans its least to its greatest value (and 0) in 15 steps."""
    N, K = w.shape
    groups = -(-K // group)
    v = torch.nn.functional.pad(w.float(), (0, groups * group - K)).view(N, groups, group)
    low, high = v.amin(dim=2).clamp(max=0), v.amax(dim=2).clamp(min=0)
    scale = ((high - low) / 15).clamp(min=1e-6).to(dtype)
    zero = (-low / scale.float()).round().clamp(0, 15)
    code = (v / scale.float()[..., None] + zero[..., None]).round().clamp(0, 15)
    code = code.to(torch.uint8).view(N, -1)[:, :K + K % 2]
    # rows of whole 16 bytes, scales and zero points [group][out]
    bq = torch.zeros(N, -(-code.shape[1] // 32) * 16, dtype=torch.uint8, device=w.device)
    bq[:, :code.shape[1] // 2] = code[:, 0::2] | code[:, 1::2] << 4
    wide = torch.zeros(groups, -(-N // 16) * 16, dtype=dtype, device=w.device)
    bscale, bzero = wide[:, :N], wide.to(torch.uint8)[:, :N]
    bscale.copy_(scale.T)
    bzero.copy_(zero.T)
    return {"bq": bq[:, :(K + 1) // 2], "bscale": bscale, "N": N, "group": group, "bzero": bzero}


class Stack:
    """`blocks` blocks with random weights; x and h are of `dtype`."""

    def __init__(self, blocks, dim, hidden, *, group=128, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device=device)

        self.scale, self.dim, self.dtype = blocks ** -0.5, dim, dtype
        self.first = 1 + 0.1 * normal(dim)  # pre-norm of the first block
        self.up, self.down, self.norms = [], [], []
        for _ in range(blocks):
            self.up.append(quantise(normal(hidden, dim) * dim ** -0.5, group, dtype))
            self.down.append(quantise(normal(dim, hidden) * hidden ** -0.5, group, dtype))
            self.norms.append({"post_weight": 1 + 0.1 * normal(dim),
                               "gate": (0.5 + 0.1 * normal(dim)).to(dtype),
                               "pre_weight": 1 + 0.1 * normal(dim)})

    def block(self, i, h):
        """The block's output, before its norms."""
        return tg.gemm_w4(tg.gemm_w4(h, relu=True, **self.up[i]), **self.down[i])

    def run(self, x):
        """(x, h) after the last block and its norms, for the rows of x."""
        _, h = tg.norm_residual(x, pre_weight=self.first)
        for i, norm in enumerate(self.norms):
            x, h = tg.norm_residual(self.block(i, h), x, scale=self.scale, **norm)
        return x, h


class Token:
    """The stack on one row, as a graph: step(x) gives h."""

    def __init__(self, stack):
        self.x = torch.zeros(1, stack.dim, dtype=stack.dtype, device=stack.first.device)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            stack.run(self.x)  # the workspaces of this stream come before the capture
        stream.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=stream):
            _, self.h = stack.run(self.x)

    def step(self, x):
        self.x.copy_(x)
        self.graph.replay()
        return self.h


def tune(stack, x, target, rate):
    """A step on mean((h - target)²) / 2 in the last block's norms; returns the loss."""
    _, h = tg.norm_residual(x, pre_weight=stack.first)
    for i, norm in enumerate(stack.norms[:-1]):
        x, h = tg.norm_residual(stack.block(i, h), x, scale=stack.scale, **norm)
    norm, o = stack.norms[-1], stack.block(len(stack.norms) - 1, h)
    _, h = tg.norm_residual(o, x, scale=stack.scale, **norm)
    error = h.float() - target.float()
    dh = (error / error.shape[0]).to(h.dtype)  # of the mean over rows, summed over columns
    grads = tg.norm_residual_backward(None, dh, o, x, scale=stack.scale, **norm)
    norm["post_weight"] -= rate * grads.post_weight
    norm["pre_weight"] -= rate * grads.pre_weight
    norm["gate"] -= rate * grads.gate
    return float((error * error).mean()) / 2


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--dim", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=16384)
    ap.add_argument("--blocks", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=512)
    a = ap.parse_args()
    stack = Stack(a.blocks, a.dim, a.hidden)
    x = torch.randn(a.prompt, a.dim, device="cuda").to(stack.dtype)

    def timed(what, f, reps=20):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(reps):
            f()
        torch.cuda.synchronize()
        print(f"{what}: {(time.perf_counter() - t) / reps * 1e6:.1f} us")

    timed(f"{a.prompt} rows through {a.blocks} blocks", lambda: stack.run(x))
    token = Token(stack)
    timed("one row, as a graph", lambda: token.step(x[:1]))
    target = stack.run(x)[1].float() * 1.5
    losses = [tune(stack, x, target, 0.2) for _ in range(5)]
    print("loss of five steps:", " ".join(f"{v:.4f}" for v in losses))
    tg.sync_status()


if __name__ == "__main__":
    main()
