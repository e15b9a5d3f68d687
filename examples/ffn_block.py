"""Training steps of a feed-forward block, sharded over emulated ranks.

    y = x + W2 gelu(W1 rms_norm(x) + b1) + b2,   loss = mean((y - target)^2) / 2

What a rank of a sharded job does with one parameter group, through the public
calls: the all-gather places the bf16 parameters (tide_ag_place), the operators
run the block forward and backward on the rank's own tokens, the reduce-scatter
sums the bf16 gradients into fp32 shards (tide_rs_reduce), and each rank
updates its shard.  All N = M*L ranks live on this GPU and take turns.

Between forward and backward a rank keeps the block's input, the normalised
input and the pre-activation in 8 bits, and nothing else of their size.

    python examples/ffn_block.py [--tokens T] [--width D] [--inner F] [--nodes M] [--gpus L] [--steps K]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fsdp_layout_aware_gb300 as tide  # noqa: E402

BF = torch.bfloat16
EPS = 1e-5


class Block:
    """One rank's buffers and its forward and backward pass."""

    def __init__(self, tokens, width, inner):
        def new(*shape, dtype=BF):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        self.n, self.a, self.y = new(tokens, width), new(tokens, inner), new(tokens, width)
        self.dz, self.dn, self.dx = new(tokens, inner), new(tokens, width), new(tokens, width)
        self.rstd = new(tokens, dtype=torch.float32)
        self.x8, self.n8 = (tide.Checkpoint8.empty(tokens, width) for _ in range(2))
        self.z8 = tide.Checkpoint8.empty(tokens, inner)

    def forward(self, x, params):
        g, w1, b1, w2, b2 = params
        tide.tide_rms_norm(x, g, EPS, y=self.n, rstd=self.rstd, y8=self.n8)
        tide.tide_checkpoint_store(x, self.x8)
        tide.tide_linear(self.n, w1, self.a, bias=b1, act="gelu", z=self.z8)
        tide.tide_linear(self.a, w2, self.y, bias=b2, residual=x)
        return self.y

    def backward(self, dy, params, grads):
        g, w1, _, w2, _ = params
        dg, dw1, db1, dw2, db2 = grads
        tide.tide_linear_grad_weight(dy, self.z8, dw2, db=db2, act="gelu")
        tide.tide_linear_grad_input(dy, w2, self.dz, act="gelu", z=self.z8)
        tide.tide_linear_grad_weight(self.dz, self.n8, dw1, db=db1)
        tide.tide_linear_grad_input(self.dz, w1, self.dn)
        tide.tide_rms_norm_backward(self.dn, self.x8, g, self.rstd, self.dx, dweight=dg, dres=dy)
        return self.dx

    def kept_bytes(self):
        return sum(c.codes.numel() + c.scales.numel() for c in (self.x8, self.n8, self.z8)) + 4 * self.rstd.numel()


def pack(plan, tensors):
    """The ranks' padded, packed fp32 shards of full parameters."""
    shards = torch.zeros(plan.N, plan.S, device="cuda")
    for p, t in enumerate(tensors):
        flat = torch.zeros(plan.N * plan.e[p], device="cuda")
        flat[:t.numel()] = t.reshape(-1)
        shards[:, plan.o[p]:plan.o[p] + plan.e[p]] = flat.view(plan.N, plan.e[p])
    return shards


def train(tokens=256, width=512, inner=1536, nodes=1, gpus=4, steps=8, lr=2.0, seed=0, say=print):
    """Losses of `steps` steps."""
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    shapes = [(width,), (inner, width), (inner,), (width, inner), (width,)]
    first = [torch.ones(width, device="cuda"), randn(inner, width) / width ** 0.5, torch.zeros(inner, device="cuda"),
             randn(width, inner) / inner ** 0.5, torch.zeros(width, device="cuda")]
    mix = randn(width, width) / width ** 0.5  # the map to learn
    xs = [randn(tokens, width).to(BF) for _ in range(nodes * gpus)]
    losses = []
    with tide.TidePlan(shapes, nodes * gpus, nodes, gpus) as plan:
        plan.set_option(tide.TIDE_OPT_RS_AVERAGE, 1)
        master = pack(plan, first)
        reduced = [torch.empty(plan.S, device="cuda") for _ in range(plan.N)]
        placed = [torch.empty(plan.N * plan.e[p], dtype=BF, device="cuda") for p in range(plan.P)]
        params = [b[:t.numel()].view(t.shape) for b, t in zip(placed, first)]
        grads = [[torch.empty(s, dtype=BF, device="cuda") for s in shapes] for _ in range(plan.N)]
        flat_grads = [g for rank in grads for g in rank]
        block = Block(tokens, width, inner)
        for step in range(steps):
            shards = master.to(BF)
            plan.ag_place(list(shards), placed, 2)
            total = 0.0
            for rank, x in enumerate(xs):
                diff = block.forward(x, params).float() - torch.tanh(x.float() @ mix)
                total += 0.5 * diff.square().mean().item() / plan.N
                block.backward((diff / diff.numel() * tokens).to(BF), params, grads[rank])
            plan.rs_reduce(flat_grads, reduced)
            for rank in range(plan.N):
                master[rank].sub_(reduced[rank], alpha=lr / tokens)
            losses.append(total)
            say(f"step {step}: loss {total:.5f}")
        tide.tide_ops_check()
        plan.check()
        plain = 2 * tokens * (2 * width + inner) + 4 * tokens
        say(f"kept between forward and backward: {block.kept_bytes()} bytes a rank ({plain} in bf16)")
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 256), ("width", 512), ("inner", 1536), ("nodes", 1), ("gpus", 4), ("steps", 8)):
        ap.add_argument("--" + name, type=int, default=value)
    train(**vars(ap.parse_args()))


if __name__ == "__main__":
    main()
