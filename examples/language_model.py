"""Training steps of a small language model, sharded over emulated ranks.

    x = scale * E[ids],   y = x + W2 gelu(W1 rms_norm(x) + b1) + b2,   z = H rms_norm(y)
    loss = -mean over the tokens of log softmax(z)[next id]

What a rank of a sharded job does from the ids of its batch to the update of its
shard, through the public calls: the all-gather places the bf16 parameters
(tide_ag_place), the token embedding, the feed-forward block (ffn_block.py), the
output's linear layer and the log probabilities run forward and backward, the
reduce-scatter averages the bf16 gradients into fp32 shards (tide_rs_reduce),
and the shards' global norm clips them before the update.  All N = M*L ranks live
on this GPU and take turns; the norm is one call over all ranks' shards, which a job on
N GPUs joins from the ranks' norms.

    python examples/language_model.py [--tokens T] [--vocab V] [--width D] [--inner F] [--nodes M] [--gpus L] [--steps K]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import fsdp_layout_aware_gb300 as tide  # noqa: E402
from ffn_block import BF, EPS, Block, pack  # noqa: E402

PADDING = -1  # a place without a token: no input, no loss, no gradient


class Model:
    """One rank's buffers, and its loss and gradients for a batch of ids."""

    def __init__(self, tokens, vocab, width, inner):
        def new(*shape, dtype=BF):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        self.scale = width ** 0.5
        self.block = Block(tokens, width, inner)
        self.x, self.n, self.dn, self.dy = (new(tokens, width) for _ in range(4))
        self.logits = new(tokens, vocab)  # and their gradient, in place
        self.rstd, self.logp, self.lse, self.dlogp = (new(tokens, dtype=torch.float32) for _ in range(4))

    def loss(self, ids, targets, params):
        """Minus the log probabilities' mean over the targets that are not padding, on the GPU."""
        table, *ffn, g, head = params
        tide.tide_embedding(ids, table, self.x, scale=self.scale)
        self.y = self.block.forward(self.x, ffn)
        tide.tide_rms_norm(self.y, g, EPS, y=self.n, rstd=self.rstd)
        tide.tide_linear(self.n, head, self.logits)
        tide.tide_log_probs(self.logits, targets, self.logp, lse=self.lse)
        self.count = (targets != PADDING).sum().clamp(min=1)
        return -self.logp.sum() / self.count

    def backward(self, ids, targets, params, grads):
        """Gradients of the last loss."""
        _, *ffn, g, head = params
        dtable, *dffn, dg, dhead = grads
        self.dlogp.copy_((-1.0 / self.count).expand_as(self.dlogp))
        tide.tide_log_probs_backward(self.logits, self.lse, self.logits, targets=targets, dlogp=self.dlogp)
        tide.tide_linear_grad_weight(self.logits, self.n, dhead)
        tide.tide_linear_grad_input(self.logits, head, self.dn)
        tide.tide_rms_norm_backward(self.dn, self.y, g, self.rstd, self.dy, dweight=dg)
        dx = self.block.backward(self.dy, ffn, dffn)
        tide.tide_embedding_backward(ids, dx, dtable, scale=self.scale)


def shapes_of(vocab, width, inner):
    return [(vocab, width), (width,), (inner, width), (inner,), (width, inner), (width,), (width,), (vocab, width)]


def train(tokens=256, vocab=1000, width=256, inner=512, nodes=1, gpus=4, steps=8, lr=0.5, max_norm=1.0, seed=0, say=print):
    """(loss, norm) of `steps` steps."""
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    shapes = shapes_of(vocab, width, inner)
    first = [randn(*s) / s[-1] ** 0.5 if len(s) == 2 else torch.zeros(*s, device="cuda") for s in shapes]
    first[1].fill_(1.0), first[6].fill_(1.0)  # the norms' weights
    # A batch a rank: ids that follow one another by a fixed rule, the last quarter of it padding.
    rule = torch.randperm(vocab, generator=gen, device="cuda")
    batches = []
    for _ in range(nodes * gpus):
        ids = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
        ids[3 * tokens // 4:] = PADDING
        batches.append((ids, torch.where(ids == PADDING, PADDING, rule[ids.clamp(min=0)])))
    history = []
    with tide.TidePlan(shapes, nodes * gpus, nodes, gpus) as plan:
        plan.set_option(tide.TIDE_OPT_RS_AVERAGE, 1)
        master = pack(plan, first)
        reduced = [torch.empty(plan.S, device="cuda") for _ in range(plan.N)]
        shards = tide.TensorList(reduced)
        norm = torch.empty(1, device="cuda")
        placed = [torch.empty(plan.N * plan.e[p], dtype=BF, device="cuda") for p in range(plan.P)]
        params = [b[:t.numel()].view(t.shape) for b, t in zip(placed, first)]
        grads = [[torch.empty(s, dtype=BF, device="cuda") for s in shapes] for _ in range(plan.N)]
        flat_grads = [g for rank in grads for g in rank]
        model = Model(tokens, vocab, width, inner)
        for step in range(steps):
            plan.ag_place(list(master.to(BF)), placed, 2)
            total = 0.0
            for rank, (ids, targets) in enumerate(batches):
                total += model.loss(ids, targets, params).item() / plan.N
                model.backward(ids, targets, params, grads[rank])
            plan.rs_reduce(flat_grads, reduced)
            tide.tide_grad_norm(shards, norm)
            tide.tide_grad_clip(shards, norm, max_norm)
            for rank in range(plan.N):
                master[rank].sub_(reduced[rank], alpha=lr)
            history.append((total, norm.item()))
            say(f"step {step}: loss {total:.5f}, gradient norm {norm.item():.4f}")
        tide.tide_ops_check()
        plan.check()
    return history


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 256), ("vocab", 1000), ("width", 256), ("inner", 512), ("nodes", 1), ("gpus", 4), ("steps", 8)):
        ap.add_argument("--" + name, type=int, default=value)
    train(**vars(ap.parse_args()))


if __name__ == "__main__":
    main()
