"""A sharded training step with 8-bit floating-point matrices and Muon, on one GPU.

    python examples/matrix_step.py [--steps 40]

A next-token model (an embedding, two matrices with a rectifier between them) is trained on a random walk
over tokens.  W ranks are simulated the way the library's own tests do it: their buffers are
slices of one GPU's memory and the collectives are copies.  Every step
  1. each rank quantizes its rows of both matrices in tiles (quant_f8); codes and exponents one after
     the other are the gathered matrix, which the products take as it is;
  2. each rank runs its tokens forward: activations quantized along rows and columns at once, the
     products from 8-bit blocks (matmul_f8);
  3. and backward: the input gradient from the transposed tiles (transpose_f8), the weight gradients
     from both operands along their columns, added to the fp32 gradient (micro-batches);
  4. the averaged gradients' squared norm (grad_sumsq) clips two optimizers: Muon steps the matrices, each
     on the rank that owns it, AdamW the embedding.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_communication_amd as zpq  # noqa: E402


def gathered(weight, ranks):
    """The matrix as the all-gather leaves it: every rank's rows (whole tiles, but for the last) in tiles."""
    rows = -(-weight.shape[0] // (128 * ranks)) * 128
    sent = [zpq.quant_f8(w, tile=True) for w in weight.split(rows)]
    return torch.cat([c.view(torch.uint8) for c, _ in sent]).view(torch.float8_e4m3fn), torch.cat([s for _, s in sent])


class Linear:
    """y = x w^T from a gathered matrix [outputs, inputs], and its backward pass."""

    def __init__(self, w, inputs, grad):
        self.w, self.inputs, self.grad = w, inputs, grad

    def forward(self, x):
        rows, self.x = zpq.quant_f8(x, along="both")
        return zpq.matmul_f8(rows, self.w)

    def backward(self, dy, need_input=True):
        rows, cols = zpq.quant_f8(dy, along="both", dtype=torch.float8_e5m2)
        zpq.matmul_f8(cols, self.x, out=self.grad, accumulate=True)
        return zpq.matmul_f8(rows, zpq.transpose_f8(*self.w, cols=self.inputs)) if need_input else None


def forward_backward(ids, target, table, one, two, grads, scale):
    """Loss of a batch; adds the gradients of `scale` times its sum to grads."""
    e = zpq.embedding(ids, table, out_dtype=torch.bfloat16)
    h = one.forward(e)
    r = torch.relu(h)
    logp = torch.log_softmax(two.forward(r).float(), 1)
    d = logp.exp()
    d.scatter_add_(1, target[:, None], torch.full_like(d[:, :1], -1.0))
    dr = two.backward((d * scale).bfloat16())
    de = one.backward(torch.where(h > 0, dr, torch.zeros_like(dr)))
    zpq.embedding_grad(ids, de, table.shape[0], out=grads[0], accumulate=True)
    return -logp.gather(1, target[:, None]).mean()


def train(steps=40, vocab=500, dim=96, hidden=320, batch=256, ranks=4, micro=2, lr=0.02, seed=0):
    """Losses of each step, averaged over ranks and micro-batches."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    table, first, second = rand(vocab, dim), rand(hidden, dim) / math.sqrt(dim), rand(vocab, hidden) / math.sqrt(hidden)
    grads = [torch.zeros_like(t) for t in (table, first, second)]
    # a rank owns whole matrices: here rank 0 the first, rank 1 the second
    muon = [zpq.Muon([p], [g], lr=lr, momentum=0.9) for p, g in zip((first, second), grads[1:])]
    adam = zpq.AdamW([table], grads[:1], lr=lr, betas=(0.9, 0.95), weight_decay=0.0)
    losses = []
    for step in range(1, steps + 1):
        weights = gathered(first, ranks), gathered(second, ranks)
        for g in grads:
            g.zero_()
        loss = torch.zeros((), device="cuda")
        for _ in range(ranks * micro):
            ids = torch.randint(0, vocab, (batch,), generator=gen, device="cuda")
            target = (ids * 7 + torch.randint(0, 3, (batch,), generator=gen, device="cuda")) % vocab
            one, two = Linear(weights[0], dim, grads[1]), Linear(weights[1], hidden, grads[2])
            loss += forward_backward(ids, target, table, one, two, grads, 1 / (batch * ranks * micro))
        losses.append(loss.item() / (ranks * micro))
        total = adam.grad_sumsq()
        for m in muon:
            m.grad_sumsq(out=total, accumulate=True)
        for m in muon:
            m.step(sumsq=total, max_norm=1.0)
        adam.step(step, sumsq=total, max_norm=1.0)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    losses = train(steps=ap.parse_args().steps)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i + 1:4d}  loss {losses[i]:.4f}")
    print(f"step {len(losses):4d}  loss {losses[-1]:.4f}")
