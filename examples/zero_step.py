"""A sharded training step around qwZ and qgZ, on one GPU.

    python examples/zero_step.py [--steps 60] [--state-bits 8]

A next-token model (an embedding table and an output matrix) is trained on a
random walk over tokens.  W = L * N ranks are simulated the way the
library's own tests do it: a rank's buffers are slices of one GPU's memory and the
collectives are copies.  Every rank
  1. quantizes its slice of the fp16 weights (quant_i8); the slices' codes and
     scales, one after the other, are the gathered buffer;
  2. looks its tokens up straight in the gathered INT8 table (embedding_i8); the
     output matrix is dequantized (dequant_i8);
  3. computes the loss and, by hand, the gradients: of the table from the
     tokens (embedding_grad), of the matrix by products;
  4. reorders and quantizes them (qgz_reorder_quant_i4), and after each hop
     reduces what it received (qgz_dequant_reduce_requant_i4);
  5. adds its slice's squared norm to the others' (grad_sumsq) and steps its
     slice (AdamW), which writes the fp16 weights of the next step.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_communication_amd as zpq  # noqa: E402

QW, QG = 256, 64                       # quantization blocks of weights and gradients


class Rank:
    """One rank's slice of the flat weights: fp32 master, fp16 copy, gradient,
    optimizer.  A slice may end in the middle of a tensor: it is stepped as the
    pieces of the tensors that it holds, each with its tensor's weight decay."""

    def __init__(self, flat, first, size, tensors, lr, state_bits, seed):
        self.master = flat[first:first + size].clone()
        self.half = self.master.half()
        self.grad = torch.zeros(size, dtype=torch.float16, device="cuda")
        cuts = [(max(a, first) - first, min(b, first + size) - first, decay) for a, b, decay in tensors
                if a < first + size and b > first]
        part = lambda x: [x[a:b] for a, b, _ in cuts]  # noqa: E731
        self.opt = zpq.AdamW(part(self.master), part(self.grad), copies=part(self.half), lr=lr, betas=(0.9, 0.95),
                             weight_decay=[d for _, _, d in cuts], state_bits=state_bits, seed=seed)


def train(steps=60, vocab=500, dim=96, batch=512, local_ranks=2, nodes=2, lr=3e-2, state_bits=8, seed=0):
    """Losses of each step, averaged over the ranks."""
    L, N = local_ranks, nodes
    W = L * N
    gen = torch.Generator(device="cuda").manual_seed(seed)
    table, matrix = vocab * dim, dim * vocab
    whole = W * QW * QG                                        # any slice is whole blocks of both kinds
    n = -(-(table + matrix) // whole) * whole
    S = n // W
    flat = torch.zeros(n, device="cuda")
    flat[:table + matrix] = torch.randn(table + matrix, generator=gen, device="cuda") * 0.02
    tensors = [(0, table, 0.0), (table, table + matrix, 0.01), (table + matrix, n, 0.0)]
    ranks = [Rank(flat, r * S, S, tensors, lr, state_bits, seed) for r in range(W)]
    scale = math.sqrt(dim)
    losses = []
    for step in range(1, steps + 1):
        # 1: all ranks' codes and scales, as the all-gather leaves them
        sent = [zpq.quant_i8(r.half, QW) for r in ranks]
        codes, scales = torch.cat([c for c, _ in sent]), torch.cat([s for _, s in sent])
        # (the matrix starts inside a block: dequantize from the block's start)
        lead = table % QW
        b0 = (table - lead) // QW
        rest = zpq.dequant_i8(codes[table - lead:].clone(), scales[b0:].clone(), QW, torch.float16)
        out = rest[lead:lead + matrix].view(dim, vocab)

        received, loss_sum = [], 0.0
        for r in range(W):
            x = torch.randint(0, vocab, (batch,), generator=gen, device="cuda")
            y = (x * 7 + torch.randint(0, 3, (batch,), generator=gen, device="cuda")) % vocab
            # 2, 3: forward and backward
            h = zpq.embedding_i8(x, codes, scales, vocab, dim, block=QW, scale=scale, out_dtype=torch.float16)
            logits = (h @ out).float()
            logp = torch.log_softmax(logits, 1)
            loss_sum += -logp.gather(1, y[:, None]).mean().item()
            d = logp.exp()
            d.scatter_add_(1, y[:, None], torch.full_like(d[:, :1], -1.0))
            d = d.half()                                       # batch times the mean's gradient
            g = torch.zeros(n, dtype=torch.float16, device="cuda")
            zpq.embedding_grad(x, d @ out.t().contiguous(), vocab, scale=scale / batch, out=g[:table].view(vocab, dim))
            g[table:table + matrix] = (h.t().contiguous() @ d / batch).reshape(-1)
            received.append(zpq.qgz_reorder_quant_i4(g, L, N, QG))
        losses.append(loss_sum / W)

        # 4, hop 1: rank j of a node receives chunk j of every rank of its node
        c = n // L
        between = []
        for r in range(W):
            node, j = divmod(r, L)
            got = [received[node * L + i] for i in range(L)]
            between.append(zpq.qgz_dequant_reduce_requant_i4(
                torch.cat([a.view(L, -1)[j] for a, _ in got]), torch.cat([b.view(L, -1)[j] for _, b in got]), L, c, QG))
        # hop 2: rank j of node m receives position m of every node's rank j
        for r in range(W):
            m, j = divmod(r, L)
            got = [between[i * L + j] for i in range(N)]
            zpq.qgz_dequant_reduce_requant_i4(
                torch.cat([a.view(N, -1)[m] for a, _ in got]), torch.cat([b.view(N, -1)[m] for _, b in got]), N, S, QG,
                divisor=float(W), out=ranks[r].grad)

        # 5: the norm is the sum over the ranks (an all-reduce of one number)
        total = torch.zeros(1, dtype=torch.float64, device="cuda")
        for r in ranks:
            r.opt.grad_sumsq(out=total, accumulate=True)
        for r in ranks:
            r.opt.step(step, sumsq=total, max_norm=1.0)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    losses = train(steps=a.steps, state_bits=a.state_bits)
    for i in range(0, len(losses), max(1, len(losses) // 12)):
        print(f"step {i + 1:4d}  loss {losses[i]:.4f}")
    print(f"step {len(losses):4d}  loss {losses[-1]:.4f}  (uniform over the 3 successors: {math.log(3):.4f})")
