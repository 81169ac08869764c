"""Training steps of a tiny tied-embedding model over W virtual ranks.

Each rank looks its tokens up (``embedding``), normalises the rows keeping 8
bits of them (``layer_norm_checkpoint8``), and predicts every next token with
the table itself (``cross_entropy``, which keeps no logits; padding has targets
outside the table).  The loss's gradient follows at once
(``cross_entropy_backward``), so that the normalised rows themselves need not be
kept: the layer norm's gradient takes their 8-bit form
(``layer_norm_backward_checkpoint8``), its weight and bias gradients going
straight into the rank's gradient tensors.  The table's gradient from the
projection is the base that the lookup's gradient is added to in place
(``embedding_backward``), and one ``FusionPlan`` averages everything over the
ranks.

    python examples/data_parallel_step.py [steps]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import collective_reduction_virtual_gb300 as vc  # noqa: E402

RANKS, TOKENS, VOCAB, WIDTH = 4, 512, 257, 192


def batch(g):
    """Tokens that mostly follow a rule (the next one is 3 times this one plus
    1), and padding (-1) at the end of some rows."""
    t = torch.empty(8, TOKENS // 8 + 1, dtype=torch.int64, device="cuda")
    t[:, 0] = torch.randint(0, VOCAB, (8,), generator=g, device="cuda")
    for k in range(1, t.shape[1]):
        t[:, k] = (3 * t[:, k - 1] + 1) % VOCAB
    noise = torch.rand(t.shape, generator=g, device="cuda") < 0.05
    t[noise] = torch.randint(0, VOCAB, (int(noise.sum()),), generator=g, device="cuda")
    t[-1, -5:] = -1
    return t[:, :-1].contiguous(), t[:, 1:].contiguous()


def gradients(params, grads, tokens, targets):
    """One rank's loss (a tensor), its gradients written to `grads`."""
    table, weight, bias = params
    scale = math.sqrt(WIDTH)
    x = vc.embedding(tokens, table, scale=scale)
    y, rstd, kept = vc.layer_norm_checkpoint8(x, weight, bias)
    del x
    counted = torch.where(tokens >= 0, targets, -1)
    share = 1.0 / ((counted >= 0).sum())
    losses, lse = vc.cross_entropy(y, table, counted)
    dy, _ = vc.cross_entropy_backward(share, y, table, counted, lse, dtable=grads[0])
    del y  # the kept form is all that the rest of the backward pass needs of it
    dx, _, _ = vc.layer_norm_backward_checkpoint8(dy, kept, rstd, weight, dx=dy, dweight=grads[1],
                                                  dbias=grads[2])
    vc.embedding_backward(dx, tokens, VOCAB, scale=scale, base=grads[0], out=grads[0])
    return losses.sum() * share


def train(steps=60, rate=0.5):
    """The mean loss over the ranks at each step."""
    g = torch.Generator(device="cuda")
    g.manual_seed(20261202)
    params = [torch.randn(VOCAB, WIDTH, generator=g, device="cuda") * 0.02,
              torch.ones(WIDTH, device="cuda"), torch.zeros(WIDTH, device="cuda")]
    data = [batch(g) for _ in range(RANKS)]
    grads = [[torch.empty_like(p) for p in params] for _ in range(RANKS)]
    average = vc.FusionPlan(grads, grads, op="avg", ring_order=True)
    losses = []
    for _ in range(steps):
        losses.append(sum(gradients(params, grads[u], *data[u]) for u in range(RANKS)) / RANKS)
        average()
        for p, d in zip(params, grads[0]):  # every rank holds the same averages
            p.sub_(d, alpha=rate)
    return [float(v) for v in losses], grads


if __name__ == "__main__":
    history, _ = train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
    for step in range(0, len(history), max(1, len(history) // 10)):
        print(f"step {step:4d}  loss {history[step]:.4f}")
    print(f"last       loss {history[-1]:.4f}")
