"""A data-parallel training step made of this package's calls, on one GPU.

P nodes, whose batches and gradients sit next to each other, train a residual
block y = layer_norm(x W1 + x) W2 towards a random block of the same form:

  layer_norm, layer_norm_backward   the block's norm; the gradients of its weight
                                    and bias go straight into the nodes' rows
  topk_ef, sparse_reduce            each node sends its largest gradients; the
                                    rest stays in its residual
  momentum_step                     momentum and update from the reduced sum
  orthogonal_step                   W1 and W2 move along orthogonalised updates,
                                    the norm's vectors along the update itself

    python examples/training_step.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_gradient_reduction_amd as sg

NODES, ROWS, WIDTH, OUT = 4, 256, 256, 64
LR, MU = 0.01, 0.9


def train(steps=40, seed=0):
    """Trains for `steps` steps; returns the losses before each of them."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    # one flat vector: W1, W2, the norm's weight, its bias
    ends = [0]
    for size in (WIDTH * WIDTH, WIDTH * OUT, WIDTH, WIDTH):
        ends.append(ends[-1] + size)
    parts = [slice(a, b) for a, b in zip(ends, ends[1:])]
    N = ends[-1]
    matrices = [(ends[0], WIDTH, WIDTH), (ends[1], WIDTH, OUT)]
    vectors = slice(ends[2], N)

    def views(flat):
        return flat[parts[0]].view(WIDTH, WIDTH), flat[parts[1]].view(WIDTH, OUT), flat[parts[2]], flat[parts[3]]

    def start():
        flat = normal(N) * WIDTH ** -0.5
        flat[parts[2]] = 1
        flat[parts[3]] = 0
        return flat

    weights, teacher = start(), start()
    w1, w2, gain, bias = views(weights)
    x = normal(NODES, ROWS, WIDTH)
    t1, t2, tg, tb = views(teacher)
    target = sg.layer_norm(x @ t1, tg, tb, residual=x)[0] @ t2

    k = N // 10
    grad, residual = torch.zeros(NODES, N, device=dev), torch.zeros(NODES, N, device=dev)
    momentum, update = torch.zeros(N, device=dev), torch.empty(N, device=dev)
    idx = torch.empty(NODES, k, dtype=torch.int32, device=dev)
    val = torch.empty(NODES, k, device=dev)
    offsets = [p * k for p in range(NODES + 1)]
    workspace = torch.empty(sg.orthogonalize_workspace_bytes(N, matrices), dtype=torch.uint8, device=dev)
    losses = []
    for _ in range(steps):
        y, mean, rstd, total = sg.layer_norm(x @ w1, gain, bias, residual=x)
        error = y @ w2 - target
        losses.append(error.square().mean())
        derror = error * (2 / (ROWS * OUT))  # of each node's own mean
        grad[:, parts[1]] = (y.transpose(1, 2) @ derror).view(NODES, -1)
        dtotal, _, _ = sg.layer_norm_backward(derror @ w2.t(), total, gain, mean, rstd, nodes=NODES,
                                              dweight=grad[:, parts[2]], dbias=grad[:, parts[3]])
        grad[:, parts[0]] = (x.transpose(1, 2) @ dtotal).view(NODES, -1)

        sg.topk_ef(grad, residual, k, out_idx=idx, out_val=val)
        reduced = sg.sparse_reduce(offsets, idx.view(-1), val.view(-1), N, delta=0.3)
        sg.momentum_step(reduced, momentum, MU, scale=1 / NODES, nesterov=True, update=update)
        sg.orthogonal_step(weights, update, matrices, lr=LR, workspace=workspace)
        weights[vectors] -= LR * update[vectors]
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    got = train(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
    for step in range(0, len(got), 5):
        print(f"step {step:3d}  loss {got[step]:.4f}")
    print(f"last      loss {got[-1]:.4f}")
