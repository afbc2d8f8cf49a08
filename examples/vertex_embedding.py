"""Learns vertex embeddings of a graph from its two-step neighbourhoods.

The sparse product C = A A of an R-MAT graph counts the two-step paths between its
vertices. Its rows, as ``binding.spgemm`` leaves them on the GPU, teach a softmax over
all vertices (``losses.distillation``: the class table is one row a vertex, the
logarithm of a count is the teacher's value), and a neighbour of each vertex is its label.
Neither the logits (vertices x vertices) nor their gradient is ever stored whole.

    python examples/vertex_embedding.py [--scale 14] [--edge-factor 8] [--dim 64] [--batch 2048] [--steps 100]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from sparse_gemm_irregular_gm_gb300 import binding, inputs, losses  # noqa: E402


def rows_of(C, host_row_ptr, first, last):
    """Rows [first, last) of a device CSR as one of their own (row pointers from 0)."""
    lo, hi = int(host_row_ptr[first]), int(host_row_ptr[last])
    return binding.DeviceCSR(last - first, C.n_cols, C.row_ptr[first:last + 1] - lo, C.col[lo:hi], C.val[lo:hi])


def train(scale=14, edge_factor=8, dim=64, batch=2048, steps=100, temperature=1.0, rate=0.05, seed=1, report=None):
    """Returns the batches' mean losses, one a step."""
    A = inputs.rmat(scale, edge_factor, seed=seed, values="ones")
    dA = binding.to_device(A, dtype="float32")
    C = binding.spgemm(dA, dA)
    C.val.log_()  # paths are at least 1
    n = A.n_rows
    row_ptr = C.row_ptr.cpu()
    degree = dA.row_ptr[1:] - dA.row_ptr[:-1]
    g = torch.Generator(device="cuda").manual_seed(seed)
    vertex = (torch.randn(n, dim, generator=g, device="cuda") / dim ** 0.5).requires_grad_()
    classes = (torch.randn(n, dim, generator=g, device="cuda") / dim ** 0.5).requires_grad_()
    optimiser = torch.optim.Adam([vertex, classes], lr=rate)
    means = []
    for step in range(steps):
        first = step * batch % n
        last = min(n, first + batch)
        # one neighbour of each vertex as its label; vertices without any are left out
        k = (torch.rand(last - first, generator=g, device="cuda") * degree[first:last]).long()
        at = (dA.row_ptr[first:last] + k).clamp(max=dA.nnz - 1)
        target = torch.where(degree[first:last] > 0, dA.col[at].long(), -100)
        optimiser.zero_grad(set_to_none=True)
        o = losses.distillation(vertex[first:last], classes, rows_of(C, row_ptr, first, last), temperature, target=target)
        loss = 0.5 * o.kl.mean() + 0.5 * o.loss.mean()
        loss.backward()
        optimiser.step()
        means.append(loss.detach())
        if report and step % report == 0:
            print(f"step {step:4d}  divergence {o.kl.detach().mean():.4f}  cross entropy {o.loss.detach().mean():.4f}")
    losses.gm_loss_status()
    return torch.stack(means).cpu()


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("scale", 14), ("edge-factor", 8), ("dim", 64), ("batch", 2048), ("steps", 100)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    train(a.scale, a.edge_factor, a.dim, a.batch, a.steps, report=10)
