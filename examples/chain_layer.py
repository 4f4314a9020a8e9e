"""A recurrent layer whose states are coupled along a chain, trained and served.

The layer starts from the linear system h' = -T (h - x) of a chain of diffusing
cells, whose T is symmetric and tridiagonal.  bstq.solve diagonalises T once; in
T's eigenbasis the system is bstq.recur with the eigenvalues as rates.  From there
the layer is its own model: a gate for each channel, and rates that are trained
while the basis stays (Q diag(rate) Q^T keeps T's eigenvectors, not its zeros).
Training runs the recurrence, its gradients (bstq.recur_grad) and, for the two
weight matrices, updates that bstq.orthogonalize makes orthogonal.  Serving
starts from the states after a prompt and goes token by token (bstq.recur_step).

    python examples/chain_layer.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from symmetric_tridiagonal_eigensolver_gb300 import bstq  # noqa: E402


def chain_basis(cells, coupling, device):
    """Rates and eigenvectors of the chain coupling * tridiag(-1; 2; -1)."""
    d = torch.full((1, cells), 2.0 * coupling, device=device)
    e = torch.full((1, cells - 1), -coupling, device=device)
    rate, Q, info = bstq.solve(d, e, jobz=True)
    if int(info[0]) != 0:
        raise RuntimeError(f"eigensolve: info {int(info[0])}")
    return rate[0].contiguous(), Q[0].contiguous()


class ChainLayer:
    """y = recur(x W, x G) Q^T: W takes tokens to T's eigenbasis, G to the gates."""

    def __init__(self, cells, coupling, device, seed):
        g = torch.Generator(device=device).manual_seed(seed)
        self.rate, self.Q = chain_basis(cells, coupling, device)
        self.W = self.Q.clone()
        self.G = torch.randn(cells, cells, generator=g, device=device) / cells ** 0.5

    def forward(self, x, lengths=None):
        u, r = x @ self.W, x @ self.G
        h, last = bstq.recur(u, r, self.rate, lengths=lengths)
        return h @ self.Q.T, (x, u, r, h, lengths), last

    def gradients(self, dy, kept):
        x, u, r, h, lengths = kept
        du, dr, drate, _ = bstq.recur_grad(u, r, self.rate, h, dy @ self.Q, lengths=lengths)
        flat = x.flatten(0, 1).T
        return flat @ du.flatten(0, 1), flat @ dr.flatten(0, 1), drate

    def update(self, dW, dG, drate, step):
        self.W -= step * bstq.orthogonalize(dW)
        self.G -= step * bstq.orthogonalize(dG)
        self.rate = (self.rate - step * drate / (drate.abs().max() + 1e-12) * self.rate).contiguous()

    def token(self, x, state):
        """One token of every sequence; `state` is updated in place."""
        return bstq.recur_step(state, x @ self.W, x @ self.G, self.rate) @ self.Q.T


def train(steps=60, cells=64, batch=8, time=256, device="cuda"):
    """Fits a layer to another one's outputs on sequences of several lengths;
    returns the layer and the losses."""
    teacher, layer = ChainLayer(cells, 0.30, device, seed=1), ChainLayer(cells, 0.12, device, seed=2)
    g = torch.Generator(device=device).manual_seed(3)
    losses = []
    for k in range(steps):
        x = torch.randn(batch, time, cells, generator=g, device=device)
        lengths = torch.randint(time // 2, time + 1, (batch,), generator=g, device=device).to(torch.int32)
        want = teacher.forward(x, lengths)[0]
        y, kept, _ = layer.forward(x, lengths)
        count = int(lengths.sum()) * cells
        diff = y - want                       # zero beyond each length
        losses.append(float(diff.square().sum() / count))
        layer.update(*layer.gradients(2 * diff / count, kept), step=0.05 * (1 - k / steps))
    return layer, losses


def serve(layer, prompt, more):
    """Outputs for `more` (batch, time, cells) after `prompt`, token by token."""
    _, _, state = layer.forward(prompt)
    return torch.stack([layer.token(more[:, t], state) for t in range(more.shape[1])], 1)


if __name__ == "__main__":
    layer, losses = train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    x = torch.randn(4, 96, 64, device="cuda")
    whole = layer.forward(x)[0][:, 64:]
    print(f"token by token: largest difference from the whole sequence {float((serve(layer, x[:, :64], x[:, 64:]) - whole).abs().max()):.1e}")
