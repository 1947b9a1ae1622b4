"""Train a gated MLP block that keeps its activations in 8 bits.

    python examples/gated_mlp_q8.py [--tokens 4096] [--features 1024] [--hidden 2816]
                                    [--steps 20] [--micro-batches 2] [--format int8]

The block is y = (silu(x Wg) * (x Wu)) Wo.  Between its forward and its
backward pass it holds x, x Wg and x Wu as 8-bit checkpoints (a byte an element
and a thirty-second) and nothing else: the hidden activation is recomputed by
the gated unit's backward pass, straight into the 8-bit form in which the weight
gradient of Wo reads it.  All products are the library's; PyTorch holds the
memory.  The same block with everything kept in float32 runs beside it, and
the script prints both losses, what each holds, and how far the gradients of
the first step are apart.
"""

from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import dense_fp32_gemm_row_gb300 as g  # noqa: E402


def product_t(a, w):
    """``a @ w.T`` of row-major matrices."""
    m, k = a.shape
    out = torch.empty((m, w.shape[0]), device=a.device)
    g.check(g.gemm_f32_ex(0, 1, m, w.shape[0], k, 1.0, a.data_ptr(), a.stride(0), w.data_ptr(),
                          w.stride(0), 0.0, out.data_ptr(), out.stride(0),
                          stream=torch.cuda.current_stream().cuda_stream), "gemm_f32_ex")
    return out


class GatedMLP:
    """Wg and Wu side by side in one (features, 2 hidden) matrix, and Wo."""

    def __init__(self, features, hidden, format="int8", seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.format = hidden, format
        self.w_in = torch.randn((features, 2 * hidden), generator=gen, device="cuda")
        self.w_in *= features ** -0.5
        self.w_out = torch.randn((hidden, features), generator=gen, device="cuda") * hidden ** -0.5
        self.dw_in, self.dw_out = torch.zeros_like(self.w_in), torch.zeros_like(self.w_out)

    def forward(self, x):
        """y, and what the backward pass needs."""
        both = g.matmul(x, self.w_in)
        h, gate_q, up_q = g.q8_gated(both[:, :self.hidden], both[:, self.hidden:],
                                     format=self.format)
        return g.matmul(h, self.w_out), (g.q8_store(x, format=self.format), gate_q, up_q)

    def backward(self, held, dy, first):
        """Adds to (first: sets) the weights' gradients; returns dx."""
        x_q, gate_q, up_q = held
        dh = product_t(dy, self.w_out)
        both = torch.empty((dy.shape[0], 2 * self.hidden), device=dy.device)
        _, _, h_q = g.q8_gated_backward(gate_q, up_q, dh, dgate=both[:, :self.hidden],
                                        dup=both[:, self.hidden:])
        beta = 0.0 if first else 1.0
        g.q8_wgrad(h_q, dy, out=self.dw_out, beta=beta)
        g.q8_wgrad(x_q, both, out=self.dw_in, beta=beta)
        return product_t(both, self.w_in)

    def step(self, rate):
        for w, dw in ((self.w_in, self.dw_in), (self.w_out, self.dw_out)):
            w.sub_(dw, alpha=rate)


class FullMLP(GatedMLP):
    """The same with everything kept in float32, by PyTorch's autograd."""

    def gradients(self, x, target, scale):
        w_in, w_out = self.w_in.clone().requires_grad_(), self.w_out.clone().requires_grad_()
        both = x @ w_in
        gate, up = both[:, :self.hidden], both[:, self.hidden:]
        y = (torch.nn.functional.silu(gate) * up) @ w_out
        loss = ((y - target) ** 2).sum() * scale
        loss.backward()
        return float(loss.detach()), w_in.grad, w_out.grad


def train(tokens, features, hidden, steps, micro_batches, format, rate=0.2, say=print):
    """The losses of both blocks, and the relative distances of their first gradients."""
    block = GatedMLP(features, hidden, format)
    full = FullMLP(features, hidden, format)
    teacher = GatedMLP(features, hidden, format, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(2)
    scale = 1.0 / (tokens * micro_batches * features)
    losses, apart = [], None
    for i in range(steps):
        loss = loss_full = 0.0
        full.dw_in.zero_()
        full.dw_out.zero_()
        for b in range(micro_batches):
            x = torch.randn((tokens, features), generator=gen, device="cuda")
            target, _ = teacher.forward(x)
            y, held = block.forward(x)
            error = y - target
            loss += float((error * error).sum()) * scale
            block.backward(held, 2 * scale * error, first=b == 0)
            part, d_in, d_out = full.gradients(x, target, scale)
            loss_full += part
            full.dw_in += d_in
            full.dw_out += d_out
        if apart is None:
            apart = [float((p - q).norm() / q.norm())
                     for p, q in ((block.dw_in, full.dw_in), (block.dw_out, full.dw_out))]
            bits = sum(q.nbytes for q in held)
            say(f"held for the backward pass: {bits / 2**20:.1f} MiB in {format}, "
                f"{4 * tokens * (features + 3 * hidden) / 2**20:.1f} MiB in float32 (x, gate, up, h)")
            say(f"first gradients, relative distance: w_in {apart[0]:.2e}, w_out {apart[1]:.2e}")
        block.step(rate * features)
        full.step(rate * features)
        losses.append((loss, loss_full))
        say(f"step {i:3d}  loss {loss:.6f}   float32 {loss_full:.6f}")
    return losses, apart


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--features", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2816)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--micro-batches", type=int, default=2)
    ap.add_argument("--format", choices=tuple(g.Q8_FORMATS), default="int8")
    a = ap.parse_args(argv)
    train(a.tokens, a.features, a.hidden, a.steps, a.micro_batches, a.format)
    return 0


if __name__ == "__main__":
    sys.exit(main())
