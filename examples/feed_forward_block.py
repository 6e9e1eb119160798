"""A gated feed-forward block trained in bf16 with 8-bit kept activations, then served with 4-bit weights.

    y = x + act(norm(x) Wg^T) * (norm(x) Wu^T) Wd^T

Training steps keep the norm's output and the hidden activations in 8 bits between the forward and the
backward pass; serving quantizes the three trained weights (smoothing, low-rank branch, INT4) and answers
single tokens with weight-only products. Synthetic data: a fixed random block is the teacher.

    python examples/feed_forward_block.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a4_quantized_gemm_smooth_amd as w4  # noqa: E402

EPS = 1e-5


def _bytes(n):
    return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")


class Kept:
    """Activations [M, K] kept in 8 bits."""

    def __init__(self, M, K):
        sizes = w4.checkpoint_sizes(M, K)
        self.K, self.codes, self.scales = K, torch.empty(sizes["codes"], dtype=torch.int8, device="cuda"), _bytes(sizes["scales"])

    def keep(self, x):
        w4.checkpoint_pack(x, self.codes, self.scales)

    def read(self, into):
        w4.checkpoint_unpack(self.codes, self.scales, into)
        return into

    def weight_grad(self, dy, dw, ws):
        w4.checkpoint_weight_grad(dy, self.codes, self.scales, self.K, dw, ws)


class Block:
    """The block's parameters (fp32, with bf16 copies that the products read) and one batch's buffers."""

    def __init__(self, M, K, F, seed, act="silu"):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.M, self.K, self.F, self.act = M, K, F, act
        self.master = dict(wg=r(F, K) / K ** 0.5, wu=r(F, K) / K ** 0.5, wd=r(K, F) / F ** 0.5, gamma=torch.ones(K, device="cuda"),
                           beta=torch.zeros(K, device="cuda"))
        bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        f32 = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
        self.n, self.h, self.mean, self.rstd = bf(M, K), bf(M, F), f32(M), f32(M)
        self.kept_n, self.kept_h = Kept(M, K), Kept(M, F)
        self.dn, self.dx = bf(M, K), bf(M, K)
        self.grad = dict(wg=bf(F, K), wu=bf(F, K), wd=f32(K, F), gamma=f32(K), beta=f32(K))
        self.ws = _bytes(max(w4.gated_forward_bytes(M, K, F), w4.gated_backward_bytes(M, K, F), w4.layer_norm_backward_bytes(M, K),
                             w4.checkpoint_weight_grad_bytes(M, K, F)))
        self.load()

    def load(self):
        self.w = {k: v.bfloat16() if k.startswith("w") else v for k, v in self.master.items()}

    def forward(self, x):
        w = self.w
        w4.layer_norm(x, w["gamma"], w["beta"], EPS, self.n, self.mean, self.rstd)
        w4.gated_forward(self.n, w["wg"], w["wu"], self.act, self.h, self.ws)
        self.kept_n.keep(self.n)
        self.kept_h.keep(self.h)
        return x + self.h @ w["wd"].T

    def backward(self, x, dy):
        """The parameters' gradients in ``grad`` and dx, from what the forward pass kept."""
        w, g = self.w, self.grad
        self.kept_h.weight_grad(dy, g["wd"], self.ws)
        dh = dy @ w["wd"]
        n = self.kept_n.read(self.n)
        w4.gated_backward(dh, n, w["wg"], w["wu"], self.act, self.dn, g["wg"], g["wu"], self.ws)
        w4.layer_norm_backward(self.dn, x, w["gamma"], self.mean, self.rstd, self.dx, g["gamma"], g["beta"], self.ws)
        return dy + self.dx

    def step(self, rate):
        for k, v in self.master.items():
            v -= rate * self.grad[k].float()
        self.load()


class Served:
    """The trained block with its three weights in 4 bits, for single tokens."""

    def __init__(self, block, x, rank=32):
        self.gamma, self.beta = block.w["gamma"], block.w["beta"]
        block.forward(x)   # calibration: the inputs of each layer
        layers = dict(wg=block.n, wu=block.n, wd=block.h)
        self.layers = {k: self._quantize(block.w[k], calibration, rank) for k, calibration in layers.items()}

    @staticmethod
    def _quantize(w, calibration, rank):
        bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
        lam, inv = w4.smooth_factors(w4.column_absmax(bits(calibration)), w4.column_absmax(bits(w)))
        return w4.W4A4Linear.from_weights(bits(w), lam, inv, rank)

    def __call__(self, x):
        n, stats = torch.empty_like(x), torch.empty((2, x.shape[0]), device="cuda")
        w4.layer_norm(x, self.gamma, self.beta, EPS, n, stats[0], stats[1])
        g, u = self.layers["wg"].tokens(n).float(), self.layers["wu"].tokens(n).float()
        h = (g * torch.sigmoid(g) * u).bfloat16()
        return x + self.layers["wd"].tokens(h)


def main(M=1024, K=512, F=1408, steps=30, rate=0.1):
    """Trains, quantizes and serves; returns the losses and the served block's relative error."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    target = Block(M, K, F, seed=2).forward(x)
    block = Block(M, K, F, seed=3)
    losses = []
    for i in range(steps):
        y = block.forward(x)
        d = y.float() - target.float()
        losses.append(float(d.square().sum(1).mean()))
        block.backward(x, (2 / M * d).bfloat16())
        block.step(rate)
        if i % 10 == 0 or i == steps - 1:
            print(f"step {i:3d}  loss {losses[-1]:.4f}", flush=True)
    kept = sum(t.codes.numel() + t.scales.numel() for t in (block.kept_n, block.kept_h))
    print(f"kept for the backward pass: {kept / 2 ** 20:.2f} MiB in 8 bits, {M * (K + F) * 2 / 2 ** 20:.2f} MiB in bf16")
    y = block.forward(x)
    served = Served(block, x)
    worst = 0.0
    for m in (1, 4):
        z = served(x[:m])
        branch = (y[:m] - x[:m]).float()
        worst = max(worst, float(((z - x[:m]).float() - branch).norm() / branch.norm()))
    print(f"4-bit weights, 1 and 4 tokens: relative error of the block's branch {worst:.3f}")
    return losses, worst


if __name__ == "__main__":
    main()
