"""Training steps of a gated feed-forward block in MXFP4, from libfp4q's calls:

    y = x + Wd (silu(Wg n) * (Wu n)),   n = rms_norm(x) * w

with every product on FP4 operands (blocks of 32 along K), the gradients
rounded stochastically, and an AdamW step whose two moments are held in 8
bits.  Run it on an MI355X:

    python examples/gated_ffn_step.py [--tokens 2048] [--width 1024] [--hidden 2816] [--steps 20]

It fits a block to the outputs of another one and prints the loss.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_block_scaled_fp4q_amd as fq  # noqa: E402


class GatedFFN:
    """The block's parameters (fp32, with the bf16 copies that are quantised),
    its optimizer state and its step.  Gate and up rows are one [2F, H]
    matrix.  Tokens, H and F are multiples of 64."""

    def __init__(self, width, hidden, bits=8, weight_decay=0.01, device="cuda", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.H, self.F = width, hidden

        def normal(rows, cols, sd):
            return torch.randn(rows, cols, generator=g, device=device) * sd
        self.params = [normal(2 * hidden, width, width ** -0.5), normal(width, hidden, hidden ** -0.5),
                       torch.ones(width, device=device)]
        self.copies = [p.bfloat16() for p in self.params]
        self.grads = [torch.zeros_like(p) for p in self.params]
        state = [fq.adamw_state(p, bits) for p in self.params]
        m, v, ms, vs = ([s[i] for s in state] for i in range(4))
        scales = (ms, vs) if bits == 8 else (None, None)
        self.plan = fq.adamw_plan(self.params, self.grads, m, v, *scales, copies=self.copies,
                                  weight_decay=[weight_decay, weight_decay, 0.0])
        self.t = 0
        self.quantise_weights()

    def quantise_weights(self):
        """Both orientations of the matrices: rows for the forward products,
        columns for the products that bring the gradient back."""
        gu, d, _ = self.copies
        self.gu, self.guT = fq.quantize_dual(gu)
        self.d, self.dT = fq.quantize_dual(d)

    def forward(self, x):
        """x: bf16 [tokens, H].  Returns y and what the backward pass reads."""
        F = self.F
        n, _, rstd = fq.layer_norm(x, self.copies[2], kind=fq.RMS_NORM)
        nq, nT = fq.quantize_dual(n)
        (c, s) = self.gu
        h, gate, up = fq.gemm_gated(*nq, c[:F], s[:F], c[F:], s[F:], act=fq.SILU, save=True)
        hq, hT = fq.quantize_dual(h)
        y = fq.gemm(*hq, *self.d, out_dtype=torch.bfloat16).add_(x)
        return y, (x, rstd, nT, hT, gate, up)

    def backward(self, dy, kept):
        """dy: bf16 [tokens, H].  Fills the gradients and returns dx."""
        x, rstd, nT, hT, gate, up = kept
        seed = 8 * self.t
        dq, dT = fq.quantize_dual(dy, round_row=fq.SR, seed_row=seed, round_col=fq.SR, seed_col=seed + 1)
        fq.gemm(*dT, *hT, c=self.grads[1])                     # dWd = dy^T h
        dgate, dup = fq.gemm_gated_grad(*dq, *self.dT, gate, up, act=fq.SILU)
        both = dgate.as_strided((dgate.shape[0], 2 * self.F), (2 * self.F, 1))  # one [tokens, 2F] tensor
        assert dup.data_ptr() == both.data_ptr() + 2 * self.F
        gq, gT = fq.quantize_dual(both, round_row=fq.SR, seed_row=seed + 2, round_col=fq.SR,
                                  seed_col=seed + 3)
        fq.gemm(*gT, *nT, c=self.grads[0])                     # dW of gate and up
        dn = fq.gemm(*gq, *self.guT, out_dtype=torch.bfloat16)
        dx, _, _ = fq.layer_norm_grad(dn, x, self.copies[2], None, rstd, kind=fq.RMS_NORM,
                                      dweight=self.grads[2], want_bias=False)
        return dx.add_(dy)

    def update(self, lr):
        self.t += 1
        fq.adamw_step(self.plan, lr, self.t, beta1=0.9, beta2=0.95, seed=self.t)
        self.quantise_weights()


def fit(tokens=2048, width=1024, hidden=2816, steps=20, lr=1e-3, bits=8, report=print):
    """Fits a block to another's outputs; returns the losses."""
    teacher, block = GatedFFN(width, hidden, seed=1), GatedFFN(width, hidden, bits=bits, seed=2)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    losses = []
    for i in range(steps):
        x = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
        want, _ = teacher.forward(x)
        y, kept = block.forward(x)
        diff = y.float() - want.float()
        block.backward((diff / diff.numel()).bfloat16(), kept)
        block.update(lr)
        losses.append(0.5 * diff.square().mean().item())
        report(f"step {i + 1}: loss {losses[-1]:.5f}")
    return losses


def main():
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 2048), ("width", 1024), ("hidden", 2816), ("steps", 20), ("bits", 8)):
        a.add_argument(f"--{name}", type=int, default=value)
    a.add_argument("--lr", type=float, default=1e-3)
    fit(**vars(a.parse_args()))


if __name__ == "__main__":
    main()
