"""Training steps of a stack of gated feed-forward blocks in MXFP4, from
libfp4q's calls.  Block i, on the residual stream x and its normed n:

    b = Wd_i (silu(Wg_i n) * (Wu_i n))
    x = x + g_i rms_norm(b) p_i,   n = rms_norm(x) w_i

with every product on FP4 operands (blocks of 32 along K), the gradients
rounded stochastically and clipped to a global norm, and an AdamW step whose
two moments are held in 8 bits.  The line of norms, gate and sum is one call
in each direction.  Run it on an MI355X:

    python examples/gated_stack.py [--tokens 2048] [--width 1024] [--hidden 2816] [--depth 4] [--steps 20]

It fits a stack to the outputs of another one and prints loss and norm.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_block_scaled_fp4q_amd as fq  # noqa: E402

EACH = 5  # parameters of a block: gate and up rows, down, post norm, gate, next norm


class GatedStack:
    """The blocks' parameters (fp32, with the bf16 copies that the calls read),
    their optimizer state and their step; parameter 0 is the first norm's weight.
    Tokens, width and hidden are multiples of 64."""

    def __init__(self, width, hidden, depth, bits=8, weight_decay=0.01, device="cuda", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.H, self.F, self.depth = width, hidden, depth

        def normal(rows, cols, sd):
            return torch.randn(rows, cols, generator=g, device=device) * sd
        one = torch.ones(width, device=device)
        self.params, decay = [one.clone()], [0.0]
        for _ in range(depth):
            self.params += [normal(2 * hidden, width, width ** -0.5), normal(width, hidden, hidden ** -0.5),
                            one.clone(), 0.5 * one, one.clone()]
            decay += [weight_decay, weight_decay, 0.0, 0.0, 0.0]
        self.copies = [p.bfloat16() for p in self.params]
        self.grads = [torch.zeros_like(p) for p in self.params]
        state = [fq.adamw_state(p, bits) for p in self.params]
        m, v, ms, vs = ([s[i] for s in state] for i in range(4))
        scales = (ms, vs) if bits == 8 else (None, None)
        self.plan = fq.adamw_plan(self.params, self.grads, m, v, *scales, copies=self.copies, weight_decay=decay)
        self.t = 0
        self.quantise_weights()

    def quantise_weights(self):
        """Both orientations of the matrices: rows for the forward products,
        columns for the products that bring the gradient back."""
        self.gu, self.d = ([fq.quantize_dual(self.copies[1 + EACH * i + k]) for i in range(self.depth)]
                           for k in range(2))

    def join(self, i):
        """Arguments of block i's residual_norm that its gradient takes too."""
        _, _, post, gate, _ = self.copies[1 + EACH * i:1 + EACH * (i + 1)]
        return dict(kind=fq.RMS_NORM, post_kind=fq.RMS_NORM, post_weight=post, gate=gate)

    def block(self, i, nq, save):
        F, (c, s) = self.F, self.gu[i][0]
        return fq.gemm_gated(*nq, c[:F], s[:F], c[F:], s[F:], act=fq.SILU, save=save)

    def forward(self, x):
        """x: bf16 [tokens, H].  Returns the last norm's output and what the
        backward pass reads."""
        n, _, rstd = fq.layer_norm(x, self.copies[0], kind=fq.RMS_NORM)
        kept = [(x, rstd)]
        for i in range(self.depth):
            nq, nT = fq.quantize_dual(n)
            h, gate, up = self.block(i, nq, True)
            hq, hT = fq.quantize_dual(h)
            b = fq.gemm(*hq, *self.d[i][0], out_dtype=torch.bfloat16)
            x, n, stats = fq.residual_norm(x, b, self.copies[EACH * (i + 1)], **self.join(i))
            kept.append((x, b, stats, nT, hT, gate, up))
        return n, kept

    def infer(self, x):
        """The same without a gradient: the norms' outputs leave as codes, and the
        stream is summed in place."""
        x = x.clone()
        nq = fq.quantize(fq.layer_norm(x, self.copies[0], kind=fq.RMS_NORM, stats=False)[0])
        for i in range(self.depth):
            hq = fq.quantize(self.block(i, nq, False))
            b = fq.gemm(*hq, *self.d[i][0], out_dtype=torch.bfloat16)
            _, nq, _ = fq.residual_norm(x, b, self.copies[EACH * (i + 1)], x_out=x, stats=False,
                                        quantize=i + 1 < self.depth, **self.join(i))
        return nq

    def backward(self, dn, kept):
        """dn: bf16 [tokens, H].  Fills the gradients and returns dx."""
        dx, G = None, self.grads
        for i in reversed(range(self.depth)):
            x, b, stats, nT, hT, gate, up = kept[i + 1]
            at, seed = 1 + EACH * i, 4 * (self.t * self.depth + i)
            dx, db, *_ = fq.residual_norm_grad(
                dn, dx, x, b, stats, self.copies[at + 4], dx=dx, want_bias=False, dweight=G[at + 4],
                dpost_weight=G[at + 2], dgate=G[at + 3], **self.join(i))
            bq, bT = fq.quantize_dual(db, round_row=fq.SR, seed_row=seed, round_col=fq.SR, seed_col=seed + 1)
            fq.gemm(*bT, *hT, c=G[at + 1])                         # dWd = db^T h
            dgate, dup = fq.gemm_gated_grad(*bq, *self.d[i][1], gate, up, act=fq.SILU)
            both = dgate.as_strided((dgate.shape[0], 2 * self.F), (2 * self.F, 1))  # one [tokens, 2F] tensor
            assert dup.data_ptr() == both.data_ptr() + 2 * self.F
            gq, gT = fq.quantize_dual(both, round_row=fq.SR, seed_row=seed + 2, round_col=fq.SR,
                                      seed_col=seed + 3)
            fq.gemm(*gT, *nT, c=G[at])                             # dW of gate and up
            dn = fq.gemm(*gq, *self.gu[i][1], out_dtype=torch.bfloat16)
        x, rstd = kept[0]
        d0, _, _ = fq.layer_norm_grad(dn, x, self.copies[0], None, rstd, kind=fq.RMS_NORM, dweight=G[0],
                                      want_bias=False)
        return d0.add_(dx)

    def update(self, lr, max_norm=1.0):
        """An AdamW step on the gradients clipped to max_norm; returns the norm
        they had."""
        self.t += 1
        norm, scale = fq.grad_norm(self.plan, max_norm)
        fq.adamw_step(self.plan, lr, self.t, beta1=0.9, beta2=0.95, seed=self.t, grad_scale=scale)
        self.quantise_weights()
        return norm


def fit(tokens=2048, width=1024, hidden=2816, depth=4, steps=20, lr=1e-3, bits=8, report=print):
    """Fits a stack to another's outputs; returns the losses."""
    teacher, stack = (GatedStack(width, hidden, depth, bits=bits, seed=s) for s in (1, 2))
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    losses = []
    for i in range(steps):
        x = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
        n, kept = stack.forward(x)
        diff = n.float() - teacher.infer(x).float()
        stack.backward((diff / diff.numel()).bfloat16(), kept)
        norm = stack.update(lr)
        losses.append(0.5 * diff.square().mean().item())
        report(f"step {i + 1}: loss {losses[-1]:.5f}, gradient norm {norm.item():.3g}")
    return losses


def main():
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 2048), ("width", 1024), ("hidden", 2816), ("depth", 4), ("steps", 20), ("bits", 8)):
        a.add_argument(f"--{name}", type=int, default=value)
    a.add_argument("--lr", type=float, default=1e-3)
    fit(**vars(a.parse_args()))


if __name__ == "__main__":
    main()
