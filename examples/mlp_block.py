"""A pre-norm MLP block trained with FP8 products.

    y = x + W2 gelu(W1 norm(x) + b1) + b2

Forward, four launches beside the quantisation of the weights: layer norm
that leaves its rows as fp8 codes, the first product with bias and GELU in its
epilogue (keeping the value before the activation), the quantisation of its
result, and the second product with bias and residual. Backward: the second
product's gradient with the activation's in its epilogue, the bias sums, the
weights' gradients, and layer norm's with the residual stream's gradient
added. Values and weights go to e4m3, gradients to e5m2, one scale per row.

    python examples/mlp_block.py [--tokens 1024 --width 512 --hidden 2048 --steps 60]

fits the block to a random target map and prints the loss.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_scaled_gemm_gb300 as fm  # noqa: E402

ROW, GELU = fm.SCALE_ROWWISE, fm.ACT_GELU
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def product(a, bt, out_dtype=torch.bfloat16):
    """a . bt^T of two (codes, scales) pairs with rows along the contraction."""
    return fm.fp8_scaled_mm_ex(a[0], bt[0].t(), a[1], bt[1], ROW, out_dtype=out_dtype)


class MlpBlock:
    """Parameters and their gradients (fp32), and the two passes."""

    def __init__(self, width: int, hidden: int, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, scale):
            return torch.randn(*shape, generator=g, device=device) * scale
        self.params = {
            "gamma": torch.ones(width, device=device), "beta": torch.zeros(width, device=device),
            "w1": randn(hidden, width, scale=width ** -0.5), "b1": torch.zeros(hidden, device=device),
            "w2": randn(width, hidden, scale=hidden ** -0.5), "b2": torch.zeros(width, device=device),
        }
        self.grads = {}

    def forward(self, x):
        """x [tokens, width] bf16 -> y; what the backward pass needs is kept."""
        p = self.params
        w1, w2 = p["w1"].bfloat16(), p["w2"].bfloat16()
        n, mean, rstd, nq, ns = fm.fp8_layer_norm(x, p["gamma"], p["beta"], q_dtype=E4M3)
        w1q, s1 = fm.fp8_quantize(w1, ROW)
        h, z = fm.fp8_scaled_mm_epilogue(nq, w1q.t(), ns, s1, ROW, bias=p["b1"].bfloat16(), activation=GELU,
                                         return_preact=True)
        hq, hs = fm.fp8_quantize(h, ROW)
        w2q, s2 = fm.fp8_quantize(w2, ROW)
        y = fm.fp8_scaled_mm_epilogue(hq, w2q.t(), hs, s2, ROW, bias=p["b2"].bfloat16(), residual=x)
        self.kept = (x, n, mean, rstd, h, z, w1, w2)
        return y

    def backward(self, dy):
        """dy [tokens, width] bf16 -> dx; the parameters' gradients go to ``grads``."""
        x, n, mean, rstd, h, z, w1, w2 = self.kept

        def rows(t, dtype=E4M3):
            return fm.fp8_quantize(t, ROW, dtype=dtype)

        def columns(t, dtype=E4M3):
            return fm.fp8_quantize(t.t().contiguous(), ROW, dtype=dtype)
        g = self.grads
        g["b2"] = fm.fp8_act_grad(dy, None, fm.ACT_NONE, return_dz=False)[1]
        g["w2"] = product(columns(dy, E5M2), columns(h), torch.float32)
        dyq, dys = rows(dy, E5M2)
        w2q, s2 = columns(w2)
        dz = fm.fp8_scaled_mm_act_grad(dyq, w2q.t(), dys, s2, ROW, z, GELU)
        g["b1"] = fm.fp8_act_grad(dz, None, fm.ACT_NONE, return_dz=False)[1]
        g["w1"] = product(columns(dz, E5M2), columns(n), torch.float32)
        dn = product(rows(dz, E5M2), columns(w1))
        dx, g["gamma"], g["beta"] = fm.fp8_layer_norm_grad(dn, x, self.params["gamma"], mean, rstd, residual_grad=dy)
        return dx


def train(tokens: int, width: int, hidden: int, steps: int, lr: float = 3e-3, device="cuda", log=print):
    """Fit a block to a random linear map of its input with Adam (AdamW without decay); returns the losses."""
    g = torch.Generator(device=device).manual_seed(1)
    target = torch.randn(width, width, generator=g, device=device) * width ** -0.5
    block = MlpBlock(width, hidden, device)
    names = list(block.params)
    params = [block.params[k] for k in names]
    exp_avgs, exp_avg_sqs = ([torch.zeros_like(p) for p in params] for _ in range(2))
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, width, generator=g, device=device).bfloat16()
        e = block.forward(x).float() - x.float() @ target
        losses.append(float(e.square().mean()))
        block.backward((e * (2.0 / (tokens * width))).bfloat16())
        fm.fp8_adamw(params, [block.grads[k] for k in names], exp_avgs, exp_avg_sqs, step + 1, lr=lr, weight_decay=0.0)
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:4d}  loss {losses[-1]:.4f}")
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    fm.load(build_if_missing=True)
    train(a.tokens, a.width, a.hidden, a.steps)


if __name__ == "__main__":
    main()
