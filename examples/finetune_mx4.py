"""Fine-tuning a feed-forward block over a frozen 4-bit base, then answering from it.

The block is down(silu(up(X))), each linear a frozen matrix with a rank-r adapter.  Its
base is microscaled 4-bit (--base mx4: activations packed on the way in, products on the
4-bit matrix instruction) or NF4 (--base nf4: weights rebuilt in bf16).  Training draws
dropout for the adapters inside the layers and for the hidden activations in a call of
its own; no mask is stored: the backward draws the same decisions from (seed, step).  The
adapters of both linears are slices of one flat buffer, stepped by one AdamW launch.  The
targets come from the same base with a hidden low-rank change, which the adapters have to
find.  At the end the block answers token by token, without dropout.

    python examples/finetune_mx4.py [--base nf4] [--tokens 512] [--steps 60]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_lora_blockwise_amd as q  # noqa: E402


class Mx4Base:
    """W [N, K] packed along its rows for the forward and down its columns for dX."""

    def __init__(self, W):
        self.N, self.K = W.shape
        self.w = q.mx4_quantize(W)
        self.wt = q.mx4_quantize(W, transpose=True)

    def product(self, X):
        return q.mx4_matmul(*q.mx4_quantize(X), X.shape[0], *self.w, self.N, self.K)

    def forward(self, X, L1, L2, scale, **kw):
        return q.mx4_linear_fwd(X, *self.w, self.N, L1, L2, scale, **kw)

    def backward(self, X, dY, L1, L2, scale, **kw):
        return q.mx4_linear_bwd(X, dY, *self.wt, L1, L2, scale, **kw)


class Nf4Base:
    def __init__(self, W):
        self.N, self.K = W.shape
        codes, absmax = q.nf4_quantize(W)
        self.w = (codes, *q.nf4_double_quant(absmax))

    def product(self, X):
        L1 = torch.zeros(self.K, 8, dtype=torch.bfloat16, device=X.device)
        L2 = torch.zeros(8, self.N, dtype=torch.bfloat16, device=X.device)
        return q.qlora_linear_fwd(X, *self.w, self.N, L1, L2)[0]

    def forward(self, X, L1, L2, scale, **kw):
        return q.qlora_linear_fwd_dropout(X, *self.w, self.N, L1, L2, scale, **kw)

    def backward(self, X, dY, L1, L2, scale, **kw):
        return q.qlora_linear_bwd_dropout(X, dY, *self.w, L1, L2, scale, **kw)


class Block:
    def __init__(self, base, weights, r, scale=2.0, p=0.05):
        dev = weights[0].device
        self.bases = [base(W) for W in weights]
        self.scale, self.p, self.step_no = scale, p, 0
        n = sum(r * (W.shape[0] + W.shape[1]) for W in weights)
        self.param, self.m, self.v, self.grad = (torch.zeros(n, device=dev) for _ in range(4))
        self.bf = torch.zeros(n, dtype=torch.bfloat16, device=dev)
        self.L1, self.L2, self.dL1, self.dL2 = [], [], [], []
        at = 0
        for W in weights:
            N, K = W.shape
            for params, grads, shape in ((self.L1, self.dL1, (K, r)), (self.L2, self.dL2, (r, N))):
                end = at + shape[0] * shape[1]
                params.append(self.bf[at:end].view(shape))
                grads.append(self.grad[at:end].view(shape))
                if params is self.L1:
                    self.param[at:end].normal_(0, K ** -0.5)       # L2 starts at zero
                at = end
        self.bf.copy_(self.param)

    def linear(self, i, X, p, T_out):
        return self.bases[i].forward(X, self.L1[i], self.L2[i], self.scale, p=p, seed=i, offset=self.step_no,
                                     T_out=T_out)

    def __call__(self, X):
        U, _ = self.linear(0, X, 0.0, None)
        return self.linear(1, torch.nn.functional.silu(U), 0.0, None)[0]

    def train(self, X, target, lr):
        """One step; returns the mean squared error before it."""
        self.step_no += 1
        p, drop = self.p, dict(p=self.p, offset=self.step_no)
        U, T0 = self.linear(0, X, p, True)
        H = q.lora_dropout(torch.nn.functional.silu(U), p, 2, self.step_no)
        Y, T1 = self.linear(1, H, p, True)
        err = Y.float() - target.float()
        dY = (err * (2.0 / err.numel())).to(torch.bfloat16)
        dH, _, _ = self.bases[1].backward(H, dY, self.L1[1], self.L2[1], self.scale, seed=1, T=T1, dL1=self.dL1[1],
                                          dL2=self.dL2[1], **drop)
        dS = q.lora_dropout(dH, p, 2, self.step_no)               # the same decisions as in the forward
        u = U.float()
        sig = torch.sigmoid(u)
        dU = (dS.float() * sig * (1 + u * (1 - sig))).to(torch.bfloat16)
        self.bases[0].backward(X, dU, self.L1[0], self.L2[0], self.scale, seed=0, T=T0, dX=False, dL1=self.dL1[0],
                               dL2=self.dL2[0], **drop)
        q.qlora_adamw_step(self.param, self.m, self.v, self.grad, self.step_no, lr, param_bf16=self.bf)
        return err.square().mean()


def run(base="mx4", tokens=512, width=512, hidden=1408, r=16, steps=60, lr=5e-3, answers=8, dev="cuda:0", log=print):
    """Trains and answers; returns (first loss, last loss, answers token by token, the same as one batch)."""
    torch.manual_seed(0)
    kind = {"mx4": Mx4Base, "nf4": Nf4Base}[base]
    weights = [torch.randn(n, k, device=dev).mul_(k ** -0.5).to(torch.bfloat16)
               for n, k in ((hidden, width), (width, hidden))]
    block = Block(kind, weights, r)
    change = [torch.randn(W.shape[1], 4, device=dev) @ torch.randn(4, W.shape[0], device=dev) * (0.25 / W.shape[1] ** 0.5)
              for W in weights]

    def teacher(X):
        U = block.bases[0].product(X).float() + X.float() @ change[0]
        H = torch.nn.functional.silu(U).to(torch.bfloat16)
        return block.bases[1].product(H).float() + H.float() @ change[1]

    losses, t0 = [], 0.0
    for step in range(steps):
        if step == 1:                                             # the first one sets the libraries up
            torch.cuda.synchronize()
            t0 = time.perf_counter()
        X = torch.randn(tokens, width, device=dev).to(torch.bfloat16)
        losses.append(block.train(X, teacher(X), lr))
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:3d}  mean squared error {losses[-1].item():.4f}")
    torch.cuda.synchronize()
    if steps > 1:
        log(f"{tokens} tokens a step: {1e3 * (time.perf_counter() - t0) / (steps - 1):.2f} ms")
    X = torch.randn(answers, width, device=dev).to(torch.bfloat16)
    alone = torch.cat([block(X[i:i + 1]) for i in range(answers)])
    return losses[0].item(), losses[-1].item(), alone, block(X)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--base", choices=("mx4", "nf4"), default="mx4")
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    first, last, alone, batch = run(a.base, a.tokens, steps=a.steps)
    rel = ((alone - batch).float().norm() / batch.float().norm()).item()
    print(f"loss {first:.4f} -> {last:.4f}; token by token against one batch: relative difference {rel:.1e}")


if __name__ == "__main__":
    main()
