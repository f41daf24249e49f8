"""One transformer block around the MoE layer, trained for a few steps on synthetic data.

    h   = x + (x W_o^T + b_o)           dense projection, its residual in the epilogue
    y   = MoE(h)                        routed and shared experts
    out = h + dropout(y)                mask from (seed, step), never stored
    loss = mean (out - target)^2 / 2 + balance loss and z-loss of the router

Every product, the dropout, the balance loss and all gradients run in the library; torch holds the
buffers, forms the difference to the target and applies plain gradient descent.

    python examples/train_block.py [--steps 20] [--tokens 512]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Block:
    def __init__(self, spec, seq_len, p=0.1, coef_balance=0.01, coef_z=1e-3, lr=0.5, seed=0, device="cuda"):
        import routing_shared_expert_gb300 as moe
        from workloads import make_inputs
        self.moe, self.spec, self.seq_len, self.p = moe, spec, seq_len, p
        self.coef_balance, self.coef_z, self.lr = coef_balance, coef_z, lr
        T, d = spec.T, spec.d_model
        weights = make_inputs(spec, device, seed=seed)
        self.x = weights["x"]
        # the weights move every step, so the layer reads the bf16 down projections as they are
        self.layer = moe.MoELayer(moe.config_from_spec(spec, h_format="bf16"), weights, device, staged_buffers=False)
        self.weights = {k: v for k, v in weights.items() if k != "x"}
        g = torch.Generator(device=device).manual_seed(seed + 1)
        self.W_o = (torch.randn((d, d), generator=g, device=device) * d ** -0.5).bfloat16()
        self.b_o = torch.zeros(d, device=device)
        self.target = torch.randn((T, d), generator=g, device=device)
        self.proj = moe.make_linear_config(T, d, d, dw_dtype="f32")
        self.proj_ws = moe.alloc_linear_workspace(self.proj, device)
        self.bal_ws = moe.alloc_balance_loss_workspace(self.layer.cfg, seq_len, device)
        self.rng = torch.tensor([seed, 0], dtype=torch.int64, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        bf16 = dict(dtype=torch.bfloat16, device=device)
        self.h, self.dx = torch.empty((T, d), **bf16), torch.empty((T, d), **bf16)
        self.out, self.dy = torch.empty((T, d), **f32), torch.empty((T, d), **f32)
        self.dW_o, self.db_o = torch.empty((d, d), **f32), torch.empty(d, **f32)
        self.dlogits, self.bal = torch.empty((T, spec.N), **f32), torch.empty(3, **f32)

    def forward(self):
        m = self.moe
        m.moe_linear_forward(self.proj, self.x, self.W_o, self.b_o, self.x, None, self.h, self.proj_ws)
        y = self.layer.forward(self.h)
        m.moe_dropout_add(y, self.h, self.p, self.rng, self.out)
        m.moe_balance_loss(self.layer.cfg, self.layer.out["logits"], self.layer.out["topk_idx"], None, self.seq_len,
                           self.coef_balance, self.coef_z, None, None, None, self.bal, self.dlogits, self.bal_ws)
        return self.out

    def backward(self, dout):
        """Gradients of every weight for the gradient dout of out (fp32) and the balance loss."""
        m = self.moe
        m.moe_dropout_backward(dout, self.p, self.rng, self.dy)
        grads = dict(self.layer.backward(self.h, self.dy, router_grad=True, dlogits=self.dlogits))
        dh = (dout + grads.pop("dx")).bfloat16()
        m.moe_linear_backward(self.proj, self.x, self.W_o, None, dh, self.dx, self.dW_o, self.db_o, self.proj_ws)
        return {**{k[1:]: v for k, v in grads.items()}, "W_o": self.dW_o, "b_o": self.db_o}

    def step(self):
        """One training step; returns (data loss, balance losses) as device tensors."""
        diff = self.forward() - self.target
        loss = diff.square().mean() / 2
        # the sum over a token's features in place of the mean keeps gradients within bf16's reach
        grads = self.backward(diff / self.spec.T)
        for name, grad in grads.items():
            w = getattr(self, name, None) if name in ("W_o", "b_o") else self.weights[name]
            w.sub_(self.lr * grad.view(w.shape))
        self.rng[1] += 1          # another mask next time
        return loss, self.bal.clone()

    def status(self):
        return max(abs(self.layer.status()), abs(self.layer.backward_status()),
                   abs(self.moe.moe_read_status(self.proj_ws)), abs(self.moe.moe_read_status(self.bal_ws)))


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args(argv)
    from workloads import CONFIGS
    spec = CONFIGS["olmo"].replace(T=a.tokens, d_model=256, d_expert=128, d_shared=128, N=16, K=2, alpha=2.0)
    block = Block(spec, seq_len=128)
    losses = []
    for i in range(a.steps):
        loss, bal = block.step()
        losses.append(float(loss))
        total, lb, lz = bal.tolist()
        print(f"step {i:3d}  loss {losses[-1]:.4f}  balance {lb:.4f}  z {lz:.4f}  weighted {total:.5f}")
    assert block.status() == 0
    return losses


if __name__ == "__main__":
    main()
