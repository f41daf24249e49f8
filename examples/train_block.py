"""One transformer block around the MoE layer, trained for a few steps on synthetic data.

    h   = x + (x W_o^T + b_o)           dense projection, its residual in the epilogue
    y   = MoE(h)                        routed and shared experts
    out = h + dropout(y)                mask from (seed, step), never stored
    loss = mean (out - target)^2 / 2 + balance loss and z-loss of the router

Every product, the dropout, the balance loss and all gradients run in the library; torch holds the
buffers, forms the difference to the target, adds and converts the stream's gradient where two operators want it in
different types, and applies plain gradient descent.

With --embedded the block is fed by token numbers, normalised in front of each half, and its gradients are clipped
to a global norm:

    x   = sqrt(d) table[ids]
    h   = x + (norm_1(x) W_o^T + b_o)
    out = h + dropout(MoE(norm_2(h)))

    python examples/train_block.py [--steps 20] [--tokens 512] [--embedded]
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
            w = self.weights[name] if name in self.weights else getattr(self, name)
            w.sub_(self.lr * grad.view(w.shape))
        self.rng[1] += 1          # another mask next time
        return loss, self.bal.clone()

    def status(self):
        return max(abs(self.layer.status()), abs(self.layer.backward_status()),
                   abs(self.moe.moe_read_status(self.proj_ws)), abs(self.moe.moe_read_status(self.bal_ws)))


class EmbeddedBlock(Block):
    """The block on token numbers, with normalised halves and clipped gradients."""

    def __init__(self, spec, seq_len, vocab=1000, max_norm=1.0, eps=1e-6, seed=0, device="cuda", **kw):
        super().__init__(spec, seq_len, seed=seed, device=device, **kw)
        moe, T, d = self.moe, spec.T, spec.d_model
        self.eps, self.max_norm, self.scale = eps, max_norm, d ** 0.5
        g = torch.Generator(device=device).manual_seed(seed + 2)
        self.ids = torch.randint(0, vocab, (T,), generator=g, device=device)
        self.ids[-1] = -1            # a padded place: a row of zeros, no gradient
        self.table = torch.randn((vocab, d), generator=g, device=device) * d ** -0.5
        self.norm_1, self.norm_2 = torch.ones(d, device=device), torch.ones(d, device=device)
        f32, bf16 = dict(device=device), dict(dtype=torch.bfloat16, device=device)
        self.xn, self.hn = torch.empty((T, d), **bf16), torch.empty((T, d), **bf16)
        self.rstd_1, self.rstd_2 = torch.empty(T, **f32), torch.empty(T, **f32)
        self.dh32, self.de = torch.empty((T, d), **f32), torch.empty((T, d), **bf16)
        self.dnorm_1, self.dnorm_2 = torch.empty(d, **f32), torch.empty(d, **f32)
        self.dtable, self.grad_norm = torch.empty_like(self.table), torch.empty(2, **f32)
        self.emb_ws = moe.alloc_embedding_workspace(T, vocab, d, device)
        self.norm_ws = moe.alloc_layernorm_workspace(T, d, device)
        self.clip_ws = moe.alloc_grad_norm_workspace(device)

    def forward(self):
        m = self.moe
        m.moe_embedding_forward(self.ids, self.table, self.scale, self.x, self.emb_ws)
        m.moe_layernorm_forward(self.x, None, self.norm_1, None, self.eps, None, self.xn, None, self.rstd_1, kind="rms")
        m.moe_linear_forward(self.proj, self.xn, self.W_o, self.b_o, self.x, None, self.h, self.proj_ws)
        m.moe_layernorm_forward(self.h, None, self.norm_2, None, self.eps, None, self.hn, None, self.rstd_2, kind="rms")
        y = self.layer.forward(self.hn)
        m.moe_dropout_add(y, self.h, self.p, self.rng, self.out)
        m.moe_balance_loss(self.layer.cfg, self.layer.out["logits"], self.layer.out["topk_idx"], None, self.seq_len,
                           self.coef_balance, self.coef_z, None, None, None, self.bal, self.dlogits, self.bal_ws)
        return self.out

    def backward(self, dout):
        """Gradients of every weight for the gradient dout of out and the balance loss, clipped together."""
        m = self.moe
        m.moe_dropout_backward(dout, self.p, self.rng, self.dy)
        grads = dict(self.layer.backward(self.hn, self.dy, router_grad=True, dlogits=self.dlogits))
        # the stream's own gradient passes beside the layer and joins behind the normalisation
        m.moe_layernorm_backward(self.h, self.norm_2, None, self.rstd_2, grads.pop("dx"), dout, self.dh32, self.dnorm_2,
                                 None, self.norm_ws, kind="rms")
        dh = self.dh32.bfloat16()
        m.moe_linear_backward(self.proj, self.xn, self.W_o, None, dh, self.dx, self.dW_o, self.db_o, self.proj_ws)
        m.moe_layernorm_backward(self.x, self.norm_1, None, self.rstd_1, self.dx, dh, self.de, self.dnorm_1, None,
                                 self.norm_ws, kind="rms")
        m.moe_embedding_backward(self.ids, self.de, self.scale, self.dtable, self.emb_ws)
        grads = {**{k[1:]: v for k, v in grads.items()}, "W_o": self.dW_o, "b_o": self.db_o, "norm_1": self.dnorm_1,
                 "norm_2": self.dnorm_2, "table": self.dtable}
        m.moe_clip_grad_norm(list(grads.values()), self.max_norm, None, self.grad_norm, self.clip_ws)
        return grads

    def status(self):
        return max(super().status(), *(abs(self.moe.moe_read_status(w)) for w in (self.emb_ws, self.norm_ws, self.clip_ws)))


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--embedded", action="store_true")
    a = ap.parse_args(argv)
    from workloads import CONFIGS
    spec = CONFIGS["olmo"].replace(T=a.tokens, d_model=256, d_expert=128, d_shared=128, N=16, K=2, alpha=2.0)
    block = (EmbeddedBlock if a.embedded else Block)(spec, seq_len=128)
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
