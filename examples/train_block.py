"""A block that is trained: linear attention with a decay for each head, the
fast-weight layer as its MLP, the norms and residual adds around both, and AdamW
with 8-bit states.

    x1 = x + Wo linear_attention(Wq n, Wk n, Wv n),  n = norm(x)
    y  = x1 + layer(H = norm(x1), X0 = x),           loss = |y - target|^2 / (2 rows)

Forward, backward and step are the library's; the projections are torch's. Its
gradients are written out, call by call, as a framework's own would be.

    python examples/train_block.py --config qwen3_4b_8k --steps 10
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import test_layer_gate_amd as ttt  # noqa: E402
import synth  # noqa: E402

MLP = ("Wg", "Wu", "W_down0", "taps", "W_target")


class TrainBlock:
    """weights: Wqkv [(heads + 2 kv_heads) dim, d], Wo [d, heads dim], norm1
    and norm2 [d] and the layer's Wg, Wu, W_down0, taps and W_target, all of one
    type. bits: of AdamW's states; bf16 weights have float32 masters."""

    def __init__(self, weights, eta, chunk, heads, kv_heads, dim, *, bits=8):
        self.w, self.eta, self.chunk, self.bits = weights, eta, chunk, bits
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        half = torch.arange(1, kv_heads + 1, dtype=torch.float32, device="cuda")
        self.log_decay = -torch.exp2(-1 - 8 * half / kv_heads)     # from two tokens or so to some 500
        params = list(weights.values())
        self.masters = [p.float() for p in params] if params[0].dtype == torch.bfloat16 else None
        self.state = ttt.adamw_state(params, bits)
        self.steps = 0

    def gradients(self, x, target):
        """x, target [B, T, d], T a multiple of the chunk -> loss (on the GPU),
        the gradients of the weights (float32) and of x."""
        w = self.w
        B, T, d = x.shape
        h, g, D = self.heads, self.kv_heads, self.dim
        mlp = [w[k] for k in MLP]

        _, n = ttt.block_norm(x, pre=w["norm1"])
        n = n.reshape(B * T, d)
        qkv = (n @ w["Wqkv"].t()).reshape(B, T, h + 2 * g, D)
        q, k, v = qkv[:, :, :h], qkv[:, :, h:h + g], qkv[:, :, h + g:]
        o = ttt.linear_attention(q, k, v, self.log_decay).reshape(B * T, h * D)
        f = (o @ w["Wo"].t()).reshape(B, T, d)
        x1, n2 = ttt.block_norm(x, f, pre=w["norm2"])
        y2, _, saved = ttt.layer_forward_train(n2, x, *mlp, self.eta, self.chunk)
        y, _ = ttt.block_norm(x1, y2)

        dy = y.float() - target.float()
        loss = dy.square().sum() / (2 * B * T)
        dy = (dy / (B * T)).to(x.dtype)

        grads = ttt.layer_backward(n2, x, *mlp, self.eta, self.chunk, dy, saved=saved)
        dn2 = grads.pop("dH").to(x.dtype)
        dx0 = grads.pop("dX0")
        b = ttt.block_norm_backward(dy, dn2, x1, f, pre=w["norm2"])
        grads["dnorm2"] = b["dpre"]
        df = b["df"].reshape(B * T, d)
        grads["dWo"] = (df.t() @ o).float()
        do = (df @ w["Wo"]).reshape(B, T, h, D)
        dqkv = torch.cat(ttt.linear_attention_backward(do, q, k, v, self.log_decay)[:3], 2).reshape(B * T, -1)
        grads["dWqkv"] = (dqkv.t() @ n).float()
        dn = (dqkv @ w["Wqkv"]).reshape(B, T, d)
        b = ttt.block_norm_backward(b["dx"], dn, x, pre=w["norm1"])
        grads["dnorm1"] = b["dpre"]
        return loss, {k: grads["d" + k] for k in w}, b["dx"] + dx0.to(x.dtype)

    def step(self, x, target, *, lr=1e-3, max_norm=1.0, **kw):
        """One step of AdamW; the loss before it."""
        loss, grads, _ = self.gradients(x, target)
        grads = list(grads.values())
        self.steps += 1
        ttt.adamw_step(list(self.w.values()), grads, self.state, lr=lr, step=self.steps, bits=self.bits,
                       masters=self.masters, norm=ttt.grad_norm(grads), max_norm=max_norm, **kw)
        return loss


def random_block(config, batch, seq_len, heads, kv_heads, dim, seed=0, **kw):
    """A block with random weights at a configuration of synth, and its inputs
    x [batch, seq_len, d]."""
    cfg = synth.CONFIGS[config]
    dtype = torch.float32 if cfg.dtype == "f32" else torch.bfloat16
    given = synth.make_inputs(cfg, batch=batch, seq_len=seq_len, seed=seed)
    r = torch.Generator("cuda").manual_seed(seed)
    d = cfg.d_model

    def weight(n, m):
        return (torch.randn((n, m), generator=r, device="cuda") * m ** -0.5).to(dtype)
    weights = dict(Wqkv=weight((heads + 2 * kv_heads) * dim, d), Wo=weight(d, heads * dim),
                   norm1=torch.ones(d, dtype=dtype, device="cuda"), norm2=torch.ones(d, dtype=dtype, device="cuda"),
                   **{k: torch.from_numpy(given[k]).to(dtype).cuda().contiguous() for k in MLP})
    block = TrainBlock(weights, cfg.eta, cfg.chunk, heads, kv_heads, dim, **kw)
    return block, torch.from_numpy(given["X0"]).to(dtype).cuda()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--config", default="qwen3_4b_8k", choices=sorted(synth.CONFIGS))
    ap.add_argument("--batch", type=int, default=1)
    ap.add_argument("--tokens", type=int, default=8192, help="of each sequence, a multiple of the chunk")
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--lr", type=float, default=1e-3)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--dim", type=int, default=128)
    a = ap.parse_args()
    block, x = random_block(a.config, a.batch, a.tokens, a.heads, a.kv_heads, a.dim, bits=a.bits)
    if a.tokens % block.chunk:
        ap.error(f"--tokens must be a multiple of the chunk, {block.chunk}")
    target = torch.roll(x, -1, 1)
    for s in range(a.steps):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        loss = block.step(x, target, lr=a.lr)
        torch.cuda.synchronize()
        print(f"step {s + 1}: loss {float(loss):.5f}, {1e3 * (time.perf_counter() - t0):.1f} ms", flush=True)


if __name__ == "__main__":
    main()
