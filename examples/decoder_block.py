"""A decoder block whose attention keeps its keys and values in the paged 4-bit
cache and whose MLP is the fast-weight layer: a prompt is taken in segments, as
a server would, then tokens one at a time.

    x1 = x + Wo attention(rotary(Wq n), rotary(Wk n), Wv n),  n = norm(x)
    y  = x1 + layer(H = norm(x1), X0 = x0)

kv_append rotates a segment's queries and keys and puts keys and values into
the cache in one launch; kv_attention reads them there; block_norm adds what it
returns and takes the next norm in one pass; the layer carries its state from
segment to segment and into decode_step. The projections are torch's.

    python examples/decoder_block.py --tokens 16384 --new 64
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import test_layer_gate_amd as ttt  # noqa: E402
import synth  # noqa: E402


class DecoderBlock:
    """batch sequences of up to max_len tokens. mlp: the layer's Wg, Wu, taps,
    W_target and W_down0; attn: Wq, Wk, Wv [heads * dim, d_model] and Wo
    [d_model, heads * dim]."""

    def __init__(self, attn, mlp, eta, chunk, batch, max_len, heads, kv_heads, dim, *, page=64,
                 base=1e6, scaling=None):
        self.w, self.mlp, self.eta, self.chunk = attn, mlp, eta, chunk
        self.batch, self.heads, self.kv_heads, self.dim = batch, heads, kv_heads, dim
        self.dtype = attn["Wq"].dtype
        self.Wqkv = torch.cat([attn["Wq"], attn["Wk"], attn["Wv"]]).t().contiguous()
        self.rope = ttt.rope_table(max_len, dim, base, **(scaling or {}))
        per = -(-max_len // page)
        self.pages = ttt.kv_pages(batch * per, page, kv_heads, dim)
        # the sequences' pages in turn, as they come when sequences grow together
        self.table = torch.arange(batch * per, dtype=torch.int32, device="cuda").reshape(per, batch).t().contiguous()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.seen = 0
        W = mlp["W_down0"].float()
        self.W_state = W.expand(batch, *W.shape).contiguous().clone()
        self.decode_state = None

    def attention(self, x):
        """x [batch, T, d] -> x1 = x + attention and norm(x1), the T tokens appended."""
        B, T, d = x.shape
        h, g, D = self.heads, self.kv_heads, self.dim
        x = x.contiguous()  # (of several sequences' segments, rows that are not evenly apart)
        n = ttt.block_norm(x, pre=True)[1]
        qkv = (n.reshape(B * T, d) @ self.Wqkv).reshape(B * T, h + 2 * g, D)
        q, k, v = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
        self.seen += T
        self.lens += T
        # q is rotated in place, in the projection's own rows
        ttt.kv_append(self.pages, self.table, self.lens, k, v, q=q, q_out=q, rope_table=self.rope)
        o = ttt.kv_attention(q, self.pages, self.table, self.lens, max_new=T, max_kv=self.seen)
        return ttt.block_norm(x, (o.reshape(B * T, h * D) @ self.w["Wo"].t()).reshape(B, T, d), pre=True)

    def segment(self, x, x0):
        """The next T tokens of every sequence, T a multiple of the chunk."""
        if x.shape[1] % self.chunk or self.decode_state is not None:
            raise ValueError("segments are whole chunks, and come before decoding")
        x1, h = self.attention(x)
        m = self.mlp
        return x1 + ttt.layer_forward_continue(h, x0, None, m["Wg"], m["Wu"], self.W_state, m["taps"],
                                               m["W_target"], self.eta, self.chunk, pad="chunk")

    def step(self, x, x0):
        """One token of every sequence: x, x0 [batch, d]."""
        m = self.mlp
        if self.decode_state is None:
            f, d = m["Wg"].shape
            f32 = [int(t.dtype == torch.float32) for t in (x, m["Wg"])]
            desc = ttt.make_desc(self.batch, 1, d, f, m["taps"].shape[0], *f32, 0, ttt._binding.FLAG_PAD_CHUNK)
            self.decode_state = torch.empty(ttt.decode_state_size(desc, self.chunk), dtype=torch.uint8, device="cuda")
            ttt.decode_begin(self.W_state, self.chunk, self.decode_state, act_dtype=x.dtype,
                             weight_dtype=m["Wg"].dtype, conv_k=m["taps"].shape[0])
        x1, h = (t[:, 0] for t in self.attention(x[:, None]))
        return x1 + ttt.decode_step(h, x0, m["Wg"], m["Wu"], m["taps"], m["W_target"], self.eta, self.chunk,
                                    self.seen - 1, self.W_state, self.decode_state)


def random_block(config, batch, max_len, heads, kv_heads, dim, seed=0, seq_len=64, **kw):
    """A block with random weights at a configuration of synth, and its inputs
    x0 [batch, seq_len, d]."""
    cfg = synth.CONFIGS[config]
    dtype = torch.float32 if cfg.dtype == "f32" else torch.bfloat16
    x = synth.make_inputs(cfg, batch=batch, seq_len=seq_len, seed=seed)
    mlp = {k: torch.from_numpy(x[k]).to(dtype).cuda().contiguous() for k in ("Wg", "Wu", "taps", "W_target", "W_down0")}
    r = torch.Generator("cuda").manual_seed(seed)
    d = cfg.d_model

    def weight(n, m):
        return (torch.randn((n, m), generator=r, device="cuda") * m ** -0.5).to(dtype)
    attn = dict(Wq=weight(heads * dim, d), Wk=weight(kv_heads * dim, d), Wv=weight(kv_heads * dim, d),
                Wo=weight(d, heads * dim))
    block = DecoderBlock(attn, mlp, cfg.eta, cfg.chunk, batch, max_len, heads, kv_heads, dim, **kw)
    return block, torch.from_numpy(x["X0"]).to(dtype).cuda()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--config", default="qwen3_4b_64k", choices=sorted(synth.CONFIGS))
    ap.add_argument("--batch", type=int, default=1)
    ap.add_argument("--tokens", type=int, default=16384, help="the prompt's, a multiple of the chunk")
    ap.add_argument("--segment", type=int, default=4096)
    ap.add_argument("--new", type=int, default=64)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--dim", type=int, default=128)
    a = ap.parse_args()
    block, x0 = random_block(a.config, a.batch, a.tokens + a.new, a.heads, a.kv_heads, a.dim, seq_len=a.tokens + a.new)
    chunk = block.chunk
    if a.tokens % chunk or a.segment % chunk or a.tokens < chunk:
        ap.error(f"--tokens and --segment must be multiples of the chunk, {chunk}")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for s in range(0, a.tokens, a.segment):
        part = x0[:, s:min(s + a.segment, a.tokens)].contiguous()
        y = block.segment(part, part)
    torch.cuda.synchronize()
    t1 = time.perf_counter()
    for t in range(a.tokens, a.tokens + a.new):
        part = x0[:, t].contiguous()
        y = block.step(part, part)
    torch.cuda.synchronize()
    t2 = time.perf_counter()
    n = a.batch
    print(f"{a.config}, {n} x {a.tokens} tokens in segments of {a.segment}: {1e3 * (t1 - t0):.1f} ms, "
          f"{n * a.tokens / (t1 - t0):.0f} tokens/s (first calls included)")
    if a.new:
        print(f"{a.new} single tokens: {1e6 * (t2 - t1) / a.new:.0f} us each; cache {block.pages.numel() / 1e6:.1f} MB")
    print(f"last outputs finite: {bool(torch.isfinite(y).all())}")


if __name__ == "__main__":
    main()
