"""One decoder layer end to end: 4-bit projections, rotary positions, paged KV cache,
attention, the routed expert FFN and sampling of this package.

A prompt goes in by chunks into a cache of 4-bit codes, is branched into continuations
that share its pages, each continuation draws a few tokens, one is dropped and the
pages are brought together:

    python examples/decoder_layer.py

Weights are random (there is no model behind them); residual additions are the
only arithmetic done outside of the package's kernels.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bounded_expert_cache_gb300 as bec
import workloads as W


def random_q4_0(rows: int, cols: int, seed: int) -> torch.Tensor:
    """A random Q4_0 matrix [rows, cols] in split-plane layout, on the GPU."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, rows * cols // 2, dtype=np.uint8)
    scales = rng.uniform(0.5, 1.0, rows * cols // 32) / (4.6 * np.sqrt(cols))
    return torch.from_numpy(np.concatenate([codes, scales.astype(np.float16).view(np.uint8)])).cuda()


class DecoderLayer:
    """x -> h = x + O(attention(QKV(x))) -> h + experts(h), fp32 stream, bf16 cache.

    rot: a bec.Rotary that queries and keys are turned by. bits: 4 for a cache of 4-bit
    codes. vocab: tokens that next_token draws from.
    """

    def __init__(self, w: W.Workload, heads: int, kv_heads: int, head_dim: int, window: int = 0, sinks: int = 0,
                 pages: int = 64, page_tokens: int = 16, max_seqs: int = 8, max_tokens: int = 128,
                 rot: bec.Rotary | None = None, bits: int = 0, vocab: int = 0):
        self.w, self.heads, self.kv_heads, self.head_dim = w, heads, kv_heads, head_dim
        self.window, self.sinks, self.rot, self.vocab = window, sinks, rot, vocab
        self.n_qkv = (heads + 2 * kv_heads) * head_dim
        self.w_qkv = random_q4_0(self.n_qkv, w.hidden, 1)
        self.w_o = random_q4_0(w.hidden, heads * head_dim, 2)
        if vocab:
            self.w_vocab = random_q4_0(vocab, w.hidden, 3)
            self.embedding = torch.randn((vocab, w.hidden), device="cuda")
        self.kv = bec.KvCache.empty(1, pages, kv_heads, page_tokens, head_dim, max_seqs, pages, bits=bits)
        # the expert FFN, its experts in a bounded cache of slots
        self.store = torch.empty((1, w.n_experts, w.payload_bytes), dtype=torch.uint8, pin_memory=True)
        W.fill_store(w, self.store.numpy())
        self.moe = bec.Context(1, w.n_experts, w.top_k, w.hidden, w.inter, w.shared_inter, w.quant, w.slots,
                               max_tokens=max_tokens)
        self.moe.bind_store(self.store)
        self.w_router = torch.from_numpy(W.router_weights(w, 0)).cuda()
        self.plan = bec.Plan(w.n_experts, w.top_k, max_tokens)
        self.trace = {}  # the last step's intermediate tensors

    def _step(self, x, seqs, n_new, cu, attend):
        T = x.shape[0]
        H, Hkv, D = self.heads, self.kv_heads, self.head_dim
        qkv = bec.quant_linear(x, self.w_qkv, bec.Q4_0, self.n_qkv,
                               y=torch.empty((T, self.n_qkv), dtype=torch.bfloat16, device=x.device))
        q = qkv[:, :H * D].unflatten(1, (H, D))
        k = qkv[:, H * D:(H + Hkv) * D].unflatten(1, (Hkv, D))
        v = qkv[:, (H + Hkv) * D:].unflatten(1, (Hkv, D))
        self.kv.reserve(seqs, n_new)
        if self.rot is None:
            self.kv.write(0, k, v, seqs, cu)
        else:
            q = self.kv.write_rotary(0, q, k, v, seqs, cu, self.rot)
        a = attend(q)
        h = x + bec.quant_linear(a.flatten(1), self.w_o, bec.Q4_0, self.w.hidden,
                                 y=torch.empty((T, self.w.hidden), device=x.device))
        idx = torch.empty((T, self.w.top_k), dtype=torch.int32, device=x.device)
        wt = torch.empty((T, self.w.top_k), device=x.device)
        y = torch.empty((T, self.w.hidden), device=x.device)
        self.moe.layer_forward(0, h, self.w_router, None, idx, wt, self.plan, y)
        self.trace = dict(x=x, qkv=qkv, q=q, attention=a, h=h, idx=idx, y=y)
        return h + y

    def prefill(self, x, seqs, n_new):
        """Chunks of several sequences in one call: x [sum(n_new), hidden]."""
        cu = torch.zeros(len(n_new) + 1, dtype=torch.int32, device=x.device)
        cu[1:] = torch.cumsum(n_new, 0)
        return self._step(x, seqs, n_new, cu, lambda q: self.kv.attn_prefill(
            0, q, seqs, cu, window=self.window, sinks=self.sinks))

    def decode(self, x, seqs):
        """One new token of each sequence: x [len(seqs), hidden]."""
        ones = torch.ones_like(seqs)
        cu = torch.arange(len(seqs) + 1, dtype=torch.int32, device=x.device)
        return self._step(x, seqs, ones, cu, lambda q: self.kv.attn_decode(
            0, q, seqs, window=self.window, sinks=self.sinks))

    def next_token(self, x, **kept):
        """One token of each row of x, and its probability among those that are kept (bec.sample)."""
        x = x / x.pow(2).mean(-1, keepdim=True).sqrt()
        logits = bec.quant_linear(x, self.w_vocab, bec.Q4_0, self.vocab,
                                  y=torch.empty((x.shape[0], self.vocab), device=x.device))
        u = torch.rand(x.shape[0], device=x.device)
        self.trace.update(logits=logits, u=u)
        return bec.sample(logits, u, **kept)

    def check(self):
        self.kv.check_errors()
        self.moe.check_device_errors()

    def close(self):
        self.moe.close()


def main():
    torch.manual_seed(0)
    w = W.WORKLOADS["tiny"]
    layer = DecoderLayer(w, heads=4, kv_heads=2, head_dim=64, window=64, sinks=4, rot=bec.Rotary(64), bits=4, vocab=1000)
    i32 = dict(dtype=torch.int32, device="cuda")
    kept = dict(temperature=0.8, top_k=40, top_p=0.95)

    prompt = layer.embedding[torch.randint(layer.vocab, (150,), device="cuda")]
    for chunk in prompt.split(100):
        out = layer.prefill(chunk, torch.tensor([0], **i32), torch.tensor([chunk.shape[0]], **i32))
    layer.check()
    print(f"prompt of 150 tokens in 2 chunks: {int((layer.kv.ref > 0).sum())} pages in use")

    branches = torch.tensor([1, 2, 3], **i32)
    layer.kv.fork(torch.zeros(3, **i32), branches)
    token, prob = layer.next_token(out[-1:].expand(3, -1), **kept)
    drawn = [token]
    for _ in range(20):
        x = layer.decode(layer.embedding[token], branches)
        token, prob = layer.next_token(x, **kept)
        drawn.append(token)
    layer.check()
    print(f"3 branches of 20 tokens: {int((layer.kv.ref > 0).sum())} pages in use, "
          f"{int((layer.kv.ref > 1).sum())} of them shared, lengths {layer.kv.lens.tolist()[:4]}")
    for i, line in enumerate(torch.stack(drawn, 1).tolist()):
        print(f"  branch {i + 1} drew {line[:8]} ..., the last with probability {prob[i].item():.3f}")

    layer.kv.free(torch.tensor([0, 2], **i32))
    layer.kv.compact()
    x = layer.decode(layer.embedding[token[[0, 2]]], torch.tensor([1, 3], **i32))
    layer.check()
    used = torch.nonzero(layer.kv.ref).flatten().tolist()
    print(f"prompt and a branch dropped, pages brought together: {len(used)} pages in use, the last is {used[-1]}; "
          f"output rms {x.pow(2).mean().sqrt().item():.3f}")
    layer.close()


if __name__ == "__main__":
    main()
