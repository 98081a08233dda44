"""The example decoder layer with rotary positions, a cache of 4-bit codes and drawn
tokens: each of these stages in 64 bits on what the one before it gave."""
import os
import sys

import pytest
import torch

import workloads as W
from test_gpu_kv import BF16, i32, worst
from test_gpu_kv4 import Codes, rows_ref
from test_gpu_rotary import codes_of, rounding, split, turned
from test_gpu_sample import outcomes

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("dim,interleaved,window", [(64, False, 0), (26, True, 24)])
def test_layer_with_rotary_codes_and_drawn_tokens(dim, interleaved, window):
    import bounded_expert_cache_gb300 as bec
    from decoder_layer import DecoderLayer
    torch.manual_seed(5)
    w = W.WORKLOADS["tiny"]
    H, Hkv, D, sinks = 4, 2, 64, 3
    rot = bec.Rotary(dim, interleaved=interleaved, factor=4.0, context=64)
    layer = DecoderLayer(w, heads=H, kv_heads=Hkv, head_dim=D, window=window, sinks=sinks, rot=rot, bits=4, vocab=777)
    kv, held = layer.kv, [0] * 8

    def check(out, seqs, counts, chunk):
        layer.check()
        t = layer.trace
        qkv = t["qkv"].unflatten(1, (-1, D))
        at = 0
        for s, n in zip(seqs, counts):
            held[s] += n
            assert int(kv.lens[s]) == held[s]
            rows = slice(at, at + n)
            pos = torch.arange(held[s] - n, held[s], device="cuda", dtype=torch.int32)
            y, tol = turned(qkv[rows, :H], pos, rot)
            assert worst(t["q"][rows], y, tol + rounding(y, BF16)) <= 1.0
            j = torch.arange(held[s], device="cuda")
            p, place = kv.table[s, j // kv.k.shape[3]].long(), j % kv.k.shape[3]
            K, V = [], []
            for pool, parts in ((kv.k, K), (kv.v, V)):
                codes, meta = split(pool[0], D)
                codes, meta = codes[p, :, place], meta[p, :, place]
                parts += Codes.parts(codes, meta)
                if parts is V:  # as they were given
                    want = codes_of(qkv[rows, H + Hkv:].float())
                    assert torch.equal(codes[-n:], want[0]) and torch.equal(meta[-n:], want[1])
            ref, tol = rows_ref(t["q"][rows], K, V, held[s], window, sinks, D ** -0.5, BF16, chunk)
            assert worst(t["attention"][rows], ref, tol) <= 1.0
            at += n
        assert torch.isfinite(out).all()

    for seqs, counts in (([0, 4], [50, 11]), ([0], [40])):
        x = layer.embedding[torch.randint(layer.vocab, (sum(counts),), device="cuda")]
        out = layer.prefill(x, i32(seqs), i32(counts))
        check(out, seqs, counts, True)
    kv.fork(i32([0, 0]), i32([1, 2]))
    held[1] = held[2] = held[0]
    x = out[-3:]
    for _ in range(3):
        token, prob = layer.next_token(x, temperature=0.7, top_k=50, top_p=0.9, min_p=0.01)
        z, u = layer.trace["logits"].double().cpu().numpy(), layer.trace["u"].tolist()
        for r in range(3):
            f32 = torch.tensor([0.7, 0.9, 0.01]).double().tolist()
            want = outcomes(z[r], u[r], f32[0], 50, f32[1], f32[2])
            assert int(token[r]) in [a[0] for a in want]
            assert min(abs(float(prob[r]) - a[1]) for a in want) <= 2.0 ** -23
        x = layer.decode(layer.embedding[token], i32([1, 2, 4]))
        check(x, [1, 2, 4], [1, 1, 1], False)
    kv.free(i32([0, 2]))
    kv.compact()
    x = layer.decode(layer.embedding[token[[0, 2]]], i32([1, 4]))
    check(x, [1, 4], [1, 1], False)
    layer.close()
