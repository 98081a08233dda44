"""The example decoder layer: its projections, attention and experts run
together, each stage checked in 64 bits on the inputs it was given."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
import workloads as W

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

U24, U8 = 2.0 ** -24, 2.0 ** -8


def unpack_q4_0(w, rows, cols):
    """Q4_0 matrix in 64 bits from its packed bytes."""
    raw = w.cpu().numpy()
    codes = raw[:rows * cols // 2].reshape(rows, cols // 32, 16).astype(np.int64)
    d = raw[rows * cols // 2:].view(np.float16).astype(np.float64).reshape(rows, cols // 32, 1)
    return (np.concatenate([codes & 15, codes >> 4], axis=2) - 8) * d


def close(got, ref, tol):
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)


class Check:
    def __init__(self, layer, w):
        self.layer, self.w = layer, w
        n, h = layer.n_qkv, w.hidden
        self.wq = unpack_q4_0(layer.w_qkv, n, h).reshape(n, h)
        self.wo = unpack_q4_0(layer.w_o, h, layer.heads * layer.head_dim).reshape(h, -1)
        self.experts = [oracle.expert_matrices(layer.store[0, e].numpy(), w.hidden, w.inter, w.quant)
                        for e in range(w.n_experts)]

    def step(self, rows):
        """rows[i]: (keys, values, position) of row i's sequence, up to and with its own token."""
        L, t = self.layer, {k: v.double().cpu().numpy() for k, v in self.layer.trace.items()}
        H, Hkv, D = L.heads, L.kv_heads, L.head_dim
        ref = t["x"] @ self.wq.T
        tol = 200 * U24 * (np.abs(t["x"]) @ np.abs(self.wq).T)
        close(t["qkv"], ref, tol + 1.01 * U8 * np.abs(ref))
        q = t["qkv"][:, :H * D].reshape(-1, H, D)
        for i, (keys, vals, pos) in enumerate(rows):
            see = [j for j in range(pos + 1) if not L.window or pos - j < L.window or j < L.sinks]
            for h in range(H):
                k, v = keys[see, h // (H // Hkv)], vals[see, h // (H // Hkv)]
                s = k @ q[i, h] * D ** -0.5
                p = np.exp(s - s.max())
                p /= p.sum()
                A = p @ np.abs(v)
                delta = 2 * (D + 8) * U24 * np.max(np.abs(k) @ np.abs(q[i, h])) * D ** -0.5
                o = p @ v
                close(t["attention"][i, h], o, (2 * delta + 200 * U24 + U8) * A + 1.01 * U8 * np.abs(o))
        a = t["attention"].reshape(len(q), -1)
        ref = t["x"] + a @ self.wo.T
        close(t["h"], ref, 200 * U24 * (np.abs(a) @ np.abs(self.wo).T + np.abs(ref)))
        # the experts, on the h they were given
        idx, wt, _ = oracle.route(t["h"], W.router_weights(self.w, 0), None, self.w.top_k)
        assert np.array_equal(t["idx"].astype(np.int64), idx)
        y = oracle.moe_layer(t["h"], idx, wt, lambda e: self.experts[e], None)
        rel = np.linalg.norm(t["y"] - y) / np.linalg.norm(y)
        assert rel <= 5e-3, rel
        return t["qkv"]


@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
def test_decoder_layer_stage_by_stage(window, sinks):
    from decoder_layer import DecoderLayer
    torch.manual_seed(3)
    w = W.WORKLOADS["tiny"]
    layer = DecoderLayer(w, heads=4, kv_heads=2, head_dim=64, window=window, sinks=sinks)
    H, Hkv, D = 4, 2, 64
    chk = Check(layer, w)
    i32 = dict(dtype=torch.int32, device="cuda")
    hist = {}  # sequence -> list of (k, v) per token

    def add(seq, qkv_row):
        k = qkv_row[H * D:(H + Hkv) * D].reshape(Hkv, D)
        v = qkv_row[(H + Hkv) * D:].reshape(Hkv, D)
        hist.setdefault(seq, []).append((k, v))

    def run(kind, x, seqs, counts):
        s = torch.tensor(seqs, **i32)
        out = layer.decode(x, s) if kind == "decode" else layer.prefill(x, s, torch.tensor(counts, **i32))
        layer.check()
        qkv = layer.trace["qkv"].double().cpu().numpy()
        at, rows = 0, []
        for seq, n in zip(seqs, counts):
            for i in range(n):
                add(seq, qkv[at + i])
            K = np.stack([t[0] for t in hist[seq]])
            V = np.stack([t[1] for t in hist[seq]])
            rows += [(K, V, len(K) - n + i) for i in range(n)]
            at += n
        chk.step(rows)
        return out

    run("prefill", torch.randn((61, w.hidden), device="cuda"), [0, 4], [50, 11])
    run("prefill", torch.randn((40, w.hidden), device="cuda"), [0], [40])
    layer.kv.fork(torch.tensor([0, 0], **i32), torch.tensor([1, 2], **i32))
    hist[1], hist[2] = list(hist[0]), list(hist[0])
    for _ in range(3):
        run("decode", torch.randn((3, w.hidden), device="cuda"), [1, 2, 4], [1, 1, 1])
    layer.kv.free(torch.tensor([0, 2], **i32))
    layer.kv.compact()
    for _ in range(2):
        run("decode", torch.randn((2, w.hidden), device="cuda"), [4, 1], [1, 1])
    used = torch.nonzero(layer.kv.ref).flatten().tolist()
    assert used[-1] < len(used) + 2  # pages taken after compact are the lowest free ones
    layer.close()


def test_example_runs(capsys):
    import decoder_layer
    decoder_layer.main()
    out = capsys.readouterr().out
    assert "3 branches of 20 tokens" in out and "brought together" in out
