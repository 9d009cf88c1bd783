"""A decoder layer served from FP4 weights and an NVFP4 cache of keys and values:

    y      = norm(x)                                       the layer's first norm
    q,k,v  = y . W_qkv^T                                   one projection; k, v into the cache's pages,
    a      = attention(rope(norm(q)), cache)               normalised and rotated on the way
    h, y   = x + a . W_o^T, norm(h)                        the residual sum and the second norm
    out    = h + down(silu(gate(y)) * up(y))               (its sum is the next layer's residual_norm)

    python examples/decoder_layer.py [--prompt 500] [--batch 8] [--steps 20] ...

It takes a prompt through the layer in two chunks, then a batch of sequences token by token from a
CUDA graph, and prints the time of each.  Weights and inputs are random."""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import fp4_weight_only_nvfp4_gb300 as vt  # noqa: E402

EPS = 1e-6


def _quantized(n, k, dev):
    codes, scales, glob = vt.quantize((torch.randn(n, k, device=dev) * k ** -0.5).bfloat16(), vt.NVFP4)
    return codes, scales, float(glob)


class Layer:
    """The weights, a cache of `pages` pages, and workspaces for up to max_tokens tokens of max_batch
    sequences."""

    def __init__(self, hidden, inner, q_heads, kv_heads, head_dim, pages, page_size, max_tokens, max_batch, positions,
                 device="cuda"):
        self.hidden, self.inner, self.q_heads, self.kv_heads, self.dim = hidden, inner, q_heads, kv_heads, head_dim
        one = lambda n, k: vt.PackedWeight.from_codes(*_quantized(n, k, device), vt.NVFP4, n, k)
        self.W_qkv = one((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.W_o = one(hidden, q_heads * head_dim)
        self.W_gate_up = vt.PackedWeight.gate_up(_quantized(inner, hidden, device), _quantized(inner, hidden, device),
                                                 vt.NVFP4, inner, hidden, paired=True)
        self.W_down = one(hidden, inner)
        ones = lambda n: 1 + 0.1 * torch.randn(n, device=device)
        self.norm1, self.norm2, self.q_norm, self.k_norm = (ones(n) for n in (hidden, hidden, head_dim, head_dim))
        # keys are normalised: their largest value follows from the norm's weights; values are measured
        glob = torch.full((kv_heads,), 8.0 / (6 * 448), device=device)
        self.cache = vt.KVCache.empty(pages, page_size, kv_heads, head_dim, glob, glob.clone())
        self.table = vt.rope_table(positions, head_dim, device=device)
        self.ws = [W.new_workspace(max_tokens) for W in (self.W_qkv, self.W_o, self.W_gate_up, self.W_down)]
        self.ws_attention = vt.attention_workspace(max_tokens, max_batch, q_heads, self.cache)

    def buffers(self, tokens):
        dev = self.norm1.device
        rows = lambda n: torch.empty(tokens, n, dtype=torch.bfloat16, device=dev)
        return {"y": rows(self.hidden), "qkv": rows((self.q_heads + 2 * self.kv_heads) * self.dim),
                "a": rows(self.q_heads * self.dim), "o": rows(self.hidden), "h": rows(self.hidden),
                "act": rows(self.inner), "mlp": rows(self.hidden)}

    def __call__(self, x, b, slots, positions, tables, lens, starts=None):
        """x [tokens, hidden] bf16 -> (h, mlp): the layer's output is their sum, which the next layer's
        residual_norm takes.  Every step's result stays in b."""
        T = x.shape[0]
        heads = lambda t: t.view(T, -1, self.dim)
        vt.residual_norm(x, None, self.norm1, eps=EPS, out=(None, b["y"]))
        vt.w4a16_gemm(b["y"], self.W_qkv, out=b["qkv"], workspace=self.ws[0])
        q, k, v = heads(b["qkv"]).split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        vt.kv_append(q, k, v, self.cache, slots, positions, self.table, self.q_norm, self.k_norm, EPS, out=q)
        vt.paged_attention(q, self.cache, tables, lens, starts, out=heads(b["a"]), workspace=self.ws_attention)
        vt.w4a16_gemm(b["a"], self.W_o, out=b["o"], workspace=self.ws[1])
        vt.residual_norm(b["o"], x, self.norm2, eps=EPS, out=(b["h"], b["y"]))
        vt.w4a16_gemm_silu_mul(b["y"], self.W_gate_up, out=b["act"], workspace=self.ws[2])
        vt.w4a16_gemm(b["act"], self.W_down, out=b["mlp"], workspace=self.ws[3])
        return b["h"], b["mlp"]


def _slots(tables, seq, at, page_size):
    return tables[seq, at // page_size].long() * page_size + at % page_size


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("prompt", 500), ("batch", 8), ("steps", 20), ("hidden", 2048), ("inner", 4096),
                        ("q-heads", 16), ("kv-heads", 4), ("head-dim", 128), ("page-size", 16)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    torch.manual_seed(0)
    dev, page = "cuda", a.page_size
    longest = a.prompt + a.steps
    each = -(-longest // page)
    layer = Layer(a.hidden, a.inner, a.q_heads, a.kv_heads, a.head_dim, (a.batch + 1) * each, page,
                  max(a.prompt, a.batch), a.batch + 1, longest)
    tables = torch.randperm((a.batch + 1) * each, device=dev).to(torch.int32).view(a.batch + 1, each)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
    clock = lambda: torch.cuda.Event(enable_timing=True)

    # a prompt in two chunks, the last sequence's
    half = a.prompt // 2
    for begin, end in ((0, half), (half, a.prompt)):
        if end == begin:
            continue
        at = torch.arange(begin, end, device=dev)
        x, b = torch.randn(end - begin, a.hidden, device=dev).bfloat16(), layer.buffers(end - begin)
        call = lambda: layer(x, b, _slots(tables, a.batch, at, page), at.to(torch.int32), tables[a.batch:], i32(end),
                             i32(0, end - begin))
        call()
        t0, t1 = clock(), clock()
        t0.record(), call(), t1.record()
        t1.synchronize()
        print(f"chunk of {end - begin} behind {begin}: {t0.elapsed_time(t1) * 1e3:.1f} us")

    # a batch, one token each, replayed from a graph
    x, b = torch.randn(a.batch, a.hidden, device=dev).bfloat16(), layer.buffers(a.batch)
    lens, slots = torch.ones(a.batch, dtype=torch.int32, device=dev), torch.zeros(a.batch, dtype=torch.int64, device=dev)
    positions, seq = torch.zeros(a.batch, dtype=torch.int32, device=dev), torch.arange(a.batch, device=dev)
    run = lambda: layer(x, b, slots, positions, tables[:a.batch], lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    t0, t1 = clock(), clock()
    t0.record()
    for step in range(a.steps):
        positions.fill_(step), lens.fill_(step + 1)
        slots.copy_(_slots(tables, seq, torch.full_like(seq, step), page))
        graph.replay()
        x.copy_(b["h"] + b["mlp"])
    t1.record()
    t1.synchronize()
    print(f"{a.steps} steps of {a.batch} sequences: {t0.elapsed_time(t1) * 1e3 / max(1, a.steps):.1f} us each, "
          f"rms of the output {x.float().square().mean().sqrt().item():.3f}")
    assert vt.workspace_status(layer.ws_attention) == 0


if __name__ == "__main__":
    main()
