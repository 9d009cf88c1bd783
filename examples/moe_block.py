"""A mixture-of-experts block with a low-rank adapter per request, served from FP4 weights:

    y   = x . W_o^T + adapter(x)          the shared projection and each request's adapter
    ids = top-k of y . W_router^T         the experts of every token
    out = sum_j w_j * down_j(silu(gate_j(y)) * up_j(y))

    python examples/moe_block.py [--tokens 300] [--experts 32] [--topk 4] ...

It runs the block on a prompt's worth of tokens and on a batch of single tokens replayed from a
CUDA graph, and prints the time of each.  Weights and inputs are random."""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import fp4_weight_only_nvfp4_gb300 as vt  # noqa: E402


def _quantized(n, k, sigma, dev):
    codes, scales, glob = vt.quantize((torch.randn(n, k, device=dev) * sigma).bfloat16(), vt.NVFP4)
    return codes, scales, float(glob)


def _stacked(E, n, k, dev):
    parts = [_quantized(n, k, k ** -0.5, dev) for _ in range(E)]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]), [p[2] for p in parts]


class Block:
    """The weights, and buffers for up to max_tokens tokens (zeroed or made once)."""

    def __init__(self, hidden, inner, experts, topk, adapters, rank, max_tokens, device="cuda"):
        self.topk, self.experts, self.hidden = topk, experts, hidden
        one = lambda n: vt.PackedWeight.from_codes(*_quantized(n, hidden, hidden ** -0.5, device),
                                                   vt.NVFP4, n, hidden)
        self.W_o, self.W_router = one(hidden), one(experts)
        self.gate, self.up = _stacked(experts, inner, hidden, device), _stacked(experts, inner, hidden, device)
        self.down = _stacked(experts, hidden, inner, device)
        self.W_gate_up = vt.PackedWeight.grouped_gate_up(self.gate, self.up, vt.NVFP4, experts, inner, hidden)
        self.W_down = vt.PackedWeight.grouped(*self.down, vt.NVFP4, experts, hidden, inner)
        self.adapters = vt.LoraAdapters(
            (torch.randn(adapters, rank, hidden, device=device) * hidden ** -0.5).bfloat16(),
            (torch.randn(adapters, hidden, rank, device=device) * rank ** -0.5).bfloat16(),
            torch.full((adapters,), 0.5, device=device))
        self.ws_o, self.ws_router = self.W_o.new_workspace(max_tokens), self.W_router.new_workspace(max_tokens)
        self.ws_route = vt.group_workspace(max_tokens, topk, max(experts, adapters), device)
        self.ws_ffn = vt.moe_ffn_workspace(self.W_gate_up, self.W_down, max_tokens, topk)

    def buffers(self, tokens):
        dev = self.W_o.packed.device
        rows = lambda n: torch.empty(tokens, n, dtype=torch.bfloat16, device=dev)
        return {"y": rows(self.hidden), "logits": rows(self.experts), "out": rows(self.hidden),
                "requests": vt.RowGroups.empty(tokens, 1, self.adapters.L, dev),
                "routes": vt.RowGroups.empty(tokens, self.topk, self.experts, dev, weights=True)}

    def __call__(self, x, adapter_ids, b):
        """x [tokens, hidden] bf16, adapter_ids int32 [tokens, 1] (-1: none) -> b["out"]."""
        vt.w4a16_gemm(x, self.W_o, out=b["y"], workspace=self.ws_o)
        vt.group_rows(adapter_ids, self.adapters.L, out=b["requests"], workspace=self.ws_route)
        vt.lora_add(x, self.adapters, b["requests"], b["y"], out=b["y"])
        vt.w4a16_gemm(b["y"], self.W_router, out=b["logits"], workspace=self.ws_router)
        vt.moe_route(b["logits"], self.topk, out=b["routes"], workspace=self.ws_route)
        return vt.moe_ffn(b["y"], self.W_gate_up, self.W_down, b["routes"], out=b["out"],
                          workspace=self.ws_ffn)

    def graph(self, x, adapter_ids, b):
        """The call on these buffers as a CUDA graph (the current contents of x and adapter_ids
        are used at every replay)."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self(x, adapter_ids, b)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self(x, adapter_ids, b)
        return g


def _ms(f, n=20):
    f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        f()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / n


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 300), ("batch", 8), ("hidden", 2048), ("inner", 768),
                        ("experts", 32), ("topk", 4), ("adapters", 8), ("rank", 16)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    torch.manual_seed(0)
    block = Block(a.hidden, a.inner, a.experts, a.topk, a.adapters, a.rank, max(a.tokens, a.batch))
    for name, tokens in (("prompt", a.tokens), ("decode", a.batch)):
        x = torch.randn(tokens, a.hidden, device="cuda").bfloat16()
        ids = (torch.arange(tokens, dtype=torch.int32, device="cuda") % (a.adapters + 1) - 1)[:, None]
        b = block.buffers(tokens)
        if name == "decode":
            ms = _ms(block.graph(x, ids, b).replay)
        else:
            ms = _ms(lambda: block(x, ids, b))
        print(f"{name}: {tokens} tokens, {ms * 1e3:.1f} us, rms of the output "
              f"{b['out'].float().square().mean().sqrt().item():.3f}")
    assert vt.workspace_status(block.ws_ffn) == 0


if __name__ == "__main__":
    main()
