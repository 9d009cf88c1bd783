"""GPU: the cache, its attention and the norms with the products between them, as a decoder layer runs
them (examples/decoder_layer.py): every step against its definition, from the step's own inputs."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from layer_helpers import F, attention, head_norm, quantise, rotate, values
from rows_helpers import assert_close, f64

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def _rms(x, w, eps):
    return x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * w


def _product(y, x, W):
    """bf16(x . w^T): w as fp32, the fp32 sum off by K 2^-23 of the terms' absolute values, activations to 2^-20."""
    w = f64(W.dequant())
    ref, size = f64(x) @ w.T, np.abs(f64(x)) @ np.abs(w).T
    assert_close(y, ref, (x.shape[1] * 2.0 ** -23 + 2.0 ** -20) * size)


def _norm(y, h, w):
    """bf16(norm(h) * w) of an h that is itself within half a bf16 step of the kernel's (see residual_norm)."""
    ref = _rms(f64(h), f64(w), 1e-6)
    assert_close(y, ref, (h.shape[1] * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -7) * np.abs(ref))


def _check(layer, x, b, k_raw, slots, positions, tables, lens, starts, k, v):
    """The buffers of one call against the definitions; k, v: the cache's values [slots, heads, D] before, brought up
    to date."""
    T, D, Hq, Hkv = x.shape[0], layer.dim, layer.q_heads, layer.kv_heads
    page = layer.cache.page_size
    table = layer.table.cpu().numpy()[positions.cpu().numpy()]
    cos, sin = np.split(table, 2, axis=1)
    raw = k_raw.float().cpu().numpy().reshape(T, Hq + 2 * Hkv, D)
    q, kk, vv = raw[:, :Hq], raw[:, Hq:Hq + Hkv], raw[:, Hq + Hkv:]
    q, kk = (rotate(head_norm(t, w.cpu().numpy(), 1e-6), cos, sin, False) for t, w in ((q, layer.q_norm), (kk, layer.k_norm)))
    got = b["qkv"].view(T, -1, D)[:, :Hq]
    assert torch.equal(got.cpu(), torch.from_numpy(q).to(torch.bfloat16))
    for into, t, g in ((k, kk, layer.cache.k_scale), (v, vv, layer.cache.v_scale)):
        g = g.cpu().numpy()[None, :, None]
        into[slots.cpu().numpy()] = values(*quantise(t, g), g.astype(np.float64))
    ref, err = attention(f64(got), k, v, tables.cpu().numpy(), lens.cpu().numpy(), None if starts is None else starts.cpu().numpy(),
                         page, D ** -0.5)
    assert_close(b["a"].view(T, Hq, D), ref, err)
    _product(b["o"], b["a"], layer.W_o)
    h = f64(x) + f64(b["o"])
    assert_close(b["h"], h, 2.0 ** -22 * (np.abs(f64(x)) + np.abs(f64(b["o"]))))
    _norm(b["y"], b["h"], layer.norm2)
    _product(b["mlp"], b["act"], layer.W_down)


def test_chunks_then_single_tokens():
    from decoder_layer import Layer, _slots
    torch.manual_seed(1)
    page, pages, hidden = 16, 24, 256
    layer = Layer(hidden, 320, 6, 2, 64, pages, page, 130, 3, 200)
    cache = layer.cache
    slots_all = pages * page
    k = np.full((slots_all, 2, 64), np.nan)
    v = k.copy()
    tables = torch.randperm(pages, device="cuda").to(torch.int32).view(3, 8)
    lens = [0, 0, 0]

    def call(rows):
        """rows[s] more tokens for each sequence s."""
        T = sum(rows)
        at = torch.cat([torch.arange(l, l + r) for l, r in zip(lens, rows)]).cuda()
        seq = torch.repeat_interleave(torch.arange(3), torch.tensor(rows)).cuda()
        for s, r in enumerate(rows):
            lens[s] += r
        slots, positions = _slots(tables, seq, at, page), at.to(torch.int32)
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        starts = None if rows == [1, 1, 1] else torch.tensor(np.cumsum([0] + rows), dtype=torch.int32, device="cuda")
        x, b = torch.randn(T, hidden, device="cuda").bfloat16(), layer.buffers(T)
        # the projection's output before the rotation in its place
        y = vt.residual_norm(x, None, layer.norm1, eps=1e-6)[1]
        _norm(y, x, layer.norm1)
        raw = vt.w4a16_gemm(y, layer.W_qkv)
        _product(raw, y, layer.W_qkv)
        layer(x, b, slots, positions, tables, n, starts)
        _check(layer, x, b, raw, slots, positions, tables, n, starts, k, v)

    call([60, 1, 37])    # prompts of different lengths
    call([1, 1, 1])      # a token each
    call([30, 2, 0])     # a chunk beside two drafted tokens
    call([1, 1, 1])
    assert vt.workspace_status(layer.ws_attention) == 0


def test_the_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_layer.py"), "--prompt", "90", "--batch", "3",
                        "--steps", "5", "--hidden", "512", "--inner", "640", "--q-heads", "8", "--kv-heads", "2"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "chunk of 45 behind 45" in r.stdout and "steps of 3 sequences" in r.stdout
