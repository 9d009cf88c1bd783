"""GPU: the example block, each stage against fp64 on the inputs that the stage had."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from rows_helpers import BF16, assert_close, f64, products64, silu_mul64, weight64

pytestmark = pytest.mark.gpu
EXAMPLE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "moe_block.py")


def _example():
    spec = importlib.util.spec_from_file_location("moe_block", EXAMPLE)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _w64(part, e):
    return weight64(vt.NVFP4, part[0][e].cpu().numpy(), part[1][e].cpu().numpy(), np.float32(part[2][e]))


@pytest.mark.parametrize("hidden,inner", [(256, 96), (96, 256)])
def test_block(hidden, inner):
    torch.manual_seed(3)
    tokens, E, topk, L, R = 45, 6, 3, 4, 16
    block = _example().Block(hidden, inner, E, topk, L, R, tokens)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    ids = (torch.arange(tokens, dtype=torch.int32, device="cuda") % (L + 1) - 1)[:, None]
    b = block.buffers(tokens)
    block(x, ids, b)
    torch.cuda.synchronize()
    assert vt.workspace_status(block.ws_ffn) == 0

    # the adapters: rows of no request keep the projection, the others differ from it
    plain = vt.w4a16_gemm(x, block.W_o, workspace=block.ws_o)
    none = ids[:, 0].cpu().numpy() < 0
    assert torch.equal(b["y"][torch.from_numpy(none).cuda()], plain[torch.from_numpy(none).cuda()])
    A, B = f64(block.adapters.A), f64(block.adapters.B)
    ref, err = f64(plain).copy(), 2.0 ** -20 * np.abs(f64(plain))
    for m in np.nonzero(~none)[0]:
        a = int(ids[m, 0])
        v, va = A[a] @ f64(x[m]), np.abs(A[a]) @ np.abs(f64(x[m]))
        ref[m] += 0.5 * B[a] @ v
        err[m] += 0.5 * np.abs(B[a]) @ ((hidden + R) * 2.0 ** -23 * va + 2.0 ** -15 * np.abs(v))
    assert_close(b["y"], ref, err)

    # the experts, on the routes that the router chose from the logits it was given
    chosen, w = f64(b["routes"].ids).astype(int), f64(b["routes"].weights)
    assert np.array_equal(chosen, np.argsort(-f64(b["logits"]), axis=1, kind="stable")[:, :topk])
    y = f64(b["y"])
    ref, err = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    for e in range(E):
        for m, j in zip(*np.nonzero(chosen == e)):
            hh, herr = silu_mul64(y[m:m + 1], _w64(block.gate, e), _w64(block.up, e))
            herr = herr + BF16 * (np.abs(hh) + herr)  # h is bf16
            d, derr = products64(hh, _w64(block.down, e))
            derr = derr + herr @ np.abs(_w64(block.down, e)).T
            ref[m] += w[m, j] * d[0]
            err[m] += w[m, j] * (derr[0] + (BF16 + topk * 2.0 ** -22) * (np.abs(d[0]) + derr[0]))
    assert_close(b["out"], ref, err)

    # replayed from a graph on new inputs: the same bits as the call
    g = block.graph(x, ids, b)
    x.copy_(torch.randn_like(x))
    ids.copy_(ids.flip(0))
    g.replay()
    torch.cuda.synchronize()
    got = b["out"].clone()
    block(x, ids, b)
    assert torch.equal(got, b["out"])


def test_buffers_made_for_a_call_belong_to_its_stream():
    """Results of calls that make their own buffers on a side stream, while the current stream
    keeps allocating and overwriting memory."""
    torch.manual_seed(4)
    block = _example().Block(256, 96, 6, 3, 4, 16, 40)
    x = torch.randn(40, 256, device="cuda").bfloat16()
    logits = torch.randn(40, 6, device="cuda")
    want = vt.moe_ffn(x, block.W_gate_up, block.W_down, vt.moe_route(logits, 3))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        routes = vt.moe_route(logits, 3, stream=side)
        out = vt.moe_ffn(x, block.W_gate_up, block.W_down, routes, stream=side)
        for n in (1 << 12, 1 << 16, 1 << 20):
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        side.synchronize()
        assert torch.equal(out, want)


def test_the_example_runs(capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["moe_block.py", "--tokens", "70", "--hidden", "256", "--inner",
                                     "96", "--experts", "5", "--topk", "2"])
    _example().main()
    out = capsys.readouterr().out
    assert "prompt: 70 tokens" in out and "decode: 8 tokens" in out
