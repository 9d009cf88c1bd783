"""GPU: the norms around a block with its gate and residual sum, against fp64."""
import numpy as np
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt
from rows_helpers import acts, f64

pytestmark = pytest.mark.gpu


def _rms(x, w, eps):
    return x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * w


def _ref(x, r, w, pw, gate, scale, eps):
    a = f64(x)
    a = a if pw is None else _rms(a, f64(pw), eps)
    a = a if gate is None else a * f64(gate)
    h = a * scale + (0 if r is None else f64(r))
    # fp32: the sum of squares to H 2^-23 (half of it in its root), and a few roundings each
    unit = x.shape[1] * 2.0 ** -23 + 2.0 ** -20
    dh = unit * np.abs(a * scale) + 2.0 ** -22 * np.abs(h)
    y = _rms(h, f64(w), eps)
    # y also moves with its row's h: by dh itself and through the row's root mean square
    root = np.sqrt((h ** 2).mean(-1, keepdims=True) + eps)
    dy = (unit + np.sqrt((dh ** 2).mean(-1, keepdims=True)) / root) * np.abs(y) + dh / root * np.abs(f64(w))
    return h, dh, y, dy


def _near(got, ref, err):
    half = torch.finfo(got.dtype).eps / 2
    assert (np.abs(f64(got) - ref) <= err + half * (np.abs(ref) + err) + 2.0 ** -133).all()


CASES = [(1, 1), (1, 7), (3, 64), (1, 4096), (203, 2560), (17, 5120), (5, 8192), (2, 8200), (4, 16384), (3, 16383),
         (9, 2049), (33, 520)]


@pytest.mark.parametrize("T,H", CASES)
@pytest.mark.parametrize("post,gate,fp32,weights", [(False, None, False, "bf16"), (True, "channel", True, "fp32"),
                                                    (True, "token", False, "bf16"), (False, "channel", False, "fp32")])
def test_norms(T, H, post, gate, fp32, weights):
    rng = np.random.default_rng(T * 7 + H)
    kind = torch.float32 if weights == "fp32" else torch.bfloat16
    x, r = acts(rng, T, H), acts(rng, T, H).to(torch.float32 if fp32 else torch.bfloat16)
    w, pw = (1 + 0.2 * acts(rng, H).float()).to(kind), (0.5 + 0.1 * acts(rng, H).float()).to(kind)
    g = {None: None, "channel": acts(rng, H), "token": acts(rng, T, H)}[gate]
    on = lambda t: None if t is None else t.cuda()
    h, y = vt.residual_norm(x.cuda(), r.cuda(), w.cuda(), on(pw) if post else None, on(g), scale=0.7, eps=1e-5)
    hr, dh, yr, dy = _ref(x, r, w, pw if post else None, g, 0.7, 1e-5)
    assert h.dtype == r.dtype and y.dtype == torch.bfloat16
    _near(h, hr, dh)
    _near(y, yr, dy)


@pytest.mark.parametrize("H", [96, 97, 4096])
def test_strides_offsets_and_places(H):
    """Views of wider buffers, at odd offsets, and outputs in the inputs' place: equal values, and
    nothing beside the rows is touched."""
    rng = np.random.default_rng(H)
    T = 5
    x, r, g, w = acts(rng, T, H).cuda(), acts(rng, T, H).cuda(), acts(rng, T, H).cuda(), acts(rng, H).cuda()
    want = vt.residual_norm(x, r, w, w, g)
    for off, wide in ((0, 8), (8, 24), (1, 3), (3, 8)):
        buf = [torch.full((T, H + wide + off), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(5)]
        vx, vr, vg, vh, vy = (b[:, off:off + H] for b in buf)
        vx.copy_(x), vr.copy_(r), vg.copy_(g)
        h, y = vt.residual_norm(vx, vr, w, w, vg, out=(vh, vy))
        for got, ref in zip((h, y), want):  # another layout of the row sums in another order
            assert torch.allclose(got.float(), ref.float(), rtol=2.0 ** -7, atol=1e-5)
        if off == 0:
            assert torch.equal(h, want[0]) and torch.equal(y, want[1]) or H % 8
        again = vt.residual_norm(vx, vr, w, w, vg, out=(vr, vx))
        assert torch.equal(again[0], h) and torch.equal(again[1], y)
        for b in buf:
            assert (b[:, :off] == 7).all() and (b[:, off + H:] == 7).all()


def test_without_a_residual_and_special_rows():
    rng = np.random.default_rng(1)
    x, w = acts(rng, 6, 256), acts(rng, 256)
    x[1], x[2, 5], x[3, 7], x[4] = 0, float("nan"), float("inf"), x[4] * 1e-30
    h, y = vt.residual_norm(x.cuda(), None, w.cuda(), eps=1e-6)
    assert h is None
    _, _, ref, dy = _ref(x[[0, 4, 5]], None, w, None, None, 1.0, 1e-6)
    _near(y[[0, 4, 5]], ref, dy)
    assert (y[1] == 0).all() and y[2].isnan().all() and y[3, 7].isnan()
    assert vt.residual_norm(x.cuda()[:0], None, w.cuda())[1].shape == (0, 256)


def test_another_stream_and_a_graph():
    rng = np.random.default_rng(2)
    x, r, w = acts(rng, 40, 1024).cuda(), acts(rng, 40, 1024).cuda(), acts(rng, 1024).cuda()
    want = vt.residual_norm(x, r, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = vt.residual_norm(x, r, w, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph, out = torch.cuda.CUDAGraph(), (torch.empty_like(x), torch.empty_like(x))
    with torch.cuda.graph(graph):
        vt.residual_norm(x, r, w, out=out)
    x.neg_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, vt.residual_norm(x, r, w)))


@pytest.mark.parametrize("H", [96, 97])
def test_rows_more_than_32_bits_apart(H):
    rng = np.random.default_rng(H)
    T = 9
    x, r, g = (acts(rng, T, H).cuda() for _ in range(3))
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    want = vt.residual_norm(x, r, w, post_weight=w, gate=g)
    wide = torch.empty((T, 1 << 30), dtype=torch.bfloat16, device="cuda")
    part = [wide[:, 1000 * i:1000 * i + H] for i in range(5)]
    for a, b in zip(part, (x, r, g)):
        a.copy_(b)
    got = vt.residual_norm(part[0], part[1], w, post_weight=w, gate=part[2], out=(part[3], part[4]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
