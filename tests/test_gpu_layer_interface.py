"""GPU: what the binding of the cache, its attention and the norms refuses."""
import pytest
import torch

import fp4_weight_only_nvfp4_gb300 as vt

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _cache(heads=2, dim=64, page=16, pages=4):
    g = torch.full((heads,), 0.01, device="cuda")
    return vt.KVCache.empty(pages, page, heads, dim, g, g.clone())


def _rows(*shape, dtype=BF, device="cuda"):
    return torch.zeros(*shape, dtype=dtype, device=device)


def test_cache_and_append():
    c, x, slots = _cache(), _rows(3, 2, 64), torch.arange(3, device="cuda")
    ok = dict(q=x, k=x.clone(), v=x.clone(), cache=c, slots=slots)
    vt.kv_append(**ok)
    table, pos = vt.rope_table(8, 64), torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad, match in ((dict(q=x.float()), "bf16"), (dict(k=_rows(3, 1, 64)), "k must be"), (dict(v=_rows(2, 2, 64)), "v must be"),
                       (dict(slots=slots.int()), "slots"), (dict(slots=slots[:2]), "slots"), (dict(slots=slots.cpu()), "CUDA"),
                       (dict(k=x.cpu()), "CUDA"), (dict(q=_rows(3, 64, 2).transpose(1, 2)), "side by side"),
                       (dict(q=_rows(2, 64)[:1].expand(3, 2, 64)), "side by side"), (dict(q=_rows(1, 2, 64).expand(3, 2, 64)), "overlapping"), (dict(positions=pos), "go together"),
                       (dict(positions=pos, table=table.double()), "fp32"), (dict(positions=pos.long(), table=table), "positions"),
                       (dict(positions=pos, table=table.cpu()), "CUDA"),
                       (dict(q_norm=_rows(64), k_norm=_rows(64, dtype=torch.float32)), "k_norm"),
                       (dict(q_norm=_rows(64, dtype=torch.float16), k_norm=_rows(64)), "bf16 or fp32"), (dict(q_norm=_rows(32), k_norm=_rows(64)), "q_norm"),
                       (dict(q=None, out=x), "no out"), (dict(out=_rows(3, 2, 64, dtype=torch.float32)), "out")):
        with pytest.raises(ValueError, match=match):
            vt.kv_append(**{**ok, **bad})
    for bad in (dict(q=_rows(3, 3, 64)), dict(q_norm=_rows(64)), dict(positions=pos, table=_rows(8, 8, dtype=torch.float32)),
                dict(q=torch.zeros(3 * 130, dtype=BF, device="cuda").as_strided((3, 2, 64), (130, 64, 1)))):
        with pytest.raises(vt.VtError):
            vt.kv_append(**{**ok, **bad})
    with pytest.raises(ValueError, match="k_codes"):
        c.put(slots, _rows(3, 2, 31, dtype=torch.uint8), *(_rows(3, 2, n, dtype=torch.uint8) for n in (4, 32, 4)))
    with pytest.raises(ValueError, match="slots"):
        c.get(slots[None])
    with pytest.raises(ValueError, match="k must be"):
        vt.kv_read(c, slots, out=(x[:2], x))
    with pytest.raises(ValueError, match="k_scale"):
        vt.KVCache.empty(4, 16, 3, 64, c.k_scale, c.v_scale)
    with pytest.raises(ValueError, match="data must be"):
        vt.KVCache(c.data[:, :-1], 16, 2, 64, c.k_scale, c.v_scale)
    with pytest.raises(vt.VtError, match="multiples of 128"):
        vt.KVCache(c.data.view(-1)[64:64 + c.data.shape[1]][None], 16, 2, 64, c.k_scale, c.v_scale).get(slots)


def test_attention():
    c, q = _cache(), _rows(3, 4, 64)
    tables, lens = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    ok = dict(q=q, cache=c, tables=tables, lens=lens)
    assert not vt.paged_attention(**ok).any()
    for bad, match in ((dict(q=q[0]), r"\[T, q_heads"), (dict(q=_rows(3, 4, 128)), "q must be"), (dict(tables=tables.long()), "tables"),
                       (dict(tables=tables[0]), "tables"), (dict(tables=tables.cpu()), "tables"), (dict(lens=lens[:2]), "lens"),
                       (dict(lens=lens.long()), "lens"), (dict(starts=lens), "starts"), (dict(sinks=_rows(4)), "sinks"),
                       (dict(sinks=_rows(3, dtype=torch.float32)), "sinks"), (dict(out=_rows(3, 4, 128)), "out"),
                       (dict(workspace=_rows(10)), "workspace"), (dict(tables=tables.expand(3, 2).t().contiguous().t()), "tables")):
        with pytest.raises(ValueError, match=match):
            vt.paged_attention(**{**ok, **bad})
    for bad in (dict(q=_rows(3, 3, 64)), dict(q=_rows(2, 4, 64)), dict(window=-1), dict(scale=float("nan")),
                dict(q=_rows(3, 130, 64)), dict(workspace=torch.zeros(4096, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(vt.VtError):
            vt.paged_attention(**{**ok, **bad})
    assert vt.paged_attention(q[:0], c, tables[:0], lens[:0]).shape == (0, 4, 64)


def test_norms():
    x, w = _rows(3, 32), _rows(32)
    for bad, match in ((dict(x=x.float()), "x must be"), (dict(x=x.cpu()), "CUDA"), (dict(residual=x[:2]), "residual"), (dict(residual=x.half()), "residual"),
                       (dict(weight=w[:31]), "weight"), (dict(weight=w.half()), "bf16 or fp32"), (dict(post_weight=w.float()), "post_weight"),
                       (dict(gate=w[:31]), "gate"), (dict(gate=_rows(2, 32)), "gate"), (dict(out=(None, x)), "go together"), (dict(out=(x.float(), x)), "h must be"),
                       (dict(residual=x.t().contiguous().t()), "unit inner stride")):
        with pytest.raises(ValueError, match=match):
            vt.residual_norm(**{**dict(x=x, residual=x.clone(), weight=w), **bad})
    for bad in (dict(eps=-1.0), dict(scale=float("inf"))):
        with pytest.raises(vt.VtError):
            vt.residual_norm(x, x.clone(), w, **bad)
    with pytest.raises(vt.VtError, match="H must be"):
        vt.residual_norm(_rows(1, 16385), None, _rows(16385))
