"""Cases for what stands between the FP4 products of a decoder layer, served from a paged cache of
keys and values held in NVFP4: what each operator reads, computes and returns.

  norm    h = residual + scale * gate * norm(x), y = norm(h): the norms after one block and before
          the next, with the gate and the residual sum between them
  append  per-head norms of q and k, the position rotation, and k and v quantised into the cache's
          pages (the appended values are read back)
  decode  attention of one row per sequence over the cache
  extend  causal attention of chunks of rows, appended last, over the cache

`run` computes them either in plain torch (fp32, rounded once at the end) or, with `own`, by the
framework's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TABLE = 32768  # positions of the rotation's table


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of one sequence: latency only
        dict(name="norm 1", op="norm", T=1, H=4096, post=False, gate="none", fp32=False, scale=1.0),
        # a decode batch of odd size between two blocks with norms on both sides
        dict(name="norm 203", op="norm", T=203, H=2560, post=True, gate="channel", fp32=True, scale=0.5),
        # a long prefill chunk with a gate for every token
        dict(name="norm 8192", op="norm", T=8192, H=5120, post=True, gate="token", fp32=False, scale=1.0),
        # a decode step of an odd batch: one token of every sequence, the last rows are padding
        dict(name="append 37", op="append", T=37, pad=3, Hq=32, Hkv=8, D=128, rot=128, norm=True, page=16),
        # a prefill chunk, heads of 256 with a quarter of them rotated
        dict(name="append 8192", op="append", T=8192, pad=0, Hq=24, Hkv=4, D=256, rot=64, norm=True, page=64),
        # one sequence of a few hundred tokens: latency only
        dict(name="decode 1", op="decode", B=1, L=391, Hq=32, Hkv=8, D=128, page=16, window=0, sinks=False),
        # a serving batch of ragged lengths
        dict(name="decode 64", op="decode", B=64, L=8192, Hq=32, Hkv=4, D=128, page=64, window=0, sinks=False),
        # one long document
        dict(name="decode long", op="decode", B=1, L=131071, Hq=24, Hkv=4, D=256, page=64, window=0, sinks=False),
        # many short sequences, heads of 64 with sinks and a sliding window
        dict(name="decode 251", op="decode", B=251, L=1500, Hq=64, Hkv=8, D=64, page=32, window=1024, sinks=True),
        # a few drafted tokens for each of a batch of sequences
        dict(name="extend 4x31", op="extend", B=31, n=4, past=4000, Hq=32, Hkv=8, D=128, page=16, window=0, sinks=False),
        # chunks of several prompts, each behind what is in the cache, with a window and sinks
        dict(name="extend 2900", op="extend", B=5, n=900, past=2500, Hq=64, Hkv=8, D=64, page=32, window=512, sinks=True),
        # one long prompt from its first token on
        dict(name="extend 8192", op="extend", B=1, n=8192, past=0, Hq=32, Hkv=4, D=128, page=64, window=0, sinks=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "decode", "extend", "decode", "extend"])
    if op == "norm":
        H = rng.choice([8 * rng.randint(64, 1024), rng.randint(500, 8192)])
        T = min(_log(rng, 1, 8192), 8192 * 5120 // H)
        return dict(op=op, T=T, H=H, post=rng.random() < 0.5, gate=rng.choice(["none", "channel", "token"]),
                    fp32=rng.random() < 0.4, scale=rng.choice([1.0, 0.5, 0.22]))
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        T = _log(rng, 1, 8192)
        while T * (Hq + 2 * Hkv) * D > 8192 * 32 * 256:
            T = max(1, T // 2)
        return dict(op=op, T=T, pad=rng.randint(0, min(5, T - 1)), Hq=Hq, Hkv=Hkv, D=D,
                    rot=D // rng.choice([1, 2, 4]), norm=rng.random() < 0.5, page=page)
    window, sinks = rng.choice([0, 0, _log(rng, 16, 2000)]), rng.random() < 0.3
    if op == "decode":
        B = _log(rng, 1, 256)
        L = _log(rng, 1, 131071)
        while B * L * Hkv * D > 64 * 8192 * 4 * 128:
            L = max(1, L // 2)
        return dict(op=op, B=B, L=L, Hq=Hq, Hkv=Hkv, D=D, page=page, window=window, sinks=sinks)
    B = _log(rng, 1, 32)
    n = _log(rng, 1, 8192)
    past = rng.choice([0, _log(rng, 1, 16000)])
    while B * n * Hq * D * (n / 2 + past) > 8192 * 32 * 128 * 4096 or B * (n + past) * Hkv * D > 64 * 8192 * 512 \
            or B * n * Hq * (n + past) > 8192 * 32 * 8192:
        n, past = max(1, n // 2), past // 2
    return dict(op=op, B=B, n=n, past=past, Hq=Hq, Hkv=Hkv, D=D, page=page, window=window, sinks=sinks)


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(case):
    """(rows, length with them) of every sequence: ragged, the first the longest."""
    if case["op"] == "decode":
        return [(1, max(1, case["L"] - (b * 977) % max(1, (3 * case["L"]) // 4))) for b in range(case["B"])]
    n, past = case["n"], case["past"]
    rows = [max(1, n - (b * 389) % max(1, n // 2)) for b in range(case["B"])] if n > 8 else [n] * case["B"]
    return [(r, r + max(0, past - (b * 577) % max(1, past // 2 + 1))) for b, r in enumerate(rows)]


def _quantise(x, g):
    """x fp32 [..., D] in NVFP4 with the globals g: codes [..., D/2] (low nibble = even), scale bytes.
    Every operation is rounded on its own, in fp32."""
    v = x.unflatten(-1, (-1, 16))
    top = v.abs().amax(-1, keepdim=True)
    byte = torch.clamp(top / (6 * g), max=448.0).to(torch.float8_e4m3fn)
    unit = byte.float() * g
    q = (v / torch.where(unit == 0, 1.0, unit)).abs()
    code = (q > 0.25).to(torch.uint8)
    code += q >= 0.75
    code += q > 1.25
    code += q >= 1.75
    code += q > 2.5
    code += q >= 3.5
    code += q > 5
    code += 8 * (v < 0).to(torch.uint8)
    code = torch.where(unit == 0, 0, code).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte.view(torch.uint8).squeeze(-1)


def _spread(g, rows, heads, D):
    """Keys or values as models have them: a few channels of every head much larger than the others."""
    x = torch.randn(rows, heads, D, generator=g, device=DEV)
    x *= 0.6 + 2.4 * (torch.rand(heads, D, generator=g, device=DEV) > 0.95)
    return x


def _globals(g, heads):
    """fp32 [heads], as calibration on a few thousand tokens gives them."""
    return (9.0 + 4 * torch.rand(heads, generator=g, device=DEV)) / (6 * 448)


def _cache(s, g, case, lens):
    """The cache's pages and the table of each sequence's (-1 behind its last)."""
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    each = [-(-n // page) for n in lens]
    pages = sum(each)
    s["tables"] = torch.full((len(lens), max(each)), -1, dtype=torch.int32, device=DEV)
    mine = torch.arange(max(each), device=DEV) < torch.tensor(each, device=DEV)[:, None]
    s["tables"][mine] = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    s["k_scale"], s["v_scale"] = _globals(g, Hkv), _globals(g, Hkv)
    for k, w in (("k", s["k_scale"]), ("v", s["v_scale"])):
        s[k] = _quantise(_spread(g, pages * page, Hkv, D), w[:, None, None])
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if own:
        import fp4_weight_only_nvfp4_gb300 as vt
        s["cache"] = vt.KVCache.empty(pages, page, Hkv, D, s["k_scale"], s["v_scale"])
        s["cache"].put(torch.arange(pages * page, device=DEV), *s["k"], *s["v"])


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        s["x"] = (torch.randn(T, H, generator=g, device=DEV) * 2).to(torch.bfloat16)
        s["residual"] = torch.randn(T, H, generator=g, device=DEV).to(torch.float32 if case["fp32"] else torch.bfloat16)
        s["weight"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16)
        s["post_weight"] = (0.3 + 0.05 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16) if case["post"] else None
        shape = {"none": None, "channel": (H,), "token": (T, H)}[case["gate"]]
        s["gate_by"] = None if shape is None else torch.sigmoid(torch.randn(shape, generator=g, device=DEV)).to(torch.bfloat16)
        if own:
            s["h"], s["y"] = torch.empty_like(s["residual"]), torch.empty_like(s["x"])
        return s
    if case["op"] == "append":
        T, Hq, Hkv, D, page = (case[k] for k in ("T", "Hq", "Hkv", "D", "page"))
        # one projection's output holds q, k and v side by side
        s["qkv"] = _spread(g, T, Hq + 2 * Hkv, D).to(torch.bfloat16)
        s["q_norm"], s["k_norm"] = ((1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) for _ in range(2))
        s["positions"] = torch.randint(0, TABLE, (T,), generator=g, device=DEV, dtype=torch.int32)
        half = case["rot"] // 2
        angle = torch.arange(TABLE, device=DEV, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        s["table"] = torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()
        s["pages"] = -(-T // page) + 3
        s["slots"] = torch.randperm(s["pages"] * page, generator=g, device=DEV)[:T].contiguous()
        s["slots"][T - case["pad"]:] = -1
        s["k_scale"], s["v_scale"] = _globals(g, Hkv), _globals(g, Hkv)
        if own:
            import fp4_weight_only_nvfp4_gb300 as vt
            s["cache"] = vt.KVCache.empty(s["pages"], page, Hkv, D, s["k_scale"], s["v_scale"])
            s["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        return s
    Hq, D = case["Hq"], case["D"]
    rows = _rows(case)
    _cache(s, g, case, [n for _, n in rows])
    T = sum(r for r, _ in rows)
    s["most"] = max(r for r, _ in rows)
    s["q"] = (1.3 * torch.randn(T, Hq, D, generator=g, device=DEV)).to(torch.bfloat16)
    s["scale"] = D ** -0.5
    s["sink"] = torch.randn(Hq, generator=g, device=DEV) + 1 if case["sinks"] else None
    ends = torch.cumsum(torch.tensor([0] + [r for r, _ in rows], device=DEV), 0)
    s["starts"] = ends.to(torch.int32)
    if own:
        import fp4_weight_only_nvfp4_gb300 as vt
        s["out"] = torch.empty_like(s["q"])
        s["workspace"] = vt.attention_workspace(T, case["B"], Hq, s["cache"])
    return s


# ------------------------------------------------------------------------ the plain forms
def _rms(x, w):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _head_norm(x, w):
    """The norm of each head: its sum of squares in fp64, then fp32 with every operation rounded on
    its own, since the quantiser's borders follow."""
    ms = x.double().square().sum(-1, keepdim=True).float() / x.shape[-1]
    return x * (1 / torch.sqrt(ms + EPS)) * w.float()


def _rotate(x, cos, sin):
    half = cos.shape[-1]
    a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _e2m1():
    return torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=DEV)


def _values(codes, scales, g):
    """What codes [..., D/2] and scale bytes stand for, fp32."""
    v = _e2m1()
    x = torch.stack([v[(codes & 15).int()], v[(codes >> 4).int()]], -1).flatten(-2).unflatten(-1, (-1, 16))
    return (x * scales.view(torch.float8_e4m3fn).float()[..., None] * g).flatten(-2)


def _paged(s, name):
    """Every sequence's keys or values, fp32 [B, Hkv, places, D]."""
    page, Hkv = s["page"], s["Hkv"]
    at = s["tables"].clamp(min=0).long()
    codes, scales = (t.unflatten(0, (-1, page))[at].flatten(1, 2) for t in s[name])
    return _values(codes, scales, s[name + "_scale"][:, None, None]).transpose(1, 2)


def _plain(s):
    if s["op"] == "norm":
        a = s["x"].float()
        if s["post_weight"] is not None:
            a = _rms(a, s["post_weight"])
        if s["gate_by"] is not None:
            a = a * s["gate_by"].float()
        h = s["residual"].float() + s["scale"] * a
        return {"h": h.to(s["residual"].dtype), "y": _rms(h, s["weight"]).to(torch.bfloat16)}
    Hq, Hkv = s["Hq"], s["Hkv"]
    if s["op"] == "append":
        q, k, v = s["qkv"].float().split([Hq, Hkv, Hkv], 1)
        if s["norm"]:
            q, k = _head_norm(q, s["q_norm"]), _head_norm(k, s["k_norm"])
        cos, sin = s["table"][s["positions"].long()][:, None].chunk(2, -1)
        q, k = _rotate(q, cos, sin), _rotate(k, cos, sin)
        there = (s["slots"] >= 0)[:, None, None]
        k, v = (torch.where(there, _values(*_quantise(x, g[:, None, None]), g[:, None, None]), 0.0).to(torch.bfloat16)
                for x, g in ((k, s["k_scale"]), (v, s["v_scale"])))
        return {"q": q.to(torch.bfloat16), "k": k, "v": v}
    # rows of every sequence side by side: [B, Hkv, most * group, D]
    B, D, group, most = s["B"], s["D"], Hq // Hkv, s["most"]
    starts, lens = s["starts"].long(), s["lens"].long()
    n = starts[1:] - starts[:-1]
    i = torch.arange(most, device=DEV)
    at = torch.where(i < n[:, None], starts[:-1, None] + i, 0)
    q = s["q"].float()[at].unflatten(2, (Hkv, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    w = torch.matmul(q, _paged(s, "k").transpose(2, 3)).unflatten(2, (most, group)).mul_(s["scale"])
    j = torch.arange(w.shape[-1], device=DEV)
    pos = (lens - n)[:, None] + i
    seen = j <= pos[..., None]
    if s["window"]:
        seen &= j > pos[..., None] - s["window"]
    w.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].view(1, Hkv, 1, group, 1)
        top = torch.maximum(top, sink)
    top = torch.where(top == -math.inf, 0.0, top)
    w = w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(sink - top)
    o = torch.matmul(w.flatten(2, 3), _paged(s, "v")).unflatten(2, (most, group)) / total
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)
    return {"o": o[i < n[:, None]].to(torch.bfloat16)}


def run(state):
    if not own:
        return _plain(state)
    import fp4_weight_only_nvfp4_gb300 as vt
    s = state
    if s["op"] == "norm":
        h, y = vt.residual_norm(s["x"], s["residual"], s["weight"], post_weight=s["post_weight"], gate=s["gate_by"],
                                scale=s["scale"], eps=EPS, out=(s["h"], s["y"]))
        return {"h": h, "y": y}
    if s["op"] == "append":
        q, k, v = s["qkv"].split([s["Hq"], s["Hkv"], s["Hkv"]], 1)
        q = vt.kv_append(q, k, v, s["cache"], s["slots"], s["positions"], s["table"],
                         q_norm=s["q_norm"] if s["norm"] else None, k_norm=s["k_norm"] if s["norm"] else None,
                         eps=EPS, out=s["out"])
        k, v = vt.kv_read(s["cache"], s["slots"])
        return {"q": q, "k": k, "v": v}
    more = {} if s["op"] == "decode" else {"starts": s["starts"]}
    return {"o": vt.paged_attention(s["q"], s["cache"], s["tables"], s["lens"], scale=s["scale"], window=s["window"],
                                    sinks=s["sink"], out=s["out"], workspace=s["workspace"], **more)}


# --------------------------------------------------------------------- the path's own work
def work(case):
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        gate = {"none": 0, "channel": 2 * H, "token": 2 * T * H}[case["gate"]]
        return {"bytes": T * H * (4 + (8 if case["fp32"] else 4)) + gate + (4 if case["post"] else 2) * H,
                "flops": T * H * (14 if case["post"] else 10)}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        T = case["T"]
        # q, k and v in, q out, the cache written, read again, and its values out
        return {"bytes": T * D * (4 * Hq + 4 * Hkv + 4 * Hkv * 9 / 16 + 4 * Hkv) + 4 * T * (3 + case["rot"]),
                "flops": T * D * (8 * Hq + 16 * Hkv)}
    size, seen = 0, 0
    for r, n in _rows(case):
        first = n - r  # the position of the sequence's first row
        reach = case["window"] or n
        size += n - max(0, first - reach + 1)
        full = max(0, min(r, reach - first - 1))  # rows that see less than `reach` keys
        seen += full * first + full * (full + 1) // 2 + (r - full) * reach
    T = sum(r for r, _ in _rows(case))
    return {"bytes": 4 * T * Hq * D + size * Hkv * 2 * D * 9 / 16, "flops": 4 * seen * Hq * D}


# --------------------------------------------------------- the same from the definition, fp64
def _bits(codes, scales, g):
    """Values in fp64 from the bit fields of codes [..., D/2] and scale bytes."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    exp, man = (c >> 1) & 3, (c & 1).double()
    x = torch.where(exp == 0, 0.5 * man, torch.exp2((exp - 1).double()) * (1 + 0.5 * man))
    x = torch.where(c >= 8, -x, x)
    b = scales.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    unit = torch.where(e == 0, m * 2.0 ** -9, torch.exp2((e - 7).double()) * (1 + m / 8)) * g
    return x * unit.repeat_interleave(16, -1)


def _nearest(x, grid):
    """The nearest of an ascending grid to each x, halfway ones to the even index."""
    i = torch.bucketize(x, (grid[1:] + grid[:-1]) / 2)  # a value on a border counts to the lower one
    j = (i + 1).clamp(max=len(grid) - 1)
    tie = (j > i) & (x == (grid[i] + grid[j]) / 2) & (i % 2 == 1)
    return grid[torch.where(tie, j, i)]


def _exact_values(x, g):
    e = torch.arange(16, device=DEV, dtype=torch.float64)[:, None]
    m = torch.arange(8, device=DEV, dtype=torch.float64)
    units = torch.where(e == 0, m / 512, torch.exp2(e - 7) * (1 + m / 8)).flatten()[:-1]
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    v = x.unflatten(-1, (-1, 16))
    unit = _nearest(v.abs().amax(-1, keepdim=True) / (6 * g), units) * g
    return torch.where(unit == 0, 0.0, _nearest((v / unit).abs(), grid) * unit * v.sign()).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    rms = lambda x, w: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()  # noqa: E731
    if case["op"] == "norm":
        a = s["x"].double()
        a = a if s["post_weight"] is None else rms(a, s["post_weight"])
        a = a if s["gate_by"] is None else a * s["gate_by"].double()
        h = s["residual"].double() + case["scale"] * a
        return {"h": h, "y": rms(h, s["weight"])}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        x = s["qkv"].double()
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        if case["norm"]:
            q, k = rms(q, s["q_norm"]), rms(k, s["k_norm"])
        half = case["rot"] // 2
        t = s["table"].double()[s["positions"].long()][:, None]
        turn = torch.complex(t[..., :half], t[..., half:])

        def rope(y):
            z = torch.complex(y[..., :half], y[..., half:2 * half]) * turn
            return torch.cat([z.real, z.imag, y[..., 2 * half:]], -1)

        away = s["slots"] < 0
        out = {"q": rope(q)}
        for n, y, g in (("k", rope(k), s["k_scale"]), ("v", v, s["v_scale"])):
            out[n] = _exact_values(y, g.double()[:, None, None])
            out[n][away] = 0
        return out
    if work(case)["flops"] > 2e12:
        return None
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    row = 0
    for b, (r, n) in enumerate(_rows(case)):
        j = torch.arange(n, device=DEV)
        place = s["tables"][b].long()[j // case["page"]] * case["page"] + j % case["page"]
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            k, v = (_bits(s[x][0][place, h], s[x][1][place, h], s[x + "_scale"][h].double()) for x in ("k", "v"))
            for at in range(0, r, 1024):  # rows at a time
                i = torch.arange(at, min(r, at + 1024), device=DEV)
                away = j > (n - r + i)[:, None]
                if case["window"]:
                    away |= j <= (n - r + i)[:, None] - case["window"]
                w = torch.einsum("ihd,jd->hij", s["q"][row + i, heads].double(), k) * s["scale"]
                w.masked_fill_(away, -math.inf)
                if s["sink"] is not None:
                    w = torch.cat([w, s["sink"][heads].double()[:, None, None].expand(-1, i.numel(), 1)], 2)
                w = torch.softmax(w, 2)[..., :n]
                o[row + i, heads] = torch.einsum("hij,jd->ihd", w, v)
        row += r
    return {"o": o}
