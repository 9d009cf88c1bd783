"""Cases for the operators of a mixture-of-experts block on packed FP4 weights, and of the
low-rank adapters beside its shared projections: what each reads, computes and returns.

  route    router logits -> the experts of each token, their weights, and the (token, expert)
           pairs grouped by expert
  gate_up  the experts' fused gate and up products over those ragged groups, with
           silu(gate) * up as the output
  down     the experts' down products over the groups, and each token's weighted sum of them
  lora     y + scale_a * (x A_a^T) B_a^T, with an adapter of its own for every request

`run` computes them either in plain torch (fp32, rounded once at the end) or, with `own`, by the
framework's entry points.
"""
import math

import torch

own = False

NVFP4, MXFP4 = 0, 1
GROUP = {NVFP4: 16, MXFP4: 32}
FMT = {"nvfp4": NVFP4, "mxfp4": MXFP4}
DEV = "cuda"


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a small batch: latency only
        dict(name="route 8", op="route", M=8, E=128, topk=8),
        # a long prefill chunk
        dict(name="route 8192", op="route", M=8192, E=128, topk=8),
        # a single token: 8 experts of 128, each with one row
        dict(name="gate_up 1", op="gate_up", fmt="nvfp4", M=1, E=128, topk=8, I=768, H=2048),
        # a decode batch of odd size: nearly every expert is read for a few rows each
        dict(name="gate_up 77", op="gate_up", fmt="nvfp4", M=77, E=128, topk=8, I=768, H=2048),
        # a prefill chunk over fewer, larger MXFP4 experts, sizes off the tiles' multiples
        dict(name="gate_up 1021 mx", op="gate_up", fmt="mxfp4", M=1021, E=24, topk=3, I=1440, H=2592),
        # a long prefill chunk: products bound by the tensor cores
        dict(name="gate_up 4096", op="gate_up", fmt="nvfp4", M=4096, E=128, topk=8, I=768, H=2048),
        # the second half of the same layers: two tokens, a decode batch, a long chunk
        dict(name="down 2", op="down", fmt="nvfp4", M=2, E=128, topk=8, I=768, H=2048),
        dict(name="down 150 mx", op="down", fmt="mxfp4", M=150, E=24, topk=3, I=1440, H=2592),
        dict(name="down 4096", op="down", fmt="nvfp4", M=4096, E=128, topk=8, I=768, H=2048),
        # one request with its adapter, beside the output projection
        dict(name="lora 1", op="lora", M=1, requests=1, L=16, R=16, K=4096, N=4096),
        # a decode batch: nearly as many adapters as tokens, ranks that differ
        dict(name="lora 96", op="lora", M=96, requests=96, L=64, R=64, K=5120, N=6144),
        # a mixed prefill batch of a few long requests, some without an adapter
        dict(name="lora 5003", op="lora", M=5003, requests=11, L=8, R=32, K=4096, N=5120),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "gate_up", "down", "lora", "gate_up", "down", "lora"])
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256])
        return dict(op=op, M=_log(rng, 1, 8192), E=E, topk=rng.randint(1, 8))
    if op == "lora":
        M = _log(rng, 1, 5000)
        requests = M if M <= 128 and rng.random() < 0.6 else min(M, _log(rng, 1, 24))
        return dict(op=op, M=M, requests=requests, L=_log(rng, 1, 12 if requests < M else 96),
                    R=rng.choice([8, 16, 24, 32, 64]), K=8 * rng.randint(64, 640),
                    N=rng.randint(512, 5120))
    fmt = rng.choice(["nvfp4", "mxfp4"])
    E = rng.choice([8, 16, 24, 60, 64, 128])
    topk = rng.randint(1, min(8, E))
    I, H = 32 * rng.randint(8, 40), 32 * rng.randint(16, 72)
    M = _log(rng, 1, 4096)
    while M * topk * I * H > 4096 * 8 * 768 * 2048 or E * I * H > 128 * 768 * 2048:
        I, M = max(256, (I // 64) * 32), max(1, M // 2)
    return dict(op=op, fmt=fmt, M=M, E=E, topk=topk, I=I, H=H)


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _logits(g, M, E):
    """Router logits: every expert has a popularity of its own, as trained routers have."""
    return 1.5 * torch.randn(M, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)


def _top(x, k):
    """The k largest of each row, the largest first, equal values by the lowest index."""
    v, i = torch.sort(x, dim=1, descending=True, stable=True)
    return v[:, :k], i[:, :k].to(torch.int32)


def _grouped(ids, E):
    """Pairs (row-major in ids) in increasing expert order, and where each expert's begin."""
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices.to(torch.int32)
    ends = torch.cumsum((flat[:, None] == torch.arange(E, device=DEV)).sum(0), 0)
    return order, torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), ends]).to(torch.int32)


def _weight(g, fmt, E, N, K):
    """Gaussian weights quantised to the block format: codes [E, N, K/2] (low nibble = even k),
    scale bytes [E, N, K/group] and one global per expert."""
    sigma = 0.02 + 0.002 * (torch.arange(E) % 5)
    w = torch.randn(E, N, K // GROUP[fmt], GROUP[fmt], generator=g, device=DEV) * sigma.to(DEV)[:, None, None, None]
    top = w.abs().amax(-1, keepdim=True)
    if fmt == NVFP4:
        glob = 5.5 * sigma / (6 * 448)
        s = (top / (6 * glob.to(DEV)[:, None, None, None])).clamp(max=448).to(torch.float8_e4m3fn)
        scales, unit = s.view(torch.uint8), s.float() * glob.to(DEV)[:, None, None, None]
    else:
        x = torch.ceil(torch.log2(top / 6))
        glob, scales, unit = torch.ones(E), (x + 127).to(torch.uint8), torch.exp2(x)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = torch.bucketize((w / unit).abs(), mid, out_int32=True).to(torch.uint8) + 8 * (w < 0).to(torch.uint8)
    code = code.view(E, N, K)
    codes, scales = code[:, :, 0::2] | (code[:, :, 1::2] << 4), scales.squeeze(-1).contiguous()
    return codes, scales, glob


def _ranks(case):
    """The adapters' ranks: the largest, half and a quarter of it in turn."""
    return [max(1, case["R"] >> (a % 3)) for a in range(case["L"])]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "route":
        s["logits"] = _logits(g, case["M"], case["E"])
    elif case["op"] == "lora":
        M, L, R, K, N = (case[k] for k in ("M", "L", "R", "K", "N"))
        ranks = torch.tensor(_ranks(case), dtype=torch.int32, device=DEV)
        live = (torch.arange(R, device=DEV) < ranks[:, None]).to(torch.bfloat16)
        s["x"] = torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16)
        s["y"] = torch.randn(M, N, generator=g, device=DEV).to(torch.bfloat16)
        s["A"] = (torch.randn(L, R, K, generator=g, device=DEV) / K ** 0.5).to(torch.bfloat16) * live[:, :, None]
        s["B"] = (torch.randn(L, N, R, generator=g, device=DEV) / R ** 0.5).to(torch.bfloat16) * live[:, None, :]
        s["scale"] = 0.5 + torch.rand(L, generator=g, device=DEV)
        # requests are contiguous runs of tokens; one in nine has no adapter (-1)
        of = torch.randint(0, L, (case["requests"],), generator=g, device=DEV, dtype=torch.int32)
        of[4::9] = -1
        if case["requests"] == M:
            ids = of
        else:
            cut = torch.sort(torch.rand(case["requests"] - 1, generator=g, device=DEV)).values * M
            ids = of[torch.bucketize(torch.arange(M, device=DEV) + 0.5, cut)]
        s["ids"] = ids.contiguous()
        rows = (ids[:, None] == torch.arange(L, device=DEV)).sum(0)
        s["most"] = max(1, int(rows.max()))
        if own:
            import fp4_weight_only_nvfp4_gb300 as vt
            s["adapters"] = vt.LoraAdapters(s["A"], s["B"], s["scale"], ranks)
            s["groups"] = vt.group_rows(s["ids"], L)
            s["out"] = torch.empty_like(s["y"])
    else:
        fmt = FMT[case["fmt"]]
        M, E, topk, I, H = (case[k] for k in ("M", "E", "topk", "I", "H"))
        top, s["ids"] = _top(_logits(g, M, E), topk)
        s["ids"] = s["ids"].contiguous()
        s["weights"] = torch.softmax(top, dim=1)
        s["order"], s["offsets"] = _grouped(s["ids"], E)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        if case["op"] == "gate_up":
            s["x"] = torch.randn(M, H, generator=g, device=DEV).to(torch.bfloat16)
            s["gate"], s["up"] = _weight(g, fmt, E, I, H), _weight(g, fmt, E, I, H)
        else:
            # what silu(gate) * up looks like: mostly small, a few large
            a, b = (torch.randn(M * topk, I, generator=g, device=DEV) for _ in range(2))
            s["x"] = (torch.nn.functional.silu(a) * b).to(torch.bfloat16)
            s["w"] = _weight(g, fmt, E, H, I)
        if own:
            import fp4_weight_only_nvfp4_gb300 as vt
            if case["op"] == "gate_up":
                s["W"] = vt.PackedWeight.grouped_gate_up(*((c, sc, gl.tolist()) for c, sc, gl in (s["gate"], s["up"])),
                                                         fmt, E, I, H)
                s["out"] = torch.empty(M * topk, I, dtype=torch.bfloat16, device=DEV)
            else:
                c, sc, gl = s["w"]
                s["W"] = vt.PackedWeight.grouped(c, sc, gl.tolist(), fmt, E, H, I)
                s["out"] = torch.empty(M, H, dtype=torch.bfloat16, device=DEV)
            s["groups"] = vt.RowGroups(s["ids"], s["order"], s["offsets"], s["weights"])
            s["workspace"] = s["W"].ragged_workspace(M, topk)
    if own and case["op"] == "route":
        import fp4_weight_only_nvfp4_gb300 as vt
        s["out"] = vt.RowGroups.empty(case["M"], case["topk"], case["E"], DEV, weights=True)
        s["workspace"] = vt.group_workspace(case["M"], case["topk"], case["E"], DEV)
    return s


# ------------------------------------------------------------------------ the plain forms
def _e2m1(device):
    return torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=device)


def _dequant(fmt, codes, scales, glob):
    v = _e2m1(codes.device)
    w = torch.stack([v[(codes & 15).long()], v[(codes >> 4).long()]], -1).flatten(-2)
    if fmt == NVFP4:
        unit = scales.view(torch.float8_e4m3fn).float() * glob.to(w.device)[:, None, None]
    else:
        unit = torch.exp2(scales.float() - 127)
    return (w.unflatten(-1, (-1, GROUP[fmt])) * unit[..., None]).flatten(-2)


def _slots(order, offsets, E, most):
    """Where each grouped row stands in an [E, most] arrangement of the groups."""
    i = torch.arange(order.numel(), device=order.device)
    e = torch.bucketize(i, offsets[1:].long(), right=True)
    return e * most + i - offsets.long()[e]


def _products(s, rows, w, E):
    """rows (in group order) times each one's expert, fp32."""
    at = _slots(s["order"], s["offsets"], E, s["most"])
    a = torch.zeros(E * s["most"], rows.shape[1], device=rows.device)
    a[at] = rows.float()
    return torch.bmm(a.view(E, s["most"], -1), w.transpose(1, 2)).flatten(0, 1)[at]


def _plain(s):
    if s["op"] == "route":
        top, ids = _top(s["logits"], s["topk"])
        e = torch.exp(top - top[:, :1])
        order, offsets = _grouped(ids, s["E"])
        return {"ids": ids, "weights": e / e.sum(1, keepdim=True), "order": order, "offsets": offsets}
    if s["op"] == "lora":
        L, R = s["L"], s["R"]
        ids = s["ids"].long()
        has = ids >= 0
        order = torch.sort(torch.where(has, ids, L), stable=True).indices
        begin = torch.cumsum((ids[:, None] == torch.arange(L, device=ids.device)).sum(0), 0)
        begin = torch.cat([torch.zeros(1, dtype=torch.int64, device=ids.device), begin])
        # every token's place in an [L + 1, most] arrangement; tokens without an adapter share the last
        key = torch.where(has, ids, L)[order]
        at = torch.where(key < L, key * s["most"] + torch.arange(ids.numel(), device=ids.device) - begin[key], L * s["most"])
        x = torch.zeros(L * s["most"] + 1, s["K"], device=ids.device)
        x[at] = s["x"].float()[order]
        v = torch.bmm(x[:-1].view(L, s["most"], -1), s["A"].float().transpose(1, 2)) * s["scale"][:, None, None]
        d = torch.zeros(L * s["most"] + 1, s["N"], device=ids.device)
        d[:-1] = torch.bmm(v, s["B"].float().transpose(1, 2)).flatten(0, 1)
        d[-1] = 0
        y = s["y"].float()
        y[order] += d[at]
        return {"y": y.to(torch.bfloat16)}
    fmt, E = FMT[s["fmt"]], s["E"]
    if s["op"] == "gate_up":
        rows = s["x"][s["order"].long() // s["topk"]]
        gate = _products(s, rows, _dequant(fmt, *s["gate"]), E)
        up = _products(s, rows, _dequant(fmt, *s["up"]), E)
        return {"h": (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)}
    d = _products(s, s["x"], _dequant(fmt, *s["w"]), E)
    pairs = torch.empty_like(d)
    pairs[s["order"].long()] = d
    y = (pairs.view(s["M"], s["topk"], -1) * s["weights"][:, :, None]).sum(1)
    return {"y": y.to(torch.bfloat16)}


def run(state):
    if not own:
        return _plain(state)
    import fp4_weight_only_nvfp4_gb300 as vt
    s = state
    if s["op"] == "route":
        r = vt.moe_route(s["logits"], s["topk"], out=s["out"], workspace=s["workspace"])
        return {"ids": r.ids, "weights": r.weights, "order": r.order, "offsets": r.offsets}
    if s["op"] == "lora":
        return {"y": vt.lora_add(s["x"], s["adapters"], s["groups"], s["y"], out=s["out"])}
    if s["op"] == "gate_up":
        return {"h": vt.w4a16_gemm_ragged_silu_mul(s["x"], s["W"], s["groups"], out=s["out"], workspace=s["workspace"])}
    return {"y": vt.w4a16_gemm_ragged_combine(s["x"], s["W"], s["groups"], out=s["out"], workspace=s["workspace"])}


# --------------------------------------------------------------------- the path's own work
def _in_use(n, each, of):
    """Distinct members of `of` that n draws of `each` at a time are expected to touch."""
    return of * (1 - (1 - each / of) ** n)


def work(case):
    if case["op"] == "route":
        M, E, k = case["M"], case["E"], case["topk"]
        return {"bytes": 4 * M * E + 12 * M * k + 4 * (E + 1), "flops": M * E + 4 * M * k}
    if case["op"] == "lora":
        M, K, N, r = case["M"], case["K"], case["N"], _ranks(case)
        mean = sum(r) / len(r)
        share = 1 - len(range(4, case["requests"], 9)) / case["requests"]  # tokens with an adapter
        used = _in_use(share * case["requests"], 1, case["L"])
        return {"bytes": 2 * M * (share * K + 2 * N) + 2 * used * mean * (K + N) + 4 * M,
                "flops": 2 * share * M * mean * (K + N)}
    M, E, k, I, H = (case[x] for x in ("M", "E", "topk", "I", "H"))
    each = 0.5 + 1 / GROUP[FMT[case["fmt"]]]
    used = _in_use(M, k, E)
    if case["op"] == "gate_up":
        return {"bytes": used * 2 * I * H * each + 2 * M * H + 2 * M * k * I + 4 * M * k,
                "flops": 4 * M * k * I * H}
    return {"bytes": used * I * H * each + 2 * M * k * I + 2 * M * H + 8 * M * k, "flops": 2 * M * k * I * H}


# --------------------------------------------------------- the same from the definition, fp64
def _exact_weight(fmt, codes, scales, glob, e):
    """One expert's weight in fp64 from the bit fields of its codes and scales."""
    c = torch.empty(codes.shape[1], codes.shape[2] * 2, dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = (codes[e] & 15).long(), (codes[e] >> 4).long()
    exp, man = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(exp == 0, 0.5 * man, torch.exp2((exp - 1).double()) * (1 + 0.5 * man))
    val = torch.where(c >= 8, -mag, mag)
    b = scales[e].long()
    if fmt == NVFP4:
        ex, m = (b >> 3) & 15, (b & 7).double()
        unit = torch.where(ex == 0, m * 2.0 ** -9, torch.exp2((ex - 7).double()) * (1 + m / 8))
        unit = torch.where(b >= 128, -unit, unit) * float(glob[e])
    else:
        unit = torch.exp2((b - 127).double())
    return val * unit.repeat_interleave(GROUP[fmt], 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        l = s["logits"].double()
        idx = torch.argsort(l, dim=1, descending=True, stable=True)[:, :case["topk"]]
        w = torch.softmax(torch.gather(l, 1, idx), dim=1)
        return {"ids": idx.to(torch.int32), "weights": w, "order": None, "offsets": None}
    if case["op"] == "lora":
        y, ids = s["y"].double(), s["ids"]
        for a in range(case["L"]):
            m = torch.nonzero(ids == a).flatten()
            y[m] += s["scale"][a].double() * (s["x"][m].double() @ s["A"][a].double().T @ s["B"][a].double().T)
        return {"y": y}
    fmt, k = FMT[case["fmt"]], case["topk"]
    begin, order = s["offsets"].tolist(), s["order"].long()
    if case["op"] == "gate_up":
        h = torch.zeros(case["M"] * k, case["I"], dtype=torch.float64, device=DEV)
        for e in range(case["E"]):
            i = slice(begin[e], begin[e + 1])
            if begin[e + 1] > begin[e]:
                x = s["x"][order[i] // k].double()
                g = x @ _exact_weight(fmt, *s["gate"], e).T
                h[i] = g * torch.sigmoid(g) * (x @ _exact_weight(fmt, *s["up"], e).T)
        return {"h": h}
    y = torch.zeros(case["M"], case["H"], dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        i = slice(begin[e], begin[e + 1])
        if begin[e + 1] > begin[e]:
            d = s["x"][i].double() @ _exact_weight(fmt, *s["w"], e).T
            y.index_add_(0, order[i] // k, d * s["weights"].flatten()[order[i]].double()[:, None])
    return {"y": y}
