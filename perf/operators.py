"""Cases of the expert-layer operators: routing, the way of the tokens to their experts and
back, and the FP8 product with FP32 block scales.

The operators, as a mixture-of-experts layer uses them:

* routing: scores of a token over all experts, top-k inside the best expert groups,
  renormalised weights, and the gradient of the logits;
* dispatch: the map from routed slots to expert-ordered rows, and the token rows quantized
  into them (FP8 with an FP32 scale per 1x128 block, or MXFP4 as the framework's path has it);
* product: expert-grouped E4M3 x E4M3 with FP32 scales per 1x128 block of the activations
  and per 128x128 block of the weights;
* combine: the weighted sum of a token's expert rows, and its gradients.

``run`` computes them in plain torch operations where ``own`` is false and through the
framework's entry points where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
TINY = 2.0 ** -100          # floor under a block's amax (FP8 with FP32 scales)


def listed():
    return [
        # one token of a running request is routed: a call's latency (256 experts in 8 groups,
        # sigmoid scores with a balance bias, the router of the framework's 671B setting)
        {"name": "route one token", "op": "route", "tokens": 1, "experts": 256, "groups": 8, "kept": 4, "best": 2,
         "k": 8, "score": "sigmoid", "bias": True, "f32": True},
        # a batch of prompts through the same router
        {"name": "route prompts", "op": "route", "tokens": 32768, "experts": 256, "groups": 8, "kept": 4, "best": 2,
         "k": 8, "score": "sigmoid", "bias": True, "f32": True},
        # a softmax router without groups over an odd number of experts, BF16 logits (ties)
        {"name": "route softmax odd", "op": "route", "tokens": 5003, "experts": 60, "groups": 1, "kept": 1, "best": 1,
         "k": 4, "score": "softmax", "bias": False, "f32": False},
        # the router's gradient in a training step
        {"name": "route backward", "op": "route_back", "tokens": 16384, "experts": 256, "k": 8, "score": "softmax",
         "f32": True},
        # a decoding batch: map and FP8 rows for 32 experts
        {"name": "dispatch decode", "op": "dispatch", "tokens": 64, "experts": 32, "first": 0, "local": 32, "k": 8,
         "width": 7168, "format": "fp8"},
        # prompts: 65536 routed rows of the hidden width
        {"name": "dispatch prompts", "op": "dispatch", "tokens": 8192, "experts": 32, "first": 0, "local": 32, "k": 8,
         "width": 7168, "format": "fp8"},
        # one rank's share of 256 experts, MXFP4 codes, then the FP8 rows of the forward product
        {"name": "dispatch share mxfp4", "op": "dispatch", "tokens": 4001, "experts": 256, "first": 64, "local": 64,
         "k": 8, "width": 2048, "format": "mxfp4"},
        # a decoding batch: a few rows for each of 32 experts, the weights are the traffic
        {"name": "product decode", "op": "product", "experts": 32, "rows": 128, "n": 4096, "width": 7168},
        # prompts: the up projection of 8 experts
        {"name": "product prompts", "op": "product", "experts": 8, "rows": 32768, "n": 4096, "width": 7168},
        # odd sizes: features and width that end inside a scale block
        {"name": "product odd", "op": "product", "experts": 3, "rows": 1501, "n": 1352, "width": 1744},
        # the layer's output for prompts, beside a shared expert's output
        {"name": "combine prompts", "op": "combine", "tokens": 8192, "experts": 32, "first": 0, "local": 32, "k": 8,
         "width": 7168, "base": True},
        # its gradients: of the expert rows and of the weights
        {"name": "combine backward", "op": "combine_back", "tokens": 4099, "experts": 64, "first": 0, "local": 64,
         "k": 6, "width": 2048},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_back", "dispatch", "dispatch", "product", "product", "combine",
                     "combine_back"])
    if op in ("route", "route_back"):
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        experts = groups * rng.randint(max(1, 8 // groups), max(2, 384 // groups))
        kept = rng.randint(max(1, groups // 2), groups)
        k = rng.randint(1, min(16, kept * (experts // groups)))
        tokens = _log(rng, 1, 32768)
        score = rng.choice(["softmax", "sigmoid"])
        if op == "route_back":              # (of one renormalised weight it would be zero)
            return {"op": op, "tokens": tokens, "experts": experts, "k": max(2, k), "score": score,
                    "f32": rng.random() < 0.5}
        return {"op": op, "tokens": tokens, "experts": experts, "groups": groups, "kept": kept,
                "best": min(rng.choice([1, 2]), experts // groups), "k": k, "score": score,
                "bias": rng.random() < 0.5, "f32": rng.random() < 0.5}
    if op == "product":
        experts = _log(rng, 1, 32)
        width = 16 * _log(rng, 8, 512)
        n = 8 * _log(rng, 16, 512)
        rows = _log(rng, 1, 16384)
        return {"op": op, "experts": experts, "rows": rows, "n": n, "width": width}
    experts = _log(rng, 2, 256)
    local = experts if rng.random() < 0.6 else rng.randint(1, experts)
    first = rng.randint(0, experts - local)
    k = rng.randint(1, min(8, experts))
    tokens = _log(rng, 1, 8192)
    case = {"op": op, "tokens": tokens, "experts": experts, "first": first, "local": local, "k": k}
    if op == "dispatch":
        case["format"] = rng.choice(["fp8", "fp8", "mxfp4"])
        case["width"] = 128 * _log(rng, 1, 56) if case["format"] == "mxfp4" else 16 * _log(rng, 8, 448)
    else:
        case["width"] = 8 * _log(rng, 16, 896)
        if op == "combine":
            case["base"] = rng.random() < 0.5
    return case


# ---- inputs ------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 2654435761 % (1 << 62))


def _logits(case, g):
    """Router logits: experts of unequal popularity, tokens of unequal sharpness."""
    t, e = case["tokens"], case["experts"]
    pull = torch.randn(e, device=DEV, generator=g) * 0.5
    sharp = torch.rand(t, 1, device=DEV, generator=g) + 0.7
    return (torch.randn(t, e, device=DEV, generator=g) * sharp + pull).to(
        torch.float32 if case["f32"] else torch.bfloat16)


def _undecided(case, logits, bias):
    """Rows whose choice hangs on less than the rounding of a 32-bit score: two different
    neighbours in the order of the groups or of the experts closer than 2^-15."""
    e, ng, k = case["experts"], case.get("groups", 1), case["k"]
    l64 = logits.double()
    c = torch.softmax(l64, 1) if case["score"] == "softmax" else torch.sigmoid(l64)
    if bias is not None:
        c = c + bias.double()

    def close(v, n):
        v = v[:, :n + 1]
        gap = v[:, :-1] - v[:, 1:]
        return ((gap > 0) & (gap < 2.0 ** -15 * v[:, :-1].abs().clamp_min(1e-12))).any(1)

    bad = torch.zeros(c.shape[0], dtype=torch.bool, device=DEV)
    if ng > 1:
        gs = c.view(-1, ng, e // ng).sort(2, descending=True).values[:, :, :case["best"]].sum(2)
        gv, gi = gs.sort(dim=1, descending=True, stable=True)
        bad |= close(gv, case["kept"])
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, gi[:, :case["kept"]], True)
        c = c.masked_fill(~keep.repeat_interleave(e // ng, 1), -math.inf)
    v = c.sort(1, descending=True).values
    return bad | close(v.nan_to_num(neginf=-1e30), min(k, e - 1))


def _router_inputs(case, g):
    logits = _logits(case, g)
    bias = torch.randn(case["experts"], device=DEV, generator=g) * 0.05 if case.get("bias") else None
    for _ in range(6):                      # rows that rounding decides are drawn again
        bad = _undecided(case, logits, bias)
        logits = torch.where(bad[:, None], _logits(case, g), logits)
    return logits, bias


def _slots(case, g):
    """Routed ids [T, k]: distinct experts of a token, some experts far busier than others,
    one token in fifty masked out (ids -1)."""
    t, e, k = case["tokens"], case["experts"], case["k"]
    pull = torch.randn(e, device=DEV, generator=g) * 0.7
    ids = (torch.rand(t, e, device=DEV, generator=g).clamp_min(1e-9).log().neg().log().neg() + pull).topk(k, 1).indices
    ids = ids.to(torch.int32)
    dead = torch.rand(t, device=DEV, generator=g) < 0.02
    return ids.masked_fill_(dead[:, None], -1)


def _rows(t, k, g):
    """BF16 activations: unit scale, a few loud channels, tokens of unequal size."""
    loud = 1 + 15 * (torch.rand(k, device=DEV, generator=g) < 0.004)
    size = torch.exp(0.5 * torch.randn(t, 1, device=DEV, generator=g))
    return (torch.randn(t, k, device=DEV, generator=g) * loud * size).to(torch.bfloat16)


def _blocks(x):
    """[..., K] -> [..., ceil(K/128), 128], zero past K."""
    k = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, -k % 128))
    return x.view(*x.shape[:-1], -1, 128)


def _counts(case, seed):
    """Rows of each expert: unequal shares that add up to `rows`, some of them zero."""
    r = torch.Generator().manual_seed(int(seed) + 977)
    share = torch.softmax(0.4 * torch.randn(case["experts"], generator=r), 0)
    pick = torch.multinomial(share, case["rows"], replacement=True, generator=r)
    return torch.bincount(pick, minlength=case["experts"]).tolist()


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("route", "route_back"):
        t, e, k = case["tokens"], case["experts"], case["k"]
        s["logits"], s["bias"] = _router_inputs(case, g)
        if op == "route":
            s["mask"] = (torch.rand(t, device=DEV, generator=g) >= 0.02).to(torch.uint8)
            s["ids"] = torch.empty((t, k), dtype=torch.int32, device=DEV)
            s["weights"] = torch.empty((t, k), dtype=torch.float32, device=DEV)
        else:
            order = s["logits"].float().sort(dim=1, descending=True, stable=True).indices
            s["ids"] = order[:, :k].to(torch.int32).contiguous()
            s["dweights"] = torch.randn(t, k, device=DEV, generator=g)
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    if op == "product":
        m, n, k, e = case["rows"], case["n"], case["width"], case["experts"]
        counts = _counts(case, seed)
        s["most"] = max(counts)
        s["offs"] = torch.tensor([0] + counts, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)
        kb, nb = -(-k // 128), -(-n // 128)
        x = _rows(m, k, g).float()
        sa = _blocks(x).abs().amax(-1).clamp_min(TINY) / 448
        s["a"] = (x / sa.repeat_interleave(128, 1)[:, :k]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        s["sa"] = sa.contiguous()
        # weights as a checkpoint holds them: every 128x128 block filled to E4M3's range
        w = torch.empty((e, n, k), dtype=torch.uint8, device=DEV)
        for i in range(e):
            v = torch.randn(n, k, device=DEV, generator=g)
            w[i] = (v * (448 / 4.5)).clamp(-448, 448).to(E4M3).view(torch.uint8)
        s["w"] = w
        s["sw"] = (torch.rand(e, nb, kb, device=DEV, generator=g) + 0.5) * (4.5 / 448 / math.sqrt(k))
        s["y"] = torch.zeros((m, n), dtype=torch.bfloat16, device=DEV)
        return s
    t, k, width, local = case["tokens"], case["k"], case["width"], case["local"]
    cap = t * k
    s["ids"] = _slots(case, g)
    s["offs"] = torch.zeros(local + 1, dtype=torch.int32, device=DEV)
    s["pos"] = torch.zeros((t, k), dtype=torch.int32, device=DEV)
    s["src"] = torch.full((cap,), -1, dtype=torch.int32, device=DEV)
    if op == "dispatch":
        s["x"] = _rows(t, width, g)
        # the workspace that a program keeps for the map (int32 words)
        s["ws"] = torch.empty(128 * (local + 1) + 64, dtype=torch.int32, device=DEV)
        s["y"] = torch.zeros((cap, width), dtype=torch.uint8, device=DEV)
        if case["format"] == "fp8":
            s["ys"] = torch.zeros((cap, -(-width // 128)), dtype=torch.float32, device=DEV)
        else:
            s["codes"] = torch.zeros((cap, width // 2), dtype=torch.uint8, device=DEV)
            s["scales"] = torch.zeros((cap, width // 32), dtype=torch.uint8, device=DEV)
            s["ys"] = torch.zeros((cap, width // 128), dtype=torch.uint8, device=DEV)
        return s
    s["offs"], s["pos"], s["src"] = _map(case, s["ids"])
    s["y"] = _rows(cap, width, g)
    w = torch.rand(t, k, device=DEV, generator=g) + 0.1
    s["weights"] = 2.5 * w / w.sum(1, keepdim=True)
    if op == "combine":
        s["base"] = _rows(t, width, g) if case["base"] else None
        s["out"] = torch.empty((t, width), dtype=torch.bfloat16, device=DEV)
    else:
        s["dout"] = _rows(t, width, g)
        s["dy"] = torch.zeros((cap, width), dtype=torch.bfloat16, device=DEV)
        s["dweights"] = torch.zeros((t, k), dtype=torch.float32, device=DEV)
    return s


# ---- plain forms -------------------------------------------------------------------------

def _route(case, logits, bias, mask):
    e, ng, k = case["experts"], case["groups"], case["k"]
    x = logits.float()
    if case["score"] == "softmax":
        x = torch.exp(x - x.amax(1, keepdim=True))
        score = x / x.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-x))
    c = score if bias is None else score + bias
    if ng > 1:
        best = c.view(-1, ng, e // ng).sort(2, descending=True).values[:, :, :case["best"]].sum(2)
        top = best.sort(dim=1, descending=True, stable=True).indices[:, :case["kept"]]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, top, True)
        c = torch.where(keep.repeat_interleave(e // ng, 1), c, -math.inf)
    ids = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    w = 2.5 * w / (w.sum(1, keepdim=True) + 1e-20)
    live = mask.bool()[:, None]
    return torch.where(live, ids, -1).to(torch.int32), torch.where(live, w, 0.0)


def _route_back(case, logits, ids, dw):
    x = logits.float()
    at = ids.long()
    if case["score"] == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-x))
    s = p.gather(1, at)
    d = s.sum(1, keepdim=True) + 1e-20
    ds = 2.5 * (dw - (dw * s).sum(1, keepdim=True) / d) / d
    if case["score"] == "softmax":
        full = torch.zeros_like(p).scatter_(1, at, ds)
        out = p * (full - (ds * s).sum(1, keepdim=True))
    else:
        out = torch.zeros_like(p).scatter_(1, at, ds * s * (1 - s))
    return out.to(logits.dtype)


def _map(case, ids):
    first, local = case["first"], case["local"]
    e = ids.reshape(-1) - first
    here = (e >= 0) & (e < local)
    key = torch.where(here, e, local)
    order = key.sort(stable=True).indices
    count = torch.zeros(local + 1, dtype=torch.int32, device=ids.device).index_add_(
        0, key, torch.ones_like(key))
    offs = torch.cat([count.new_zeros(1), count[:local].cumsum(0, dtype=torch.int32)])
    rows = torch.arange(e.numel(), dtype=torch.int32, device=ids.device)
    pos = torch.empty_like(rows).scatter_(0, order, rows)
    pos = torch.where(here, pos, -1).view(ids.shape)
    src = torch.where(rows < offs[local], order.to(torch.int32), -1)
    return offs, pos, src


def _fp8(x):
    """E4M3 bytes and FP32 scales of 1x128 blocks."""
    k = x.shape[1]
    b = _blocks(x.float())
    amax = b.abs().amax(-1, keepdim=True).clamp_min(TINY)
    q = (b * (448 / amax)).clamp(-448, 448).to(E4M3)
    return q.view(torch.uint8).view(x.shape[0], -1)[:, :k], (amax / 448)[..., 0]


def _fp4_as_fp8(x):
    """MXFP4 of 32-blocks (exponent floor(log2 amax) - 2, nearest even, saturating), then
    E4M3 under the largest of four block exponents."""
    t, k = x.shape
    b = x.float().view(t, k // 128, 4, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - 2 + 127, 0).clamp(0, 254)
    v = torch.ldexp(b, 127 - e)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp_max(6)
    top = e.amax(2, keepdim=True)
    y = torch.ldexp(torch.copysign(a, v), e - top).to(E4M3)
    return y.view(torch.uint8).view(t, k), top.view(t, k // 128).to(torch.uint8)


def _spread(rows, src, k):
    """Token rows into expert order; zero where no slot is."""
    token = src.clamp_min(0).long() // k
    return torch.where((src >= 0)[:, None], rows[token], torch.zeros((), dtype=rows.dtype, device=rows.device))


def _product(s):
    case, offs, most = s["case"], s["offs"].long(), s["most"]
    m, n, k = case["rows"], case["n"], case["width"]
    a = s["a"].view(E4M3).float() * s["sa"].repeat_interleave(128, 1)[:, :k]
    w = s["w"].view(E4M3).float()
    w *= s["sw"].repeat_interleave(128, 2)[:, :, :k].repeat_interleave(128, 1)[:, :n]
    at = offs[:-1, None] + torch.arange(most, device=DEV)
    rows = torch.arange(m, device=DEV)
    expert = (rows[:, None] >= offs[None, 1:]).sum(1)
    y = torch.bmm(a[at.clamp_max(m - 1)], w.transpose(1, 2))
    return y[expert, rows - offs[expert]].to(torch.bfloat16)


def _taken(y, pos):
    return torch.where((pos >= 0)[..., None], y[pos.clamp_min(0).long()].float(), 0.0)


def run(s):
    if own:
        import block_scaled_precision_bf16tofp4row_amd as mx
    case = s["case"]
    op = case["op"]
    if op == "route":
        if own:
            mx.mxfp4_route_topk(s["logits"], s["ids"], s["weights"], bias=s["bias"], row_mask=s["mask"],
                                n_group=case["groups"], topk_group=case["kept"], group_best=case["best"],
                                score=case["score"], renorm=True, scale=2.5)
            return {"ids": s["ids"], "weights": s["weights"]}
        ids, w = _route(case, s["logits"], s["bias"], s["mask"])
        return {"ids": ids, "weights": w}
    if op == "route_back":
        if own:
            mx.mxfp4_route_topk_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"], score=case["score"],
                                         renorm=True, scale=2.5)
            return s["dlogits"]
        return _route_back(case, s["logits"], s["ids"], s["dweights"])
    if op == "dispatch":
        k, fp8 = case["k"], case["format"] == "fp8"
        if own:
            mx.mxfp4_expert_map(s["ids"], s["offs"], s["pos"], s["ws"], src=s["src"], first_expert=case["first"])
            if fp8:
                mx.mxfp4_dispatch_fp8_rows(s["x"], s["pos"], s["y"], s["ys"])
            else:
                mx.mxfp4_dispatch_rows(s["x"], s["pos"], s["codes"], s["scales"])
                mx.mxfp4_to_fp8_rows(s["codes"], s["scales"], s["y"], s["ys"], s["offs"])
            offs, pos, src, y, ys = s["offs"], s["pos"], s["src"], s["y"], s["ys"]
        else:
            offs, pos, src = _map(case, s["ids"])
            y, ys = _fp8(s["x"]) if fp8 else _fp4_as_fp8(s["x"])
            y, ys = _spread(y, src, k), _spread(ys, src, k)
        return {"offs": offs, "pos": pos, "src": src, "y": y.view(E4M3),
                "scales": ys if fp8 else ys.view(torch.float8_e8m0fnu)}
    if op == "product":
        if own:
            mx.mxfp4_fp8_block_gemm(s["a"], s["sa"], s["w"], s["sw"], s["y"], s["offs"])
            return s["y"]
        return _product(s)
    if op == "combine":
        if own:
            mx.mxfp4_combine_rows(s["y"], s["pos"], s["out"], weights=s["weights"], base=s["base"])
            return s["out"]
        out = (_taken(s["y"], s["pos"]) * s["weights"][..., None]).sum(1)
        return (out if s["base"] is None else out + s["base"].float()).to(torch.bfloat16)
    if own:
        mx.mxfp4_combine_rows_backward(s["dout"], s["y"], s["pos"], s["weights"], s["dy"], s["dweights"])
        return {"dy": s["dy"], "dweights": s["dweights"]}
    dout = s["dout"].float()
    dweights = (_taken(s["y"], s["pos"]) * dout[:, None]).sum(2)
    src = s["src"]
    weight = torch.where(src >= 0, s["weights"].reshape(-1)[src.clamp_min(0).long()], 0.0)
    dy = (dout[src.clamp_min(0).long() // case["k"]] * weight[:, None]).to(torch.bfloat16)
    return {"dy": dy, "dweights": dweights}


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("route", "route_back"):
        t, e, k = case["tokens"], case["experts"], case["k"]
        el = 4 if case["f32"] else 2
        if op == "route":
            return {"bytes": t * (e * el + 8 * k + 1) + (4 * e if case["bias"] else 0), "flops": 6 * t * e}
        return {"bytes": t * (2 * e * el + 8 * k), "flops": 8 * t * e}
    if op == "product":
        m, n, k, g = case["rows"], case["n"], case["width"], case["experts"]
        kb, nb = -(-k // 128), -(-n // 128)
        live = min(g, m)
        return {"bytes": m * k + 4 * m * kb + live * (n * k + 4 * nb * kb) + 2 * m * n, "flops": 2 * m * n * k}
    t, k, w = case["tokens"], case["k"], case["width"]
    rows = max(1, t * k * case["local"] // case["experts"])
    if op == "dispatch":
        index = 8 * t * k + 4 * rows + 4 * (case["local"] + 1)
        if case["format"] == "fp8":
            return {"bytes": index + 2 * t * w + rows * (w + 4 * -(-w // 128)), "flops": 4 * t * w}
        return {"bytes": index + 2 * t * w + rows * (2 * (w // 2 + w // 32) + w + w // 128), "flops": 4 * t * w}
    if op == "combine":
        return {"bytes": 2 * rows * w + 8 * t * k + 2 * t * w * (2 if case["base"] else 1), "flops": 2 * rows * w}
    return {"bytes": 4 * rows * w + 12 * t * k + 2 * t * w, "flops": 3 * rows * w}


# ---- the definitions in 64 bits --------------------------------------------------------------

def _exact_blocks(x, size):
    """Each value's block maximum along the row, blocks of `size`, in the row's layout."""
    k = x.shape[1]
    m = torch.cat([x.abs(), x.new_zeros(x.shape[0], -k % size)], 1).unflatten(1, (-1, size)).amax(2)
    return m


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        e, ng, k, t = case["experts"], case["groups"], case["k"], case["tokens"]
        l64 = s["logits"].double()
        score = torch.softmax(l64, 1) if case["score"] == "softmax" else torch.sigmoid(l64)
        c = score if s["bias"] is None else score + s["bias"].double()
        out = torch.zeros((t, e), dtype=torch.bool, device=DEV)
        if ng > 1:
            val = torch.stack([v.topk(case["best"], 1).values.sum(1) for v in c.chunk(ng, 1)], 1)
            for _ in range(case["kept"]):   # argmax takes the first of equal values
                i = val.argmax(1)
                val[torch.arange(t), i] = -math.inf
            out = (val > -math.inf).repeat_interleave(e // ng, 1)
        left = c.masked_fill(out, -math.inf)
        ids = []
        for _ in range(k):
            i = left.argmax(1)
            ids.append(i)
            left[torch.arange(t), i] = -math.inf
        ids = torch.stack(ids, 1)
        w = score.gather(1, ids)
        w = 2.5 * w / (w.sum(1, keepdim=True) + 1e-20)
        dead = s["mask"] == 0
        ids[dead] = -1
        w[dead] = 0
        return {"ids": ids, "weights": w}
    if op == "route_back":
        l64 = s["logits"].double().requires_grad_()
        score = torch.softmax(l64, 1) if case["score"] == "softmax" else torch.sigmoid(l64)
        w = score.gather(1, s["ids"].long())
        w = 2.5 * w / (w.sum(1, keepdim=True) + 1e-20)
        return torch.autograd.grad(w, l64, s["dweights"].double())[0]
    if op == "product":
        k, n = case["width"], case["n"]
        a = s["a"].view(E4M3).double()
        for b in range(s["sa"].shape[1]):
            a[:, 128 * b:128 * b + 128] *= s["sa"][:, b:b + 1].double()
        y = torch.empty((case["rows"], n), dtype=torch.float64, device=DEV)
        at = s["offs"].tolist()
        rn, rk = torch.arange(n, device=DEV) // 128, torch.arange(k, device=DEV) // 128
        for g in range(case["experts"]):
            if at[g] < at[g + 1]:
                w = s["w"][g].view(E4M3).double() * s["sw"][g].double()[rn][:, rk]
                y[at[g]:at[g + 1]] = a[at[g]:at[g + 1]] @ w.t()
        return y
    # the map, slot by slot on the host
    t, k = case["tokens"], case["k"]
    lists = [[] for _ in range(case["local"])]
    for slot, e in enumerate(s["ids"].reshape(-1).tolist()):
        if case["first"] <= e < case["first"] + case["local"]:
            lists[e - case["first"]].append(slot)
    flat = [slot for v in lists for slot in v]
    src = torch.full((t * k,), -1, dtype=torch.int64)
    src[:len(flat)] = torch.tensor(flat, dtype=torch.int64)
    pos = torch.full((t * k,), -1, dtype=torch.int64)
    pos[src[:len(flat)]] = torch.arange(len(flat))
    src, pos = src.to(DEV), pos.view(t, k).to(DEV)
    live = len(flat)
    if op == "dispatch":
        offs = torch.tensor([0] + [len(v) for v in lists]).cumsum(0)
        x = s["x"].double()
        rows = src[:live] // k
        y = torch.zeros((t * k, case["width"]), dtype=torch.float64, device=DEV)
        if case["format"] == "fp8":
            sc = _exact_blocks(x, 128).clamp_min(TINY) / 448
            q = x / sc.repeat_interleave(128, 1)[:, :case["width"]]
            y[:live] = q[rows]
            scales = torch.zeros((t * k, sc.shape[1]), dtype=torch.float64, device=DEV)
            scales[:live] = sc[rows]
        else:
            m = _exact_blocks(x, 32)
            e = torch.where(m > 0, torch.floor(torch.log2(m.clamp_min(1e-300))) - 2, -127.0).clamp_min(-127)
            v = x / torch.exp2(e).repeat_interleave(32, 1)
            grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
            a = v.abs().clamp_max(6)
            hi = torch.searchsorted(grid, a).clamp_max(7)
            lo = (hi - 1).clamp_min(0)
            up, down = grid[hi] - a, a - grid[lo]
            code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
            top = e.unflatten(1, (-1, 4)).amax(2)
            val = torch.sign(v) * grid[code] * torch.exp2(e - top.repeat_interleave(4, 1)).repeat_interleave(32, 1)
            y[:live] = val[rows]
            scales = torch.full((t * k, top.shape[1]), 2.0 ** -127, dtype=torch.float64, device=DEV)
            scales[:live] = torch.exp2(top)[rows]
        return {"offs": offs, "pos": pos, "src": src, "y": y, "scales": scales}
    here = pos >= 0
    w = s["weights"].double()
    if op == "combine":
        out = torch.zeros((t, case["width"]), dtype=torch.float64, device=DEV)
        if s["base"] is not None:
            out += s["base"].double()
        for j in range(k):
            at = here[:, j]
            out[at] += w[at, j:j + 1] * s["y"][pos[at, j]].double()
        return out
    dout = s["dout"].double()
    dy = torch.zeros((t * k, case["width"]), dtype=torch.float64, device=DEV)
    dw = torch.zeros((t, k), dtype=torch.float64, device=DEV)
    for j in range(k):
        at = here[:, j]
        dy[pos[at, j]] = dout[at] * w[at, j:j + 1]
        dw[at, j] = (dout[at] * s["y"][pos[at, j]].double()).sum(1)
    return {"dy": dy, "dweights": dw}
