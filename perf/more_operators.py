"""Cases of the feed-forward operators around the FP8 product with FP32 block scales.

The operators, as an expert or a dense feed-forward layer uses them:

* gated: gate and up projections, activation and product in one call, act(g) u of
  h = [g, u] = A W^T + bias, as BF16 rows (with h kept for the gradient) or as E4M3 rows with
  an FP32 scale per 1x128 block, the operand of the down projection;
* gated gradient: the product of the output's gradient with the transposed down projection
  and the gradient of h from it, in one call, as BF16 or as E4M3 rows with FP32 scales;
* product with an epilogue: act(A W^T + bias) + residual;
* its gradient: of the pre-activation rows and of each expert's bias.

``run`` computes them in plain torch operations where ``own`` is false and through the
framework's entry points where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
TINY = 2.0 ** -100          # floor under a block's amax


def listed():
    return [
        # a running request: one token through a dense (shared) expert of the framework's 671B
        # setting, added to the residual stream; a call's latency
        {"name": "ffn one token", "op": "ffn", "experts": 1, "rows": 1, "inner": 2048, "width": 7168, "act": "silu",
         "bias": False, "residual": True},
        # a decoding batch: a few rows for each of 32 experts, the weights are the traffic
        {"name": "ffn decode", "op": "ffn", "experts": 32, "rows": 128, "inner": 2048, "width": 7168, "act": "silu",
         "bias": False, "residual": False},
        # prompts: the rows of 8 experts, up and down
        {"name": "ffn prompts", "op": "ffn", "experts": 8, "rows": 32768, "inner": 2048, "width": 7168, "act": "silu",
         "bias": False, "residual": False},
        # the forward of a training step: h is kept for the gradient, the output stays BF16
        {"name": "gated training", "op": "gated", "experts": 8, "rows": 16384, "inner": 2048, "width": 7168,
         "act": "silu", "bias": False},
        # odd sizes (an inner width and a width that end inside a scale block), biases
        {"name": "gated odd", "op": "gated", "experts": 3, "rows": 1501, "inner": 680, "width": 1744, "act": "gelu",
         "bias": True},
        # the backward of that step: BF16 gradients of h, and the activations again, for the
        # weights' gradients
        {"name": "gated backward", "op": "gated_back", "experts": 8, "rows": 16384, "inner": 2048, "width": 7168,
         "act": "silu"},
        {"name": "gated backward odd", "op": "gated_back", "experts": 5, "rows": 1203, "inner": 456, "width": 1040,
         "act": "gelu_tanh"},
        # the gradient that only passes through (frozen experts): FP8 all the way to the tokens
        {"name": "ffn backward", "op": "ffn_back", "experts": 8, "rows": 4096, "inner": 2048, "width": 7168,
         "act": "silu"},
        # one token through a dense projection with a bias, added to the residual stream
        {"name": "dense one token", "op": "dense", "experts": 1, "rows": 1, "inner": 7168, "width": 2048, "act": "none",
         "bias": True, "residual": True, "keep": False},
        # a dense layer of a training step on 8192 tokens: the pre-activation is kept
        {"name": "dense training", "op": "dense", "experts": 1, "rows": 8192, "inner": 4096, "width": 7168,
         "act": "gelu", "bias": True, "residual": False, "keep": True},
        # the gradients behind it: of the rows and of 8 experts' biases
        {"name": "dense backward", "op": "dense_back", "experts": 8, "rows": 32768, "inner": 4096, "act": "gelu",
         "fp8": False},
        # few rows, an odd width, FP8 rows for the product that follows
        {"name": "dense backward odd", "op": "dense_back", "experts": 3, "rows": 77, "inner": 1360, "act": "silu",
         "fp8": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "gated", "gated", "gated_back", "gated_back", "ffn_back", "dense", "dense",
                     "dense_back"])
    case = {"op": op, "experts": _log(rng, 1, 32), "rows": _log(rng, 1, 16384), "inner": 8 * _log(rng, 4, 256)}
    case["act"] = rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"])
    if op == "dense_back":
        case["inner"] = 16 * _log(rng, 2, 256)
        case["fp8"] = rng.random() < 0.5
        return case
    case["width"] = 16 * _log(rng, 8, 512)
    if op == "ffn":
        case["inner"] = 16 * _log(rng, 2, 128)
    if op == "ffn_back":
        case["inner"] = 128 * _log(rng, 1, 16)
    if op == "dense":
        case["inner"] = 8 * _log(rng, 16, 512)
        case["act"] = rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu"])
        case["keep"] = case["act"] != "none" and rng.random() < 0.5
    if op in ("ffn", "gated", "dense"):
        case["bias"] = rng.random() < 0.5
    if op in ("ffn", "dense"):
        case["residual"] = rng.random() < 0.5
    return case


# ---- inputs ------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 2654435761 % (1 << 62))


def _rows(t, k, g):
    """BF16 activations: unit scale, a few loud channels, tokens of unequal size."""
    loud = 1 + 15 * (torch.rand(k, device=DEV, generator=g) < 0.004)
    size = torch.exp(0.5 * torch.randn(t, 1, device=DEV, generator=g))
    return (torch.randn(t, k, device=DEV, generator=g) * loud * size).to(torch.bfloat16)


def _counts(case, seed):
    """Rows of each expert: unequal shares that add up to `rows`, some of them zero."""
    r = torch.Generator().manual_seed(int(seed) + 977)
    share = torch.softmax(0.4 * torch.randn(case["experts"], generator=r), 0)
    pick = torch.multinomial(share, case["rows"], replacement=True, generator=r)
    return torch.bincount(pick, minlength=case["experts"]).tolist()


def _weights(e, n, k, g, parts=1):
    """[e, parts n, k] as a checkpoint holds them: every 128x128 block of a part filled to
    E4M3's range, the product of unit rows of about unit size."""
    w = torch.empty((e, parts * n, k), dtype=torch.uint8, device=DEV)
    for i in range(e):
        v = torch.randn(parts * n, k, device=DEV, generator=g)
        w[i] = (v * (448 / 4.5)).clamp(-448, 448).to(E4M3).view(torch.uint8)
    s = torch.rand(e, parts * -(-n // 128), -(-k // 128), device=DEV, generator=g) + 0.5
    return w, s * (4.5 / 448 / math.sqrt(k))


def _operand(m, k, g):
    """E4M3 rows with FP32 scales per 1x128 block."""
    x = _rows(m, k, g).float()
    s = _blocks(x).abs().amax(-1).clamp_min(TINY) / 448
    q = (x / s.repeat_interleave(128, 1)[:, :k]).clamp(-448, 448).to(E4M3).view(torch.uint8)
    return q, s.contiguous()


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device=DEV)


def _fp8_rows(m, k):
    return (torch.zeros((m, k), dtype=torch.uint8, device=DEV), torch.zeros((m, -(-k // 128)), device=DEV))


def _work_buffer():
    """The workspace that a program keeps for the calls of few rows, or of many for the biases."""
    return torch.empty(1 << 25, dtype=torch.uint8, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    op, e, m, n = case["op"], case["experts"], case["rows"], case["inner"]
    counts = _counts(case, seed)
    s = {"case": case, "most": max(counts)}
    s["offs"] = torch.tensor([0] + counts, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)
    s["ws"] = _work_buffer()
    if op == "dense_back":
        s["dout"] = _rows(m, n, g)
        s["pre"] = (1.5 * torch.randn(m, n, device=DEV, generator=g)).to(torch.bfloat16)
        s["dbias"] = torch.zeros((e, n), device=DEV)
        if case["fp8"]:
            s["q"], s["qs"] = _fp8_rows(m, n)
        else:
            s["dpre"] = _bf(m, n)
        return s
    k = case["width"]
    s["a"], s["sa"] = _operand(m, k, g)
    if op in ("gated", "ffn"):
        s["w"], s["sw"] = _weights(e, n, k, g, 2)
        s["bias"] = 0.3 * torch.randn(e, 2 * n, device=DEV, generator=g) if case["bias"] else None
        if op == "gated":
            s["h"], s["out"] = _bf(m, 2 * n), _bf(m, n)
        else:
            s["w2"], s["sw2"] = _weights(e, k, n, g)
            s["bias2"] = 0.3 * torch.randn(e, k, device=DEV, generator=g) if case["bias"] else None
            s["residual"] = _rows(m, k, g) if case["residual"] else None
            s["q"], s["qs"] = _fp8_rows(m, n)
            s["y"] = _bf(m, k)
    elif op == "dense":
        s["w"], s["sw"] = _weights(e, n, k, g)
        s["bias"] = 0.3 * torch.randn(e, n, device=DEV, generator=g) if case["bias"] else None
        s["residual"] = _rows(m, n, g) if case["residual"] else None
        s["pre"] = _bf(m, n) if case["keep"] else None
        s["y"] = _bf(m, n)
    else:
        # a: the gradient's rows, of the down projection's width; w: that projection transposed
        s["w"], s["sw"] = _weights(e, n, k, g)
        s["h"] = (1.5 * torch.randn(m, 2 * n, device=DEV, generator=g)).to(torch.bfloat16)
        if op == "gated_back":
            s["dh"], s["out"] = _bf(m, 2 * n), _bf(m, n)
        else:
            s["w2"], s["sw2"] = _weights(e, k, 2 * n, g)
            s["q"], s["qs"] = _fp8_rows(m, 2 * n)
            s["y"] = _bf(m, k)
    return s


# ---- plain forms -------------------------------------------------------------------------

def _blocks(x):
    """[..., K] -> [..., ceil(K/128), 128], zero past K."""
    x = torch.nn.functional.pad(x, (0, -x.shape[-1] % 128))
    return x.view(*x.shape[:-1], -1, 128)


def _deq(w, s, parts=1):
    """FP32 weights of E4M3 bytes [E, parts N, K] and scales per 128x128 block of a part."""
    e, rows, k = w.shape
    v = w.view(E4M3).float().view(e * parts, rows // parts, k)
    s = s.reshape(e * parts, -1, s.shape[2])
    v *= s.repeat_interleave(128, 2)[:, :, :k].repeat_interleave(128, 1)[:, :rows // parts]
    return v.view(e, rows, k)


def _expert_of(s):
    rows = torch.arange(s["case"]["rows"], device=DEV)
    return (rows[:, None] >= s["offs"].long()[None, 1:]).sum(1)


def _product(s, a, sa, w):
    """FP32 rows of E4M3 rows and their scales times each expert's FP32 weights, padded to the
    expert with the most rows."""
    offs, (m, k) = s["offs"].long(), a.shape
    x = a.view(E4M3).float() * sa.repeat_interleave(128, 1)[:, :k]
    at = offs[:-1, None] + torch.arange(s["most"], device=DEV)
    y = torch.bmm(x[at.clamp_max(m - 1)], w.transpose(1, 2))
    expert = _expert_of(s)
    return y[expert, torch.arange(m, device=DEV) - offs[expert]]


def _fp8(x):
    """E4M3 bytes and FP32 scales of 1x128 blocks of FP32 rows."""
    k = x.shape[1]
    b = _blocks(x)
    amax = b.abs().amax(-1, keepdim=True).clamp_min(TINY)
    q = (b * (448 / amax)).clamp(-448, 448).to(E4M3)
    return q.view(torch.uint8).view(x.shape[0], -1)[:, :k].contiguous(), (amax / 448)[..., 0]


def _act(x, name):
    if name == "silu":
        return x / (1 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x.clamp_min(0) if name == "relu" else x


def _slope(x, name):
    """The activation's derivative."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) * math.sqrt(0.5 / math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x * x * x))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)
    return (x > 0).to(x.dtype) if name == "relu" else torch.ones_like(x)


def _gated(s):
    """FP32 h and act(g) u."""
    h = _product(s, s["a"], s["sa"], _deq(s["w"], s["sw"], 2))
    if s["bias"] is not None:
        h += s["bias"][_expert_of(s)]
    gate, up = h.chunk(2, 1)
    return h, _act(gate, s["case"]["act"]) * up


def _gated_back(s):
    """FP32 gradient of h, and act(g) u."""
    name = s["case"]["act"]
    d = _product(s, s["a"], s["sa"], _deq(s["w"], s["sw"]))
    gate, up = s["h"].float().chunk(2, 1)
    a = _act(gate, name)
    return torch.cat([d * up * _slope(gate, name), d * a], 1), a * up


def _part_scales(s):
    """The gated weights' scales.  Where blocks over the joined features would be as many, the call
    asks for the parts' shape."""
    sw = s["sw"]
    return sw.view(sw.shape[0], 2, -1, sw.shape[2]) if s["case"]["inner"] % 128 > 64 else sw


def run(s):
    if own:
        import block_scaled_precision_bf16tofp4row_amd as mx
    case = s["case"]
    op, bf = case["op"], torch.bfloat16
    if op == "gated":
        if own:
            mx.mxfp4_fp8_gated_gemm(s["a"], s["sa"], s["w"], _part_scales(s), s["offs"], out=s["out"], h=s["h"],
                                    bias=s["bias"], act=case["act"])
            return {"h": s["h"], "out": s["out"]}
        h, out = _gated(s)
        return {"h": h.to(bf), "out": out.to(bf)}
    if op == "ffn":
        if own:
            mx.mxfp4_fp8_gated_gemm(s["a"], s["sa"], s["w"], _part_scales(s), s["offs"], q=s["q"], q_scales=s["qs"],
                                    bias=s["bias"], act=case["act"], workspace=s["ws"])
            mx.mxfp4_fp8_block_gemm_act(s["q"], s["qs"], s["w2"], s["sw2"], s["y"], s["offs"], bias=s["bias2"],
                                        residual=s["residual"])
            return s["y"]
        y = _product(s, *_fp8(_gated(s)[1]), _deq(s["w2"], s["sw2"]))
        if s["bias2"] is not None:
            y += s["bias2"][_expert_of(s)]
        return (y if s["residual"] is None else y + s["residual"].float()).to(bf)
    if op == "gated_back":
        if own:
            mx.mxfp4_fp8_gated_gemm_backward(s["a"], s["sa"], s["w"], s["sw"], s["h"], s["offs"], dh=s["dh"],
                                             out=s["out"], act=case["act"])
            return {"dh": s["dh"], "out": s["out"]}
        dh, out = _gated_back(s)
        return {"dh": dh.to(bf), "out": out.to(bf)}
    if op == "ffn_back":
        if own:
            mx.mxfp4_fp8_gated_gemm_backward(s["a"], s["sa"], s["w"], s["sw"], s["h"], s["offs"], dq=s["q"],
                                             dq_scales=s["qs"], act=case["act"], workspace=s["ws"])
            mx.mxfp4_fp8_block_gemm_act(s["q"], s["qs"], s["w2"], s["sw2"], s["y"], s["offs"])
            return s["y"]
        return _product(s, *_fp8(_gated_back(s)[0]), _deq(s["w2"], s["sw2"])).to(bf)
    if op == "dense":
        if own:
            mx.mxfp4_fp8_block_gemm_act(s["a"], s["sa"], s["w"], s["sw"], s["y"], s["offs"], bias=s["bias"],
                                        residual=s["residual"], pre=s["pre"], act=case["act"])
            return {"y": s["y"], "pre": s["pre"]} if case["keep"] else s["y"]
        pre = _product(s, s["a"], s["sa"], _deq(s["w"], s["sw"]))
        if s["bias"] is not None:
            pre += s["bias"][_expert_of(s)]
        y = _act(pre, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(bf), "pre": pre.to(bf)} if case["keep"] else y.to(bf)
    if own:
        if case["fp8"]:
            mx.mxfp4_act_rows_backward(s["dout"], s["pre"], s["offs"], q=s["q"], q_scales=s["qs"], dbias=s["dbias"],
                                       act=case["act"], workspace=s["ws"])
            return {"q": s["q"].view(E4M3), "scales": s["qs"], "dbias": s["dbias"]}
        mx.mxfp4_act_rows_backward(s["dout"], s["pre"], s["offs"], dpre=s["dpre"], dbias=s["dbias"], act=case["act"],
                                   workspace=s["ws"])
        return {"dpre": s["dpre"], "dbias": s["dbias"]}
    d = s["dout"].float() * _slope(s["pre"].float(), case["act"])
    mine = _expert_of(s)[None] == torch.arange(case["experts"], device=DEV)[:, None]
    dbias = mine.float() @ d
    if case["fp8"]:
        q, scales = _fp8(d)
        return {"q": q.view(E4M3), "scales": scales, "dbias": dbias}
    return {"dpre": d.to(bf), "dbias": dbias}


# ---- what a pass cannot do without ---------------------------------------------------------

def _product_work(m, n, k, e):
    """Bytes of the operands (each live expert's weights once) and operations of a product."""
    kb, nb = -(-k // 128), -(-n // 128)
    return m * k + 4 * m * kb + min(e, m) * (n * k + 4 * nb * kb), 2 * m * n * k


def work(case):
    op, e, m, n = case["op"], case["experts"], case["rows"], case["inner"]
    live = min(e, m)
    if op == "dense_back":
        size = n + 4 * -(-n // 128) if case["fp8"] else 2 * n
        return {"bytes": m * (4 * n + size) + 4 * e * n, "flops": 12 * m * n}
    k = case["width"]
    bias = 4 * live if case.get("bias") else 0
    if op == "dense":
        b, f = _product_work(m, n, k, e)
        rows = 1 + (1 if case["residual"] else 0) + (1 if case["keep"] else 0)
        return {"bytes": b + 2 * m * n * rows + bias * n, "flops": f}
    if op in ("gated", "ffn"):
        b, f = _product_work(m, 2 * n, k, e)
        if op == "gated":
            return {"bytes": b + 6 * m * n + 2 * bias * n, "flops": f}
        mid = m * n + 4 * m * -(-n // 128)              # written here, read by the second product
        b2, f2 = _product_work(m, k, n, e)
        return {"bytes": b + mid + b2 + 2 * m * k * (2 if case["residual"] else 1) + bias * (2 * n + k),
                "flops": f + f2}
    b, f = _product_work(m, n, k, e)
    if op == "gated_back":
        return {"bytes": b + 10 * m * n, "flops": f}
    b2, f2 = _product_work(m, k, 2 * n, e)
    return {"bytes": b + 4 * m * n + 2 * m * n + 8 * m * -(-n // 128) + b2 + 2 * m * k, "flops": f + f2}


# ---- the definitions in 64 bits --------------------------------------------------------------

def _exact_product(s, a, w, sw, parts=1):
    """float64 rows `a` by each expert's weights, expert by expert; features of each of `parts`
    equal parts are scaled by blocks of their own."""
    e, n, k = w.shape
    sw = sw.reshape(e, parts, -1, sw.shape[2]).double()
    at = s["offs"].tolist()
    y = torch.empty((a.shape[0], n), dtype=torch.float64, device=DEV)
    cols = torch.arange(k, device=DEV) // 128
    feats = torch.arange(n // parts, device=DEV) // 128
    for i in range(e):
        if at[i] < at[i + 1]:
            full = torch.cat([sw[i, p][feats][:, cols] for p in range(parts)])
            y[at[i]:at[i + 1]] = a[at[i]:at[i + 1]] @ (w[i].view(E4M3).double() * full).t()
    return y


def _exact_rows(a, sa):
    x = a.view(E4M3).double()
    for b in range(sa.shape[1]):
        x[:, 128 * b:128 * b + 128] *= sa[:, b:b + 1].double()
    return x


def _exact_fp8(x):
    """The values that E4M3 rows with 1x128 scales hold, and x under the scales unrounded."""
    out, raw, scales = torch.empty_like(x), torch.empty_like(x), []
    for c in range(0, x.shape[1], 128):
        v = x[:, c:c + 128]
        sc = v.abs().amax(1, keepdim=True).clamp_min(TINY) / 448
        r = v / sc
        step = torch.exp2(torch.frexp(r.abs().clamp_min(2.0 ** -6)).exponent.double() - 4)
        out[:, c:c + 128] = torch.round(r / step) * step * sc
        raw[:, c:c + 128] = r
        scales.append(sc)
    return out, raw, torch.cat(scales, 1)


def _exact_act(x, name):
    """An activation and its derivative (by automatic differentiation)."""
    f = {"silu": lambda v: v * torch.sigmoid(v), "gelu": lambda v: v * torch.special.ndtr(v),
         "gelu_tanh": lambda v: v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)),
         "relu": torch.relu, "none": lambda v: v * 1}[name]
    x = x.detach().requires_grad_()
    y = f(x)
    return y.detach(), torch.autograd.grad(y.sum(), x)[0]


def _exact_bias(s, y, bias):
    at = s["offs"].tolist()
    for i in range(s["case"]["experts"]):
        if bias is not None:
            y[at[i]:at[i + 1]] += bias[i].double()
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op, n, name = case["op"], case["inner"], case["act"]
    if op == "dense_back":
        d = s["dout"].double() * _exact_act(s["pre"].double(), name)[1]
        at = s["offs"].tolist()
        dbias = torch.stack([d[at[i]:at[i + 1]].sum(0) for i in range(case["experts"])])
        if case["fp8"]:
            _, raw, scales = _exact_fp8(d)
            return {"q": raw, "scales": scales, "dbias": dbias}
        return {"dpre": d, "dbias": dbias}
    a = _exact_rows(s["a"], s["sa"])
    if op in ("gated", "ffn"):
        h = _exact_bias(s, _exact_product(s, a, s["w"], s["sw"], 2), s["bias"])
        out = _exact_act(h[:, :n], name)[0] * h[:, n:]
        if op == "gated":
            return {"h": h, "out": out}
        y = _exact_bias(s, _exact_product(s, _exact_fp8(out)[0], s["w2"], s["sw2"]), s["bias2"])
        return y if s["residual"] is None else y + s["residual"].double()
    y = _exact_product(s, a, s["w"], s["sw"])
    if op == "dense":
        pre = _exact_bias(s, y, s["bias"])
        out = _exact_act(pre, name)[0]
        if s["residual"] is not None:
            out = out + s["residual"].double()
        return {"y": out, "pre": pre} if case["keep"] else out
    act, slope = _exact_act(s["h"][:, :n].double(), name)
    up = s["h"][:, n:].double()
    dh = torch.cat([y * up * slope, y * act], 1)
    if op == "gated_back":
        return {"dh": dh, "out": act * up}
    return _exact_product(s, _exact_fp8(dh)[0], s["w2"], s["sw2"])
