"""A mixture-of-experts layer on the library's calls, for prompts and for decoding, and its
gradients.

    python examples/expert_layer.py            # both, on synthetic data, with times

Forward: the router chooses k of E experts per token, the map gives every choice a row in
expert order, the token rows are quantized into those rows (E4M3, an FP32 scale per 1x128
block), two expert products with 128x128-scaled E4M3 weights around a gated SiLU, and the
expert rows come back to their tokens under the router's weights.  Buffers are sized once for
the most tokens of a call, nothing reads a count on the host, so a layer can be captured into
a graph.  With fused=True the first product, the activation and the quantization are one call,
and so are the down projection's transposed product and the activation's gradient on the way
back; without it the activation is plain torch between two products, from the BF16 rows.

Backward: of the layer's output to the routing weights and router logits and to the tokens.
The activation gradients run through the same product on the transposed weights (kept beside
the weights).  A fused layer also gives the weights' gradients: the BF16 rows that its calls
leave behind, and the tokens gathered in expert order, go through the column quantizer into
mxfp4_fp8_grouped_gemm_wgrad (features and widths that are multiples of 256).

FeedForward is the same block for every token (a dense layer, or the expert that all tokens
share), with biases and the residual added in the second product.
"""
from __future__ import annotations

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_bf16tofp4row_amd as mx  # noqa: E402


def quantize_weights(w: torch.Tensor):
    """[G, N, K] -> E4M3 bytes and an FP32 scale per 128x128 block."""
    G, N, K = w.shape
    nb, kb = (N + 127) // 128, (K + 127) // 128
    full = torch.zeros((G, nb * 128, kb * 128), dtype=torch.float32, device=w.device)
    full[:, :N, :K] = w
    blocks = full.view(G, nb, 128, kb, 128)
    scale = blocks.abs().amax((2, 4)).clamp_min(2.0 ** -100) / 448
    q = (blocks / scale[:, :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(G, nb * 128, kb * 128)[:, :N, :K].contiguous(), scale.contiguous()


class ExpertLayer:
    """w_up [E, 2 I, H] (gate and up features), w_down [E, H, I], router [E, H], bias [E]."""

    def __init__(self, w_up, w_down, router, bias, k, n_group=1, topk_group=1, scale=1.0, fused=False):
        self.fused = fused
        if fused and w_down.shape[2] % 128:
            raise ValueError("the fused gradients take inner widths that are multiples of 128")
        self.up, self.up_s = quantize_weights(w_up)
        self.down, self.down_s = quantize_weights(w_down)
        # for the gradients: 128x128 blocks are the same blocks transposed
        self.up_t, self.up_ts = self.up.transpose(1, 2).contiguous(), self.up_s.transpose(1, 2).contiguous()
        self.down_t, self.down_ts = self.down.transpose(1, 2).contiguous(), self.down_s.transpose(1, 2).contiguous()
        self.router, self.bias = router, bias
        self.E, self.H, self.I, self.k = w_up.shape[0], w_up.shape[2], w_down.shape[2], k
        self.how = dict(n_group=n_group, topk_group=topk_group, group_best=min(2, self.E // n_group), score="sigmoid",
                        scale=scale)

    def plan(self, T: int, device="cuda"):
        """The buffers of calls on up to T tokens."""
        rows = T * self.k
        bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=device)      # noqa: E731
        b = {}
        b["ids"], b["w"] = mx.alloc_route_outputs(T, self.k, device)
        b["offs"], b["pos"], b["ws"] = mx.alloc_expert_map_outputs(T, self.k, self.E, device)
        b["x"], b["xs"] = mx.alloc_fp8_rows_f32_outputs(rows, self.H, device)
        b["h"], b["a"], b["y"] = bf(rows, 2 * self.I), bf(rows, self.I), bf(rows, self.H)
        b["aq"], b["as"] = mx.alloc_fp8_rows_f32_outputs(rows, self.I, device)
        b["out"] = bf(T, self.H)
        b["logits"] = torch.empty((T, self.E), device=device)
        # rows that no token has keep what the buffers hold: make that finite once
        b["h"].zero_()
        if self.fused:
            sizes = self.E, rows, self.I, self.H
            b["fws"] = torch.empty(max(mx.mxfp4_fp8_gated_gemm_workspace(*sizes),
                                       mx.mxfp4_fp8_gated_gemm_backward_workspace(*sizes)), dtype=torch.uint8, device=device)
            b["dh"], b["dy"] = bf(rows, 2 * self.I).zero_(), bf(rows, self.H).zero_()
            b["a"].zero_()
        return b

    def part(self, b, T: int):
        """The part of a plan that T tokens use: every buffer's first rows."""
        if T > b["out"].shape[0]:
            raise ValueError(f"{T} tokens, planned for {b['out'].shape[0]}")
        rows = {"offs": None, "ws": None, "fws": None} | dict.fromkeys(("ids", "w", "pos", "out", "logits"), T)
        return {name: v[:rows.get(name, T * self.k)] for name, v in b.items() if isinstance(v, torch.Tensor)}

    def forward(self, x, plan, row_mask=None, shared=None, keep=True):
        """x [T, H] BF16 -> [T, H]; shared: a shared expert's output, added in.  keep: for the
        gradients (without it a fused layer writes no BF16 rows between its products)."""
        b = self.part(plan, x.shape[0])
        # the tokens whose rows the plan holds for backward, and for weight_gradients
        plan["kept"], plan["graded"] = x.shape[0] if keep or not self.fused else None, None
        torch.matmul(x.float(), self.router.t(), out=b["logits"])
        mx.mxfp4_route_topk(b["logits"], b["ids"], b["w"], bias=self.bias, row_mask=row_mask, **self.how)
        mx.mxfp4_expert_map(b["ids"], b["offs"], b["pos"], b["ws"])
        mx.mxfp4_dispatch_fp8_rows(x, b["pos"], b["x"], b["xs"])
        if self.fused:
            mx.mxfp4_fp8_gated_gemm(b["x"], b["xs"], self.up, self.up_s, b["offs"], q=b["aq"], q_scales=b["as"],
                                    h=b["h"] if keep else None, workspace=b["fws"])
        else:
            mx.mxfp4_fp8_block_gemm(b["x"], b["xs"], self.up, self.up_s, b["h"], b["offs"])
            gate, up = b["h"].chunk(2, 1)
            torch.mul(torch.nn.functional.silu(gate), up, out=b["a"])
            mx.mxfp4_bf16_to_fp8_rows_f32(b["a"], b["aq"], b["as"], b["offs"])
        mx.mxfp4_fp8_block_gemm(b["aq"], b["as"], self.down, self.down_s, b["y"], b["offs"])
        mx.mxfp4_combine_rows(b["y"], b["pos"], b["out"], weights=b["w"], base=shared)
        return b["out"]

    def backward(self, dout, plan):
        """After forward: the gradients of the tokens (through the experts) and of the logits."""
        T = dout.shape[0]
        if plan.get("kept") != T:
            raise ValueError(f"the plan keeps no rows of a forward call on {T} tokens")
        plan["graded"] = T if self.fused else None
        b = self.part(plan, T)
        dy = b["dy"] if self.fused else torch.zeros_like(b["y"])
        dw = torch.empty_like(b["w"])
        mx.mxfp4_combine_rows_backward(dout, b["y"], b["pos"], b["w"], dy, dw)
        dlogits = torch.empty_like(b["logits"])
        mx.mxfp4_route_topk_backward(b["logits"], b["ids"], dw, dlogits, score="sigmoid", scale=self.how["scale"])
        qy, sy = mx.alloc_fp8_rows_f32_outputs(T * self.k, self.H)
        mx.mxfp4_bf16_to_fp8_rows_f32(dy, qy, sy, b["offs"])
        q, s = mx.alloc_fp8_rows_f32_outputs(T * self.k, 2 * self.I)
        if self.fused:
            mx.mxfp4_fp8_gated_gemm_backward(qy, sy, self.down_t, self.down_ts, b["h"], b["offs"], dh=b["dh"], dq=q,
                                             dq_scales=s, out=b["a"], workspace=b["fws"])
        else:
            da = torch.zeros_like(b["a"])
            mx.mxfp4_fp8_block_gemm(qy, sy, self.down_t, self.down_ts, da, b["offs"])
            gate, up = b["h"].float().chunk(2, 1)
            sig = torch.sigmoid(gate)
            dh = torch.cat([da.float() * up * sig * (1 + gate * (1 - sig)), da.float() * gate * sig], 1).bfloat16()
            mx.mxfp4_bf16_to_fp8_rows_f32(dh, q, s, b["offs"])
        dxr = torch.zeros_like(b["y"])
        mx.mxfp4_fp8_block_gemm(q, s, self.up_t, self.up_ts, dxr, b["offs"])
        dx = torch.empty((T, self.H), dtype=torch.bfloat16, device=dout.device)
        mx.mxfp4_combine_rows(dxr, b["pos"], dx)                 # the dispatch's gradient: the plain sum
        return dx, dlogits


    def weight_gradients(self, x, plan):
        """After backward of a fused layer: the gradients of w_up and w_down."""
        if plan.get("graded") != x.shape[0]:
            raise ValueError(f"the plan keeps no rows of a fused layer's backward call on {x.shape[0]} tokens")
        b = self.part(plan, x.shape[0])
        rows, E = b["y"].shape[0], self.E
        xr = torch.zeros_like(b["y"])             # the tokens in expert order
        here = b["pos"] >= 0
        xr[b["pos"][here].long()] = x[here.nonzero()[:, 0]]
        grads = []
        for left, right in ((b["dh"], xr), (b["dy"], b["a"])):
            N, K = left.shape[1], right.shape[1]
            lt, ls = mx.alloc_cols_outputs(rows, N, E)
            rt, rs = mx.alloc_cols_outputs(rows, K, E)
            mx.mxfp4_bf16_to_fp8_cols_ragged(left, lt, ls, b["offs"])
            mx.mxfp4_bf16_to_fp8_cols_ragged(right, rt, rs, b["offs"])
            dw = torch.empty((E, N, K), dtype=torch.bfloat16, device=x.device)
            mx.mxfp4_fp8_grouped_gemm_wgrad(lt, ls, rt, rs, dw, b["offs"], M_cap=rows, N=N, K=K)
            grads.append(dw)
        return grads


class FeedForward:
    """The gated block for every token, y = W_down (silu(g) u) + b_down + residual with
    [g, u] = W_up x + b_up: w_up [2 I, H], w_down [H, I], b_up [2 I], b_down [H] (FP32)."""

    def __init__(self, w_up, w_down, b_up, b_down):
        self.up, self.up_s = quantize_weights(w_up[None])
        self.down, self.down_s = quantize_weights(w_down[None])
        self.up_t, self.up_ts = self.up.transpose(1, 2).contiguous(), self.up_s.transpose(1, 2).contiguous()
        self.down_t, self.down_ts = self.down.transpose(1, 2).contiguous(), self.down_s.transpose(1, 2).contiguous()
        self.b_up, self.b_down = b_up, b_down
        self.H, self.I = w_down.shape
        if self.I % 128:
            raise ValueError("inner widths are multiples of 128")

    def plan(self, T: int, device="cuda"):
        """The buffers of calls on T tokens, no more and no fewer (the offsets say T)."""
        bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=device)      # noqa: E731
        b = {"offs": torch.tensor([0, T], dtype=torch.int32, device=device)}
        b["h"], b["dh"], b["y"], b["dx"] = bf(T, 2 * self.I), bf(T, 2 * self.I), bf(T, self.H), bf(T, self.H)
        for name, width in (("x", self.H), ("a", self.I), ("dy", self.H), ("dh8", 2 * self.I)):
            b[name], b[name + "_s"] = mx.alloc_fp8_rows_f32_outputs(T, width, device)
        b["ws"] = torch.empty(max(mx.mxfp4_fp8_gated_gemm_workspace(1, T, self.I, self.H),
                                  mx.mxfp4_fp8_gated_gemm_backward_workspace(1, T, self.I, self.H),
                                  mx.mxfp4_act_rows_backward_workspace(1, T, max(2 * self.I, self.H))),
                              dtype=torch.uint8, device=device)
        return b

    def planned(self, b, rows):
        """The plan b, if the rows are those it is for: the calls go by its offsets."""
        if rows.shape != b["y"].shape:
            raise ValueError(f"rows {tuple(rows.shape)}, planned for {tuple(b['y'].shape)}")
        return b

    def forward(self, x, plan, residual=None):
        """x [T, H] BF16 -> [T, H]."""
        b = self.planned(plan, x)
        b["kept"] = True
        mx.mxfp4_bf16_to_fp8_rows_f32(x, b["x"], b["x_s"], b["offs"])
        mx.mxfp4_fp8_gated_gemm(b["x"], b["x_s"], self.up, self.up_s, b["offs"], q=b["a"], q_scales=b["a_s"], h=b["h"],
                                bias=self.b_up, workspace=b["ws"])
        mx.mxfp4_fp8_block_gemm_act(b["a"], b["a_s"], self.down, self.down_s, b["y"], b["offs"], bias=self.b_down,
                                    residual=residual)
        return b["y"]

    def backward(self, dout, plan):
        """After forward: the gradients of x (the residual's is dout), of b_up and of b_down."""
        b = self.planned(plan, dout)
        if "kept" not in b:
            raise ValueError("the plan keeps no rows of a forward call")
        db_up, db_down = torch.empty_like(self.b_up)[None], torch.empty_like(self.b_down)[None]
        mx.mxfp4_act_rows_backward(dout, None, b["offs"], q=b["dy"], q_scales=b["dy_s"], dbias=db_down, workspace=b["ws"])
        mx.mxfp4_fp8_gated_gemm_backward(b["dy"], b["dy_s"], self.down_t, self.down_ts, b["h"], b["offs"], dh=b["dh"],
                                         dq=b["dh8"], dq_scales=b["dh8_s"], workspace=b["ws"])
        mx.mxfp4_act_rows_backward(b["dh"], None, b["offs"], dbias=db_up, workspace=b["ws"])
        mx.mxfp4_fp8_block_gemm_act(b["dh8"], b["dh8_s"], self.up_t, self.up_ts, b["dx"], b["offs"])
        return b["dx"], db_up[0], db_down[0]


def random_layer(E, H, I, k, n_group=1, topk_group=1, seed=0, device="cuda", fused=False):
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=device)     # noqa: E731
    return ExpertLayer(r(E, 2 * I, H) / H ** 0.5, r(E, H, I) / I ** 0.5, r(E, H) / H ** 0.5, 0.05 * r(E), k,
                       n_group, topk_group, scale=2.5, fused=fused)


def main():
    for fused in (False, True):
        layer = random_layer(E=32, H=7168, I=2048, k=8, n_group=8, topk_group=4, fused=fused)
        for T in (8192, 64, 1):
            x = torch.randn(T, layer.H, device="cuda").bfloat16()
            b = layer.plan(T)
            layer.forward(x, b, keep=False)
            n = 5 if T > 1000 else 50
            torch.cuda.synchronize()
            t = time.perf_counter()
            for _ in range(n):
                layer.forward(x, b, keep=False)
            torch.cuda.synchronize()
            print(f"{T} tokens{', fused' if fused else ''}: forward {(time.perf_counter() - t) / n * 1e6:.0f} us")
        x = torch.randn(4096, layer.H, device="cuda").bfloat16()
        b = layer.plan(4096)
        dout = torch.randn_like(layer.forward(x, b))
        layer.backward(dout, b)
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(5):
            dx, dlogits = layer.backward(dout, b)
        torch.cuda.synchronize()
        print(f"backward of 4096 tokens{', fused' if fused else ''}: {(time.perf_counter() - t) / 5 * 1e6:.0f} us",
              tuple(dx.shape), tuple(dlogits.shape))
    dw_up, dw_down = layer.weight_gradients(x, b)
    print("weight gradients:", tuple(dw_up.shape), tuple(dw_down.shape))


if __name__ == "__main__":
    main()
