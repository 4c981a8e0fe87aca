"""A mixture-of-experts layer on the library's calls, for prompts and for decoding, and its
gradients.

    python examples/expert_layer.py            # both, on synthetic data, with times

Forward: the router chooses k of E experts per token, the map gives every choice a row in
expert order, the token rows are quantized into those rows (E4M3, an FP32 scale per 1x128
block), two expert products with 128x128-scaled E4M3 weights around a gated SiLU, and the
expert rows come back to their tokens under the router's weights.  The activation itself is
plain torch.  Buffers are sized once for the most tokens of a call, nothing reads a count on
the host, so a layer can be captured into a graph.

Backward: of the layer's output to the routing weights and router logits and to the tokens.
The activation gradients run through the same product on the transposed weights (kept beside
the weights).  Weight gradients are not shown: mxfp4_fp8_grouped_gemm_wgrad computes them from
the column layouts of the MXFP4 path or of BF16 rows in expert order, which the FP8 dispatch
here does not make.
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

    def __init__(self, w_up, w_down, router, bias, k, n_group=1, topk_group=1, scale=1.0):
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
        return b

    def part(self, b, T: int):
        """The part of a plan that T tokens use: every buffer's first rows."""
        if T > b["out"].shape[0]:
            raise ValueError(f"{T} tokens, planned for {b['out'].shape[0]}")
        rows = {"offs": None, "ws": None} | dict.fromkeys(("ids", "w", "pos", "out", "logits"), T)
        return {name: v[:rows.get(name, T * self.k)] for name, v in b.items()}

    def forward(self, x, plan, row_mask=None, shared=None):
        """x [T, H] BF16 -> [T, H]; shared: a shared expert's output, added in."""
        b = self.part(plan, x.shape[0])
        torch.matmul(x.float(), self.router.t(), out=b["logits"])
        mx.mxfp4_route_topk(b["logits"], b["ids"], b["w"], bias=self.bias, row_mask=row_mask, **self.how)
        mx.mxfp4_expert_map(b["ids"], b["offs"], b["pos"], b["ws"])
        mx.mxfp4_dispatch_fp8_rows(x, b["pos"], b["x"], b["xs"])
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
        b = self.part(plan, T)
        dy, da = torch.zeros_like(b["y"]), torch.zeros_like(b["a"])
        dw = torch.empty_like(b["w"])
        mx.mxfp4_combine_rows_backward(dout, b["y"], b["pos"], b["w"], dy, dw)
        dlogits = torch.empty_like(b["logits"])
        mx.mxfp4_route_topk_backward(b["logits"], b["ids"], dw, dlogits, score="sigmoid", scale=self.how["scale"])
        q, s = mx.alloc_fp8_rows_f32_outputs(T * self.k, self.H)
        mx.mxfp4_bf16_to_fp8_rows_f32(dy, q, s, b["offs"])
        mx.mxfp4_fp8_block_gemm(q, s, self.down_t, self.down_ts, da, b["offs"])
        gate, up = b["h"].float().chunk(2, 1)
        sig = torch.sigmoid(gate)
        dh = torch.cat([da.float() * up * sig * (1 + gate * (1 - sig)), da.float() * gate * sig], 1).bfloat16()
        q, s = mx.alloc_fp8_rows_f32_outputs(T * self.k, 2 * self.I)
        mx.mxfp4_bf16_to_fp8_rows_f32(dh, q, s, b["offs"])
        dxr = torch.zeros_like(b["y"])
        mx.mxfp4_fp8_block_gemm(q, s, self.up_t, self.up_ts, dxr, b["offs"])
        dx = torch.empty((T, self.H), dtype=torch.bfloat16, device=dout.device)
        mx.mxfp4_combine_rows(dxr, b["pos"], dx)                 # the dispatch's gradient: the plain sum
        return dx, dlogits


def random_layer(E, H, I, k, n_group=1, topk_group=1, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=device)     # noqa: E731
    return ExpertLayer(r(E, 2 * I, H) / H ** 0.5, r(E, H, I) / I ** 0.5, r(E, H) / H ** 0.5, 0.05 * r(E), k,
                       n_group, topk_group, scale=2.5)


def main():
    layer = random_layer(E=32, H=7168, I=2048, k=8, n_group=8, topk_group=4)
    for T in (8192, 64, 1):
        x = torch.randn(T, layer.H, device="cuda").bfloat16()
        b = layer.plan(T)
        layer.forward(x, b)
        n = 5 if T > 1000 else 50
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            layer.forward(x, b)
        torch.cuda.synchronize()
        print(f"{T} tokens: forward {(time.perf_counter() - t) / n * 1e6:.0f} us")
    x = torch.randn(4096, layer.H, device="cuda").bfloat16()
    b = layer.plan(4096)
    out = layer.forward(x, b)
    dx, dlogits = layer.backward(torch.randn_like(out), b)
    print("backward of 4096 tokens:", tuple(dx.shape), tuple(dlogits.shape))


if __name__ == "__main__":
    main()
