"""A mixture-of-experts layer on the library's operators: training step and
int8 serving.

    out[t] = sum_j weights[t, j] * (silu(x[t] W1[e]) W2[e]),   e = ids[t, j]

Run it for the time of each path at a prompt and at a decode step:

    python examples/moe_layer.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from tiled_staged_matmul_gb300 import binding as tsm


class MoELayer:
    """Experts W1 (groups x width x hidden) and W2 (groups x hidden x width),
    f16; ``capacity`` rows are kept for each expert, choices past it dropped."""

    def __init__(self, W1, W2, capacity):
        self.W1, self.W2, self.capacity = W1, W2, capacity
        self.groups = W1.shape[0]

    # ------------------------------------------------------------- training

    def forward(self, x, ids, weights):
        """out, and what ``backward`` needs."""
        slots, counts = tsm.moe_route(ids, self.groups, self.capacity)
        # (The weights' gradients read the rows past an expert's last, too:
        # zeros, which the outputs allocated by these calls start as.)
        rows = tsm.moe_dispatch(x, slots, self.groups, self.capacity)
        h = tsm.grouped_gemm(rows, self.W1, counts, out_dtype=x.dtype)
        a = torch.nn.functional.silu(h)
        y = tsm.grouped_gemm(a, self.W2, counts, out_dtype=x.dtype)
        out = tsm.moe_combine(y, slots, weights)
        return out, (slots, counts, rows, h, a, y, weights)

    def backward(self, dout, saved):
        """Gradients of x, the routing weights, W1 and W2."""
        slots, counts, rows, h, a, y, weights = saved
        dy, dweights = tsm.moe_combine_grad(dout, y, slots, weights)
        da = tsm.grouped_gemm(dy, self.W2.transpose(1, 2).contiguous(), counts)
        s = torch.sigmoid(h.float())
        dh = (da * s * (1 + h.float() * (1 - s))).to(h.dtype)
        drows = tsm.grouped_gemm(dh, self.W1.transpose(1, 2).contiguous(), counts, out_dtype=dout.dtype)
        dx = tsm.moe_dispatch_grad(drows, slots)
        dW2 = tsm.gemm(a.transpose(1, 2).contiguous(), dy)
        dW1 = tsm.gemm(rows.transpose(1, 2).contiguous(), dh)
        return dx, dweights, dW1, dW2

    # -------------------------------------------------------------- serving

    def quantise(self):
        """Both weights as int8 with a scale per expert and column, once."""
        def columns(W):
            q, scales = tsm.quantize_rows(W.transpose(1, 2).contiguous())
            return q.transpose(1, 2).contiguous(), scales
        self.q1, self.s1 = columns(self.W1)
        self.q2, self.s2 = columns(self.W2)

    def serve(self, x, ids, weights):
        """The layer on int8 products: the tokens are quantised before they are
        copied to their experts (a quarter to half of the bytes), the hidden
        rows in between."""
        slots, counts = tsm.moe_route(ids, self.groups, self.capacity)
        q, scales = tsm.quantize_rows(x)
        shape = (self.groups, self.capacity)
        rows = tsm.moe_dispatch(q, slots, *shape, torch.empty((*shape, q.shape[1]), dtype=q.dtype, device=x.device))
        rscales = tsm.moe_dispatch(scales[:, None], slots, *shape,
                                   torch.empty((*shape, 1), device=x.device))[..., 0]
        a = tsm.grouped_gemm_s8(rows, self.q1, rscales, self.s1, counts, activation="silu", out_dtype=x.dtype)
        qa, ascales = tsm.quantize_rows(a, counts)
        y = tsm.grouped_gemm_s8(qa, self.q2, ascales, self.s2, counts, out_dtype=x.dtype)
        return tsm.moe_combine(y, slots, weights)


def main():
    width, hidden, groups, topk = 2048, 1408, 64, 6
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")
    W1 = (rand(groups, width, hidden) * width ** -0.5).half()
    W2 = (rand(groups, hidden, width) * hidden ** -0.5).half()

    def microseconds(f):
        for _ in range(3):
            f()
        times = []
        for _ in range(10):
            e0, e1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            e0.record()
            f()
            e1.record()
            torch.cuda.synchronize()
            times.append(e0.elapsed_time(e1) * 1e3)
        return sorted(times)[len(times) // 2]

    for tokens, capacity in ((4096, 512), (32, 32)):
        layer = MoELayer(W1, W2, capacity)
        layer.quantise()
        x = rand(tokens, width).half()
        weights, ids = torch.softmax(rand(tokens, groups), 1).topk(topk)
        ids = ids.int()
        weights = (weights / weights.sum(1, keepdim=True)).contiguous()
        out, saved = layer.forward(x, ids, weights)
        served = layer.serve(x, ids, weights)
        err = float((served.float() - out.float()).norm() / out.float().norm())
        print(f"{tokens} tokens: forward {microseconds(lambda: layer.forward(x, ids, weights)):.0f} us, "
              f"backward {microseconds(lambda: layer.backward(out, saved)):.0f} us, "
              f"int8 {microseconds(lambda: layer.serve(x, ids, weights)):.0f} us "
              f"({err:.4f} of the f16 result's norm away)")


if __name__ == "__main__":
    main()
