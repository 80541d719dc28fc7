"""A routed layer with adapters, from the segmented products: training and serving.

    python examples/routed_layer.py [--tokens 2048] [--steps 5]

Training: each token goes to `fan` of the experts, y = sum_f gate_f * (x W_g^T)
over its experts g.  RoutedLinear is the whole differentiable layer: group_rows
plans the batch, gemm_f16_grouped_nt gathers the tokens and runs the experts,
and its backward pass runs gemm_f16_grouped_nn (by the tokens) and
gemm_f16_grouped_tn (by the weights).  Serving: the same batch through one
shared projection with a low-rank adapter per request (gemm_f16_lora_nt),
sixteen requests of one token each, captured into a HIP graph.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_fp16_gemm_f16_amd as g  # noqa: E402


class RoutedLinear(torch.autograd.Function):
    """y[t] = sum_f gates[t, f] * (x[t] @ w[ids[t, f]].T), fp32 [tokens, N].

    x fp16 [tokens, K], w fp16 [experts, N, K], ids int32 [tokens, fan] (an id
    outside the experts drops the token there), gates fp32 [tokens, fan].
    Gradients: x and w in fp32 sums rounded to their own type, gates in fp32.
    """

    @staticmethod
    def forward(ctx, x, w, ids, gates):
        tokens, fan = ids.shape
        order, inverse, offsets = g.group_rows(ids, w.shape[0])
        rows = g.gemm_f16_grouped_nt(x, w, offsets, index=order, fan=fan, out_dtype=torch.float32)
        each = rows[inverse.long()].view(tokens, fan, -1)  # back in the tokens' order
        ctx.save_for_backward(x, w, gates, order, inverse, offsets, each)
        return (each * gates[:, :, None]).sum(1)

    @staticmethod
    def backward(ctx, dy):
        x, w, gates, order, inverse, offsets, each = ctx.saved_tensors
        tokens, fan = gates.shape
        token = torch.div(order, fan, rounding_mode="floor").long()
        # the gradient of each routed row, in the experts' order; fp16 as the products' operand
        d_rows = (dy[token] * gates.reshape(-1)[order.long()][:, None]).to(torch.float16)
        dx = g.gemm_f16_grouped_nn(d_rows, w, offsets, out_dtype=torch.float32)
        dx = dx[inverse.long()].view(tokens, fan, -1).sum(1).to(x.dtype)
        dw = g.gemm_f16_grouped_tn(d_rows, x[token], offsets, out_dtype=torch.float32).to(w.dtype)
        return dx, dw, None, (each * dy[:, None, :]).sum(2)


def train(tokens=2048, width=512, out=768, experts=8, fan=2, steps=5, seed=0):
    """A few steps towards a random target; returns the losses."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, width, generator=gen, device="cuda").half()
    target = torch.randn(tokens, out, generator=gen, device="cuda")
    logits = torch.randn(tokens, experts, generator=gen, device="cuda")
    gates, ids = torch.softmax(logits, 1).topk(fan, 1)
    master = torch.randn(experts, out, width, generator=gen, device="cuda") * width**-0.5
    losses = []
    for _ in range(steps):
        w = master.half().requires_grad_()
        y = RoutedLinear.apply(x, w, ids.to(torch.int32), gates)
        loss = (y - target).square().mean()
        (loss * 1024.0).backward()  # the gradient's rows are fp16: scaled into its range
        master -= 500.0 * w.grad.float() / 1024.0
        losses.append(float(loss.detach()))
    return losses


def serve(requests=16, width=1024, out=1024, adapters=4, rank=16, seed=1):
    """One token of each request through a captured step, twice, the second time with
    other requests; returns (results, the same by plain products in fp32)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).half()

    w = normal(out, width, std=width**-0.5)
    down, up = normal(adapters, rank, width, std=width**-0.5), normal(adapters, out, rank, std=rank**-0.5)
    x = torch.zeros(requests, width, dtype=torch.float16, device="cuda")
    ids = torch.zeros(requests, dtype=torch.int32, device="cuda")

    def step():
        order, _, offsets = g.group_rows(ids, adapters)
        return g.gemm_f16_lora_nt(x, w, down, up, ids, order, offsets)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    results, plain = [], []
    for _ in range(2):
        x.copy_(normal(requests, width, std=1.0))
        ids.copy_(torch.randint(-1, adapters, (requests,), generator=gen, device="cuda"))
        graph.replay()
        results.append(y.clone())
        want = x.float() @ w.float().t()
        for s in range(adapters):
            mine = ids == s
            want[mine] += x[mine].float() @ down[s].float().t() @ up[s].float().t()
        plain.append(want)
    return results, plain


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args()
    losses = train(tokens=a.tokens, steps=a.steps)
    print("training loss:", " ".join(f"{v:.4f}" for v in losses))
    for got, want in zip(*serve()):
        print(f"serving: largest difference from fp32 {float((got.float() - want).abs().max()):.5f}")


if __name__ == "__main__":
    main()
