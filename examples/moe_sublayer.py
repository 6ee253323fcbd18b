"""A mixture-of-experts sublayer on the library's operators: trained, then run token by token.

    python examples/moe_sublayer.py [--tokens 4096] [--width 1024] [--hidden 512] [--experts 32] [--steps 30]

    out = x + sum over the chosen experts e of  p_e W2_e relu(W1_e norm(x))^2

The forward pass is layer norm, routing, two experts' products and combine; the
backward pass calls each operator's gradient.  The experts' stacks are moved by
their orthogonalized momentum, the rest by plain gradients.  The data is a
fixed random sublayer of the same form, so the loss can fall.  Afterwards one
token at a time goes through the trained sublayer as a captured HIP graph.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import newton_schulz_07_amd as ns  # noqa: E402


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight):
        y, mean, rstd = ns.ns_layer_norm(x, weight)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dweight, _ = ns.ns_layer_norm_backward(dy.contiguous(), x, weight, mean, rstd, bias=False)
        return dx, dweight


class Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k):
        r = ns.ns_route(logits, top_k)
        ctx.save_for_backward(logits, r.ids)
        ctx.mark_non_differentiable(r.offsets, r.rows, r.slots)
        return r.weights, r.offsets, r.rows, r.slots

    @staticmethod
    def backward(ctx, dweights, *_):
        logits, ids = ctx.saved_tensors
        return ns.ns_route_backward(logits, ids, dweights.contiguous()), None


class Gathered(torch.autograd.Function):
    """x[rows[i]] W_e^T: the first product, which reads the tokens where they are."""

    @staticmethod
    def forward(ctx, x, w, offsets, rows, slots):
        ctx.save_for_backward(x, w, offsets, rows, slots)
        return ns.ns_experts_product(x, w, offsets, rows)

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets, rows, slots = ctx.saved_tensors
        dy = dy.contiguous()
        dw = ns.ns_experts_weight_grad(dy, x, offsets, rows)
        return ns.ns_experts_combine(ns.ns_experts_input_grad(dy, w, offsets), slots), dw, None, None, None


class Sorted(torch.autograd.Function):
    """x[i] W_e^T on rows that are sorted already."""

    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return ns.ns_experts_product(x, w, offsets)

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        return ns.ns_experts_input_grad(dy, w, offsets), ns.ns_experts_weight_grad(dy, x, offsets), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, slots):
        ctx.save_for_backward(y, weights, slots)
        return ns.ns_experts_combine(y, slots, weights)

    @staticmethod
    def backward(ctx, dout):
        y, weights, slots = ctx.saved_tensors
        dy, dweights = ns.ns_experts_combine_backward(dout.contiguous(), y, slots, weights)
        return dy, dweights, None


class Sublayer(torch.nn.Module):
    def __init__(self, width, hidden, experts, top_k, dtype=torch.bfloat16, device="cuda", seed=0):
        super().__init__()
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, scale, kind):
            return torch.nn.Parameter((torch.randn(*shape, generator=g) * scale).to(device, kind))

        self.top_k = top_k
        self.gamma = torch.nn.Parameter(torch.ones(width, device=device))
        self.router = normal(width, experts, scale=width ** -0.5, kind=torch.float32)
        self.w1 = normal(experts, hidden, width, scale=width ** -0.5, kind=dtype)
        self.w2 = normal(experts, width, hidden, scale=hidden ** -0.5, kind=dtype)

    def forward(self, x):
        h = Norm.apply(x, self.gamma)
        weights, offsets, rows, slots = Route.apply(h.float() @ self.router, self.top_k)
        z = torch.relu(Gathered.apply(h, self.w1, offsets, rows, slots))
        return x + Combine.apply(Sorted.apply(z * z, self.w2, offsets), weights, slots)


def train(model, target, tokens, steps, lr=0.02, seed=1):
    """The loss of each step."""
    width = model.gamma.numel()
    g = torch.Generator(device=model.gamma.device).manual_seed(seed)
    stacks = [model.w1, model.w2]
    momentum = [torch.zeros_like(w) for w in stacks]
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=g, device=model.gamma.device).to(model.w1.dtype)
        with torch.no_grad():
            want = target(x)
        out = model(x)
        loss = (out.float() - want.float()).square().mean()
        model.zero_grad(set_to_none=True)
        loss.backward()
        with torch.no_grad():
            for w, m in zip(stacks, momentum):
                m.mul_(0.9).add_(w.grad)
            for w, u in zip(stacks, ns.orthogonalize_grouped(momentum)):
                w.sub_(u, alpha=lr)
            for p in (model.gamma, model.router):
                p.sub_(p.grad, alpha=lr)
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


class Decoder:
    """One token at a time through a captured graph."""

    def __init__(self, model):
        self.x = torch.zeros(1, model.gamma.numel(), device=model.gamma.device, dtype=model.w1.dtype)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream), torch.no_grad():
            model(self.x)  # makes the workspaces
            stream.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph, stream=stream):
                self.out = model(self.x)
        torch.cuda.current_stream().wait_stream(stream)

    def __call__(self, x):
        self.x.copy_(x)
        self.graph.replay()
        return self.out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in dict(tokens=4096, width=1024, hidden=512, experts=32, top_k=4, steps=30).items():
        ap.add_argument("--" + name.replace("_", "-"), type=int, default=value)
    a = ap.parse_args(argv)
    model = Sublayer(a.width, a.hidden, a.experts, a.top_k)
    target = Sublayer(a.width, a.hidden, a.experts, a.top_k, seed=7)
    begin = time.perf_counter()
    losses = train(model, target, a.tokens, a.steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps, {time.perf_counter() - begin:.2f} s")

    decode = Decoder(model)
    worst = 0.0
    for i in range(8):
        x = torch.randn(1, a.width, device="cuda").to(model.w1.dtype)
        got = decode(x).clone()
        with torch.no_grad():
            worst = max(worst, (got.float() - model(x).float()).abs().max().item())
    torch.cuda.synchronize()
    begin = time.perf_counter()
    for _ in range(200):
        decode(x)
    torch.cuda.synchronize()
    print(f"token by token: {(time.perf_counter() - begin) / 200 * 1e6:.1f} us each, largest difference from eager {worst}")
    return losses, worst


if __name__ == "__main__":
    main()
