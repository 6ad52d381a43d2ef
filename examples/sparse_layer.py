"""A sparse transformer layer: attention over selected key blocks, then routed experts.

Both halves are products with a matrix that the layer itself chooses in every call
(queries x key blocks, tokens x slots). The script runs one training step on a
prompt, then the last tokens of the same prompt one at a time over a cache, and
compares the two.

    python examples/sparse_layer.py [--tokens 1024] [--device cuda:0]

The projections and the experts' own products are plain torch; the layer has no
normalisation and its gradients stop at its input's projections.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import sparse_dense_matrix_gb300 as sdm  # noqa: E402


class SparseLayer:
    def __init__(self, heads=8, kv_heads=2, dim=64, block=16, n=4, experts=8, k=2, inner=256,
                 device="cuda:0", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.block, self.n, self.experts, self.k = block, n, experts, k
        H = self.hidden = heads * dim

        def weight(*shape):
            w = torch.randn(*shape, generator=g, device=device) * shape[-2] ** -0.5
            return w.to(torch.bfloat16)

        self.w_qkv = weight(H, (heads + 2 * kv_heads) * dim)
        self.w_out, self.w_gate = weight(H, H), weight(H, experts)
        self.w_up, self.w_down = weight(experts, H, inner), weight(experts, inner, H)

    def qkv(self, x):
        B, T, _ = x.shape
        y = (x @ self.w_qkv).view(B, T, -1, self.dim)
        return y.split([self.heads, self.kv_heads, self.kv_heads], dim=2)   # views of one tensor

    def route(self, h):
        """The k best experts of each token, their weights, and the sorted routes."""
        top = torch.topk((h @ self.w_gate).float(), self.k, dim=1)
        weights = torch.softmax(top.values, dim=1)
        return sdm.ExpertRoutes(top.indices.to(torch.int32), self.experts), weights

    def run_experts(self, xs, offsets):
        ys = torch.zeros_like(xs)
        at = offsets.tolist()
        for e in range(self.experts):
            rows = slice(at[e], at[e + 1])
            ys[rows] = torch.relu(xs[rows] @ self.w_up[e]) @ self.w_down[e]
        return ys

    def mlp(self, h):
        routes, weights = self.route(h)
        xs = routes.dispatch(h)
        ys = self.run_experts(xs, routes.offsets)
        return routes.combine(ys, weights), (routes, weights, xs, ys)

    def prompt(self, x):
        """x [B, T, H] -> the layer's output, and what the backward pass and a cache need."""
        B, T, H = x.shape
        q, k, v = self.qkv(x)
        means = sdm.block_means(k, self.block)
        sel = sdm.select_blocks(q, means, self.n, self.block, T)
        out, lse = sel.attend(q, k, v)
        h = x + out.view(B, T, H) @ self.w_out
        y, kept = self.mlp(h.view(B * T, H))
        return h + y.view(B, T, H), (q, k, v, means, sel, out, lse, *kept)

    def prompt_backward(self, grad, saved):
        """Gradients of q, k, v, the experts' inputs' rows, and the router's weights."""
        q, k, v, _, sel, out, lse, routes, weights, xs, ys = saved
        B, T, H = grad.shape
        rows = grad.reshape(B * T, H)
        dys, dweights = routes.combine_backward(rows, ys, weights)
        dxs = torch.zeros_like(xs)
        at = routes.offsets.tolist()
        for e in range(self.experts):
            r = slice(at[e], at[e + 1])
            up = xs[r] @ self.w_up[e]
            dxs[r] = torch.where(up > 0, dys[r] @ self.w_down[e].T, 0) @ self.w_up[e].T
        dh = rows + routes.dispatch_backward(dxs)
        dout = (dh @ self.w_out.T).view(B, T, self.heads, self.dim)
        dq, dk, dv = sel.backward(dout, q, k, v, out, lse)
        return {"dq": dq, "dk": dk, "dv": dv, "dh": dh.view(B, T, H), "dweights": dweights}

    def token(self, x, cache_k, cache_v, means, lengths):
        """One more token of each sequence: x [B, 1, H]. The caches hold lengths[b] keys
        and are written at that position; lengths and means are brought up to date."""
        B = x.shape[0]
        q, k, v = self.qkv(x)
        b, at = torch.arange(B, device=x.device), lengths.long()
        cache_k[b, at], cache_v[b, at] = k[:, 0], v[:, 0]
        lengths += 1
        sdm.block_means(cache_k, self.block, lengths, out=means, new_keys=1)
        sel = sdm.select_blocks(q, means, self.n, self.block, cache_k.shape[1], lengths)
        out, _ = sel.attend(q, cache_k, cache_v)
        h = x + out.view(B, 1, -1) @ self.w_out
        y, _ = self.mlp(h.view(B, -1))
        return h + y.view(B, 1, -1)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--device", default="cuda:0")
    a = ap.parse_args()
    torch.manual_seed(0)
    layer = SparseLayer(device=a.device)
    B, T, H = a.batch, a.tokens, layer.hidden
    x = torch.randn(B, T, H, device=a.device).bfloat16()

    y, saved = layer.prompt(x)
    grads = layer.prompt_backward(torch.randn_like(y), saved)
    print("training step:", {n: round(g.float().norm().item(), 3) for n, g in grads.items()})

    # the last tokens again, one at a time, over a cache of the ones before
    last = min(8, T)
    k, v, means = saved[1].clone(), saved[2].clone(), saved[3]
    k[:, T - last:] = v[:, T - last:] = 0
    lengths = torch.full((B,), T - last, dtype=torch.int32, device=a.device)
    means = sdm.block_means(k, layer.block, lengths)
    worst = 0.0
    for t in range(T - last, T):
        one = layer.token(x[:, t:t + 1], k, v, means, lengths)
        worst = max(worst, (one[:, 0].float() - y[:, t].float()).abs().max().item())
    sdm.dynamic_sync()
    print(f"token by token: largest difference {worst:.3g} in values up to "
          f"{y.float().abs().max().item():.3g}")
    return grads, worst, y


if __name__ == "__main__":
    main()
