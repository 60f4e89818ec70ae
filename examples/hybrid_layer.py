"""A layer of a hybrid mixture-of-experts decoder over GGUF-packed weights: linear attention, then experts. A prompt
is taken in one call, then tokens one at a time.

    x --(norm)--(Q8_0 product)--> q | k | v | decays --(linear attention)--(Q8_0 product, added)--> x
    x --(norm)--(F16 product)--> logits --(choice of experts)--(experts' network, Q4_K / Q6_K, added)--> x

The norms and the decays' softplus are torch; the other steps are calls of the library: matmul, linear_attend, matmul,
matmul, route_experts, experts_ffn. The decoding step is captured into a CUDA graph once and replayed per token; what
the layer remembers, a matrix per sequence and head, is on the device and does not grow.

    python examples/hybrid_layer.py [--tokens 64] [--prompt 2000]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_weight_gguf_gb300 as q  # noqa: E402
import qmm_synth  # noqa: E402


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class HybridLayer:
    """n_heads value heads and n_qk query / key heads of head_dim, n_experts networks of n_ff units of which every
    position takes top_k, over `width` activations."""

    def __init__(self, width, n_heads, n_qk, head_dim, n_experts, top_k, n_ff, n_seqs, seed=0, device="cuda:0"):
        rng = np.random.default_rng(seed)
        self.width, self.n_heads, self.n_qk, self.head_dim = width, n_heads, n_qk, head_dim
        self.n_experts, self.top_k, self.n_ff = n_experts, top_k, n_ff
        self.n_qkv = (2 * n_qk + n_heads) * head_dim + n_heads

        def weights(fmt, k, n):
            return torch.from_numpy(self._weights(fmt, k, n, rng)).to(device)

        self.w_qkv, self.w_out = weights("q8_0", width, self.n_qkv), weights("q8_0", n_heads * head_dim, width)
        self.w_router = weights("f16", width, n_experts)
        self.w_gate, self.w_up = (weights("q4_k", width, n_ff * n_experts) for _ in range(2))
        self.w_down = weights("q6_k", n_ff, width * n_experts)
        self.decay_bias = torch.linspace(-6.0, 0.0, n_heads, device=device)  # slow heads and fast ones
        self.state = torch.zeros(n_seqs, n_heads, head_dim, head_dim, device=device)

    @staticmethod
    def _weights(fmt, k, n, rng):
        # rows scaled so that activations keep their size from one product to the next
        if fmt == "f16":
            return qmm_synth.gen_weights(fmt, k, n, rng, std=k ** -0.5)
        block, places = {"q8_0": (34, (0,)), "q4_k": (144, (0, 2)), "q6_k": (210, (208,))}[fmt]
        w = qmm_synth.gen_weights(fmt, k, n, rng).reshape(-1, block)
        size = {"q8_0": 10.0, "q4_k": 3.0, "q6_k": 3.0}[fmt]
        for at in places:
            d = np.ascontiguousarray(w[:, at:at + 2]).view(np.float16).astype(np.float32) / (size * k ** 0.5)
            w[:, at:at + 2] = d.astype(np.float16).view(np.uint8)
        return w.reshape(-1)

    def __call__(self, x):
        """x [n_seqs, n_new, width], changed in place; the state goes on by n_new positions per sequence."""
        n_seqs, n_new, _ = x.shape
        rows, h, n, d = x.view(-1, self.width), self.n_heads, self.n_qk, self.head_dim
        made = q.matmul("q8_0", self.w_qkv, norm(rows), self.width, self.n_qkv).view(n_seqs, n_new, -1)
        heads = made[..., :(2 * n + h) * d].unflatten(-1, (-1, d))
        decay = -torch.nn.functional.softplus(made[..., -h:] + self.decay_bias)
        # keys of unit length: what a position adds to the state stays bounded
        keys = torch.nn.functional.normalize(heads[..., n:2 * n, :], dim=-1)
        o = q.linear_attend(heads[..., :n, :], keys, heads[..., 2 * n:, :], decay, self.state)
        q.matmul("q8_0", self.w_out, o.view(-1, h * d), h * d, self.width, y=rows, accumulate=True)

        normed = norm(rows)
        logits = q.matmul("f16", self.w_router, normed, self.width, self.n_experts)
        ids, weights = q.route_experts(logits.view(-1, self.n_experts), self.top_k)
        q.experts_ffn("swiglu", "q4_k", self.w_gate, self.w_up, "q6_k", self.w_down, normed, ids, weights,
                      self.width, self.n_ff, self.n_experts, y=rows, accumulate=True)
        return x


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=2000)
    ap.add_argument("--seqs", type=int, default=1)
    a = ap.parse_args()
    layer = HybridLayer(2048, 16, 16, 128, 64, 8, 768, a.seqs)
    torch.manual_seed(1)
    prompt = torch.randn(a.seqs, a.prompt, 2048, device="cuda:0")
    x = layer(prompt)[:, -1:].contiguous()
    layer(x)                                     # first calls set up what the library owns
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        layer(x)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.tokens):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    q.qmm_device_status()
    print(f"{a.tokens} tokens of {a.seqs} sequences after a prompt of {a.prompt}: "
          f"{begin.elapsed_time(end) * 1e3 / a.tokens:.1f} us per token, |x| {x.norm().item() / x.numel() ** 0.5:.3f}")


if __name__ == "__main__":
    main()
