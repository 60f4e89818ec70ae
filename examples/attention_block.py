"""The attention half of a decoder layer over GGUF-packed weights and a paged,
quantised key-value cache: a prompt is taken in one chunk, then tokens one at
a time.

    x --(norm)--(Q4_K product)--> q | k | v --(rotary, packed into pages)-->
      attention --(Q4_K product, added)--> x

The norm is torch; the other steps are calls of the library: matmul, kv_append,
attend, matmul. The decoding step is captured into a CUDA graph once and
replayed per token; page table and lengths live on the device, so the graph does
not change.

    python examples/attention_block.py [--tokens 64] [--cache q8_0]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_weight_gguf_gb300 as q  # noqa: E402
import qmm_synth  # noqa: E402


class AttentionBlock:
    """n_heads query and n_kv key / value heads of head_dim over `width` activations."""

    def __init__(self, width, n_heads, n_kv, head_dim, n_seqs, max_len, cache="q8_0", page=64, seed=0,
                 device="cuda:0"):
        rng = np.random.default_rng(seed)
        self.width, self.n_heads, self.n_kv, self.head_dim = width, n_heads, n_kv, head_dim
        self.n_qkv = (n_heads + 2 * n_kv) * head_dim
        self.w_qkv, self.w_out = (self._weights(k, n, rng, device) for k, n in
                                  ((width, self.n_qkv), (n_heads * head_dim, width)))
        per = -(-max_len // page)
        self.cache = q.KvCache.empty(cache, cache, n_seqs * per, page, n_kv, head_dim, device=device)
        # pages dealt out in an arbitrary order, as after some sequences came and went
        order = rng.permutation(n_seqs * per).astype(np.int32).reshape(n_seqs, per)
        self.page_table = torch.from_numpy(order).to(device)
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device=device)
        self.rope = q.rope_table(max_len, head_dim, device=device)

    @staticmethod
    def _weights(k, n, rng, device):
        # rows scaled so that activations keep their size from one product to the next
        w = qmm_synth.gen_weights("q4_k", k, n, rng).reshape(-1, 144)
        scales = w[:, :4].copy().view(np.float16)
        w[:, :4] = (scales.astype(np.float32) / (3.0 * k ** 0.5)).astype(np.float16).view(np.uint8)
        return torch.from_numpy(w.reshape(-1)).to(device)

    def __call__(self, x, workspace=None):
        """x [n_seqs, n_new, width] with the attention's output added in place; the cache grows by
        n_new positions per sequence."""
        n_seqs, n_new, _ = x.shape
        rows = x.view(-1, self.width)
        normed = rows * torch.rsqrt(rows.square().mean(-1, keepdim=True) + 1e-6)
        qkv = q.matmul("q4_k", self.w_qkv, normed, self.width, self.n_qkv)
        heads = qkv.view(n_seqs, n_new, -1, self.head_dim)
        h, n = self.n_heads, self.n_kv
        self.lens += n_new
        turned = q.kv_append(self.cache, heads[:, :, h:h + n], heads[:, :, h + n:], self.page_table, self.lens,
                             q=heads[:, :, :h], rope=self.rope)
        o = q.attend(self.cache, turned, self.page_table, self.lens, workspace=workspace)
        q.matmul("q4_k", self.w_out, o.view(-1, h * self.head_dim), h * self.head_dim, self.width, y=rows,
                 accumulate=True)
        return x


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=200)
    ap.add_argument("--seqs", type=int, default=2)
    ap.add_argument("--cache", default="q8_0", choices=("f16", "bf16", "q8_0", "q4_0"))
    a = ap.parse_args()
    block = AttentionBlock(4096, 32, 8, 128, a.seqs, a.prompt + a.tokens + 8, a.cache)
    torch.manual_seed(1)
    prompt = torch.randn(a.seqs, a.prompt, 4096, device="cuda:0")
    x = block(prompt)[:, -1:].contiguous()
    block(x)                                     # first calls set up what the library owns
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        block(x)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.tokens):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    q.qmm_device_status()
    held = block.lens.tolist()
    print(f"{a.tokens} tokens of {a.seqs} sequences, {a.cache} cache, lengths {held}: "
          f"{begin.elapsed_time(end) * 1e3 / a.tokens:.1f} us per token, |x| {x.norm().item() / x.numel() ** 0.5:.3f}")


if __name__ == "__main__":
    main()
