"""One attention layer served as the library is used: 4-bit weights, a quantised key/value cache, and a
batch of answers to one prompt.

The prompt is read once (its tokens' keys and values go to shared pages), then every answer decodes token by
token: fused projections (hqq_gemv_w4a16), hqq_kv_write, hqq_kv_attention_shared, output projection.
The check at the end reads the cache back (hqq_kv_read) and repeats the last step's attention densely in
fp32.

    python examples/decode_layer.py [--prompt 700] [--answers 16] [--steps 40]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import weight_only_quantization_amd as hq  # noqa: E402


class QuantizedLinear:
    """W [N, K] in 4 bits, groups of 64; y = x @ W^T."""

    def __init__(self, w):
        self.n, self.k = w.shape
        self.q = hq.hqq_quantize(w, nbits=4, group_size=64)

    def __call__(self, x):
        return hq.hqq_gemv_w4a16(self.q.packed, self.q.delta, self.q.zero, self.n, self.k, 64, x)


class Layer:
    """Attention layer over pages of its own; `pages` hands out page ids in order."""

    def __init__(self, hidden=1024, heads=8, kv_heads=2, dim=128, nbits=4, num_pages=256, page_size=64, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5).half()

        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.qkv = QuantizedLinear(weight((heads + 2 * kv_heads) * dim, hidden))
        self.out = QuantizedLinear(weight(hidden, heads * dim))
        self.cache = hq.hqq_kv_cache(num_pages, kv_heads, dim, nbits=nbits, page_size=page_size)
        self.free = 0

    def pages(self, tokens):
        n = -(-tokens // self.cache.page_size)
        ids = torch.arange(self.free, self.free + n, dtype=torch.int32, device="cuda")
        self.free += n
        if self.free > self.cache.num_pages:
            raise ValueError("the cache has %d pages, %d are needed" % (self.cache.num_pages, self.free))
        return ids

    def project(self, x):
        """Queries, keys and values: slices of the fused projection, used where they lie."""
        y = self.qkv(x).view(x.shape[0], -1, self.dim)
        return y[:, :self.heads], y[:, self.heads:self.heads + self.kv_heads], y[:, self.heads + self.kv_heads:]

    def slots(self, table, positions):
        """Slot of position positions[i] on the pages table[i] (or the one list table)."""
        page, size = positions // self.cache.page_size, self.cache.page_size
        ids = table[page] if table.dim() == 1 else table.gather(1, page[:, None])[:, 0]
        return ids.long() * size + positions % size

    def read_prompt(self, x):
        """The prompt's tokens into pages of their own; returns the pages and the layer's output."""
        n = x.shape[0]
        pages = self.pages(n)
        q, k, v = self.project(x)
        hq.hqq_kv_write(self.cache, k, v, self.slots(pages, torch.arange(n, device="cuda")))
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        o = hq.hqq_kv_attention(self.cache, q, pages[None], lens, max_len=n)
        return pages, self.out(o.view(n, -1))

    def step(self, x, prompt_pages, prompt_len, table, lens, max_len):
        """One token of every answer; lens: cached tokens of each answer before this one."""
        q, k, v = self.project(x)
        hq.hqq_kv_write(self.cache, k, v, self.slots(table, lens.long()))
        lens += 1
        o = hq.hqq_kv_attention_shared(self.cache, q, prompt_pages, prompt_len, table, lens, max_len=max_len)
        return q, o, self.out(o.view(x.shape[0], -1))


def dense_attention(layer, q, prompt_pages, prompt_len, table, lens):
    """The step's attention in fp32 on the cache read back."""
    out = torch.empty(q.shape, device="cuda")
    for b, n in enumerate(lens.tolist()):
        at = torch.cat((layer.slots(prompt_pages, torch.arange(prompt_len, device="cuda")),
                        layer.slots(table[b], torch.arange(n, device="cuda"))))
        k, v = (x.float().repeat_interleave(layer.heads // layer.kv_heads, 1) for x in hq.hqq_kv_read(layer.cache, at))
        p = torch.softmax((q[b].float()[:, None] * k.transpose(0, 1)).sum(-1) * layer.dim ** -0.5, -1)
        out[b] = (p[..., None] * v.transpose(0, 1)).sum(1)
    return out


def main(prompt=700, answers=16, steps=40, nbits=4, seed=0):
    hidden = 1024
    layer = Layer(hidden=hidden, nbits=nbits, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(prompt, hidden, generator=gen, device="cuda").half()
    prompt_pages, _ = layer.read_prompt(x)
    table = layer.pages(answers * -(-steps // layer.cache.page_size) * layer.cache.page_size).view(answers, -1)
    lens = torch.zeros(answers, dtype=torch.int32, device="cuda")
    x = torch.randn(answers, hidden, generator=gen, device="cuda").half()
    for i in range(steps):
        q, o, y = layer.step(x, prompt_pages, prompt, table, lens, max_len=i + 1)
        x = (x + y).float()
        x = (x * x.square().mean(-1, keepdim=True).rsqrt()).half()  # the model's norm, here without a weight
    want = dense_attention(layer, q, prompt_pages, prompt, table, lens)
    err = float((o.float() - want).norm() / want.norm())
    print("%d answers of %d tokens to a prompt of %d: last step's attention is %.2e off the dense one" % (answers, steps, prompt, err))
    return err


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--answers", type=int, default=16)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--nbits", type=int, default=4, choices=(4, 8))
    a = ap.parse_args()
    main(a.prompt, a.answers, a.steps, a.nbits)
