"""Decoding with drafted trees on the quantised cache: each step verifies a tree of drafted tokens per answer in one pass, keeps the
accepted path, and the cache's pages are shared, copied and moved together as answers fork and end.

A step: hqq_kv_tree_plan (masks, rotary positions and slots from the drafts' parents), then in every layer the fused projection,
hqq_kv_write_rope and hqq_kv_attention_tree, then hqq_kv_accept for all layers.  (A model would choose the
accepted path from its logits; here it is the path to the last draft.)  In the end the answers fork in two
(hqq_kv_fork), half of them leave, and hqq_kv_compact moves the others' pages together.
The check decodes the accepted tokens one by one into a second cache: the bytes that both caches stand for have to be
the same, and the attention of each accepted draft the one of its token.

    python examples/draft_layer.py [--answers 8] [--drafts 16] [--steps 6]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import weight_only_quantization_amd as hq  # noqa: E402
from examples.decode_layer import QuantizedLinear  # noqa: E402

PAGE = 64


class Layer:
    def __init__(self, gen, hidden, heads, kv_heads, dim, num_pages, nbits):
        def weight(n, k):
            return (torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5).half()

        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.qkv = QuantizedLinear(weight((heads + 2 * kv_heads) * dim, hidden))
        self.out = QuantizedLinear(weight(hidden, heads * dim))
        self.cache = hq.hqq_kv_cache(num_pages, kv_heads, dim, nbits=nbits, page_size=PAGE)

    def project(self, x):
        y = self.qkv(x).view(x.shape[0], -1, self.dim)
        return y[:, :self.heads], y[:, self.heads:self.heads + self.kv_heads], y[:, self.heads + self.kv_heads:]


def trees(gen, answers, drafts):
    """Parents of the drafts of every answer (the first follows the answer so far), and the path to the last draft."""
    parents = [[-1] + [int(torch.randint(max(0, t - 4), t, (1,), generator=gen)) for t in range(1, drafts)] for _ in range(answers)]
    paths = []
    for p in parents:
        path = [drafts - 1]
        while p[path[-1]] >= 0:
            path.append(p[path[-1]])
        paths.append(path[::-1])
    return parents, paths


def step(layers, caches, x, parents, paths, table, lens, drafts, rope, max_len):
    """One verified draft of every answer.  Returns the new lengths, and per layer what the check needs."""
    i32 = dict(dtype=torch.int32, device="cuda")
    lens = lens + drafts                                     # the drafts are cached behind the answers
    mask, positions, slots = hq.hqq_kv_tree_plan(torch.tensor(parents, **i32).view(-1), table, lens, PAGE)
    seen = []
    for layer in layers:
        q, k, v = layer.project(x)
        turned = hq.hqq_kv_write_rope(layer.cache, q, k, v, positions, slots, rope)
        o = hq.hqq_kv_attention_tree(layer.cache, turned, mask, table, lens, max_len=max_len)
        seen.append((q, k, v, o))
        y = x + layer.out(o.view(x.shape[0], -1))
        x = (y.float() * y.float().square().mean(-1, keepdim=True).rsqrt()).half()  # the model's norm, here without a weight
    most = max(map(len, paths))
    accepted = torch.tensor([p + [-1] * (most - len(p)) for p in paths], **i32)
    lens = hq.hqq_kv_accept(caches, table, lens, accepted, torch.tensor([len(p) for p in paths], **i32), tokens=drafts)
    return lens, seen


def slots_of(table, length):
    at = torch.arange(length, device="cuda")
    return table[at // PAGE].long() * PAGE + at % PAGE


def one_by_one(layers, plain, seen, paths, table, before, drafts, rope):
    """The accepted tokens decoded one at a time into the caches `plain`: the largest relative distance of an accepted draft's attention
    from its token's."""
    worst = 0.0
    for layer, cache, (q, k, v, o) in zip(layers, plain, seen):
        for b, path in enumerate(paths):
            for j, t in enumerate(path):
                at = b * drafts + t
                pos = before[b] + j
                slot = table[b, pos // PAGE].long()[None] * PAGE + pos % PAGE
                turned = hq.hqq_kv_write_rope(cache, q[at:at + 1], k[at:at + 1], v[at:at + 1], torch.tensor([pos], device="cuda"), slot, rope)
                want = hq.hqq_kv_attention(cache, turned, table[b:b + 1], torch.tensor([pos + 1], dtype=torch.int32, device="cuda")).float()
                worst = max(worst, float((o[at].float() - want[0]).norm() / want.norm()))
    return worst


def same(cache, plain, table, other, lens):
    """Whether the tokens of each row of `table` in cache are those of `other` in plain."""
    for row, old, n in zip(table, other, lens):
        if n and not all(torch.equal(a, b) for a, b in zip(hq.hqq_kv_read(cache, slots_of(row, n)), hq.hqq_kv_read(plain, slots_of(old, n)))):
            return False
    return True


def main(answers=8, drafts=16, steps=6, num_layers=2, nbits=4, seed=0):
    hidden, heads, kv_heads, dim = 512, 8, 2, 128
    gen, host = torch.Generator(device="cuda").manual_seed(seed), torch.Generator().manual_seed(seed + 1)
    cols = -(-steps * drafts // PAGE) + 1
    num_pages = answers * cols + 2 * answers
    layers = [Layer(gen, hidden, heads, kv_heads, dim, num_pages, nbits) for _ in range(num_layers)]
    caches = hq.KVLayers([layer.cache for layer in layers])
    plain = [hq.hqq_kv_cache(num_pages, kv_heads, dim, nbits=nbits, page_size=PAGE) for _ in layers]
    rope = hq.hqq_rope_table(dim, scaling="bands", factor=4.0, original_len=2048)
    ids = torch.randperm(num_pages, generator=host).to(torch.int32).cuda()
    table, fresh = ids[:answers * cols].view(answers, cols), ids[answers * cols:]
    lens = torch.zeros(answers, dtype=torch.int32, device="cuda")
    worst = 0.0
    for _ in range(steps):
        before = lens.tolist()
        parents, paths = trees(host, answers, drafts)
        x = torch.randn(answers * drafts, hidden, generator=gen, device="cuda").half()
        lens, seen = step(layers, caches, x, parents, paths, table, lens, drafts, rope, cols * PAGE)
        worst = max(worst, one_by_one(layers, plain, seen, paths, table, before, drafts, rope))
    count = lens.tolist()
    equal = all(same(layer.cache, p, table, table, count) for layer, p in zip(layers, plain))

    # every answer goes on twice; then every other one of them leaves
    twice = torch.arange(answers, dtype=torch.int32, device="cuda").repeat_interleave(2)
    forked, fork_lens = hq.hqq_kv_fork(caches, table, lens, twice, fresh)
    equal = equal and all(same(layer.cache, p, forked, table[twice.long()], fork_lens.tolist()) for layer, p in zip(layers, plain))
    left, left_lens = forked[1::2].contiguous(), fork_lens[1::2].contiguous()
    moved, used = hq.hqq_kv_compact(caches, left, left_lens)
    equal = equal and all(same(layer.cache, p, moved, table, left_lens.tolist()) for layer, p in zip(layers, plain))
    equal = equal and int(used) == sum(-(-n // PAGE) for n in count) and int(moved.max()) < int(used)
    print("%d answers of %d tokens, %d drafts a step: accepted drafts' attention at most %.2e off one by one, caches %s"
          % (answers, sum(count), drafts, worst, "equal" if equal else "DIFFER"))
    return worst, equal


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--answers", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=16)
    ap.add_argument("--steps", type=int, default=6)
    ap.add_argument("--nbits", type=int, default=4, choices=(4, 8))
    a = ap.parse_args()
    main(a.answers, a.drafts, a.steps, nbits=a.nbits)
