"""Steps of a served layer that check drafted tokens, built from the library's operators:

    x -> residual addition + RMS norm, MXFP8 output   (rmsnorm_quantize_fp8)
      -> query/key/value projection, W4A8             (gemm_w4a8)
      -> rotation by position, write to the cache     (rope_append)
      -> attention of each sequence's tree of tokens  (tree_attention)
      -> output projection, W4A8                      (quantize_fp8, gemm_w4a8)
      -> logits, W4A8, and a token drawn at each node (gemm_w4a8, sample)

Each step checks a tree of drafted tokens per sequence: from the root on, the
child that holds the drawn token is accepted, and the accepted tokens' keys and
values are written again, at the positions where the sequence continues.  A
prompt is a chain of tokens over what the cache holds.  Weights, embeddings and
drafts are random (there is no checkpoint): the acceptance is not of interest,
and a narrow vocabulary makes it happen at all.

    python examples/draft_step.py [--fmt mxfp4] [--batch 4] [--prompt 200] [--steps 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from decode_layer import Layer, Pages, mxq  # noqa: E402

TREE = [-1, 0, 0, 1, 1, 2, 2, 3]  # parents: the last token, two guesses, two after each, one more


class DraftLayer(Layer):
    def __init__(self, hidden, heads, kv_heads, dim, pages, page_size, fmt, vocab, seed=0):
        super().__init__(hidden, heads, kv_heads, dim, pages, page_size, fmt, seed)
        g = torch.Generator(device="cuda").manual_seed(seed + 7)
        self.embedding = torch.randn(vocab, hidden, generator=g, device="cuda").bfloat16()
        self.head = mxq.quantize((torch.randn(vocab, hidden, generator=g, device="cuda") / hidden ** 0.5).bfloat16())
        self.freqs = 10000.0 ** (-torch.arange(dim // 2, device="cuda", dtype=torch.float32) / (dim // 2))

    def check(self, tokens, slots, positions, table, context, mask):
        """(outputs [batch * n, hidden], projected q, k, v) of n tokens a sequence."""
        x = self.embedding[tokens]
        q, k, v, _ = self.project(x, None)
        turned = mxq.rope_append(self.cache, q, k, v, slots, positions, self.freqs)
        o = mxq.tree_attention(turned, self.cache, table, context, mask)
        return x + self.output(o), (q, k, v)

    def draw(self, x, u, **settings):
        a, s, _ = mxq.rmsnorm_quantize_fp8(x, self.norm)
        return mxq.sample(mxq.gemm_w4a8(a, s, *self.head), u, **settings)[0]


def run(fmt="mxfp8", batch=4, prompt=200, steps=8, vocab=64, hidden=1024, heads=16, kv_heads=4, dim=64, page_size=16, seed=0):
    """Prompts, then steps; the accepted tokens of each sequence."""
    g = torch.Generator().manual_seed(seed)
    n = len(TREE)
    pages = Pages(batch, batch * (-(-(prompt + n * (steps + 1)) // page_size) + 1), page_size)
    layer = DraftLayer(hidden, heads, kv_heads, dim, len(pages.free), page_size, fmt, vocab, seed)
    depth = [0] * n
    for j, parent in enumerate(TREE[1:], 1):
        depth[j] = depth[parent] + 1
    last, taken = [], [[] for _ in range(batch)]
    for b in range(batch):
        # the prompt but for its last token, which is the first tree's root
        tokens = torch.randint(vocab, (max(1, prompt * (b + 1) // batch),), generator=g)
        last.append(int(tokens[-1]))
        for at in range(0, len(tokens) - 1, 64):
            part = tokens[at:min(at + 64, len(tokens) - 1)]
            slots = torch.tensor(pages.grow(b, len(part))).cuda()
            table, lens = pages.tables()
            layer.check(part.cuda(), slots, torch.arange(at, at + len(part)).cuda(), table[b:b + 1],
                        torch.tensor([at], dtype=torch.int32).cuda(), mxq.tree_mask(list(range(-1, len(part) - 1))))
    mask = mxq.tree_mask([TREE] * batch)
    for _ in range(steps):
        context = list(pages.lens)
        tokens = torch.randint(vocab, (batch, n), generator=g)
        tokens[:, 0] = torch.tensor(last)
        slots = [pages.grow(b, n) for b in range(batch)]
        positions = torch.tensor([[c + d for d in depth] for c in context]).flatten().cuda()
        table, _ = pages.tables()
        x, (q, k, v) = layer.check(tokens.flatten().cuda(), torch.tensor(slots).flatten().cuda(), positions, table,
                                   torch.tensor(context, dtype=torch.int32).cuda(), mask)
        drawn = layer.draw(x, torch.rand(batch * n, generator=g).cuda(), temperature=1.0, top_k=20, top_p=0.95).view(batch, n).tolist()
        rows, to = [], []
        for b in range(batch):
            node, path = 0, [0]
            while True:
                token = drawn[b][node]
                taken[b].append(token)
                child = [j for j in range(n) if TREE[j] == node and int(tokens[b, j]) == token]
                if not child:
                    break
                node = child[0]
                path.append(node)
            last[b] = token
            rows += [b * n + j for j in path]
            to += slots[b][:len(path)]
            pages.lens[b] = context[b] + len(path)
            while len(pages.lists[b]) > -(-pages.lens[b] // page_size):
                pages.free.append(pages.lists[b].pop())
        rows = torch.tensor(rows).cuda()
        mxq.rope_append(layer.cache, q[rows], k[rows], v[rows], torch.tensor(to).cuda(), positions[rows], layer.freqs)
    return taken, pages.lens


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--fmt", default="mxfp8", choices=["mxfp8", "mxfp4"])
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--prompt", type=int, default=200)
    p.add_argument("--steps", type=int, default=8)
    a = p.parse_args()
    taken, lens = run(a.fmt, a.batch, a.prompt, a.steps)
    for t, n in zip(taken, lens):
        print(f"{len(t) / a.steps:.2f} tokens a step, {n} in the cache: {t}")


if __name__ == "__main__":
    main()
