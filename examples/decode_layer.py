"""One attention layer of a served model, built from the library's operators:

    x -> residual addition + RMS norm, MXFP8 output   (rmsnorm_quantize_fp8)
      -> query/key/value projection, W4A8             (gemm_w4a8)
      -> write of the new keys and values             (kv_append)
      -> attention of the new token over the cache    (paged_attention)
      -> MXFP8 of its output, output projection       (quantize_fp8, gemm_w4a8)

A prompt is processed in chunks: each chunk is written to the cache, then the
context is read back (kv_read) for a causal attention in 16-bit torch.  Decode
steps write one token per sequence and attend over the pages.  Weights are
random (there is no checkpoint), positions are not encoded.

    python examples/decode_layer.py [--fmt mxfp4] [--batch 4] [--prompt 200] [--steps 16]
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_microscaling_quantization_mxq_amd as mxq  # noqa: E402


class Pages:
    """Page tables of a batch over one pool: a sequence gets a page when its
    length reaches the next one."""

    def __init__(self, batch, pages, page_size):
        self.size = page_size
        self.free = list(range(pages))
        self.lists = [[] for _ in range(batch)]
        self.lens = [0] * batch

    def grow(self, b, tokens):
        """Slots of the next `tokens` positions of sequence b."""
        slots = []
        for pos in range(self.lens[b], self.lens[b] + tokens):
            if pos % self.size == 0:
                self.lists[b].append(self.free.pop())
            slots.append(self.lists[b][pos // self.size] * self.size + pos % self.size)
        self.lens[b] += tokens
        return slots

    def slots(self, b):
        """Slots of all positions of sequence b."""
        return [self.lists[b][p // self.size] * self.size + p % self.size for p in range(self.lens[b])]

    def tables(self):
        """(table, lens) on the device, no wider than the longest sequence needs."""
        width = max(1, max(len(p) for p in self.lists))
        table = torch.tensor([p + [-1] * (width - len(p)) for p in self.lists], dtype=torch.int32)
        return table.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda()


class Layer:
    def __init__(self, hidden, heads, kv_heads, dim, pages, page_size, fmt, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim

        def weight(n, k):
            return mxq.quantize((torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k)).bfloat16())

        self.norm = torch.ones(hidden, device="cuda", dtype=torch.bfloat16)
        self.wqkv = weight((heads + 2 * kv_heads) * dim, hidden)
        self.wo = weight(hidden, heads * dim)
        self.cache = mxq.kv_cache(pages, page_size, kv_heads, dim, fmt)

    def project(self, x, residual):
        """(q, k, v, residual) of the tokens x [n, hidden]: views of one product's output."""
        a, s, residual = mxq.rmsnorm_quantize_fp8(x, self.norm, residual)
        qkv = mxq.gemm_w4a8(a, s, *self.wqkv)
        h, kv, d = self.heads, self.kv_heads, self.dim
        return (qkv[:, :h * d].unflatten(1, (h, d)), qkv[:, h * d:(h + kv) * d].unflatten(1, (kv, d)),
                qkv[:, (h + kv) * d:].unflatten(1, (kv, d)), residual)

    def output(self, o):
        a, s = mxq.quantize_fp8(o.reshape(o.shape[0], -1))
        return mxq.gemm_w4a8(a, s, *self.wo)

    def prompt_chunk(self, x, residual, pages, b):
        """The tokens x of sequence b's prompt, after the ones it has already: causal
        attention over the cache's contents, read back to 16 bits."""
        q, k, v, residual = self.project(x, residual)
        mxq.kv_append(self.cache, k, v, torch.tensor(pages.grow(b, len(x))).cuda())
        keys, values = mxq.kv_read(self.cache, torch.tensor(pages.slots(b)).cuda())
        group = self.heads // self.kv_heads
        qf = q.float().transpose(0, 1)  # [heads, n, d]
        kf = keys.float().transpose(0, 1).repeat_interleave(group, 0)
        vf = values.float().transpose(0, 1).repeat_interleave(group, 0)
        w = qf @ kf.transpose(1, 2).contiguous() / math.sqrt(self.dim)
        n, total = len(x), kf.shape[1]
        ahead = torch.arange(total, device="cuda")[None] > torch.arange(total - n, total, device="cuda")[:, None]
        o = torch.softmax(w.masked_fill(ahead, -math.inf), -1) @ vf
        return self.output(o.transpose(0, 1).bfloat16().contiguous()), residual

    def step(self, x, residual, slots, table, lens):
        """One new token per sequence, x [batch, hidden]."""
        q, k, v, residual = self.project(x, residual)
        mxq.kv_append(self.cache, k, v, slots)
        return self.output(mxq.paged_attention(q, self.cache, table, lens)), residual


def run(fmt="mxfp8", batch=4, prompt=200, steps=16, chunk=64, hidden=1024, heads=16, kv_heads=4, dim=64, page_size=16,
        seed=0):
    """Prompts of uneven lengths in chunks, then decode steps; (outputs of each
    step, the last step's output recomputed by the prompt path)."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    longest = prompt + steps + 1
    pool = batch * (-(-longest // page_size) + 1)
    pages = Pages(batch, pool, page_size)
    layer = Layer(hidden, heads, kv_heads, dim, pool, page_size, fmt, seed)
    for b in range(batch):
        n = max(1, prompt * (b + 1) // batch)
        x = torch.randn(n, hidden, generator=g, device="cuda").bfloat16()
        for at in range(0, n, chunk):
            layer.prompt_chunk(x[at:at + chunk], None, pages, b)
    outs = []
    for _ in range(steps):
        x = torch.randn(batch, hidden, generator=g, device="cuda").bfloat16()
        before = [list(p) for p in pages.lists], list(pages.lens), list(pages.free)
        slots = torch.tensor([pages.grow(b, 1)[0] for b in range(batch)]).cuda()
        y, _ = layer.step(x, None, slots, *pages.tables())
        outs.append(y)
    # the last token again, as a prompt chunk of one: the same cache, read back
    pages.lists, pages.lens, pages.free = before
    again = torch.cat([layer.prompt_chunk(x[b:b + 1], None, pages, b)[0] for b in range(batch)])
    return outs, again


def main():
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    a.add_argument("--fmt", default="mxfp8", choices=("mxfp8", "mxfp4"))
    a.add_argument("--batch", type=int, default=4)
    a.add_argument("--prompt", type=int, default=200)
    a.add_argument("--steps", type=int, default=16)
    a = a.parse_args()
    t = time.perf_counter()
    outs, again = run(a.fmt, a.batch, a.prompt, a.steps)
    torch.cuda.synchronize()
    d = (outs[-1].float() - again.float()).norm() / again.float().norm()
    print(f"{a.fmt} cache: {a.batch} prompts of up to {a.prompt} tokens, {a.steps} decode steps in "
          f"{time.perf_counter() - t:.2f} s; last step against the prompt path: {d:.2e}")


if __name__ == "__main__":
    main()
