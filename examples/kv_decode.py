"""One attention block of a decoder served from the NVFP4 key/value cache, end to end on one GPU:

  W4A16 QKV product -> pages taken -> rotary positions and quantized append -> attention over the pages
  -> W4A16 output product

for a prefill of ragged prompts, a fork into samples, decode steps, the end of some sequences and a
compaction of the pool. Weights are random; the sizes default to the 27B-class layers of the GEMM
workloads (5120 = 40 * 128 wide, 4 KV heads).

  python examples/kv_decode.py [--prompts 4] [--tokens 512] [--samples 2] [--steps 32]
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_block_scaled_amd as nv  # noqa: E402


class Linear:
    """y = x W^T with W held in NVFP4 under its global scale."""

    def __init__(self, n, k, gen):
        w = (torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k)).to(torch.bfloat16)
        codes, scales, _, self.inv_g = nv.nvfp4_quantize(w)
        self.w, _ = nv.nvfp4_prepare_weight(codes, scales, "ue4m3")
        self.n, self.k = n, k

    def __call__(self, x):
        return nv.nvfp4_gemm_w4a16(x, self.w, self.n, self.k, alpha_dev=self.inv_g)


class Block:
    """QKV, cached attention and output product of one layer, with its pool of pages."""

    def __init__(self, hidden=5120, q_heads=40, kv_heads=4, head_dim=128, page=64, pool=256, batch=16, width=64,
                 max_pos=8192, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.page = q_heads, kv_heads, head_dim, page
        self.qkv = Linear((q_heads + 2 * kv_heads) * head_dim, hidden, gen)
        self.out = Linear(hidden, q_heads * head_dim, gen)
        self.pages = torch.zeros((pool, nv.nvfp4_kv_page_bytes(page, kv_heads, head_dim)), dtype=torch.uint8, device="cuda")
        # keys and values of normalised activations lie within a few times their deviation
        g = torch.full((kv_heads,), 2688.0 / 8.0, device="cuda")
        self.cache = nv.KVCache(self.pages, page, kv_heads, head_dim, g, g.clone())
        half = head_dim // 2
        angle = torch.arange(max_pos, device="cuda")[:, None] * 1e6 ** (-torch.arange(half, device="cuda") / half)
        self.cos, self.sin = angle.cos().contiguous(), angle.sin().contiguous()
        self.table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pool, dtype=torch.int32, device="cuda")

    def resize(self, new_lens):
        """Takes pages for sequences that grow and gives back those of sequences that shrink."""
        _, _, short = nv.nvfp4_kv_resize(self.table, self.lens, new_lens, self.refs, self.page, out_table=self.table,
                                         out_refs=self.refs)
        self.lens = new_lens
        return short

    def fork(self, parents, into):
        """Copies of sequences `parents` in the rows `into` of the table."""
        child, _, short = nv.nvfp4_kv_fork(self.pages, self.table, self.lens, self.refs, parents, self.page,
                                           out_refs=self.refs)
        self.table[into] = child
        self.lens[into] = self.lens[parents.long()]
        return short

    def compact(self):
        _, _, live = nv.nvfp4_kv_compact(self.pages, self.table, self.refs, out_table=self.table, out_refs=self.refs)
        return live

    def forward(self, x, counts, start, max_q):
        """x [tokens][hidden]: counts[b] new tokens of each sequence, rows start[b] on. The cache grows by them."""
        short = self.resize(self.lens + counts)
        seq = torch.repeat_interleave(torch.arange(counts.shape[0], device="cuda"), counts.long(), output_size=x.shape[0])
        pos = (self.lens[seq] - counts[seq] + torch.arange(x.shape[0], device="cuda") - start[seq]).int()
        slots = self.table[seq, pos // self.page].long() * self.page + pos % self.page
        h, d = self.q_heads, self.head_dim
        y = self.qkv(x)
        q, k, v = (t.unflatten(1, (-1, d)) for t in y.split([h * d, self.kv_heads * d, self.kv_heads * d], 1))
        q = nv.nvfp4_kv_append(self.cache, k, v, slots, q=q, cos=self.cos, sin=self.sin, positions=pos)
        o = nv.nvfp4_kv_attention(q, self.cache, self.table, self.lens, start, max_q)
        return self.out(o.flatten(1)), q, o, short


def offsets(counts):
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--prompts", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=512, help="length of the longest prompt")
    ap.add_argument("--samples", type=int, default=2, help="samples of each prompt")
    ap.add_argument("--steps", type=int, default=32, help="timed decode steps (at least 1)")
    a = ap.parse_args(argv)
    batch = a.prompts * a.samples
    width = -(-(a.tokens + a.steps + 1) // 64) + 1
    block = Block(batch=batch, width=width, pool=batch * width + 8)
    gen = torch.Generator(device="cuda").manual_seed(1)
    hidden = block.qkv.k

    # prompts of several lengths in the first rows, all in one call
    lens = [a.tokens - (i * 37) % max(1, a.tokens // 2) for i in range(a.prompts)]
    counts = torch.tensor(lens + [0] * (batch - a.prompts), dtype=torch.int32, device="cuda")
    x = torch.randn((sum(lens), hidden), generator=gen, device="cuda").to(torch.bfloat16)
    block.forward(x, counts, offsets(counts), max(lens))

    # further samples of each prompt share its whole pages
    parents = torch.arange(batch - a.prompts, device="cuda", dtype=torch.int32) % a.prompts
    short = block.fork(parents, torch.arange(a.prompts, batch, device="cuda"))
    one = torch.ones(batch, dtype=torch.int32, device="cuda")
    start = offsets(one)
    for i in range(a.steps + 1):
        if i == 1:                                   # the first step loads kernels
            torch.cuda.synchronize()
            began = time.perf_counter()
        x = torch.randn((batch, hidden), generator=gen, device="cuda").to(torch.bfloat16)
        y, _, _, more = block.forward(x, one, start, 1)
        short = short + more
    torch.cuda.synchronize()
    took = time.perf_counter() - began

    # half of the samples end; the rest moves together
    keep = torch.arange(batch, device="cuda") % 2 == 0
    block.resize(torch.where(keep, block.lens, 0).int())
    live = block.compact()
    print(f"{batch} sequences, {a.steps} steps of one block: {1e6 * took / max(1, a.steps):.0f} us a step; "
          f"{int(live)} of {block.refs.shape[0]} pages live after packing, {int(short)} pages short; "
          f"output deviation {y.float().std().item():.3f}")
    return block


if __name__ == "__main__":
    main()
