"""A small mixture-of-experts decoder on one pool: experts and 8-bit KV pages side by side.

Each layer runs rotary positions, the write of the new keys and values, attention over the
paged cache and the paged MoE layer.  The prompts go through in one pass, the first sequence is
forked into several samples that share its pages, all of them decode, some end, and compaction
gives the pages they left back to the experts' view.

    python examples/decoder.py [--steps 48] [--samples 3]

Weights are random; nothing is downloaded.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from paged_moe_shared_gb300 import rimuru as R  # noqa: E402
from paged_moe_shared_gb300.device_pool import DevicePool  # noqa: E402


class Sequence:
    """Tokens of one request and, per layer, the pages that hold its keys and values."""

    def __init__(self, tokens, layers):
        self.tokens, self.cached = list(tokens), 0
        self.pages = [[] for _ in range(layers)]


class Decoder:
    LAYERS, HIDDEN, INTER, EXPERTS, TOP_K = 2, 512, 256, 16, 4
    HEADS, KV_HEADS, DIM, PAGE, VOCAB = 8, 2, 64, 16, 1000

    def __init__(self, expert_pages=160, seed=0, device="cuda:0"):
        self.device = device
        expert_bytes, kv_bytes = self.HIDDEN * self.INTER * 2, 2 * self.KV_HEADS * self.PAGE * self.DIM
        self.pool = DevicePool(expert_pages * expert_bytes, R.rimuru_huge_page_bytes(expert_bytes), device)
        self.ev, self.kv = self.pool.view(expert_bytes), self.pool.view(kv_bytes)
        R.rimuru_view_set_moe_shape(self.ev, self.LAYERS, self.EXPERTS, self.HIDDEN, self.INTER, self.TOP_K, 1)
        nbytes = R.rimuru_kv_scale_bytes(self.kv, self.KV_HEADS)
        self.scales = torch.empty(nbytes // 4, device=device)
        R.rimuru_view_set_kv_shape(self.kv, self.KV_HEADS, self.DIM, self.PAGE, self.scales.data_ptr(), nbytes)
        self.rope = R.rimuru_rope_create(self.DIM)

        g = torch.Generator().manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g) * shape[-2] ** -0.5).bfloat16().to(device)

        pages = self.pool.mem.view(expert_pages, expert_bytes)
        for layer in range(self.LAYERS):
            for e in range(self.EXPERTS):
                for proj in (R.PROJ_W1, R.PROJ_W3, R.PROJ_W2):
                    page = R.rimuru_page_alloc(self.ev)
                    R.rimuru_expert_map(self.ev, layer, e, proj, page)
                    rows, cols = (self.INTER, self.HIDDEN) if proj == R.PROJ_W2 else (self.HIDDEN, self.INTER)
                    pages[page].copy_(weight(rows, cols).view(torch.uint8).flatten())
        self.qkv = [weight(self.HIDDEN, (self.HEADS + 2 * self.KV_HEADS) * self.DIM) for _ in range(self.LAYERS)]
        self.wo = [weight(self.HEADS * self.DIM, self.HIDDEN) for _ in range(self.LAYERS)]
        self.router = [weight(self.HIDDEN, self.EXPERTS) for _ in range(self.LAYERS)]
        self.embed = torch.randn(self.VOCAB, self.HIDDEN, generator=g).bfloat16().to(device)
        self.work = {}

    def workspace(self, name, nbytes):
        """A 1024-byte aligned workspace that grows with need; calls on one stream share it."""
        if name not in self.work or self.work[name].numel() < nbytes + 1024:
            self.work[name] = torch.empty(nbytes + 1024, dtype=torch.uint8, device=self.device)
        return (self.work[name].data_ptr() + 1023) // 1024 * 1024, nbytes

    @staticmethod
    def norm(x):
        return torch.nn.functional.rms_norm(x, x.shape[-1:], eps=1e-6)

    def forward(self, seqs):
        """Run the tokens of every sequence that are not in the cache yet; logits of its last one."""
        new = [len(s.tokens) - s.cached for s in seqs]
        for s in seqs:
            for pages in s.pages:
                while len(pages) * self.PAGE < len(s.tokens):
                    pages.append(R.rimuru_page_alloc_near(self.kv, pages[-1]) if pages else R.rimuru_page_alloc(self.kv))
        width = max(len(s.pages[0]) for s in seqs)
        table = torch.tensor([[s.pages[layer] + [-1] * (width - len(s.pages[layer])) for s in seqs]
                              for layer in range(self.LAYERS)], dtype=torch.int32, device=self.device)
        ids = torch.tensor([t for s in seqs for t in s.tokens[s.cached:]], device=self.device)
        positions = torch.tensor([p for s in seqs for p in range(s.cached, len(s.tokens))], dtype=torch.int32,
                                 device=self.device)
        lens = torch.tensor([len(s.tokens) for s in seqs], dtype=torch.int32, device=self.device)
        cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=self.device)
        n, T, max_q, stream = len(seqs), sum(new), max(new), torch.cuda.current_stream().cuda_stream
        attn_ws = self.workspace("attention",
                                 R.rimuru_kv_attention_workspace_bytes(self.kv, self.HEADS, n, T, max_q))
        moe_ws = self.workspace("moe", R.rimuru_moe_workspace_bytes(self.ev, T))

        x = self.embed[ids]
        for layer in range(self.LAYERS):
            q, k, v = (self.norm(x) @ self.qkv[layer]).unflatten(1, (-1, self.DIM)).split(
                [self.HEADS, self.KV_HEADS, self.KV_HEADS], 1)
            arrays = [R.heads_of(q), R.heads_of(k)]
            R.rimuru_rope_apply(self.rope, positions.data_ptr(), T, self.DIM, arrays, arrays, stream)
            R.rimuru_kv_append(self.kv, R.heads_of(k), R.heads_of(v), cu.data_ptr(), lens.data_ptr(), n, T,
                               table[layer].data_ptr(), width, stream)
            out = torch.empty(T, self.HEADS, self.DIM, dtype=x.dtype, device=self.device)
            R.rimuru_kv_attention(self.kv, R.heads_of(q), R.heads_of(out), 0, cu.data_ptr(), lens.data_ptr(),
                                  n, T, max_q, table[layer].data_ptr(), width, self.DIM ** -0.5, 0,
                                  *attn_ws, stream)
            x = x + out.flatten(1) @ self.wo[layer]
            h = self.norm(x)
            logits, y = (h @ self.router[layer]).float(), torch.empty_like(h)
            R.rimuru_moe_forward(h.data_ptr(), logits.data_ptr(), T, self.ev, layer, y.data_ptr(), *moe_ws, stream)
            x = x + y
        for s in seqs:
            s.cached = len(s.tokens)
        return self.norm(x[(cu[1:] - 1).long()]) @ self.embed.T

    def fork(self, seq, n):
        """n samples that go on from `seq`, sharing its full pages; `seq` itself ends."""
        stream = torch.cuda.current_stream().cuda_stream
        kids = [Sequence(seq.tokens, self.LAYERS) for _ in range(n)]
        for layer in range(self.LAYERS):
            for kid, pages in zip(kids, R.rimuru_kv_fork(self.kv, seq.pages[layer], seq.cached, n, stream)):
                kid.pages[layer], kid.cached = list(pages), seq.cached
        self.end(seq)
        return kids

    def end(self, seq):
        """Drop a sequence's pages.  Work queued earlier on the stream may still read them."""
        for pages in seq.pages:
            for p in pages:
                R.rimuru_page_free(self.kv, p)
            pages.clear()

    def compact(self, seqs, max_moves=1 << 20):
        """Move the pages of the live sequences together; returns the number of pages moved."""
        lists = [pages for s in seqs for pages in s.pages]
        flat, moved = R.rimuru_kv_compact(self.kv, [p for pages in lists for p in pages], max_moves,
                                          torch.cuda.current_stream().cuda_stream)
        at = iter(flat)
        for pages in lists:
            pages[:] = [next(at) for _ in pages]
        return moved

    def free_expert_pages(self):
        return R.rimuru_pool_level_stats(self.pool.handle, 0)["pages_free"]

    def check(self):
        torch.cuda.synchronize()
        assert R.rimuru_get_device_error(self.ev) == R.DEV_OK and R.rimuru_get_device_error(self.kv) == R.DEV_OK

    def close(self):
        torch.cuda.synchronize()
        R.rimuru_rope_destroy(self.rope)
        self.pool.close()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=48)
    ap.add_argument("--samples", type=int, default=3)
    ap.add_argument("--requests", type=int, default=12)
    args = ap.parse_args()
    model = Decoder()
    free = [model.free_expert_pages()]
    g = torch.Generator().manual_seed(1)
    seqs = [Sequence(torch.randint(model.VOCAB, (40 + 97 * i % 300,), generator=g).tolist(), model.LAYERS)
            for i in range(args.requests)]

    logits = model.forward(seqs)  # the prompts, ragged, in one pass
    first, rest = seqs[0], seqs[1:]
    kids = model.fork(first, args.samples)
    for kid, t in zip(kids, logits[0].topk(args.samples).indices.tolist()):  # each begins with another token
        kid.tokens.append(t)
    for s, t in zip(rest, logits[1:].argmax(1).tolist()):
        s.tokens.append(t)
    live = kids + rest
    for _ in range(args.steps):
        for s, t in zip(live, model.forward(live).argmax(1).tolist()):
            s.tokens.append(t)
    free.append(model.free_expert_pages())
    for s in live[1::2]:
        model.end(s)
    live = live[::2]
    free.append(model.free_expert_pages())
    moved = model.compact(live)
    free.append(model.free_expert_pages())
    model.forward(live)
    model.check()
    print(f"{args.requests} requests, one of them as {args.samples} samples, {args.steps} steps; "
          f"{len(live)} live at the end.  Free expert-sized pages: {free[0]} before, {free[1]} while decoding, "
          f"{free[2]} once the others had ended, {free[3]} after compaction moved {moved} KV pages")
    model.close()


if __name__ == "__main__":
    main()
