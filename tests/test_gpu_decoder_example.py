"""The example decoder (rotary positions, cache, attention and MoE layer on one pool) against a
plain 64-bit decoder, through a fork, decoding, the end of a sequence and compaction."""
import os
import sys

import numpy as np
import pytest
import torch

import kv_reference as ref
from paged_moe_shared_gb300 import rimuru as R

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def bf(x):
    return x.to(torch.bfloat16).double()


def plain_logits(m, tokens):
    """Logits of every token of one sequence: full causal attention over keys and values rounded
    to the cache's codes, all experts by plain products, in 64 bits, each array that the decoder
    keeps in bf16 rounded to it (a router's near tie then falls as it does there)."""
    def norm(x):
        return bf(x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6))

    T, D, P = len(tokens), m.DIM, m.PAGE
    pages = m.pool.mem.view(-1, m.HIDDEN * m.INTER * 2)
    x = m.embed.cpu().double()[tokens]
    f, pos = ref.inv_freq(D, 10000.0, R.ROPE_PLAIN), torch.arange(T)
    table = [list(range(-(-T // P)))]
    for layer in range(m.LAYERS):
        a = bf(norm(x) @ m.qkv[layer].cpu().double()).unflatten(1, (-1, D))
        q, k, v = a.split([m.HEADS, m.KV_HEADS, m.KV_HEADS], 1)
        q, k = (bf(torch.from_numpy(ref.rope(t, pos, f, False))) for t in (q, k))
        values = np.zeros((len(table[0]), 2, m.KV_HEADS, P, D))
        scales = np.full(values.shape[:3], 2.0 ** -60)
        ref.append(values, scales, table, [0, T], [T], k, v, P)
        out = bf(ref.attention(torch.from_numpy(values), table, [T], q, [0, T], D ** -0.5, 0, P)[0])
        x = bf(x + bf(out.flatten(1) @ m.wo[layer].cpu().double()))
        h = norm(x)
        w, e = torch.softmax(bf(h @ m.router[layer].cpu().double()), -1).topk(m.TOP_K)
        w, y = w / w.sum(-1, keepdim=True), torch.zeros_like(x)
        for i in range(m.EXPERTS):
            w1, w3, w2 = (pages[R.rimuru_expert_lookup(m.ev, layer, i, p)].view(torch.bfloat16).cpu().double()
                          for p in (R.PROJ_W1, R.PROJ_W3, R.PROJ_W2))
            u = bf(torch.nn.functional.silu(h @ w1.view(m.HIDDEN, m.INTER)) * (h @ w3.view(m.HIDDEN, m.INTER))) \
                @ w2.view(m.INTER, m.HIDDEN)
            y += bf(u) * torch.where(e == i, w, 0.0).sum(-1, keepdim=True)
        x = bf(x + bf(y))
    return norm(x) @ m.embed.cpu().double().T


def close_to(got, want):
    # About ten roundings to bf16 per layer (2^-9 each, at random), which may fall the other way where
    # the sums' orders differ, and codes of the cache that do: 5 % of the row's norm.
    got = got.double().cpu()
    assert float((got - want).norm() / want.norm()) < 0.05


def test_decoder_with_fork_and_compaction():
    from decoder import Decoder, Sequence
    m = Decoder()
    start = m.free_expert_pages()
    g = torch.Generator().manual_seed(4)
    seqs = [Sequence(torch.randint(m.VOCAB, (n,), generator=g).tolist(), m.LAYERS) for n in (150, 1, 33)]
    logits = m.forward(seqs)
    for i, s in enumerate(seqs):
        close_to(logits[i], plain_logits(m, s.tokens)[-1])
    kids = m.fork(seqs[0], 3)
    assert R.rimuru_page_refs(m.kv, kids[0].pages[0][0]) == 3
    live = kids + seqs[1:]
    for step in range(20):
        for i, s in enumerate(live):
            s.tokens.append(int(logits[0].topk(3).indices[i]) if step == 0 and i < 3 else (37 * step + 11 * i) % m.VOCAB)
        logits = m.forward(live)
    for i, s in enumerate(live):
        close_to(logits[i], plain_logits(m, s.tokens)[-1])
    m.end(live.pop(1))
    m.end(live.pop(2))
    for s in live:
        s.tokens.append(5)
    before = m.forward(live)
    m.compact(live)
    for s in live:  # the same step again from the moved pages
        s.cached -= 1
    assert torch.equal(before, m.forward(live))
    m.check()
    for s in live:
        m.end(s)
    assert m.free_expert_pages() == start
    m.close()
