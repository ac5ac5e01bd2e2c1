"""The hybrid example decoder (norms with rotation, linear attention on state pages, paged attention,
MoE layers, beam selection and reordering on one pool) against a plain 64-bit decoder."""
import itertools
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


def norm(x):
    return bf(x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6))


def plain_moe(m, layer, x, swap, near):
    """`near` collects the layers where the last token's last chosen expert is ahead of the next one by
    less than rounding may move the two, so that either is right; layers in `swap` take that other one."""
    pages = m.pool.mem.view(-1, m.HIDDEN * m.INTER * 2)
    h = norm(x)
    logits = bf(h @ m.router[layer].cpu().double())
    w, e = torch.softmax(logits, -1).topk(m.TOP_K + 1)
    # logits of 2 to 4 have steps of 2^-6 in bf16, and each of the two may be a step off
    if float(logits[-1, e[-1, -2]] - logits[-1, e[-1, -1]]) < 2.0 ** -5:
        near.append(layer)
    if layer in swap:
        w[-1, -2], e[-1, -2] = w[-1, -1], e[-1, -1]
    w, e = w[:, :-1], e[:, :-1]
    w, y = w / w.sum(-1, keepdim=True), torch.zeros_like(x)
    for i in range(m.EXPERTS):
        w1, w3, w2 = (pages[R.rimuru_expert_lookup(m.ev, layer, i, p)].view(torch.bfloat16).cpu().double()
                      for p in (R.PROJ_W1, R.PROJ_W3, R.PROJ_W2))
        u = bf(torch.nn.functional.silu(h @ w1.view(m.HIDDEN, m.INTER)) * (h @ w3.view(m.HIDDEN, m.INTER))) \
            @ w2.view(m.INTER, m.HIDDEN)
        y += bf(u) * torch.where(e == i, w, 0.0).sum(-1, keepdim=True)
    return bf(x + bf(y))


def plain_linear(m, i, x):
    T, h = len(x), norm(x)
    q, k, v = bf(h @ m.lin_in[i].cpu().double()).split(
        [m.LIN_KEYS * m.KEY_DIM, m.LIN_KEYS * m.KEY_DIM, m.LIN_HEADS * m.VALUE_DIM], 1)
    q, k = (bf(torch.nn.functional.normalize(t.reshape(T, m.LIN_KEYS, m.KEY_DIM), dim=-1))
            .repeat_interleave(m.LIN_HEADS // m.LIN_KEYS, 1) for t in (q, k))
    v = v.reshape(T, m.LIN_HEADS, m.VALUE_DIM)
    f = torch.exp(-m.rate.cpu().double() * torch.nn.functional.softplus(bf(h @ m.lin_gate[i].cpu().double())))
    S, out = torch.zeros(m.LIN_HEADS, m.KEY_DIM, m.VALUE_DIM, dtype=torch.float64), []
    for t in range(T):
        S = f[t, :, None, None] * S + k[t][:, :, None] * v[t][:, None]
        out.append((q[t][:, :, None] * S).sum(1))
    return bf(x + bf(bf(torch.stack(out)).flatten(1) @ m.lin_out[i].cpu().double()))


def plain_attention(m, i, x):
    T, D, P = len(x), m.DIM, m.PAGE
    a = bf(norm(x) @ m.qkv[i].cpu().double()).unflatten(1, (-1, D))
    q, k, v = a.split([m.HEADS, m.KV_HEADS, m.KV_HEADS], 1)
    f, pos = ref.inv_freq(D, 10000.0, R.ROPE_PLAIN), torch.arange(T)

    def turn(y, w):
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.cpu().double()
        return bf(torch.from_numpy(ref.rope(y, pos, f, False)))

    q, k = turn(q, m.q_norm[i]), turn(k, m.k_norm[i])
    table = [list(range(-(-T // P)))]
    values = np.zeros((len(table[0]), 2, m.KV_HEADS, P, D))
    scales = np.full(values.shape[:3], 2.0 ** -60)
    ref.append(values, scales, table, [0, T], [T], k, v, P)
    out = bf(ref.attention(torch.from_numpy(values), table, [T], q, [0, T], D ** -0.5, 0, P)[0])
    return bf(x + bf(out.flatten(1) @ m.wo[i].cpu().double()))


def plain_logits(m, tokens, swap=(), near=None):
    near = [] if near is None else near
    x = m.embed.cpu().double()[tokens]
    for i in range(m.PAIRS):
        x = plain_moe(m, 2 * i, plain_linear(m, i, x), swap, near)
        x = plain_moe(m, 2 * i + 1, plain_attention(m, i, x), swap, near)
    return norm(x) @ m.head.cpu().double()


@pytest.mark.parametrize("beams,steps", [(4, 20), (1, 3)])
def test_beams_equal_their_tokens_run_alone(beams, steps):
    """Every beam's logits are those of its tokens from the start: its caches and states went along
    with its history through all selections, over pages that fill up on the way."""
    from hybrid_decoder import HybridDecoder
    m = HybridDecoder()
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randint(1, m.VOCAB, (n,), generator=g).tolist() for n in (37, 16, 90)]
    tokens, scores, logits = m.search(prompts, beams, steps)
    m.check()
    for r, p in enumerate(prompts):
        assert tokens[r].shape == (beams, len(p) + steps)
        assert bool((tokens[r][:, :len(p)].cpu() == torch.tensor(p)).all())
        assert len({tuple(t) for t in tokens[r].tolist()}) == beams or bool((tokens[r] == m.EOS).any())
        s = scores[r].tolist()
        assert s == sorted(s, reverse=True)
        for b in range(beams):
            got, t, near = logits[r, b].double().cpu(), tokens[r][b].tolist(), []
            wants = [plain_logits(m, t, near=near)[-1]]
            ways = [c for k in range(len(near)) for c in itertools.combinations(near, k + 1)]
            wants += [plain_logits(m, t, c)[-1] for c in ways]
            # about fourteen roundings to bf16 a pair of layers (2^-9 each, at random), which may fall the
            # other way where the sums' orders differ, and codes of the cache that do: 5 % of the row's norm
            assert min(float((got - w).norm() / w.norm()) for w in wants) < 0.05, (r, b, near)
    if beams > 1:  # beams that go on from one parent were among them
        firsts = [t[:, len(p)].unique().numel() for t, p in zip(tokens, prompts)]
        assert min(firsts) < beams
    m.close()


def test_main_runs(monkeypatch, capsys):
    import hybrid_decoder
    monkeypatch.setattr(sys, "argv", ["hybrid_decoder.py", "--requests", "2", "--beams", "3", "--steps", "18"])
    hybrid_decoder.main()
    assert capsys.readouterr().out.count("best score") == 2
