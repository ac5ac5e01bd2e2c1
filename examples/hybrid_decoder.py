"""Beam search with a small hybrid decoder on one pool: expert pages, 8-bit KV pages and the fp32 state
pages of linear-attention layers side by side.

Layers alternate: linear attention with a decay for each head, and attention over the paged cache
whose queries and keys are normalised and rotated in one pass; each is followed by a paged MoE layer.
The prompts go through in one pass.  Then each step selects the best continuations of every request
on the device, reorders the page tables of all attention layers in one launch, and lets every linear
layer read its parents' state pages and write others, so that no state is copied.

    python examples/hybrid_decoder.py [--requests 3] [--beams 4] [--steps 40]

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


class HybridDecoder:
    PAIRS, HIDDEN, INTER, EXPERTS, TOP_K = 2, 512, 256, 16, 4  # a pair: a linear layer, then a full one
    HEADS, KV_HEADS, DIM, PAGE, VOCAB = 8, 2, 64, 16, 1000
    LIN_HEADS, LIN_KEYS, KEY_DIM, VALUE_DIM = 4, 2, 64, 128
    EOS = 0

    def __init__(self, expert_pages=256, seed=0, device="cuda:0"):
        self.device = device
        expert_bytes, kv_bytes = self.HIDDEN * self.INTER * 2, 2 * self.KV_HEADS * self.PAGE * self.DIM
        state_bytes = self.LIN_HEADS * self.KEY_DIM * self.VALUE_DIM * 4
        huge = R.rimuru_huge_page_bytes(expert_bytes, state_bytes)
        self.pool = DevicePool(expert_pages * expert_bytes, huge, device)
        self.ev, self.sv, self.kv = (self.pool.view(b) for b in (expert_bytes, state_bytes, kv_bytes))
        R.rimuru_view_set_moe_shape(self.ev, 2 * self.PAIRS, self.EXPERTS, self.HIDDEN, self.INTER, self.TOP_K, 1)
        R.rimuru_view_set_state_shape(self.sv, self.LIN_HEADS, self.KEY_DIM, self.VALUE_DIM)
        nbytes = R.rimuru_kv_scale_bytes(self.kv, self.KV_HEADS)
        self.scales = torch.empty(nbytes // 4, device=device)
        R.rimuru_view_set_kv_shape(self.kv, self.KV_HEADS, self.DIM, self.PAGE, self.scales.data_ptr(), nbytes)
        self.rope = R.rimuru_rope_create(self.DIM)

        g = torch.Generator().manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g) * shape[-2] ** -0.5).bfloat16().to(device)

        pages = self.pool.mem.view(expert_pages, expert_bytes)
        for layer in range(2 * self.PAIRS):
            for e in range(self.EXPERTS):
                for proj in (R.PROJ_W1, R.PROJ_W3, R.PROJ_W2):
                    page = R.rimuru_page_alloc(self.ev)
                    R.rimuru_expert_map(self.ev, layer, e, proj, page)
                    rows, cols = (self.INTER, self.HIDDEN) if proj == R.PROJ_W2 else (self.HIDDEN, self.INTER)
                    pages[page].copy_(weight(rows, cols).view(torch.uint8).flatten())
        lin = 2 * self.LIN_KEYS * self.KEY_DIM + self.LIN_HEADS * self.VALUE_DIM
        self.lin_in = [weight(self.HIDDEN, lin) for _ in range(self.PAIRS)]
        self.lin_gate = [weight(self.HIDDEN, self.LIN_HEADS) for _ in range(self.PAIRS)]
        self.lin_out = [weight(self.LIN_HEADS * self.VALUE_DIM, self.HIDDEN) for _ in range(self.PAIRS)]
        # heads that forget within a few tokens next to heads that hardly do
        self.rate = torch.exp(torch.linspace(-5, 0, self.LIN_HEADS)).to(device)
        self.qkv = [weight(self.HIDDEN, (self.HEADS + 2 * self.KV_HEADS) * self.DIM) for _ in range(self.PAIRS)]
        self.q_norm, self.k_norm = ([(1 + 0.2 * torch.randn(self.DIM, generator=g)).bfloat16().to(device)
                                     for _ in range(self.PAIRS)] for _ in range(2))
        self.wo = [weight(self.HEADS * self.DIM, self.HIDDEN) for _ in range(self.PAIRS)]
        self.router = [weight(self.HIDDEN, self.EXPERTS) for _ in range(2 * self.PAIRS)]
        self.embed = torch.randn(self.VOCAB, self.HIDDEN, generator=g).bfloat16().to(device)
        self.head = weight(self.HIDDEN, self.VOCAB)
        self.work, self.placed = {}, []

    def workspace(self, name, nbytes):
        """A 1024-byte aligned workspace that grows with need; calls on one stream share it."""
        if name not in self.work or self.work[name].numel() < nbytes + 1024:
            self.work[name] = torch.empty(nbytes + 1024, dtype=torch.uint8, device=self.device)
        return (self.work[name].data_ptr() + 1023) // 1024 * 1024, nbytes

    def pages(self, view, *shape):
        """New pages of a view as an int32 tensor."""
        got = torch.empty(shape, dtype=torch.int32)
        for i in range(got.numel()):
            got.view(-1)[i] = page = R.rimuru_page_alloc(view)
            self.placed.append((view, page))
        return got.to(self.device)

    @staticmethod
    def norm(x):
        return torch.nn.functional.rms_norm(x, x.shape[-1:], eps=1e-6)

    def linear(self, i, x, n, T, most, cu, state_in, state_out, stream):
        h = self.norm(x)
        mix = (h @ self.lin_in[i])
        q, k, v = mix.split([self.LIN_KEYS * self.KEY_DIM, self.LIN_KEYS * self.KEY_DIM,
                             self.LIN_HEADS * self.VALUE_DIM], 1)
        q, k = (torch.nn.functional.normalize(t.reshape(T, self.LIN_KEYS, self.KEY_DIM).float(), dim=-1).to(x.dtype)
                for t in (q, k))
        v = v.view(T, self.LIN_HEADS, self.VALUE_DIM)
        g = -self.rate * torch.nn.functional.softplus((h @ self.lin_gate[i]).float())
        out = torch.empty(T, self.LIN_HEADS, self.VALUE_DIM, dtype=x.dtype, device=self.device)
        ws = self.workspace("linear", R.rimuru_linear_attention_workspace_bytes(self.sv, n, T, most))
        R.rimuru_linear_attention(self.sv, R.heads_of(q), R.heads_of(k), R.heads_of(v), R.heads_of(out), g.data_ptr(),
                                  *g.stride(), cu.data_ptr(), n, T, most, state_in.data_ptr(), state_out.data_ptr(),
                                  1.0, *ws, stream)
        return x + out.flatten(1) @ self.lin_out[i]

    def attention(self, i, x, n, T, most, cu, positions, lens, table, stream):
        q, k, v = (self.norm(x) @ self.qkv[i]).unflatten(1, (-1, self.DIM)).split(
            [self.HEADS, self.KV_HEADS, self.KV_HEADS], 1)
        arrays = [R.heads_of(q), R.heads_of(k)]
        norms = [R.head_norm_of(self.q_norm[i]), R.head_norm_of(self.k_norm[i])]
        R.rimuru_norm_rope_apply(self.rope, positions.data_ptr(), T, self.DIM, arrays, arrays, norms, stream)
        R.rimuru_kv_append(self.kv, R.heads_of(k), R.heads_of(v), cu.data_ptr(), lens.data_ptr(), n, T,
                           table[i].data_ptr(), table.shape[2], stream)
        out = torch.empty(T, self.HEADS, self.DIM, dtype=x.dtype, device=self.device)
        ws = self.workspace("attention", R.rimuru_kv_attention_workspace_bytes(self.kv, self.HEADS, n, T, most))
        R.rimuru_kv_attention(self.kv, R.heads_of(q), R.heads_of(out), 0, cu.data_ptr(), lens.data_ptr(), n, T, most,
                              table[i].data_ptr(), table.shape[2], self.DIM ** -0.5, 0, *ws, stream)
        return x + out.flatten(1) @ self.wo[i]

    def moe(self, layer, x, T, stream):
        h = self.norm(x)
        logits, y = (h @ self.router[layer]).float(), torch.empty_like(h)
        ws = self.workspace("moe", R.rimuru_moe_workspace_bytes(self.ev, T))
        R.rimuru_moe_forward(h.data_ptr(), logits.data_ptr(), T, self.ev, layer, y.data_ptr(), *ws, stream)
        return x + y

    def forward(self, ids, new, lens, table, state_in, state_out):
        """Run `ids`, the new tokens of all sequences one after another (`new` of each), where `lens`
        counts them already; logits after each sequence's last one."""
        n, T, most, stream = len(new), len(ids), max(new), torch.cuda.current_stream().cuda_stream
        cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(self.device)
        at = torch.arange(T, device=self.device) - torch.repeat_interleave(cu[1:], torch.tensor(new, device=self.device))
        positions = (torch.repeat_interleave(lens, torch.tensor(new, device=self.device)) + at).to(torch.int32)
        x = self.embed[ids]
        for i in range(self.PAIRS):
            x = self.linear(i, x, n, T, most, cu, state_in[i], state_out[i], stream)
            x = self.moe(2 * i, x, T, stream)
            x = self.attention(i, x, n, T, most, cu, positions, lens, table, stream)
            x = self.moe(2 * i + 1, x, T, stream)
        return self.norm(x[(cu[1:] - 1).long()]) @ self.head

    def search(self, prompts, beams, steps):
        """Beam search; returns for each request its beams' tokens [beams][...], their scores and the
        logits after each beam's last token."""
        dev, N, L, P = self.device, len(prompts), self.PAIRS, self.PAGE
        stream = torch.cuda.current_stream().cuda_stream
        rows = N * beams
        width = -(-(max(map(len, prompts)) + steps) // P)
        # the prompts, one sequence a request
        new = [len(p) for p in prompts]
        table = torch.full((L, N, width), -1, dtype=torch.int32, device=dev)
        for r, n in enumerate(new):
            table[:, r, :-(-n // P)] = self.pages(self.kv, L, -(-n // P))
        lens = torch.tensor(new, dtype=torch.int32, device=dev)
        state = self.pages(self.sv, L, N)
        fresh_states = [self.pages(self.sv, L, rows), self.pages(self.sv, L, rows)]
        logits = self.forward(torch.tensor(sum(prompts, []), device=dev), new, lens, table, torch.full_like(state, -1), state)
        scores = torch.zeros(N, 1, device=dev)
        done = torch.zeros(N, 1, dtype=torch.uint8, device=dev)
        tokens = [torch.tensor(p, device=dev).expand(1, -1) for p in prompts]
        # pages that hold the last tokens of a beam, by turns: one is copied into the other
        spare = [self.pages(self.kv, L, rows), self.pages(self.kv, L, rows)]
        best, parents, chosen = (torch.empty(N, beams, dtype=t, device=dev) for t in (torch.float32, torch.int32, torch.int32))
        for step in range(steps):
            had = scores.shape[1]
            ws = self.workspace("select", R.rimuru_beam_select_workspace_bytes(N, had, self.VOCAB, beams))
            R.rimuru_beam_select(R.rows_of(logits), scores.data_ptr(), done.data_ptr(), N, had, self.EOS, beams,
                                 best.data_ptr(), parents.data_ptr(), chosen.data_ptr(), *ws, stream)
            at = parents.view(-1).long()
            fresh = spare[step % 2]
            table_out = torch.full((L, rows, width), -1, dtype=torch.int32, device=dev)
            lens_out = torch.empty(rows, dtype=torch.int32, device=dev)
            R.rimuru_kv_reorder(self.kv, parents.data_ptr(), rows, lens.data_ptr(), len(lens), table.data_ptr(),
                                table_out.data_ptr(), L, width, fresh.data_ptr(), lens_out.data_ptr(), stream)
            # the new token goes into the fresh page, whether that begins with copied tokens or empty
            table_out[:, torch.arange(rows, device=dev), (lens_out // P).long()] = fresh
            tokens = [torch.cat([tokens[r][at.view(N, beams)[r] - r * had], chosen[r, :, None]], 1) for r in range(N)]
            done = (done.view(-1)[at].view(N, beams).bool() | (chosen == self.EOS)).to(torch.uint8)
            scores, table, lens = best.clone(), table_out, lens_out + 1
            state_in, state = state[:, at].contiguous(), fresh_states[step % 2]
            logits = self.forward(chosen.view(-1).long(), [1] * rows, lens, table, state_in, state)
            # pages that have filled up are other beams' history from now on
            full = [b for b, p in enumerate(prompts) if (len(p) + step + 1) % P == 0]
            for b in full:
                spare[step % 2][:, b * beams:(b + 1) * beams] = self.pages(self.kv, L, beams)
        return tokens, scores, logits.view(N, beams, -1)

    def check(self):
        torch.cuda.synchronize()
        for view in (self.ev, self.kv, self.sv):
            assert R.rimuru_get_device_error(view) == R.DEV_OK

    def close(self):
        torch.cuda.synchronize()
        for view, page in self.placed:
            R.rimuru_page_free(view, page)
        R.rimuru_rope_destroy(self.rope)
        self.pool.close()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=40)
    args = ap.parse_args()
    model = HybridDecoder()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(1, model.VOCAB, (30 + 67 * i % 200,), generator=g).tolist() for i in range(args.requests)]
    tokens, scores, _ = model.search(prompts, args.beams, args.steps)
    model.check()
    for r, p in enumerate(prompts):
        print(f"request {r}: prompt of {len(p)} tokens, best score {float(scores[r, 0]):.3f}, "
              f"continues {tokens[r][0, len(p):len(p) + 8].tolist()} ...")
    model.close()


if __name__ == "__main__":
    main()
