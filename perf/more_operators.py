"""What a hybrid decoder on a shared page pool runs next to its MoE layer and paged attention, as
cases to measure: norms of queries and keys in one pass with their rotation, linear attention with
a decay for each head on state pages, and beam search's selection with the reordering of the cache.

``listed()`` and ``draw()`` give cases, ``prepare()`` makes what a serving loop has in hand before
a call, ``run()`` is one pass: with ``own`` false in elementary torch operations, with ``own`` true
through the library.  ``exact()`` is the same from the definitions in fp64.

norm_rope: each head x of a token becomes rot_p(x / sqrt(mean(x^2) + eps) * (w + offset)).

linear: a state S [key_dim][value_dim] a head, in fp32, one page [heads][key_dim][value_dim] a
sequence.  Token by token S <- exp(g) S + k v^T and out = scale * S^T q; the page state_in[b] holds
S before the sequence's tokens (-1: zeros) and state_out[b] receives it after them.  Query/key
head h / (heads / key_heads) serves head h.

select: the n_select best of scores[b] + log_softmax(logits[b]) over the beams and the vocabulary
of each group, the lowest (beam, token) first on ties; a finished beam offers its pad token at its
own score and nothing else.

reorder: child i goes on from sequence parents[i]: its row of the page table and its length are the
parent's; a partly filled last page is copied to the child's fresh page.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of one user: q and k of one token, the whole head rotated
        dict(name="norm_rope_decode", op="norm_rope", tokens=1, q_heads=32, kv_heads=4, dim=128, rot=128,
             interleaved=False, offset=0.0, max_pos=40000, dtype="bf16"),
        # a long prefill chunk: wide heads, a quarter of each rotated, weights stored less one
        dict(name="norm_rope_prefill", op="norm_rope", tokens=8192, q_heads=16, kv_heads=2, dim=256, rot=64,
             interleaved=False, offset=1.0, max_pos=131072, dtype="bf16"),
        # one decode step of one user: latency
        dict(name="linear_decode_one", op="linear", seqs=1, min_new=1, max_new=1, heads=32, key_heads=16,
             key_dim=128, value_dim=128, constant=False, fresh=False, dtype="bf16", layout=1),
        # an ordinary decode batch: the states are nearly all that is moved
        dict(name="linear_decode_batch", op="linear", seqs=64, min_new=1, max_new=1, heads=32, key_heads=16,
             key_dim=128, value_dim=128, constant=False, fresh=False, dtype="bf16", layout=2),
        # checking a few drafted tokens for each of 16 sequences, decays fixed for each head
        dict(name="linear_verify", op="linear", seqs=16, min_new=3, max_new=5, heads=16, key_heads=16,
             key_dim=64, value_dim=128, constant=True, fresh=False, dtype="f16", layout=3),
        # one long prompt: few heads for the GPU, work along the tokens
        dict(name="linear_prompt_long", op="linear", seqs=1, min_new=8192, max_new=8192, heads=32, key_heads=16,
             key_dim=128, value_dim=128, constant=False, fresh=True, dtype="bf16", layout=4),
        # fresh ragged prompts in one batch
        dict(name="linear_prompt_ragged", op="linear", seqs=7, min_new=35, max_new=1733, heads=32, key_heads=16,
             key_dim=128, value_dim=128, constant=False, fresh=True, dtype="bf16", layout=5),
        # one user's beam step
        dict(name="select_one", op="select", groups=1, beams=4, vocab=128000, n_select=8, done=False,
             dtype="bf16", layout=6),
        # a batch of beam searches on a vocabulary of odd size, some beams finished
        dict(name="select_odd", op="select", groups=8, beams=5, vocab=50257, n_select=10, done=True,
             dtype="f32", layout=7),
        # many beam searches on a large vocabulary
        dict(name="select_batch", op="select", groups=32, beams=8, vocab=151936, n_select=16, done=False,
             dtype="bf16", layout=8),
        # the beams of one request in one layer
        dict(name="reorder_one", op="reorder", layers=1, seqs=4, width=20, pages=512, kv_heads=4, dim=128,
             page_tokens=16, layout=9),
        # every layer of a model for the beams of a small batch
        dict(name="reorder_layers", op="reorder", layers=48, seqs=32, width=130, pages=4096, kv_heads=4, dim=128,
             page_tokens=16, layout=10),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "linear", "linear", "linear", "select", "select", "reorder"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    layout = rng.randrange(1 << 20)
    if op == "norm_rope":
        kv_heads, dim = rng.choice([(4, 128), (2, 256), (8, 128), (8, 64), (1, 192), (4, 96)])
        rot = rng.choice([r for r in (dim, dim, dim // 2, dim // 4) if r % 16 == 0])
        tokens = _log_int(rng, 1, 8192 if kv_heads * dim < 1024 else 4000)
        return dict(op=op, tokens=tokens, q_heads=kv_heads * rng.choice([1, 4, 7, 8]),
                    kv_heads=kv_heads, dim=dim, rot=rot, interleaved=rng.random() < 0.4,
                    offset=rng.choice([0.0, 1.0]), max_pos=_log_int(rng, 8192, 131072),
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]) if tokens < 1500 else dtype)
    if op == "linear":
        key_heads = rng.choice([1, 2, 4, 8, 16])
        heads = key_heads * rng.choice([1, 2, 2, 4] if key_heads < 16 else [1, 2])
        base = dict(op=op, heads=heads, key_heads=key_heads, key_dim=rng.choice([64, 128, 128]),
                    value_dim=rng.choice([64, 128, 128]), constant=rng.random() < 0.3,
                    fresh=rng.random() < 0.3, dtype=dtype, layout=layout)
        kind = rng.choice(["decode", "verify", "prompt", "prompt"])
        if kind == "decode":
            return dict(base, seqs=_log_int(rng, 1, 64), min_new=1, max_new=1)
        if kind == "verify":
            most = rng.randrange(2, 17)
            return dict(base, seqs=_log_int(rng, 1, 24), min_new=rng.randrange(1, most + 1), max_new=most)
        seqs = _log_int(rng, 1, 12)
        most = _log_int(rng, 17, 8192 // seqs)
        return dict(base, seqs=seqs, min_new=rng.choice([1, max(1, most // 6), most]), max_new=most)
    if op == "select":
        groups, beams = _log_int(rng, 1, 32), rng.randrange(1, 13)
        most = min(160000, 38000000 // (groups * beams))
        return dict(op=op, groups=groups, beams=beams, vocab=_log_int(rng, 1000, most),
                    n_select=rng.choice([beams, 2 * beams, 2 * beams + 1]), done=rng.random() < 0.3,
                    dtype=rng.choice(["bf16", "f16", "f32"] if groups * beams < 100 else ["bf16"]), layout=layout)
    kv_heads, dim, page_tokens = rng.choice([(4, 128, 16), (2, 256, 16), (2, 64, 32), (1, 128, 64)])
    layers, seqs = _log_int(rng, 1, 48), _log_int(rng, 1, 32)
    return dict(op=op, layers=layers, seqs=seqs, width=_log_int(rng, 1, 130),
                pages=2 * layers * seqs + rng.randrange(16, 1000), kv_heads=kv_heads, dim=dim,
                page_tokens=page_tokens, layout=layout)


def _new(case):
    """New tokens of each sequence, by the case alone."""
    r = random.Random(case["layout"])
    return [r.randint(case["min_new"], case["max_new"]) for _ in range(case["seqs"])]


def _beams(case):
    """Parents and lengths of a reordering, by the case alone."""
    r = random.Random(case["layout"])
    n, most = case["seqs"], case["width"] * case["page_tokens"]
    lens = [r.randint(max(1, most // 2), most) for _ in range(n)]
    return [r.randrange(n) for _ in range(n)], lens


def work(case):
    """Bytes that have to be read and written once, and multiply-adds as two operations."""
    if case["op"] == "norm_rope":
        size = 4 if case["dtype"] == "f32" else 2
        heads = case["tokens"] * (case["q_heads"] + case["kv_heads"])
        return {"bytes": 2 * size * heads * case["dim"] + 4 * case["tokens"],
                "flops": heads * (4 * case["dim"] + 3 * case["rot"])}
    if case["op"] == "linear":
        T, Dk, Dv, H = sum(_new(case)), case["key_dim"], case["value_dim"], case["heads"]
        states = (1 if case["fresh"] else 2) * case["seqs"] * H * Dk * Dv * 4
        gates = 4 * H if case["constant"] else 4 * T * H
        # a token and head: k v^T into the state, and the state with q
        return {"bytes": states + gates + 2 * T * (2 * case["key_heads"] * Dk + 2 * H * Dv),
                "flops": 4 * T * H * Dk * Dv}
    if case["op"] == "select":
        size = 4 if case["dtype"] == "f32" else 2
        rows = case["groups"] * case["beams"]
        return {"bytes": rows * (size * case["vocab"] + 4) + 12 * case["groups"] * case["n_select"],
                "flops": 3 * rows * case["vocab"]}
    parents, lens = _beams(case)
    P = case["page_tokens"]
    moved = sum(lens[p] % P > 0 for p in parents)
    entries = sum(-(-lens[p] // P) for p in parents)
    page = 2 * case["kv_heads"] * (P * case["dim"] + 4)
    return {"bytes": case["layers"] * (2 * moved * page + 8 * entries), "flops": 0}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    {"norm_rope": _prepare_norm_rope, "linear": _prepare_linear, "select": _prepare_select,
     "reorder": _prepare_reorder}[case["op"]](case, gen, s)
    return s


def _workspace(s, nbytes):
    s["ws"] = torch.empty(nbytes + 1024, dtype=torch.uint8, device="cuda")
    s["ws_ptr"], s["ws_bytes"] = (s["ws"].data_ptr() + 1023) // 1024 * 1024, nbytes


def _prepare_norm_rope(case, gen, s):
    T, Hq, Hk, D, dt = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    qkv = torch.randn((T, (Hq + 2 * Hk) * D), generator=gen, device="cuda")
    # a few channels carry much larger values
    loud = 1 + 7 * (torch.rand((Hq + 2 * Hk) * D, generator=gen, device="cuda") < 0.02).float()
    qkv = (qkv * loud).to(dt)
    s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
    s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    s["wq"], s["wk"] = (((1 - case["offset"]) + 0.3 * torch.randn(D, generator=gen, device="cuda")).to(dt)
                        for _ in range(2))
    s["eps"] = 1e-6
    s["pos"] = torch.randint(0, case["max_pos"], (T,), generator=gen, device="cuda").to(torch.int32)
    s["q_out"], s["k_out"] = torch.empty(T, Hq, D, dtype=dt, device="cuda"), torch.empty(T, Hk, D, dtype=dt, device="cuda")
    s["freq"] = 1e6 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
    if own:
        from paged_moe_shared_gb300 import rimuru as R
        s["rope"] = R.rimuru_rope_create(case["rot"], R.ROPE_INTERLEAVED if case["interleaved"] else R.ROPE_HALF, 1e6)


def _prepare_linear(case, gen, s):
    H, Hk, Dk, Dv, B, dt = (case["heads"], case["key_heads"], case["key_dim"], case["value_dim"], case["seqs"],
                            DTYPES[case["dtype"]])
    new = _new(case)
    T = s["tokens"] = sum(new)
    s["max_new"] = max(new)
    s["cu"] = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    qkv = torch.randn((T, 2 * Hk * Dk + H * Dv), generator=gen, device="cuda")
    qk = qkv[:, :2 * Hk * Dk].view(T, 2 * Hk, Dk)
    qk /= qk.norm(dim=-1, keepdim=True)  # such layers normalise queries and keys
    qkv = qkv.to(dt)
    s["q"], s["k"] = qkv[:, :Hk * Dk].view(T, Hk, Dk), qkv[:, Hk * Dk:2 * Hk * Dk].view(T, Hk, Dk)
    s["v"] = qkv[:, 2 * Hk * Dk:].view(T, H, Dv)
    s["out"] = torch.empty(T, H, Dv, dtype=dt, device="cuda")
    s["scale"] = Dk ** -0.5
    # heads forget at very different rates: from a few tokens to thousands of them
    rate = torch.exp(torch.linspace(math.log(1e-3), math.log(0.7), H, device="cuda"))
    if case["constant"]:
        s["g"] = -rate
    else:
        s["g"] = -rate * torch.nn.functional.softplus(torch.randn((T, H), generator=gen, device="cuda"))
    pages = 2 * B + 3
    page_bytes = H * Dk * Dv * 4
    if own:
        from paged_moe_shared_gb300 import rimuru as R
        from paged_moe_shared_gb300.device_pool import DevicePool
        s["pool"] = DevicePool(pages * page_bytes, page_bytes, "cuda")
        mem, s["view"] = s["pool"].mem, s["pool"].view(page_bytes)
        R.rimuru_view_set_state_shape(s["view"], H, Dk, Dv)
        _workspace(s, R.rimuru_linear_attention_workspace_bytes(s["view"], B, T, s["max_new"]))
    else:
        mem = torch.empty(pages * page_bytes, dtype=torch.uint8, device="cuda")
    s["states"] = mem.view(torch.float32).view(pages, H, Dk, Dv)
    for i in range(pages):
        s["states"][i].normal_(0, 0.3, generator=gen)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    # a step writes other pages than it reads, as beams that share a parent's state need
    s["state_in"] = torch.full_like(order[:B], -1) if case["fresh"] else order[:B].clone()
    s["state_out"] = order[B:2 * B].clone()


def _prepare_select(case, gen, s):
    G, N, V, dt = case["groups"], case["beams"], case["vocab"], DTYPES[case["dtype"]]
    # a few likely tokens over a broad floor
    x = torch.randn((G * N, V), generator=gen, device="cuda") * 2.5
    s["logits"] = x.to(dt)
    s["scores"] = -20 * torch.rand((G, N), generator=gen, device="cuda") ** 2 - 1
    r = random.Random(case["layout"])
    s["done"] = None
    if case["done"]:
        s["done"] = torch.tensor([[r.random() < 0.25 for _ in range(N)] for _ in range(G)], device="cuda").to(torch.uint8)
    s["pad"] = 2
    K = case["n_select"]
    s["best"] = torch.empty(G, K, device="cuda")
    s["rows"], s["tokens"] = (torch.empty(G, K, dtype=torch.int32, device="cuda") for _ in range(2))
    if own:
        from paged_moe_shared_gb300 import rimuru as R
        _workspace(s, R.rimuru_beam_select_workspace_bytes(G, N, V, K))


def _prepare_reorder(case, gen, s):
    Hk, D, P, n, L, W = (case["kv_heads"], case["dim"], case["page_tokens"], case["seqs"], case["layers"],
                         case["width"])
    page_bytes = 2 * Hk * P * D
    pages = -(-case["pages"] // 16) * 16
    s["scales"] = torch.exp2(torch.randint(-7, -4, (pages, 2, Hk), generator=gen, device="cuda").float())
    if own:
        from paged_moe_shared_gb300 import rimuru as R
        from paged_moe_shared_gb300.device_pool import DevicePool
        s["pool"] = DevicePool(pages * page_bytes, 16 * page_bytes, "cuda")
        mem, s["view"] = s["pool"].mem, s["pool"].view(page_bytes)
        R.rimuru_view_set_kv_shape(s["view"], Hk, D, P, s["scales"].data_ptr(), s["scales"].numel() * 4)
    else:
        mem = torch.empty(pages * page_bytes, dtype=torch.uint8, device="cuda")
    s["codes"] = mem.view(pages, page_bytes)
    for i in range(0, pages, 4096):
        part = s["codes"][i:i + 4096]
        part.copy_(torch.randint(0, 0x7F, part.shape, generator=gen, device="cuda", dtype=torch.uint8))
    parents, lens = _beams(case)
    s["parents"], s["lens"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (parents, lens))
    # full pages are shared in any way; last pages and fresh ones are a sequence's own
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.randint(0, pages, (L, n, W), generator=gen, device="cuda").to(torch.int32)
    table = order[(table % max(1, pages - 2 * L * n)).long()]
    own_pages = order[pages - 2 * L * n:].view(2, L, n)
    used = -(-s["lens"] // P)
    col = torch.arange(W, device="cuda")
    table = torch.where(col == used[:, None] - 1, own_pages[0][..., None], table)
    s["table"] = torch.where(col < used[:, None], table, -1).contiguous()
    s["fresh"] = own_pages[1].contiguous()
    s["table_out"], s["lens_out"] = torch.full_like(s["table"], -1), torch.empty_like(s["lens"])


# ------------------------------------------------------------------ one pass
def run(s):
    return _RUN[s["case"]["op"], bool(own)](s)


def _plain_norm_rope(s):
    case = s["case"]
    rot = case["rot"]
    ang = s["pos"].double()[:, None, None] * s["freq"]
    cos, sin = ang.cos().float(), ang.sin().float()

    def turn(x, w):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * (w.float() + case["offset"])
        a, rest = y[..., :rot], y[..., rot:]
        if case["interleaved"]:
            u, v = a[..., 0::2], a[..., 1::2]
            a = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
        else:
            u, v = a[..., :rot // 2], a[..., rot // 2:]
            a = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
        return torch.cat([a, rest], -1).to(x.dtype)

    return turn(s["q"], s["wq"]), turn(s["k"], s["wk"])


def _own_norm_rope(s):
    from paged_moe_shared_gb300 import rimuru as R
    case = s["case"]
    norms = [R.head_norm_of(w, s["eps"], case["offset"]) for w in (s["wq"], s["wk"])]
    R.rimuru_norm_rope_apply(s["rope"], s["pos"].data_ptr(), case["tokens"], case["dim"],
                             [R.heads_of(s["q"]), R.heads_of(s["k"])],
                             [R.heads_of(s["q_out"]), R.heads_of(s["k_out"])], norms,
                             torch.cuda.current_stream().cuda_stream)
    return s["q_out"], s["k_out"]


def _plain_linear(s):
    """Chunks of 64 tokens: what a chunk's tokens give one another, and what the state before it gives."""
    case = s["case"]
    H, N = case["heads"], s["max_new"]
    i = torch.arange(N, device="cuda")
    live = i < (s["cu"][1:] - s["cu"][:-1])[:, None]                                        # [B, N]
    at = (s["cu"][:-1, None] + i).clamp(max=s["tokens"] - 1).long()
    q, k = (s[x][at].float().repeat_interleave(H // case["key_heads"], 2).transpose(1, 2) for x in "qk")
    v = s["v"][at].float().transpose(1, 2)                                                  # [B, H, N, D]
    k = torch.where(live[:, None, :, None], k, 0.0)
    g = s["g"].expand(s["tokens"], H)[at].transpose(1, 2)
    g = torch.where(live[:, None], g, 0.0).double()
    S = torch.where((s["state_in"] >= 0)[:, None, None, None], s["states"][s["state_in"].clamp(min=0).long()], 0.0)
    outs = []
    for c in range(0, N, 64):
        qc, kc, vc = (x[:, :, c:c + 64] for x in (q, k, v))
        G = g[:, :, c:c + 64].cumsum(-1)
        n = G.shape[-1]
        later = torch.arange(n, device="cuda")[:, None] < torch.arange(n, device="cuda")
        decay = torch.where(later, -math.inf, G[..., :, None] - G[..., None, :]).float().exp()
        outs.append((qc @ kc.transpose(-1, -2) * decay) @ vc + G.float().exp()[..., None] * (qc @ S))
        w = (G[..., -1:] - G).float().exp()
        S = G[..., -1].float().exp()[..., None, None] * S + (kc * w[..., None]).transpose(-1, -2) @ vc
    out = torch.cat(outs, 2).transpose(1, 2)[live] * s["scale"]
    s["states"][s["state_out"].long()] = S
    return out.to(s["v"].dtype), s["states"]


def _own_linear(s):
    from paged_moe_shared_gb300 import rimuru as R
    g = s["g"]
    R.rimuru_linear_attention(s["view"], R.heads_of(s["q"]), R.heads_of(s["k"]), R.heads_of(s["v"]),
                              R.heads_of(s["out"]), g.data_ptr(), g.stride(0) if g.dim() == 2 else 0, g.stride(-1),
                              s["cu"].data_ptr(), s["case"]["seqs"], s["tokens"], s["max_new"],
                              s["state_in"].data_ptr(), s["state_out"].data_ptr(), s["scale"], s["ws_ptr"],
                              s["ws_bytes"], torch.cuda.current_stream().cuda_stream)
    return s["out"], s["states"]


def _plain_select(s):
    case = s["case"]
    G, N, V = case["groups"], case["beams"], case["vocab"]
    x = s["logits"].double().view(G, N, V)
    top = x.amax(-1, keepdim=True)
    x -= top + (x - top).exp().sum(-1, keepdim=True).log()
    x += s["scores"].double()[..., None]
    if s["done"] is not None:
        token = torch.arange(V, device="cuda")
        only = torch.where(token == s["pad"], s["scores"].double()[..., None], -math.inf)
        x = torch.where(s["done"][..., None] != 0, only, x)
    x = x.view(G, N * V)
    best, flat = [], []
    index = torch.arange(N * V, device="cuda")
    for _ in range(case["n_select"]):
        m = x.amax(-1, keepdim=True)
        i = torch.where(x == m, index, N * V).amin(-1, keepdim=True)
        x.scatter_(1, i, -math.inf)
        best.append(m)
        flat.append(torch.where(m == -math.inf, -1, i))
    best, flat = torch.cat(best, 1), torch.cat(flat, 1)
    row = torch.arange(G, device="cuda")[:, None] * N + flat // V
    return (best.float(), torch.where(flat < 0, -1, row).to(torch.int32),
            torch.where(flat < 0, -1, flat % V).to(torch.int32))


def _own_select(s):
    from paged_moe_shared_gb300 import rimuru as R
    case = s["case"]
    R.rimuru_beam_select(R.rows_of(s["logits"]), s["scores"].data_ptr(),
                         0 if s["done"] is None else s["done"].data_ptr(), case["groups"], case["beams"],
                         s["pad"], case["n_select"], s["best"].data_ptr(), s["rows"].data_ptr(),
                         s["tokens"].data_ptr(), s["ws_ptr"], s["ws_bytes"],
                         torch.cuda.current_stream().cuda_stream)
    return s["best"], s["rows"], s["tokens"]


def _plain_reorder(s):
    P = s["case"]["page_tokens"]
    parents = s["parents"].long()
    lens = s["lens"][parents]
    used = -(-lens // P)
    table = s["table"][:, parents]                                                          # [L, n, W]
    last = (torch.arange(s["case"]["width"], device="cuda") == used[:, None] - 1) & (lens % P > 0)[:, None]
    layer, child, col = last.expand_as(table).nonzero(as_tuple=True)
    src, dst = table[layer, child, col].long(), s["fresh"][layer, child].long()
    s["codes"][dst] = s["codes"][src]
    s["scales"][dst] = s["scales"][src]
    table = torch.where(last, s["fresh"][..., None], table)
    keep = torch.arange(s["case"]["width"], device="cuda") < used[:, None]
    s["table_out"].copy_(torch.where(keep, table, s["table_out"]))
    s["lens_out"].copy_(lens)
    return s["table_out"], s["lens_out"], s["codes"], s["scales"]


def _own_reorder(s):
    from paged_moe_shared_gb300 import rimuru as R
    case = s["case"]
    R.rimuru_kv_reorder(s["view"], s["parents"].data_ptr(), case["seqs"], s["lens"].data_ptr(), case["seqs"],
                        s["table"].data_ptr(), s["table_out"].data_ptr(), case["layers"], case["width"],
                        s["fresh"].data_ptr(), s["lens_out"].data_ptr(), torch.cuda.current_stream().cuda_stream)
    return s["table_out"], s["lens_out"], s["codes"], s["scales"]


_RUN = {("norm_rope", False): _plain_norm_rope, ("norm_rope", True): _own_norm_rope,
        ("linear", False): _plain_linear, ("linear", True): _own_linear,
        ("select", False): _plain_select, ("select", True): _own_select,
        ("reorder", False): _plain_reorder, ("reorder", True): _own_reorder}


# ------------------------------------------------------------------ the definitions in fp64
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"norm_rope": _exact_norm_rope, "linear": _exact_linear, "select": _exact_select,
            "reorder": _exact_reorder}[case["op"]](s)


def _exact_norm_rope(s):
    case = s["case"]
    rot, n = case["rot"], case["rot"] // 2
    f = torch.tensor([1e6 ** (-2.0 * i / rot) for i in range(n)], dtype=torch.float64, device="cuda")
    ang = s["pos"].double()[:, None] * f
    turn = torch.polar(torch.ones_like(ang), ang)[:, None]
    got = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.double()
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["dim"] + s["eps"])
        y = y * (w.double() + case["offset"])
        re, im = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, n), slice(n, rot))
        z = torch.complex(y[..., re].contiguous(), y[..., im].contiguous()) * turn
        y[..., re], y[..., im] = z.real, z.imag
        got.append(y)
    return tuple(got)


def _exact_linear(s):
    """All pairs of a sequence's tokens at once, head by head."""
    case = s["case"]
    if sum(n * n for n in _new(case)) * case["heads"] > 1 << 32:
        return None
    per, cu = case["heads"] // case["key_heads"], s["cu"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    states = s["states"].double()
    before, after = s["state_in"].tolist(), s["state_out"].tolist()
    first = {b: states[p].clone() if p >= 0 else torch.zeros_like(states[0]) for b, p in enumerate(before)}
    for b in range(case["seqs"]):
        at = slice(cu[b], cu[b + 1])
        n = cu[b + 1] - cu[b]
        for h in range(case["heads"]):
            q, k, v = s["q"][at, h // per].double(), s["k"][at, h // per].double(), s["v"][at, h].double()
            g = (s["g"][h].expand(n) if case["constant"] else s["g"][at, h]).double()
            total = torch.cumsum(g, 0)
            pair = torch.tril(torch.exp(torch.tril(total[:, None] - total)))
            out[at, h] = s["scale"] * ((pair * (q @ k.T)) @ v + torch.exp(total)[:, None] * (q @ first[b][h]))
            left = torch.exp(total[-1] - total)
            states[after[b], h] = torch.exp(total[-1]) * first[b][h] + k.T @ (left[:, None] * v)
    return out, states


def _exact_select(s):
    case = s["case"]
    G, N, V, K = case["groups"], case["beams"], case["vocab"], case["n_select"]
    best = torch.full((G, K), -math.inf, dtype=torch.float64, device="cuda")
    rows, tokens = (torch.full((G, K), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    for g in range(G):
        x = torch.log_softmax(s["logits"][g * N:(g + 1) * N].double(), -1) + s["scores"][g, :, None].double()
        for b in range(N):
            if s["done"] is not None and s["done"][g, b]:
                x[b] = -math.inf
                x[b, s["pad"]] = s["scores"][g, b].double()
        value, index = torch.sort(x.flatten(), descending=True, stable=True)
        n = min(K, int((value > -math.inf).sum()))
        best[g, :n], rows[g, :n], tokens[g, :n] = value[:n], g * N + index[:n] // V, index[:n] % V
    return best, rows, tokens


def _exact_reorder(s):
    P = s["case"]["page_tokens"]
    parents, lens = s["parents"].tolist(), s["lens"].tolist()
    table, table_out, fresh = s["table"].cpu(), s["table_out"].cpu(), s["fresh"].cpu()
    src, dst = [], []
    for i, p in enumerate(parents):
        full, part = divmod(lens[p], P)
        table_out[:, i, :full] = table[:, p, :full]
        if part:
            src += table[:, p, full].tolist()
            dst += fresh[:, i].tolist()
            table_out[:, i, full] = fresh[:, i]
    codes, scales = s["codes"].clone(), s["scales"].double()
    codes[dst], scales[dst] = codes[src], scales[src]
    return table_out.cuda(), s["lens"][s["parents"].long()], codes, scales
