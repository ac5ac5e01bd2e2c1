"""The attention side of a shared page pool, as cases to measure: rotary positions, the 8-bit
paged key/value cache (append, page copies) and attention over it.

``listed()`` and ``draw()`` give cases, ``prepare()`` makes what a serving loop has in hand
before a call, ``run()`` is one pass: with ``own`` false in elementary torch operations in fp32,
with ``own`` true through the library.  ``exact()`` is the same from the definition in fp64.

The cache: a page holds ``page_tokens`` tokens of one layer as float8 e4m3 codes, laid out
[K, V][kv_heads][page_tokens][head_dim], and a value is its code times the fp32 power-of-two
scale of its (page, K or V, head), kept in scales[page][K, V][kv_heads].  Sequence b's token t is
slot t % page_tokens of page table[b][t // page_tokens].
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
NAN_CODE = 0x7F  # what pool bytes hold that no live token owns


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of one user: q and k of a single token, full rotary width
        dict(name="rope_decode", op="rope", tokens=1, q_heads=32, kv_heads=4, dim=128, rot=128,
             interleaved=False, scaled=False, max_pos=40000, dtype="bf16"),
        # a long prefill chunk: wide heads, a quarter of each rotated, scaled for long contexts
        dict(name="rope_prefill", op="rope", tokens=8192, q_heads=16, kv_heads=2, dim=256, rot=64,
             interleaved=True, scaled=True, max_pos=131072, dtype="bf16"),
        # the cache write of a decode step: one new token for each of 64 running sequences
        dict(name="append_decode", op="append", seqs=64, new_min=1, new_max=1, ctx_min=17,
             ctx_max=4000, kv_heads=4, q_heads=32, dim=128, page_tokens=16, dtype="bf16", layout=1),
        # the cache write of a ragged prefill batch, some of it after cached prefixes
        dict(name="append_prefill", op="append", seqs=7, new_min=301, new_max=2300, ctx_min=1,
             ctx_max=900, kv_heads=2, q_heads=16, dim=256, page_tokens=32, dtype="bf16", layout=2),
        # one user's decode step over a short conversation: latency
        dict(name="attn_decode_one", op="attn", seqs=1, ctx_min=211, ctx_max=211, q_min=1, q_max=1,
             q_heads=32, kv_heads=4, dim=128, page_tokens=16, window=0, dtype="bf16", layout=3),
        # an ordinary decode batch: 64 sequences of very different lengths
        dict(name="attn_decode_batch", op="attn", seqs=64, ctx_min=1, ctx_max=4095, q_min=1, q_max=1,
             q_heads=32, kv_heads=4, dim=128, page_tokens=16, window=0, dtype="bf16", layout=4),
        # two very long contexts, wide heads
        dict(name="attn_decode_long", op="attn", seqs=2, ctx_min=120001, ctx_max=131071, q_min=1,
             q_max=1, q_heads=16, kv_heads=2, dim=256, page_tokens=32, window=0, dtype="bf16",
             layout=5),
        # checking a few drafted tokens for each of 16 sequences
        dict(name="attn_verify", op="attn", seqs=16, ctx_min=900, ctx_max=8000, q_min=3, q_max=5,
             q_heads=32, kv_heads=4, dim=128, page_tokens=16, window=0, dtype="bf16", layout=6),
        # one 2048-token chunk of a long prompt, after 6144 cached tokens
        dict(name="attn_prefill_chunk", op="attn", seqs=1, ctx_min=6144, ctx_max=6144, q_min=2048,
             q_max=2048, q_heads=32, kv_heads=4, dim=128, page_tokens=16, window=0, dtype="bf16",
             layout=7),
        # fresh ragged prompts, wide heads, a sliding window
        dict(name="attn_prefill_ragged", op="attn", seqs=6, ctx_min=0, ctx_max=0, q_min=35,
             q_max=1733, q_heads=16, kv_heads=2, dim=256, page_tokens=32, window=1024, dtype="bf16",
             layout=8),
        # beams forked: their partly filled last pages are copied
        dict(name="pages_fork", op="pages", copies=24, pages=4096, kv_heads=4, dim=128,
             page_tokens=16),
        # a compaction before pages return to the experts: 64 MiB of live pages move
        dict(name="pages_compact", op="pages", copies=2048, pages=5000, kv_heads=2, dim=256,
             page_tokens=32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kv_heads, dim, page_tokens = rng.choice([(4, 128, 16), (2, 256, 32), (2, 256, 16), (8, 128, 16),
                                             (1, 128, 64), (8, 64, 32)])
    group = rng.choice([1, 4, 7, 8, 8, 8])
    base = dict(kv_heads=kv_heads, dim=dim)
    dtype = rng.choice(["bf16", "bf16", "f16"])
    op = rng.choice(["rope", "append", "attn", "attn", "attn", "attn", "pages"])
    if op == "rope":
        return dict(base, op=op, tokens=_log_int(rng, 1, 8192), q_heads=group * kv_heads // 2 or 1,
                    rot=rng.choice([dim, dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.5,
                    scaled=rng.random() < 0.5, max_pos=_log_int(rng, 8192, 131072), dtype=dtype)
    if op == "pages":
        copies = _log_int(rng, 1, 2048)
        return dict(base, op=op, copies=copies, pages=2 * copies + rng.randrange(1, 500),
                    page_tokens=page_tokens)
    base.update(page_tokens=page_tokens, q_heads=group * kv_heads, dtype=dtype,
                layout=rng.randrange(1 << 20))
    if op == "append":
        seqs = _log_int(rng, 1, 128)
        new = 1 if rng.random() < 0.4 else _log_int(rng, 2, max(2, 8192 // seqs))
        return dict(base, op=op, seqs=seqs, new_min=max(1, new // 3), new_max=new, ctx_min=0,
                    ctx_max=rng.randrange(1, 1500))
    window = rng.choice([0, 0, 0, _log_int(rng, 100, 5000)])
    kind = rng.choice(["decode", "decode", "verify", "prefill"])
    if kind == "decode":
        seqs = _log_int(rng, 1, 128)
        ctx = _log_int(rng, 2, max(2, min(131072, (1 << 27) // (seqs * kv_heads * dim))))
        return dict(base, op=op, seqs=seqs, ctx_min=max(1, ctx // 20), ctx_max=ctx, q_min=1, q_max=1,
                    window=window)
    if kind == "verify":
        seqs, q = _log_int(rng, 1, 32), rng.randrange(2, 17)
        ctx = _log_int(rng, 2, 16384 // (1 + seqs // 8))
        return dict(base, op=op, seqs=seqs, ctx_min=max(1, ctx // 5), ctx_max=ctx, q_min=max(1, q - 3),
                    q_max=q, window=window)
    seqs = _log_int(rng, 1, 8)
    q = _log_int(rng, 32, 4096 // seqs)
    most = (1 << 29) // (seqs * q * group * kv_heads)  # fp32 scores of the plain form
    ctx = rng.choice([0, rng.randrange(1, max(2, min(8192, most - q)))])
    return dict(base, op=op, seqs=seqs, ctx_min=ctx // 2, ctx_max=ctx, q_min=max(1, q // 6), q_max=q,
                window=window)


def _lens(case):
    """[(tokens in the cache before the pass, new tokens)] of each sequence, by the case alone."""
    r = random.Random(case["layout"])
    lo, hi = (case["new_min"], case["new_max"]) if case["op"] == "append" else (case["q_min"], case["q_max"])
    got = []
    for _ in range(case["seqs"]):
        new = r.randint(lo, hi)
        c0, c1 = case["ctx_min"], case["ctx_max"]
        ctx = r.randint(c0, c1) if c0 < 1 or case["op"] == "append" else _log_int(r, c0, c1)
        if case["op"] == "attn" and hi == 1:  # a decode step's own token is the last one cached
            ctx = max(0, ctx - 1)
        got.append((ctx, new))
    return got


def _visible(case):
    """Query-key pairs of all sequences (one head)."""
    n = 0
    w = case["window"] or 1 << 60
    for ctx, new in _lens(case):
        # query i sees min(ctx + i + 1, w) keys
        full = max(0, min(new, w - ctx))  # queries whose window is not yet full
        n += full * ctx + full * (full + 1) // 2 + (new - full) * w if full < new else \
            new * ctx + new * (new + 1) // 2
    return n


def work(case):
    """Bytes that have to be read and written once, and multiply-adds as two operations."""
    D, Hk = case["dim"], case["kv_heads"]
    if case["op"] == "rope":
        elems = case["tokens"] * (case["q_heads"] + Hk) * D
        return {"bytes": elems * 4 + case["tokens"] * 4, "flops": 3 * case["tokens"] *
                (case["q_heads"] + Hk) * case["rot"]}
    if case["op"] == "pages":
        return {"bytes": case["copies"] * (4 * case["page_tokens"] * Hk * D + 16 * Hk + 8), "flops": 0}
    lens = _lens(case)
    if case["op"] == "append":
        new = sum(n for _, n in lens)
        return {"bytes": new * Hk * D * 2 * (2 + 1), "flops": new * Hk * D * 4}
    w = case["window"] or 1 << 60
    rows = sum(n for _, n in lens) * case["q_heads"]
    keys = sum(min(ctx + n, w + n - 1) for ctx, n in lens)
    return {"bytes": rows * D * 4 + keys * Hk * D * 2, "flops": 4 * _visible(case) * case["q_heads"] * D}


# ------------------------------------------------------------------ inputs
def _rope_params(case):
    return dict(rot=case["rot"], interleaved=case["interleaved"], base=1e6,
                factor=4.0 if case["scaled"] else 1.0, orig_len=32768, low=1.0, high=32.0)


def _inv_freq(p):
    """Angle per position of each pair, and the factor on the rotated part: base^(-2i/rot); scaled,
    a pair that turns fewer than `low` times over orig_len positions is slowed by `factor`, one that
    turns more than `high` times is kept, with a linear ramp in between."""
    f = [p["base"] ** (-2.0 * i / p["rot"]) for i in range(p["rot"] // 2)]
    if p["factor"] == 1.0:
        return f, 1.0
    got = []
    for x in f:
        keep = min(1.0, max(0.0, (p["orig_len"] * x / (2 * math.pi) - p["low"]) / (p["high"] - p["low"])))
        got.append((1 - keep) * x / p["factor"] + keep * x)
    return got, 0.1 * math.log(p["factor"]) + 1.0


class _Pool:
    """Pages of one pool and their scales; with `own` also the library's pool and view."""

    def __init__(self, case, pages):
        self.page_bytes = 2 * case["kv_heads"] * case["page_tokens"] * case["dim"]
        huge = 16 * self.page_bytes
        self.pages = -(-pages // 16) * 16
        nbytes = self.pages * self.page_bytes
        self.shape = (self.pages, 2, case["kv_heads"], case["page_tokens"], case["dim"])
        self.scales = torch.ones(self.shape[:3], dtype=torch.float32, device="cuda")
        self.view = None
        if own:
            from paged_moe_shared_gb300 import rimuru as R
            from paged_moe_shared_gb300.device_pool import DevicePool
            self.pool = DevicePool(nbytes, huge, "cuda")
            self.mem = self.pool.mem
            self.view = self.pool.view(self.page_bytes)
            R.rimuru_view_set_kv_shape(self.view, case["kv_heads"], case["dim"], case["page_tokens"],
                                       self.scales.data_ptr(), self.scales.numel() * 4)
        else:
            self.mem = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        self.mem.fill_(NAN_CODE)
        self.codes = self.mem.view(torch.float8_e4m3fn).view(self.shape)

    def fill(self, ids, gen):
        """Normal values with a power-of-two spread of scales in the pages `ids`."""
        shape = (256,) + self.shape[1:]
        for i in range(0, ids.numel(), 256):
            at = ids[i:i + 256]
            n = at.numel()
            x = torch.randn(shape, generator=gen, device="cuda")[:n] * 64
            self.codes.view(torch.uint8)[at] = x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            k = torch.randint(-7, -4, (n,) + self.shape[1:3], generator=gen, device="cuda")
            self.scales[at] = torch.exp2(k.float())


def _sequences(case, gen, s):
    """Lengths, the page table and a pool whose pages hold the cached tokens; slots that no token
    owns keep the NaN code."""
    lens = _lens(case)
    P = case["page_tokens"]
    n_pages = [-(-(c + n) // P) for c, n in lens]
    width = max(n_pages) + 3
    s["pool"] = pool = _Pool(case, sum(n_pages) + 8)
    order = torch.randperm(pool.pages, generator=gen, device="cuda").to(torch.int32)
    first = torch.tensor([sum(n_pages[:i]) for i in range(len(lens))], device="cuda")
    count = torch.tensor(n_pages, device="cuda")
    col = torch.arange(width, device="cuda")
    at = (first[:, None] + col).clamp(max=pool.pages - 1)
    s["table"] = torch.where(col < count[:, None], order[at], -1).to(torch.int32).contiguous()
    live = torch.tensor([c if case["op"] == "append" else c + n for c, n in lens], device="cuda")
    used = order[:sum(n_pages)].long()
    pool.fill(used, gen)
    # slots past the live tokens of each sequence
    slot = torch.arange(P, device="cuda")
    dead = (col[None, :width, None] * P + slot >= live[:, None, None])[col.expand(len(lens), -1) < count[:, None]]
    page, slot = dead.nonzero(as_tuple=True)
    pool.codes.view(torch.uint8)[used[page], :, :, slot] = NAN_CODE
    new = torch.tensor([0] + [n for _, n in lens]).cumsum(0)
    s["cu"] = new.to(torch.int32).cuda()
    s["lens"] = torch.tensor([c + n for c, n in lens], dtype=torch.int32, device="cuda")
    s["tokens"] = int(new[-1])
    s["max_new"] = max(n for _, n in lens)
    s["max_len"] = max(c + n for c, n in lens)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    D, Hk, Hq = case["dim"], case["kv_heads"], case.get("q_heads", 0)
    if case["op"] == "pages":
        pool = s["pool"] = _Pool(case, case["pages"])
        order = torch.randperm(pool.pages, generator=gen, device="cuda").to(torch.int32)
        s["src"], s["dst"] = order[:case["copies"]].clone(), order[case["copies"]:2 * case["copies"]].clone()
        pool.fill(torch.arange(pool.pages, device="cuda"), gen)
        return s
    dt = DTYPES[case["dtype"]]
    if case["op"] == "rope":
        T = case["tokens"]
        qkv = torch.randn((T, (Hq + 2 * Hk) * D), generator=gen, device="cuda").to(dt)
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["pos"] = torch.randint(0, case["max_pos"], (T,), generator=gen, device="cuda").to(torch.int32)
        p = _rope_params(case)
        freq, s["mscale"] = _inv_freq(p)
        s["freq"] = torch.tensor(freq, dtype=torch.float32, device="cuda")
        s["q_out"], s["k_out"] = torch.empty(T, Hq, D, dtype=dt, device="cuda"), torch.empty(T, Hk, D, dtype=dt, device="cuda")
        if own:
            from paged_moe_shared_gb300 import rimuru as R
            s["rope"] = R.rimuru_rope_create(
                p["rot"], R.ROPE_INTERLEAVED if p["interleaved"] else R.ROPE_HALF, p["base"],
                R.ROPE_BY_PARTS if case["scaled"] else R.ROPE_PLAIN, p["factor"], p["orig_len"],
                p["low"], p["high"], s["mscale"])
        return s
    _sequences(case, gen, s)
    T = s["tokens"]
    qkv = torch.randn((T, (Hq + 2 * Hk) * D), generator=gen, device="cuda")
    if case["op"] == "append":
        # a few channels carry much larger values, as keys do
        loud = 1 + 7 * (torch.rand((Hq + 2 * Hk) * D, generator=gen, device="cuda") < 0.02).float()
        qkv = (qkv * loud).to(dt)
        s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["v"] = qkv[:, (Hq + Hk) * D:].view(T, Hk, D)
        return s
    s["q"] = qkv.to(dt)[:, :Hq * D].view(T, Hq, D)
    s["out"] = torch.empty(T, Hq, D, dtype=dt, device="cuda")
    s["scale"] = D ** -0.5
    if own:
        from paged_moe_shared_gb300 import rimuru as R
        nbytes = R.rimuru_kv_attention_workspace_bytes(s["pool"].view, Hq, case["seqs"], T, s["max_new"])
        s["ws"] = torch.empty(nbytes + 1024, dtype=torch.uint8, device="cuda")
        s["ws_ptr"], s["ws_bytes"] = (s["ws"].data_ptr() + 1023) // 1024 * 1024, nbytes
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _RUN[s["case"]["op"], bool(own)](s)


def _plain_rope(s):
    case = s["case"]
    rot = case["rot"]
    ang = s["pos"].float()[:, None, None] * s["freq"]
    cos, sin = ang.cos() * s["mscale"], ang.sin() * s["mscale"]

    def turn(x):
        a, rest = x[..., :rot].float(), x[..., rot:].float()
        if case["interleaved"]:
            u, v = a[..., 0::2], a[..., 1::2]
            a = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
        else:
            u, v = a[..., :rot // 2], a[..., rot // 2:]
            a = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
        return torch.cat([a, rest], -1).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _own_rope(s):
    from paged_moe_shared_gb300 import rimuru as R
    R.rimuru_rope_apply(s["rope"], s["pos"].data_ptr(), s["case"]["tokens"], s["case"]["dim"],
                        [R.heads_of(s["q"]), R.heads_of(s["k"])],
                        [R.heads_of(s["q_out"]), R.heads_of(s["k_out"])],
                        torch.cuda.current_stream().cuda_stream)
    return s["q_out"], s["k_out"]


def _places(s):
    """Sequence, position, page and slot of each new token."""
    t = torch.arange(s["tokens"], dtype=torch.int32, device="cuda")
    b = torch.searchsorted(s["cu"], t, right=True) - 1
    pos = s["lens"][b] - s["cu"][b + 1] + t
    P = s["case"]["page_tokens"]
    return b, pos, s["table"][b, pos // P].long(), (pos % P).long()


def _plain_append(s):
    pool, case = s["pool"], s["case"]
    b, pos, page, slot = _places(s)
    x = torch.stack([s["k"], s["v"]], 1).float()                                 # [T, 2, Hk, D]
    shape = pool.scales.shape
    at = page[:, None, None].expand(-1, *shape[1:])
    amax = torch.zeros(shape, device="cuda").scatter_reduce_(0, at, x.abs().amax(-1), "amax")
    m, e = torch.frexp(amax)                                                     # 448 = 0.875 * 2^9
    want = torch.exp2(torch.where(amax > 0, e - 9 + (m > 0.875).int(), -60).clamp(-60, 60).float())
    first = torch.full((pool.pages,), case["page_tokens"], device="cuda").scatter_reduce_(0, page, slot, "amin")
    new = torch.where((first > 0)[:, None, None], torch.maximum(pool.scales, want), want)
    hit = first < case["page_tokens"]
    ids = hit.nonzero()[:, 0]
    old = pool.codes[ids].float() * (pool.scales[ids] / new[ids])[..., None, None]
    kept = torch.arange(case["page_tokens"], device="cuda") < first[ids][:, None]
    codes = pool.codes.view(torch.uint8)
    codes[ids] = torch.where(kept[:, None, None, :, None], old.to(torch.float8_e4m3fn).view(torch.uint8), codes[ids])
    pool.scales.copy_(torch.where(hit[:, None, None], new, pool.scales))
    y = (x / new[page][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[page, :, :, slot] = y
    return pool.codes, pool.scales


def _own_append(s):
    from paged_moe_shared_gb300 import rimuru as R
    pool = s["pool"]
    R.rimuru_kv_append(pool.view, R.heads_of(s["k"]), R.heads_of(s["v"]), s["cu"].data_ptr(),
                       s["lens"].data_ptr(), s["case"]["seqs"], s["tokens"], s["table"].data_ptr(),
                       s["table"].stride(0), torch.cuda.current_stream().cuda_stream)
    return pool.codes, pool.scales


def _plain_attn(s):
    case, pool = s["case"], s["pool"]
    B, Hk, D, P, N = case["seqs"], case["kv_heads"], case["dim"], case["page_tokens"], s["max_new"]
    G, L = case["q_heads"] // Hk, s["max_len"]
    ids = s["table"][:, :-(-L // P)].clamp(min=0).long()
    kv = pool.codes[ids].float() * pool.scales[ids][..., None, None]             # [B, M, 2, Hk, P, D]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, B, Hk, -1, D)[..., :L, :]
    j = torch.arange(L, device="cuda")
    live = j < s["lens"][:, None]                                                # [B, L]
    v = torch.where(live[:, None, :, None], kv[1], 0.0)
    i = torch.arange(N, device="cuda")
    count = s["cu"][1:] - s["cu"][:-1]
    q = s["q"][(s["cu"][:-1, None] + i).clamp(max=s["tokens"] - 1).long()].float()  # [B, N, Hq, D]
    q = q.view(B, N, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * N, D)
    x = (q @ kv[0].transpose(-1, -2)).view(B, Hk, G, N, L)
    last = (s["lens"] - count)[:, None] + i                                      # [B, N]
    see = (j <= last[..., None]) & live[:, None]
    if case["window"]:
        see &= j > last[..., None] - case["window"]
    x = torch.where(see[:, None, None], x * s["scale"], -math.inf)
    x -= x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = x.exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hk, G * N, L) @ v).view(B, Hk, G, N, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B, N, Hk * G, D)
    return o[i < count[:, None]].to(s["q"].dtype)


def _own_attn(s):
    from paged_moe_shared_gb300 import rimuru as R
    case = s["case"]
    R.rimuru_kv_attention(s["pool"].view, R.heads_of(s["q"]), R.heads_of(s["out"]), 0,
                          s["cu"].data_ptr(), s["lens"].data_ptr(), case["seqs"], s["tokens"],
                          s["max_new"], s["table"].data_ptr(), s["table"].stride(0), s["scale"],
                          case["window"], s["ws_ptr"], s["ws_bytes"],
                          torch.cuda.current_stream().cuda_stream)
    return s["out"]


def _plain_pages(s):
    pool = s["pool"]
    codes = pool.codes.view(torch.uint8)
    src, dst = s["src"].long(), s["dst"].long()
    codes[dst] = codes[src]
    pool.scales[dst] = pool.scales[src]
    return codes, pool.scales


def _own_pages(s):
    from paged_moe_shared_gb300 import rimuru as R
    R.rimuru_kv_copy_pages(s["pool"].view, s["src"].data_ptr(), s["dst"].data_ptr(),
                           s["case"]["copies"], torch.cuda.current_stream().cuda_stream)
    return s["pool"].codes.view(torch.uint8), s["pool"].scales


_RUN = {("rope", False): _plain_rope, ("rope", True): _own_rope,
        ("append", False): _plain_append, ("append", True): _own_append,
        ("attn", False): _plain_attn, ("attn", True): _own_attn,
        ("pages", False): _plain_pages, ("pages", True): _own_pages}


# ------------------------------------------------------------------ the definition in fp64
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"rope": _exact_rope, "append": _exact_append, "attn": _exact_attn, "pages": _exact_pages}[case["op"]](s)


def _exact_rope(s):
    case = s["case"]
    rot, n = case["rot"], case["rot"] // 2
    freq, m = _inv_freq(_rope_params(case))
    turn = torch.polar(torch.full((case["tokens"], n), m, dtype=torch.float64, device="cuda"),
                       s["pos"].double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda"))
    got = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        re, im = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, n), slice(n, rot))
        z = torch.complex(y[..., re].contiguous(), y[..., im].contiguous()) * turn[:, None]
        y[..., re], y[..., im] = z.real, z.imag
        got.append(y)
    return tuple(got)


def _exact_append(s):
    """The codes' places hold the unrounded quotients of values and scales."""
    pool, case = s["pool"], s["case"]
    P, codes, scales = case["page_tokens"], pool.codes.double(), pool.scales.double()
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    for b in range(case["seqs"]):
        start = lens[b] - (cu[b + 1] - cu[b])
        for c in range(start // P, -(-lens[b] // P)):
            lo, hi = max(start, c * P), min(lens[b], (c + 1) * P)
            page, a = table[b][c], cu[b] + lo - start
            x = torch.stack([s["k"][a:a + hi - lo], s["v"][a:a + hi - lo]]).double().transpose(1, 2)  # [2, Hk, n, D]
            top = x.abs().amax((-1, -2))
            k = torch.ceil(torch.log2(top / 448))
            want = torch.where(top > 0, torch.exp2(k.clamp(-60, 60)), 2.0 ** -60)
            if lo > c * P:
                new = torch.maximum(scales[page], want)
                codes[page, :, :, :lo - c * P] *= (scales[page] / new)[..., None, None]
            else:
                new = want
            scales[page] = new
            codes[page, :, :, lo - c * P:hi - c * P] = x / new[..., None, None]
    return codes, scales


def _exact_attn(s):
    case, pool = s["case"], s["pool"]
    Hk, P = case["kv_heads"], case["page_tokens"]
    G = case["q_heads"] // Hk
    if _visible(case) * case["q_heads"] * case["dim"] > 1 << 39:
        return None
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["seqs"]):
        L, n = lens[b], cu[b + 1] - cu[b]
        ids = s["table"][b, :-(-L // P)].long()
        for h in range(Hk):
            kv = pool.codes[ids][:, :, h].double() * pool.scales[ids][:, :, h, None, None].double()
            k, v = (kv[:, w].reshape(-1, case["dim"])[:L] for w in (0, 1))
            i, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")
            hide = (j > i) | ((i - j >= case["window"]) if case["window"] else False)
            for g in range(G):
                x = s["q"][cu[b]:cu[b + 1], h * G + g].double() @ k.T * s["scale"]
                out[cu[b]:cu[b + 1], h * G + g] = torch.softmax(x.masked_fill(hide, -math.inf), -1) @ v
    return out


def _exact_pages(s):
    scales = s["pool"].scales.double()
    scales[s["dst"].long()] = scales[s["src"].long()]
    codes = s["pool"].codes.view(torch.uint8).clone()
    codes[s["dst"].long()] = codes[s["src"].long()]
    return codes, scales
