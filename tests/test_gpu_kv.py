"""Rotary positions, the 8-bit paged cache and attention over it, against 64-bit restatements."""
import math

import numpy as np
import pytest
import torch

import kv_reference as ref
from kv_reference import DEV, DT, HALF_ULP, Cache
from paged_moe_shared_gb300 import rimuru as R

pytestmark = pytest.mark.gpu


def stream():
    return torch.cuda.current_stream().cuda_stream


def qkv(T, heads, dim, dtype, seed, slack=0):
    """Arrays of one fused projection: slices with the fused row's stride."""
    g = torch.Generator().manual_seed(seed)
    row = sum(heads) * dim + slack
    x = torch.randn(T, row, generator=g).to(DT[dtype]).to(DEV)
    got, at = [], 0
    for h in heads:
        got.append(x[:, at:at + h * dim].unflatten(1, (h, dim)))
        at += h * dim
    return got


# ------------------------------------------------------------------ rope
ROPES = [
    dict(rot=128, interleaved=False, scaling=R.ROPE_PLAIN),
    dict(rot=64, interleaved=False, scaling=R.ROPE_LINEAR, factor=3.0),
    dict(rot=64, interleaved=True, scaling=R.ROPE_BASE, factor=8.0),
    dict(rot=16, interleaved=False, scaling=R.ROPE_BY_PARTS, factor=4.0, orig_len=4096.0, low=1.0, high=32.0),
    dict(rot=8, interleaved=True, scaling=R.ROPE_PLAIN),
]


def make_rope(c, mscale=1.0, base=500000.0):
    h = R.rimuru_rope_create(c["rot"], R.ROPE_INTERLEAVED if c["interleaved"] else R.ROPE_HALF, base,
                             c["scaling"], c.get("factor", 1.0), c.get("orig_len", 0.0),
                             c.get("low", 0.0), c.get("high", 0.0), mscale)
    f = ref.inv_freq(c["rot"], base, c["scaling"], c.get("factor", 1.0), c.get("orig_len", 0.0),
                     c.get("low", 0.0), c.get("high", 0.0))
    return h, f


def check_rope(x, y, pos, c, f, mscale, dtype):
    want = ref.rope(x, pos, f, c["interleaved"], mscale)
    # fp32: the angle (below pi) is rounded once, cosine and sine to an ulp or two, two products and
    # a sum: 5e-7 of |u| + |v|; the reference's own fp64 product loses at most 2^31 * 2^-53 * 2 pi
    n = c["rot"] // 2
    a = np.abs(x.double().cpu().numpy())
    iu, iv = (np.arange(n) * 2, np.arange(n) * 2 + 1) if c["interleaved"] else (np.arange(n), np.arange(n) + n)
    pair = np.zeros_like(a)
    pair[..., iu] = pair[..., iv] = a[..., iu] + a[..., iv]
    big = float(pos.abs().max()) if pos.numel() else 0.0
    tol = HALF_ULP[dtype] * np.abs(want) + (5e-7 + big * 2.0 ** -51) * abs(mscale) * pair
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= tol + 1e-30 + (6e-8 if dtype == "f16" else 0)).all(), float((err - tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("c", ROPES, ids=lambda c: f"r{c['rot']}{'i' if c['interleaved'] else 'h'}s{c['scaling']}")
@pytest.mark.parametrize("T,heads,dim", [(1, (4, 1), 128), (37, (7, 2), 256), (3, (33, 5), 136)])
def test_rope_matches_the_rotation(c, dtype, T, heads, dim):
    h, f = make_rope(c, mscale=1.25)
    q, k = qkv(T, heads, dim, dtype, seed=T + dim, slack=16)
    pos = torch.randint(0, 200000, (T,), generator=torch.Generator().manual_seed(5)).to(torch.int32).to(DEV)
    outs = [torch.empty(x.shape, dtype=x.dtype, device=DEV) for x in (q, k)]
    R.rimuru_rope_apply(h, pos.data_ptr(), T, dim, [R.heads_of(q), R.heads_of(k)],
                        [R.heads_of(o) for o in outs], stream())
    for x, y in zip((q, k), outs):
        check_rope(x, y, pos, c, f, 1.25, dtype)
    # in place gives the same bits, and leaves what lies beside the heads alone
    want = [o.clone() for o in outs]
    R.rimuru_rope_apply(h, pos.data_ptr(), T, dim, [R.heads_of(q), R.heads_of(k)],
                        [R.heads_of(q), R.heads_of(k)], stream())
    for x, y in zip((q, k), want):
        assert torch.equal(x, y)
    R.rimuru_rope_destroy(h)


def test_rope_at_extreme_positions_and_back():
    c = ROPES[0]
    h, f = make_rope(c)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 24, -(1 << 24) - 1], dtype=torch.int32, device=DEV)
    T = pos.numel()
    (q,) = qkv(T, (3,), 128, "f32", 1)
    out, back = torch.empty_like(q.contiguous()), torch.empty_like(q.contiguous())
    R.rimuru_rope_apply(h, pos.data_ptr(), T, 128, [R.heads_of(q)], [R.heads_of(out)], stream())
    check_rope(q, out, pos, c, f, 1.0, "f32")
    assert torch.equal(out[0], q[0])  # position 0 turns nothing
    neg = torch.where(pos == -2 ** 31, pos, -pos)  # int32 cannot negate -2^31: leave it out below
    R.rimuru_rope_apply(h, neg.data_ptr(), T, 128, [R.heads_of(out)], [R.heads_of(back)], stream())
    keep = (pos != -2 ** 31).cpu()
    # there and back: two rotations of 5e-7 (|u| + |v|) each, |u| + |v| below 2 * max
    assert (back.cpu()[keep] - q.cpu()[keep]).abs().max() <= 4 * 5e-7 * 2 * q.abs().max().item()
    R.rimuru_rope_destroy(h)


def test_rope_heads_outer_and_a_side_stream():
    c = ROPES[0]
    h, f = make_rope(c)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(5, 9, 128, generator=g).bfloat16().to(DEV).transpose(0, 1)  # [9 tokens, 5 heads]
    pos = torch.arange(9, dtype=torch.int32, device=DEV) * 1001
    out = torch.empty(9, 5, 128, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    R.rimuru_rope_apply(h, pos.data_ptr(), 9, 128, [R.heads_of(x)], [R.heads_of(out)], side.cuda_stream)
    side.synchronize()
    check_rope(x, out, pos, c, f, 1.0, "bf16")
    R.rimuru_rope_apply(h, 0, 0, 128, [R.heads_of(x)], [R.heads_of(out)], stream())  # no tokens
    R.rimuru_rope_destroy(h)


# ------------------------------------------------------------------ append
def run_append(c, k, v, cu, lens, table, expect=R.DEV_OK, s=None):
    cu_t = torch.tensor(cu, dtype=torch.int32, device=DEV)
    lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
    R.rimuru_kv_append(c.view, R.heads_of(k), R.heads_of(v), cu_t.data_ptr(), lens_t.data_ptr(),
                       len(lens), k.shape[0], table.data_ptr(), table.stride(0), s or stream())
    torch.cuda.synchronize()
    assert R.rimuru_get_device_error(c.view, clear=True) == expect


def same_cache(c, values, scales):
    got = c.values().numpy()
    np.testing.assert_array_equal(c.scales.cpu().double().numpy(), scales)
    np.testing.assert_array_equal(got, values)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hk,D,P", [(4, 128, 16), (2, 256, 32), (1, 64, 64), (5, 128, 32)])
def test_append_is_the_rounding_it_says(dtype, Hk, D, P):
    """Prefixes of every alignment, then more tokens of other magnitudes, to the last bit."""
    before, new = [0, 1, P - 1, P, 2 * P + 3, 0, 5], [1, 2 * P, 1, P, 3, 0, P - 5]
    c = Cache(Hk, D, P, 40)
    lens = [a + b for a, b in zip(before, new)]
    table = c.tables(lens, seed=1)
    values, scales = c.values().numpy(), c.scales.cpu().double().numpy()
    t = table.cpu().numpy()
    for step, (counts, upto, amp) in enumerate([(before, before, 1.0), (new, lens, 37.0)]):
        cu = [0] + list(np.cumsum(counts))
        _, k, v = qkv(cu[-1], (3, Hk, Hk), D, dtype, seed=step, slack=64)
        k, v = k * amp, v * (amp / 100)
        k[:, :, :3] *= 1e-4 if dtype == "f16" else 1e-9  # codes down into the subnormals and zero
        run_append(c, k, v, cu, upto, table)
        ref.append(values, scales, t, cu, upto, k, v, P)
        same_cache(c, values, scales)
    c.close()


def test_append_at_the_edges_of_the_scale_rule():
    """Magnitudes on and just past 448 * 2^k, zeros, the smallest and the largest scales."""
    c = Cache(1, 64, 16, 16)
    amps = [448.0, 449.0, 447.0, 448.0 * 2 ** -20, 0.0, 2.0 ** -100, 2.0 ** 100, 3e38, 1.0, 2.0 ** -66 * 448]
    lens = [1] * len(amps)
    table = c.tables(lens, seed=3)
    k = torch.zeros(len(amps), 1, 64, device=DEV)
    k[:, 0, 7] = torch.tensor(amps, device=DEV)
    k[:, 0, 9] = -torch.tensor(amps, device=DEV) / 3
    values, scales = c.values().numpy(), c.scales.cpu().double().numpy()
    cu = list(range(len(amps) + 1))
    run_append(c, k, -k, cu, lens, table)
    ref.append(values, scales, table.cpu().numpy(), cu, lens, k, -k, 16)
    same_cache(c, values, scales)
    c.close()


def test_append_stores_finite_values_only():
    c = Cache(2, 128, 16, 8)
    table = c.tables([5], seed=2)
    _, k, v = qkv(5, (1, 2, 2), 128, "bf16", 4)
    k, v = k.clone(), v.clone()
    k[1, 0, 3], k[2, 1, 4], v[0, 0, 0] = float("nan"), float("inf"), -float("inf")
    values, scales = c.values().numpy(), c.scales.cpu().double().numpy()
    run_append(c, k, v, [0, 5], [5], table, expect=R.DEV_NONFINITE)
    ref.append(values, scales, table.cpu().numpy(), [0, 5], [5], k, v, 16)
    same_cache(c, values, scales)
    c.close()


def test_append_touches_nothing_on_bad_tables():
    c = Cache(2, 128, 16, 8)
    _, k, v = qkv(20, (1, 2, 2), 128, "bf16", 4)
    table = c.tables([20], seed=2)
    before = c.pool.mem.clone()
    for bad, err in (((0, c.pages), R.DEV_BAD_PAGE), ((0, -5), R.DEV_BAD_PAGE)):
        t = table.clone()
        t[:, :2] = bad[1]
        run_append(c, k, v, [0, 20], [20], t, expect=err)
    run_append(c, k, v, [0, 20], [16 * table.shape[1] + 1], table, expect=R.DEV_BAD_SHAPE)
    run_append(c, k, v, [0, 20], [19], table, expect=R.DEV_BAD_SHAPE)  # fewer tokens than new ones
    assert torch.equal(before, c.pool.mem)
    c.close()


def test_append_many_sequences_of_one_token():
    c = Cache(4, 128, 16, 304)
    lens = [1 + 7 * i % 40 for i in range(150)]
    table = c.tables(lens, seed=9)
    old = [n - 1 for n in lens]
    c.fill(table, old, seed=1)
    values, scales = c.values().numpy(), c.scales.cpu().double().numpy()
    _, k, v = qkv(150, (4, 4, 4), 128, "bf16", 8)
    cu = list(range(151))
    run_append(c, k, v, cu, lens, table)
    ref.append(values, scales, table.cpu().numpy(), cu, lens, k, v, 16)
    same_cache(c, values, scales)
    c.close()


# ------------------------------------------------------------------ attention
def run_attention(c, q, cu, lens, table, scale=None, window=0, lse=True, max_q=None, expect=R.DEV_OK,
                  out=None, s=None):
    rows, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    out = torch.full((rows, Hq, D), float("nan"), dtype=q.dtype, device=DEV) if out is None else out
    st = torch.full((rows, Hq), float("nan"), device=DEV) if lse else None
    cu_t = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if max_q is None:
        max_q = 1 if cu is None else max(b - a for a, b in zip(cu, cu[1:]))
    n = R.rimuru_kv_attention_workspace_bytes(c.view, Hq, len(lens), rows, max_q)
    ws = torch.full((n + 1024,), 0xFF, dtype=torch.uint8, device=DEV)
    at = (ws.data_ptr() + 1023) // 1024 * 1024
    torch.cuda.synchronize()
    R.rimuru_kv_attention(c.view, R.heads_of(q), R.heads_of(out), st.data_ptr() if lse else 0,
                          0 if cu is None else cu_t.data_ptr(), lens_t.data_ptr(), len(lens), rows,
                          max_q, table.data_ptr(), table.stride(0), scale, window, at, n, s or stream())
    torch.cuda.synchronize()
    assert R.rimuru_get_device_error(c.view, clear=True) == expect
    return out, st


def check_attention(c, q, cu, lens, table, dtype, scale=None, window=0, **kw):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out, st = run_attention(c, q, cu, lens, table, scale, window, **kw)
    want, lse, mag, top = ref.attention(c.values(), table.cpu().numpy(), lens, q, cu, scale, window, c.P)
    # Scores: products of few-bit factors are exact in fp32, so a score is off by the roundings of
    # its sum, below 2^-17 of sum |q k|; a softmax weight is off by twice that, and weights keep at
    # least 11 bits where they meet V (2^-11 of sum p |v|, the same again for what a tile flushes);
    # the result is rounded once to its type.
    tol = HALF_ULP[dtype] * want.abs() + (2.0 ** -10 + 2.0 ** -16 * top[..., None]) * mag + 1e-7
    err = (out.double().cpu() - want).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))
    if st is not None:
        got = st.double().cpu()
        assert torch.equal(torch.isinf(got), torch.isinf(lse))
        live = torch.isfinite(lse)
        assert ((got - lse).abs()[live] <= (2.0 ** -17 * top + 2.0 ** -16)[live]).all()
    return out, st


SHAPES = [(4, 8, 128, 16), (2, 8, 256, 32), (1, 7, 64, 64), (3, 1, 128, 32), (2, 5, 256, 16), (1, 16, 128, 64)]
IDS = [f"k{a}g{b}d{c}p{d}" for a, b, c, d in SHAPES]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hk,G,D,P", SHAPES, ids=IDS)
def test_decode_over_ragged_lengths(dtype, Hk, G, D, P):
    """Lengths from zero and one up, on and around page and tile ends."""
    lens = [0, 1, P - 1, P, P + 1, 127, 128, 129, 255, 300, 511, 640, 2]
    c = Cache(Hk, D, P, sum(-(-n // P) for n in lens) + 8)
    table = c.tables(lens, seed=D)
    c.fill(table, lens, seed=P)
    (q, _) = qkv(len(lens), (Hk * G, 2), D, dtype, 3, slack=8)
    check_attention(c, q, None, lens, table, dtype)
    check_attention(c, q, None, lens, table, dtype, window=100, lse=False)
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hk,G,D,P", SHAPES, ids=IDS)
def test_a_few_queries_a_sequence(dtype, Hk, G, D, P):
    new = [1, 4, 3, 0, 7, 2, 5]
    lens = [1, 4, 130, 50, 261, 77, 6]
    cu = [0] + list(np.cumsum(new))
    c = Cache(Hk, D, P, sum(-(-n // P) for n in lens) + 8)
    table = c.tables(lens, seed=D + 1)
    c.fill(table, lens, seed=P + 1)
    q = qkv(cu[-1], (Hk * G,), D, dtype, 7)[0]
    check_attention(c, q, cu, lens, table, dtype)
    check_attention(c, q, cu, lens, table, dtype, window=33, max_q=9)
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hk,G,D,P", SHAPES, ids=IDS)
def test_prompts_and_chunks(dtype, Hk, G, D, P):
    """Fresh prompts and chunks after a prefix, lengths that end inside tiles."""
    new, ctx = [150, 1, 33, 260], [0, 40, 217, 19]
    lens = [a + b for a, b in zip(new, ctx)]
    cu = [0] + list(np.cumsum(new))
    c = Cache(Hk, D, P, sum(-(-n // P) for n in lens) + 8)
    table = c.tables(lens, seed=D + 2)
    c.fill(table, lens, seed=P + 2)
    q = qkv(cu[-1], (Hk * G, 1), D, dtype, 7)[0]
    check_attention(c, q, cu, lens, table, dtype)
    check_attention(c, q, cu, lens, table, dtype, window=64)
    c.close()


@pytest.mark.parametrize("q_len", [1, 3, 40])
def test_rows_that_see_nothing_give_zero(q_len):
    """More query rows than cached tokens: the first rows stand before position 0."""
    c = Cache(2, 128, 16, 32)
    lens = [0, 2, q_len + 5]
    cu = [0, q_len, 2 * q_len, 3 * q_len]
    table = c.tables(lens, seed=1)
    c.fill(table, lens, seed=2)
    q = qkv(cu[-1], (16,), 128, "bf16", 2)[0]
    out, st = check_attention(c, q, cu, lens, table, "bf16")
    assert (out[:q_len] == 0).all() and torch.isinf(st[:q_len]).all()
    if q_len > 2:
        assert (out[q_len:2 * q_len - 2] == 0).all()
    c.close()


@pytest.mark.parametrize("q_len", [1, 5, 70])
def test_sharp_and_flat_weights_and_uneven_scales(q_len):
    """Scores of hundreds, of zero, and pages whose value scales differ by 2^40."""
    c = Cache(2, 128, 16, 80)
    lens = [500, 333, 40 + q_len]
    cu = [0, q_len, 2 * q_len, 3 * q_len]
    table = c.tables(lens, seed=1)
    c.fill(table, lens, seed=2, spread=1)
    q = qkv(cu[-1], (16,), 128, "bf16", 2)[0]
    check_attention(c, q, cu, lens, table, "bf16", scale=4.0)
    check_attention(c, q, cu, lens, table, "bf16", scale=0.0)
    check_attention(c, q, cu, lens, table, "bf16", scale=-0.2)
    # uneven: an attended page may have any scale, from all-zero pages (2^-60) to large ones
    pages = table[0, :20].long()
    c.scales[pages, 1] = torch.exp2(torch.randint(-30, 11, (20, 2), generator=torch.Generator().manual_seed(1)).float()).to(DEV)
    c.codes()[pages[3], 1] = 0
    c.scales[pages[3], 1] = 2.0 ** -60
    check_attention(c, q, cu, lens, table, "bf16")
    c.close()


@pytest.mark.parametrize("q_len", [1, 4, 50])
def test_a_far_maximum_and_a_long_tail(q_len):
    """One key far above the rest at the start, in the middle or at the end: the many small weights
    still add up to what they weigh."""
    for where in (0, 700, 1399 - q_len):
        c = Cache(1, 128, 16, 96)
        lens = [1400]
        table = c.tables(lens, seed=1)
        c.fill(table, lens, seed=2, spread=1)
        q = qkv(q_len, (8,), 128, "bf16", 2)[0].contiguous()
        q[:] = 0.03 * q
        q[:, :, 0] = 8.0
        codes = c.codes()
        codes.view(torch.uint8)[:, 0, :, :, 0] = 0
        page, slot = int(table[0, where // 16]), where % 16
        c.scales[page, 0, 0] = 2.0 ** -5
        # score 14 * 8 / sqrt(128) = 9.9 against the others' spread around 0: e^9.9 ~ 20000 others
        codes[page, 0, 0, slot, 0] = torch.tensor(14.0 / float(c.scales[page, 0, 0])).clamp(max=448).to(ref.E4M3).view(torch.uint8)
        check_attention(c, q, [0, q_len], lens, table, "bf16")
        c.close()


def test_long_contexts_split_and_join():
    c = Cache(2, 128, 32, 1600)
    lens = [20001, 9, 30000]
    table = c.tables(lens, seed=6)
    g = torch.Generator(device=DEV).manual_seed(1)
    c.codes().copy_((torch.randn(c.codes().shape, generator=g, device=DEV) * 64).clamp(-448, 448).to(ref.E4M3).view(torch.uint8))
    c.scales.fill_(2.0 ** -6)
    q = qkv(3, (8,), 128, "bf16", 2)[0]
    check_attention(c, q, None, lens, table, "bf16")
    check_attention(c, q, None, lens, table, "bf16", window=5000)
    q = qkv(2 + 3 + 2, (8,), 128, "f16", 2)[0]
    check_attention(c, q, [0, 2, 5, 7], lens, table, "f16")
    c.close()


@pytest.mark.parametrize("q_len", [1, 6, 64])
def test_pages_past_2_31_bytes(q_len):
    """Pages of a pool larger than 4 GiB, so byte offsets pass 32 bits."""
    c = Cache(1, 128, 64, (5 << 30) // (16384 + 4096 * 4), extra_bytes=4096 * 4)
    n = 300
    table = c.tables([n], seed=1, spare=3)
    table[0, :5] = torch.tensor([c.pages - 1, 3, c.pages // 2 + 1, c.pages - 9, 70000], dtype=torch.int32)
    c.fill(table, [n], seed=2)
    q = qkv(q_len, (8,), 128, "bf16", 2)[0]
    lens, cu = [n], [0, q_len]
    out, _ = run_attention(c, q, cu, lens, table)
    ids = table[0, :5].long().cpu()
    small = c.codes()[table[0, :5].long()].contiguous().view(ref.E4M3).cpu().double() * \
        c.scales[table[0, :5].long()].cpu().double()[..., None, None]
    want, _, mag, top = ref.attention(small, np.arange(5)[None], lens, q, cu, 128 ** -0.5, 0, 64)
    tol = HALF_ULP["bf16"] * want.abs() + (2.0 ** -10 + 2.0 ** -16 * top[..., None]) * mag + 1e-7
    assert ((out.double().cpu() - want).abs() <= tol).all() and len(ids) == 5
    c.close()


@pytest.mark.parametrize("q_len", [1, 3, 48])
def test_strided_heads_outer_output_and_a_side_stream(q_len):
    c = Cache(2, 128, 16, 48)
    lens = [200, 100 + q_len]
    cu = [0, q_len, 2 * q_len]
    table = c.tables(lens, seed=4)
    c.fill(table, lens, seed=4)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(6, 2 * q_len, 128, generator=g).bfloat16().to(DEV).transpose(0, 1)
    box = torch.full((2 * q_len, 8, 256), 7.0, dtype=torch.bfloat16, device=DEV)
    out = box[:, 1:7, 64:192]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check_attention(c, q, cu, lens, table, "bf16", out=out, s=side.cuda_stream)
    box[:, 1:7, 64:192] = 7.0
    assert (box == 7.0).all()  # nothing beside the output was written
    c.close()


@pytest.mark.parametrize("q_len", [1, 4, 64])
def test_attention_reports_bad_tables_and_lengths(q_len):
    c = Cache(2, 128, 16, 32)
    lens = [100, 80]
    cu = [0, q_len, 2 * q_len]
    table = c.tables(lens, seed=4)
    c.fill(table, lens, seed=4)
    q = qkv(2 * q_len, (16,), 128, "bf16", 2)[0]
    good, _ = run_attention(c, q, cu, lens, table)
    t = table.clone()
    t[0, 2] = c.pages
    out, _ = run_attention(c, q, cu, lens, t, expect=R.DEV_BAD_PAGE)
    assert torch.equal(out[q_len:], good[q_len:])  # the other sequence is unharmed
    assert torch.isfinite(out).all()
    out, _ = run_attention(c, q, cu, [16 * table.shape[1] + 1, 80], table, expect=R.DEV_BAD_SHAPE)
    assert torch.equal(out[q_len:], good[q_len:])
    out, _ = run_attention(c, q, cu, [-3, 80], table, expect=R.DEV_BAD_SHAPE)
    assert torch.equal(out[q_len:], good[q_len:])
    c.close()


@pytest.mark.parametrize("q_len", [1, 5, 80])
def test_attention_repeats_to_the_bit_and_in_a_graph(q_len):
    c = Cache(2, 128, 16, 400)
    lens = [3000, 900 + q_len]
    cu = [0, q_len, 2 * q_len]
    table = c.tables(lens, seed=4)
    c.fill(table, lens, seed=4)
    q = qkv(2 * q_len, (16,), 128, "bf16", 2)[0]
    first, lse = run_attention(c, q, cu, lens, table)
    for _ in range(3):
        again, lse2 = run_attention(c, q, cu, lens, table)
        assert torch.equal(first, again) and torch.equal(lse, lse2)
    out = torch.zeros_like(first)
    cu_t, lens_t = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (cu, lens))
    n = R.rimuru_kv_attention_workspace_bytes(c.view, 16, 2, 2 * q_len, q_len)
    ws = torch.zeros(n + 1024, dtype=torch.uint8, device=DEV)
    at = (ws.data_ptr() + 1023) // 1024 * 1024
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.rimuru_kv_attention(c.view, R.heads_of(q), R.heads_of(out), 0, cu_t.data_ptr(), lens_t.data_ptr(),
                              2, 2 * q_len, q_len, table.data_ptr(), table.stride(0), 128 ** -0.5, 0, at, n,
                              stream())
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    # lengths are read when the kernels run: a replay serves a grown sequence
    lens_t[0] = 2990
    graph.replay()
    torch.cuda.synchronize()
    grown, _ = run_attention(c, q, cu, [2990, lens[1]], table)
    assert torch.equal(out, grown)
    c.close()


def test_a_sequence_alone_and_in_a_batch_agree():
    """Splitting the work differently changes only the order of fp32 sums."""
    c = Cache(2, 128, 16, 400)
    lens = [2500, 10, 1200, 77]
    table = c.tables(lens, seed=4)
    c.fill(table, lens, seed=4)
    q = qkv(4, (16,), 128, "bf16", 2)[0]
    both, _ = run_attention(c, q, None, lens, table)
    for b in range(4):
        one, _ = run_attention(c, q[b:b + 1], None, lens[b:b + 1], table[b:b + 1])
        d = (one[0].double() - both[b].double()).abs()
        assert (d <= 2.0 ** -7 * both[b].double().abs() + 2.0 ** -9 * both[b].abs().max()).all()
    c.close()


@pytest.mark.parametrize("G,D", [(8, 128), (7, 64), (8, 256)])
@pytest.mark.parametrize("q_len", [1, 2, 3, 16, 17, 18, 32, 33, 37])
def test_where_the_kernels_change(q_len, G, D):
    c = Cache(2, D, 16, 80)
    lens = [300, 513, q_len]
    table = c.tables(lens, seed=q_len)
    c.fill(table, lens, seed=1)
    cu = [0, q_len, 2 * q_len, 3 * q_len]
    q = qkv(cu[-1], (2 * G,), D, "bf16", q_len)[0]
    check_attention(c, q, cu, lens, table, "bf16")
    c.close()


@pytest.mark.parametrize("G,D,dtype", [(8, 128, "bf16"), (5, 64, "f16"), (8, 256, "bf16")])
@pytest.mark.parametrize("q_len", [1, 3, 40])
def test_a_wide_page_table_changes_nothing_but_the_split(q_len, G, D, dtype):
    """The bound of the lengths that the table gives decides whether units are cut."""
    lens = [0, 900, 17, 130, q_len]
    c = Cache(2, D, 16, sum(-(-n // 16) for n in lens))
    cu = [i * q_len for i in range(len(lens) + 1)]
    q = qkv(cu[-1], (2 * G,), D, dtype, q_len)[0]
    for spare in (0, 4000):
        table = c.tables(lens, seed=1, spare=spare)
        if spare == 0:
            c.fill(table, lens, seed=1)
        check_attention(c, q, cu, lens, table, dtype)
        check_attention(c, q, cu, lens, table, dtype, window=150)
    c.close()


@pytest.mark.parametrize("q_max", [1, 4, 40])
def test_many_short_sequences_and_some_without_keys_or_rows(q_max):
    rng = np.random.default_rng(q_max)
    lens = rng.choice([0, 1, 2, 15, 16, 17, 40, 127, 128, 129, 260], size=400).tolist()
    c = Cache(2, 64, 16, sum(-(-n // 16) for n in lens))
    table = c.tables(lens, seed=1)
    c.fill(table, lens, seed=2)
    n = rng.integers(0, q_max + 1, size=400) if q_max > 1 else np.ones(400, int)
    cu = [0] + np.cumsum(n).tolist()
    q = qkv(cu[-1], (6,), 64, "bf16", 3)[0]
    check_attention(c, q, cu, lens, table, "bf16", max_q=q_max)
    check_attention(c, q, cu, lens, table, "bf16", max_q=q_max, window=30)
    c.close()


# ------------------------------------------------------------------ pages
@pytest.mark.parametrize("Hk,D,P,extra", [(4, 128, 16, 0), (2, 256, 32, 32768), (1, 64, 16, 0)])
@pytest.mark.parametrize("n", [1, 7, 500])
def test_copy_pages(Hk, D, P, extra, n):
    c = Cache(Hk, D, P, 1024, extra_bytes=extra)
    g = torch.Generator(device=DEV).manual_seed(n)
    c.pool.mem.copy_(torch.randint(0, 256, c.pool.mem.shape, generator=g, device=DEV, dtype=torch.uint8))
    c.scales.copy_(torch.randn(c.scales.shape, generator=g, device=DEV))
    order = torch.randperm(c.pages, generator=g, device=DEV).to(torch.int32)
    src, dst = order[:n].clone(), order[n:2 * n].clone()
    codes, scales = c.codes().clone(), c.scales.clone()
    whole = c.pool.mem.clone().view(c.pages, c.page_bytes)
    codes[dst.long()] = codes[src.long()]
    scales[dst.long()] = scales[src.long()]
    R.rimuru_kv_copy_pages(c.view, src.data_ptr(), dst.data_ptr(), n, stream())
    torch.cuda.synchronize()
    assert torch.equal(c.codes(), codes) and torch.equal(c.scales, scales)
    used = 2 * Hk * D * P
    assert torch.equal(c.pool.mem.view(c.pages, c.page_bytes)[:, used:], whole[:, used:])
    # ids outside the view are reported and skipped
    src[0], keep = c.pages, c.pool.mem.clone()
    if n > 1:
        dst[1] = -1
    R.rimuru_kv_copy_pages(c.view, src.data_ptr(), dst.data_ptr(), n, stream())
    torch.cuda.synchronize()
    assert R.rimuru_get_device_error(c.view, clear=True) == R.DEV_BAD_PAGE
    assert torch.equal(c.pool.mem, keep)
    c.close()


def test_fork_then_diverge_and_free():
    """Children read the parent's tokens, write their own, and every page comes back."""
    c = Cache(2, 128, 16, 32)
    free0 = R.rimuru_pool_level_stats(c.pool.handle, 0)["pages_free"]
    pages = [R.rimuru_page_alloc(c.view) for _ in range(3)]
    L = 39
    table = torch.tensor([pages], dtype=torch.int32, device=DEV)
    c.fill(table, [L], seed=3)
    kids = R.rimuru_kv_fork(c.view, pages, L, 3, stream())
    assert [k[:2] for k in kids] == [pages[:2]] * 3 and len({k[2] for k in kids} | {pages[2]}) == 4
    assert R.rimuru_page_refs(c.view, pages[0]) == 4 and R.rimuru_page_refs(c.view, pages[2]) == 1
    rows = torch.tensor([pages] + kids, dtype=torch.int32, device=DEV)
    q = qkv(1, (4,), 128, "bf16", 1)[0].expand(4, 4, 128).contiguous()
    out, _ = check_attention(c, q, None, [L] * 4, rows, "bf16")
    assert (out == out[0]).all()
    # each sequence appends its own token; the shared pages stay
    shared = c.codes()[pages[:2]].clone()
    k, v = qkv(4, (2, 2), 128, "bf16", 5)
    run_append(c, k, v, [0, 1, 2, 3, 4], [L + 1] * 4, rows)
    out, _ = check_attention(c, q, None, [L + 1] * 4, rows, "bf16")
    assert not torch.equal(out[0], out[1])
    assert torch.equal(shared, c.codes()[pages[:2]])
    for row in [pages] + kids:
        for p in row:
            R.rimuru_page_free(c.view, p)
    assert R.rimuru_pool_level_stats(c.pool.handle, 0)["pages_free"] == free0
    with pytest.raises(R.RimuruError):
        R.rimuru_page_free(c.view, pages[0])
    c.close()


def test_fork_without_room_changes_nothing():
    c = Cache(1, 64, 16, 8)
    pages = [R.rimuru_page_alloc(c.view) for _ in range(6)]
    with pytest.raises(R.RimuruError) as e:
        R.rimuru_kv_fork(c.view, pages, 6 * 16 - 1, 3, stream())
    assert e.value.status == R.ERR_OOM
    assert [R.rimuru_page_refs(c.view, p) for p in pages] == [1] * 6
    assert R.rimuru_pool_level_stats(c.pool.handle, 1)["pages_owned"] == 6
    c.close()


def test_compaction_frees_huge_pages_and_keeps_every_token():
    c = Cache(2, 128, 16, 64, per_parent=8)
    rng = np.random.default_rng(0)
    for p in range(64):
        R.rimuru_page_place(c.view, p)
    live = {int(p) for q in range(8) for p in rng.choice(8, size=[2, 7, 1, 5, 3, 8, 4, 2][q], replace=False) + 8 * q}
    for p in set(range(64)) - live:
        R.rimuru_page_free(c.view, p)
    order = rng.permutation(sorted(live)).astype(int).tolist()
    seqs, lens = [order[:10], order[10:21], order[21:]], [155, 176, 16 * len(order[21:]) - 7]
    shared = seqs[0][0]
    R.rimuru_page_share(c.view, shared)
    seqs.append([shared])
    lens.append(16)
    width = max(map(len, seqs)) + 1
    table = torch.tensor([s + [-1] * (width - len(s)) for s in seqs], dtype=torch.int32, device=DEV)
    c.fill(table, lens, seed=5)
    q = qkv(4, (8,), 128, "bf16", 1)[0]
    before, _ = check_attention(c, q, None, lens, table, "bf16")
    free0 = R.rimuru_pool_level_stats(c.pool.handle, 0)["pages_free"]
    flat, moved = R.rimuru_kv_compact(c.view, table.cpu().reshape(-1).tolist(), 1000, stream())
    # 32 pages in use over 8 parents of 8: four parents suffice
    assert R.rimuru_pool_level_stats(c.pool.handle, 0)["pages_free"] == free0 + 4 and moved == 8
    assert all(a == b for a, b in zip(flat, table.cpu().reshape(-1).tolist()) if b < 0)
    t2 = torch.tensor(flat, dtype=torch.int32, device=DEV).view(4, width)
    after, _ = run_attention(c, q, None, lens, t2)
    assert torch.equal(before, after)
    assert R.rimuru_page_refs(c.view, int(t2[3, 0])) == 2 and int(t2[3, 0]) == int(t2[0, 0])
    again, moved = R.rimuru_kv_compact(c.view, flat, 1000, stream())
    assert moved == 0 and again == flat
    for p in t2.reshape(-1).tolist():
        if p >= 0:
            R.rimuru_page_free(c.view, p)
    assert R.rimuru_pool_level_stats(c.pool.handle, 0)["pages_free"] == 8
    c.close()


def test_compaction_leaves_pages_it_was_not_told_about():
    c = Cache(1, 64, 16, 16, per_parent=8)
    for p in (0, 1, 8):
        R.rimuru_page_place(c.view, p)
    flat, moved = R.rimuru_kv_compact(c.view, [0, 8], 10, stream())  # page 1 is someone else's
    assert moved == 1 and flat[0] == 0 and flat[1] // 8 == 0 and flat[1] not in (0, 1)
    flat, moved = R.rimuru_kv_compact(c.view, flat, 0, stream())
    assert moved == 0
    c.close()


def test_a_pool_shared_with_experts_gets_its_huge_pages_back():
    """KV pages cut from expert-sized huge pages: once compacted, an expert page can be placed."""
    kvp = 2 * 2 * 128 * 16
    pool_pages, per = 3, 16
    from paged_moe_shared_gb300.device_pool import DevicePool
    pool = DevicePool(pool_pages * per * kvp, per * kvp, DEV)
    ev, kv = pool.view(per * kvp), pool.view(kvp)
    scales = torch.ones(pool_pages * per, 2, 2, device=DEV)
    R.rimuru_view_set_kv_shape(kv, 2, 128, 16, scales.data_ptr(), scales.numel() * 4)
    for p in (0, 3, 16, 40):
        R.rimuru_page_place(kv, p)
    with pytest.raises(R.RimuruError):
        R.rimuru_page_alloc(ev)
    flat, moved = R.rimuru_kv_compact(kv, [0, 3, 16, 40], 8, stream())
    assert moved == 2 and {p // per for p in flat} == {0}
    R.rimuru_page_alloc(ev), R.rimuru_page_alloc(ev)
    torch.cuda.synchronize()
    pool.close()
