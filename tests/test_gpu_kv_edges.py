"""The KV operators at the edges of what they accept."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from kv_reference import DEV, Cache
from paged_moe_shared_gb300 import rimuru as R
from test_gpu_kv import check_attention, qkv, run_attention

pytestmark = pytest.mark.gpu


# One query tile whose key tiles are taken in turns: units of one key tile have no work for the second
# of the two MMA warps, which has to keep up with them all the same, whatever follows.
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (128, "f16")])
@pytest.mark.parametrize("order", ["short", "mixed", "long last"])
def test_units_of_one_key_tile_among_longer_ones(order, D, dtype):
    rng = np.random.default_rng(len(order))
    n = 900
    lens = rng.integers(1, 129, size=n)
    if order == "mixed":
        lens = np.where(rng.random(n) < 0.4, rng.integers(129, 700, size=n), lens)
    if order == "long last":
        lens[-3:] = 2000
    lens = lens.tolist()
    new = [min(x, 5) for x in lens]
    cu = [0] + np.cumsum(new).tolist()
    c = Cache(2, D, 16, sum(-(-x // 16) for x in lens))
    table = c.tables(lens, seed=1, spare=400)  # wide: the units are cut into runs of many
    c.fill(table, lens, seed=2)
    q = qkv(cu[-1], (8,), D, dtype, 3)[0]
    first, lse = check_attention(c, q, cu, lens, table, dtype, max_q=40)
    for _ in range(20):
        again, lse2 = run_attention(c, q, cu, lens, table, max_q=40)
        assert torch.equal(first, again) and torch.equal(lse, lse2)
    assert R.rimuru_get_device_error(c.view) == R.DEV_OK
    c.close()


INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("q_len", [1, 5, 40, 300])
@pytest.mark.parametrize("spare", [2, 4000])
def test_a_window_beyond_every_sequence_is_none(q_len, spare):
    """Fresh prompts, a prefix, more rows than keys; windows up to the largest int."""
    lens = [q_len, q_len + 700, max(0, q_len - 3), 0]
    cu = [i * q_len for i in range(5)]
    c = Cache(2, 128, 16, sum(-(-n // 16) for n in lens))
    table = c.tables(lens, seed=1, spare=spare)
    c.fill(table, lens, seed=2)
    q = qkv(cu[-1], (16,), 128, "bf16", 3)[0]
    none, lse = check_attention(c, q, cu, lens, table, "bf16")
    most = 16 * table.shape[1]
    for window in (q_len + 700, most - 1, most, most + 1, 1 << 30, INT_MAX - 1, INT_MAX):
        out, st = run_attention(c, q, cu, lens, table, window=window)
        assert torch.equal(out, none) and torch.equal(st, lse), window
    c.close()


@pytest.mark.parametrize("q_len", [1, 3, 40])
def test_any_upper_bound_of_the_rows_serves(q_len):
    lens = [q_len + 100, 500]
    cu = [0, q_len, 2 * q_len]
    c = Cache(2, 128, 16, sum(-(-n // 16) for n in lens))
    table = c.tables(lens, seed=1)
    c.fill(table, lens, seed=2)
    q = qkv(cu[-1], (8,), 128, "bf16", 3)[0]
    for max_q in (q_len, 2 * q_len + 1, 1 << 20, INT_MAX):
        check_attention(c, q, cu, lens, table, "bf16", max_q=max_q)
    c.close()


def test_lengths_past_the_limit_are_reported():
    c = Cache(1, 64, 16, 8)
    table = c.tables([100], seed=1)
    c.fill(table, [100], seed=2)
    q = qkv(2, (4,), 64, "bf16", 3)[0]
    good, _ = run_attention(c, q[:1], None, [100], table)
    for n in (INT_MAX, INT_MAX - 127, -3):
        out, _ = run_attention(c, q, None, [n, 100], table.expand(2, -1).contiguous(), expect=R.DEV_BAD_SHAPE)
        assert (out[0] == 0).all() and torch.isfinite(out[1]).all()
    c.close()


@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("first", [1, 3, 5])
def test_append_of_the_last_sequences_of_a_batch(first, P):
    """Offsets that do not begin at 0: the sequences before are neither read nor written."""
    before, new = [0, 2 * P, 5, 0, P - 1, 1, 3], [3 * P, 40, 2 * P + 1, 3, P + 2, 1, 0]
    lens = [a + b for a, b in zip(before, new)]
    cu = [0] + np.cumsum(new).tolist()
    c = Cache(2, 128, P, 40)
    table = c.tables(lens, seed=1)
    for b in range(len(lens)):
        c.fill(table[b:b + 1], before[b:b + 1], seed=b)
    values, scales = c.values().numpy(), c.scales.cpu().double().numpy()
    _, k, v = qkv(cu[-1], (3, 2, 2), 128, "bf16", 4)
    want = table.clone()
    table[:first] = c.pages + 5  # what lies in front of the table names no page
    cu_t = torch.tensor(cu, dtype=torch.int32, device=DEV)
    lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
    n = len(lens) - first
    R.rimuru_kv_append(c.view, R.heads_of(k), R.heads_of(v), cu_t[first:].data_ptr(), lens_t[first:].data_ptr(), n,
                       cu[-1], table[first:].data_ptr(), table.stride(0), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert R.rimuru_get_device_error(c.view, clear=True) == R.DEV_OK
    ref.append(values, scales, want.cpu().numpy()[first:], cu[first:], lens[first:], k, v, P)
    np.testing.assert_array_equal(c.scales.cpu().double().numpy(), scales)
    np.testing.assert_array_equal(c.values().numpy(), values)
    # attention takes the same offsets
    q = qkv(cu[-1], (8,), 128, "bf16", 3)[0]
    out = torch.full((cu[-1], 8, 128), 7.0, dtype=q.dtype, device=DEV)
    ws = torch.empty(R.rimuru_kv_attention_workspace_bytes(c.view, 8, n, cu[-1], max(new)) + 1024,
                     dtype=torch.uint8, device=DEV)
    R.rimuru_kv_attention(c.view, R.heads_of(q), R.heads_of(out), 0, cu_t[first:].data_ptr(),
                          lens_t[first:].data_ptr(), n, cu[-1], max(new), table[first:].data_ptr(), table.stride(0),
                          128 ** -0.5, 0, (ws.data_ptr() + 1023) // 1024 * 1024, ws.numel() - 1024,
                          torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert R.rimuru_get_device_error(c.view, clear=True) == R.DEV_OK
    assert (out[:cu[first]] == 7.0).all()
    alone = [x - cu[first] for x in cu[first:]]
    want, _ = run_attention(c, q[cu[first]:], alone, lens[first:], table[first:])
    d = (out[cu[first]:].double() - want.double()).abs()
    assert (d <= 2.0 ** -7 * want.double().abs() + 2.0 ** -9 * want.abs().max()).all()
    c.close()


# ------------------------------------------------------------------ nothing to multiply
def zero_cache(D, lens, seed=1, spare=2):
    """Pages as the append writes them for keys of zero (codes 0, scale 2^-60), and random values."""
    c = Cache(2, D, 16, sum(-(-n // 16) for n in lens))
    table = c.tables(lens, seed=seed, spare=spare)
    c.fill(table, lens, seed=seed)
    c.codes()[:, 0] = 0
    c.scales[:, 0] = 2.0 ** -60
    return c, table


ROWS = [(1, 8), (5, 3), (40, 3), (40, 8), (300, 1), (70, 16)]  # query rows, query heads per key head


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_len,G", ROWS)
def test_zero_queries_over_zero_keys_give_the_mean_of_the_values(q_len, G, dtype, D):
    """Scores of exactly 0 whatever the factors: rows of zeros, one zero head among others, scale 0,
    over keys of zero, with masked columns in every unit's last tile."""
    lens = [q_len, q_len + 203, 1000]
    cu = [i * q_len for i in range(4)]
    c, table = zero_cache(D, lens)
    q = qkv(cu[-1], (2 * G,), D, dtype, 3)[0].contiguous()
    some, none = q.clone(), torch.zeros_like(q)
    some[:, ::3] = 0
    for x in (none, some, q):
        check_attention(c, x, cu, lens, table, dtype)
        check_attention(c, x, cu, lens, table, dtype, scale=0.0)
    check_attention(c, none, cu, lens, table, dtype, window=50)
    # the smallest numbers that the types have
    tiny = torch.full_like(q, 2.0 ** -24 if dtype == "f16" else 2.0 ** -126)
    check_attention(c, tiny, cu, lens, table, dtype)
    # zero queries over other keys, and pages of zero keys among others
    c.fill(table, lens, seed=5)
    check_attention(c, none, cu, lens, table, dtype)
    check_attention(c, some, cu, lens, table, dtype, scale=0.0)
    c.codes()[::2, 0] = 0
    c.scales[::2, 0] = 2.0 ** -60
    check_attention(c, some, cu, lens, table, dtype)
    c.close()


@pytest.mark.parametrize("q_len", [1, 40, 300])
def test_a_pass_over_nothing_but_zeros_is_zero(q_len):
    """A warm-up: q = k = v = 0 through the append."""
    lens, cu = [q_len], [0, q_len]
    c = Cache(2, 128, 16, -(-q_len // 16))
    table = c.tables(lens)
    z = torch.zeros(q_len, 2, 128, dtype=torch.bfloat16, device=DEV)
    cu_t, lens_t = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (cu, lens))
    R.rimuru_kv_append(c.view, R.heads_of(z), R.heads_of(z), cu_t.data_ptr(), lens_t.data_ptr(), 1, q_len,
                       table.data_ptr(), table.stride(0), torch.cuda.current_stream().cuda_stream)
    out, lse = run_attention(c, torch.zeros(q_len, 16, 128, dtype=torch.bfloat16, device=DEV), cu, lens, table)
    assert (out == 0).all()
    want = torch.arange(1, q_len + 1, device=DEV).float().log()[:, None].expand(-1, 16)
    assert (lse - want).abs().max() <= 2.0 ** -16 * max(1.0, float(want.max()))
    c.close()


@pytest.mark.parametrize("q_len", [1, 5, 40, 300])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(q_len):
    lens, cu = [q_len + 77], [0, q_len]
    c, table = zero_cache(128, lens)
    q = qkv(q_len, (16,), 128, "bf16", 3)[0].contiguous()
    for keys in ("zero", "some"):
        if keys == "some":
            c.fill(table, lens, seed=5)
        bad = q.clone()
        bad[0, 3, 5], bad[q_len - 1, 9, 0] = float("inf"), float("nan")
        out, lse = run_attention(c, bad, cu, lens, table)
        hit = torch.zeros(q_len, 16, dtype=torch.bool, device=DEV)
        hit[0, 3] = hit[q_len - 1, 9] = True
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
        # the other rows: the tolerance of check_attention
        want, want_lse, mag, top = ref.attention(c.values(), table.cpu().numpy(), lens, q, cu, 128 ** -0.5, 0, c.P)
        tol = ref.HALF_ULP["bf16"] * want.abs() + (2.0 ** -10 + 2.0 ** -16 * top[..., None]) * mag + 1e-7
        keep = ~hit.cpu()
        assert ((out.double().cpu() - want).abs() <= tol)[keep].all()
        assert ((lse.double().cpu() - want_lse).abs() <= 2.0 ** -17 * top + 2.0 ** -16)[keep].all()
    c.close()


# ------------------------------------------------------------------ errors and streams
def busy_default_stream():
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # about 0.2 s


def test_an_error_of_the_first_call_is_kept_on_a_side_stream():
    """The default stream is busy, and a side stream does not wait for it."""
    c = Cache(2, 128, 16, 8)
    _, k, v = qkv(5, (1, 2, 2), 128, "bf16", 4)
    bad = torch.full((1, 2), c.pages + 3, dtype=torch.int32, device=DEV)
    cu_t, lens_t = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 5], [5]))
    side = torch.cuda.Stream()
    other = Cache(2, 128, 16, 8)  # loads the kernel, which would wait for the device
    R.rimuru_kv_append(other.view, R.heads_of(k), R.heads_of(v), cu_t.data_ptr(), lens_t.data_ptr(), 1, 5,
                       other.tables([5]).data_ptr(), 3, side.cuda_stream)
    busy_default_stream()
    R.rimuru_kv_append(c.view, R.heads_of(k), R.heads_of(v), cu_t.data_ptr(), lens_t.data_ptr(), 1, 5,
                       bad.data_ptr(), 2, side.cuda_stream)
    side.synchronize()
    torch.cuda.synchronize()
    assert R.rimuru_get_device_error(c.view, clear=True) == R.DEV_BAD_PAGE
    assert R.rimuru_get_device_error(c.view) == R.DEV_OK
    other.close()
    c.close()


def test_an_error_of_the_first_forward_is_kept_on_a_side_stream():
    import workloads as W
    from gpu_harness import Runner
    r, other = Runner(W.tiny(3)), Runner(W.tiny(3))
    r.logits[2, 5] = float("nan")
    side = torch.cuda.Stream()
    other.forward(side)  # loads the kernels
    busy_default_stream()
    r.forward(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert R.rimuru_get_device_error(r.ev, clear=True) == R.DEV_NONFINITE
    assert R.rimuru_get_device_error(r.ev) == R.DEV_OK
    other.close()
    r.close()


# ------------------------------------------------------------------ references
@pytest.mark.parametrize("how", ["destroy", "shrink"])
def test_the_expert_cache_drops_its_reference_only(how):
    """A slot's page that somebody else has a reference to outlives the slot, and comes back once."""
    import workloads as W
    from paged_moe_shared_gb300.device_pool import DevicePool
    shape = W.MoEShape(H=256, I=128, E=8, k=2)
    pb, n = shape.H * shape.I * 2, 12
    st = W.offload_stack(shape, 2, 4, steps=1, seed=7)
    host = torch.from_numpy(st.host_pages).pin_memory()
    pool = DevicePool(n * pb, pb, DEV)
    ev = pool.view(pb)
    R.rimuru_view_set_moe_shape(ev, 2, shape.E, shape.H, shape.I, shape.k, shape.renorm)
    off = R.rimuru_offload_create(ev, host.data_ptr(), 4, 0)
    pages = list(range(n))
    assert [R.rimuru_page_refs(ev, p) for p in pages] == [1] * n
    for p in pages:
        R.rimuru_page_share(ev, p)
    if how == "shrink":
        R.rimuru_offload_resize(off, 1)
        assert sum(R.rimuru_page_refs(ev, p) for p in pages) == 3 * 2 + 9
        R.rimuru_offload_resize(off, 1)
    R.rimuru_offload_destroy(off)
    assert [R.rimuru_page_refs(ev, p) for p in pages] == [1] * n
    for p in pages:
        R.rimuru_page_free(ev, p)
    assert [R.rimuru_page_refs(ev, p) for p in pages] == [0] * n
    p = R.rimuru_page_alloc(ev)
    assert R.rimuru_page_refs(ev, p) == 1
    R.rimuru_page_free(ev, p)
    assert R.rimuru_pool_level_stats(pool.handle, 0)["pages_free"] == n
    pool.close()


# ------------------------------------------------------------------ queries of a wide range
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_len,G", [(1, 8), (2, 8), (40, 3), (300, 1)])
@pytest.mark.parametrize("loud", [30.0, 1000.0, 4096.0, 20000.0])
def test_small_elements_beside_a_loud_one_keep_their_weight(loud, q_len, G, D, dtype):
    """One query channel far above the others, over keys that have nothing there.  With a window of
    one key the log-sum is the score itself.

    A row is scaled so that its largest magnitude lies in (224, 448], and its last part has steps of
    2^-13 (bf16) or 2^-16 (f16) there, or three significant bits: an element is off by at most 2^-14 or
    2^-17, that is 2^-14 / 224 of the largest one; times sum |k| and the scale.  The products' sum is
    off by 2^-17 of sum |q k| and the logarithm by 2^-16, as in check_attention."""
    lens = [q_len + 100, q_len]
    cu = [0, q_len, 2 * q_len]
    c = Cache(2, D, 16, sum(-(-n // 16) for n in lens))
    table = c.tables(lens, seed=1)
    c.fill(table, lens, seed=2)
    c.codes()[:, 0, :, :, D // 2 + 3] = 0
    q = qkv(cu[-1], (2 * G,), D, dtype, 3)[0].contiguous()
    q[:, :, D // 2 + 3] = loud
    scale = D ** -0.5
    _, lse = run_attention(c, q, cu, lens, table, window=1)
    values = c.values()
    _, want, _, top = ref.attention(values, table.cpu().numpy(), lens, q, cu, scale, 1, 16)
    keys = values[table.cpu().clamp(min=0).long(), 0].nan_to_num()  # [sequences, pages, heads, 16, D]
    total = keys.abs().sum(-1).amax()
    step = 2.0 ** -14 if dtype == "bf16" else 2.0 ** -17
    tol = 2.0 ** -16 + 2.0 ** -17 * top + scale * loud * step / 224 * float(total)
    err = (lse.double().cpu() - want).abs()
    assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))
    c.close()


# ------------------------------------------------------------------ rotary positions
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaling,factor", [(R.ROPE_PLAIN, 1.0), (R.ROPE_LINEAR, 64.0)])
def test_slow_pairs_turn_by_small_angles(scaling, factor, interleaved):
    """A pair (0, v) becomes (-v sin, v cos): the sine of a small angle to a few ulp of itself.  The
    angle is rounded to fp32 once, the sine is good to an ulp or two and the product is rounded: at
    most 4 ulp, 2^-22."""
    rot, T = 256, 12
    h = R.rimuru_rope_create(rot, R.ROPE_INTERLEAVED if interleaved else R.ROPE_HALF, 500000.0, scaling, factor)
    f = ref.inv_freq(rot, 500000.0, scaling, factor)
    pos = torch.tensor([1, 2, 3, 4, 5, 6, 7, 8, 9, 10, -1, -7], dtype=torch.int32, device=DEV)
    x = torch.zeros(T, 3, rot, device=DEV)
    v = torch.rand(T, 3, rot // 2, generator=torch.Generator().manual_seed(1)).to(DEV) + 0.5
    (x[..., 1::2] if interleaved else x[..., rot // 2:]).copy_(v)
    out = torch.empty_like(x)
    R.rimuru_rope_apply(h, pos.data_ptr(), T, rot, [R.heads_of(x)], [R.heads_of(out)],
                        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    ang = pos.cpu().double()[:, None] * torch.from_numpy(f)
    y = out.cpu().double()
    u, w = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:])
    want_u, want_w = -v.cpu().double() * torch.sin(ang)[:, None], v.cpu().double() * torch.cos(ang)[:, None]
    small = (ang.abs() < 1.5)[:, None].expand_as(u)  # past that a small cosine makes an ulp of the angle larger
    assert ((u - want_u).abs() <= 2.0 ** -22 * want_u.abs())[small].all(), \
        float(((u - want_u).abs() / want_u.abs())[small].max())
    small = (ang.abs() < 0.7)[:, None].expand_as(u)
    assert ((w - want_w).abs() <= 2.0 ** -22 * want_w.abs())[small].all()
    R.rimuru_rope_destroy(h)


# ------------------------------------------------------------------ head layouts
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hk,G,D", [(1, 128, 128), (2, 100, 64), (1, 33, 256), (1, 17, 128), (40, 1, 64), (1024, 1, 64)])
def test_wide_groups_and_many_heads(Hk, G, D, dtype):
    """Units of one query row, of a few, and of rows that do not fill them."""
    lens, new = [140, 3, 515], [1, 3, 9]
    cu = [0] + np.cumsum(new).tolist()
    c = Cache(Hk, D, 16, sum(-(-n // 16) for n in lens))
    q = qkv(cu[-1], (Hk * G,), D, dtype, 3)[0]
    for spare in (2, 3000):
        table = c.tables(lens, seed=1, spare=spare)
        if spare == 2:
            c.fill(table, lens, seed=2)
        check_attention(c, q, cu, lens, table, dtype)
        check_attention(c, q, cu, lens, table, dtype, window=20)
        check_attention(c, q[:3], None, lens, table, dtype)
    c.close()
