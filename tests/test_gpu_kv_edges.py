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
