"""The KV operators at the edges of what they accept."""
import numpy as np
import pytest
import torch

from kv_reference import Cache
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
