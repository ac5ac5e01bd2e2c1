"""How attention's work is cut, counted on the host: no device is touched."""
import os
import subprocess

import pytest

from paged_moe_shared_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


def test_tiles_in_closed_form_are_the_tiles_of_the_rows(tmp_path):
    """Windows up to the largest int, more rows than keys, lengths to 2^30."""
    try:
        nvcc = B.nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    exe = str(tmp_path / "split")
    r = subprocess.run([nvcc, *B.ARCH, "-std=c++17", "-O1", "-o", exe, os.path.join(HERE, "kv_split_check.cu")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_more_rows_than_an_int_can_carry_are_refused():
    from paged_moe_shared_gb300 import rimuru as R
    page = 2 * 2 * 128 * 16
    pool = R.rimuru_pool_create(64 << 20, 64 * page, 16 * page)
    kv = R.rimuru_view_create(pool, page)
    R.rimuru_view_set_kv_shape(kv, 2, 128, 16, 4096, 1 << 20)
    need = R.rimuru_kv_attention_workspace_bytes
    # a bound above the number of rows asks for no more than the rows do
    assert need(kv, 8, 1, 3, 2 ** 31 - 1) == need(kv, 8, 1, 3, 3) > 0
    for rows in (2 ** 30 + 1, 2 ** 31 - 1):
        h = R.Heads(4096, 0, 128, 8, R.BF16)
        with pytest.raises(R.RimuruError) as e:
            R.rimuru_kv_attention(kv, h, h, 0, 16, 16, 1, rows, rows, 16, 4, 1.0, 0, 4096, need(kv, 8, 1, rows, rows))
        assert e.value.status == R.ERR_UNSUPPORTED
    R.rimuru_view_destroy(kv)
    R.rimuru_pool_destroy(pool)
