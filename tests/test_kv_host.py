"""Page lists, references and host-side failures of the KV entry points; no device is touched."""
import pytest

from paged_moe_shared_gb300 import rimuru as R

BASE = 64 << 20  # a 2 MiB aligned address that is never dereferenced


@pytest.fixture
def kv():
    page = 2 * 2 * 128 * 16
    pool = R.rimuru_pool_create(BASE, 64 * page, 16 * page)
    view = R.rimuru_view_create(pool, page)
    R.rimuru_view_set_kv_shape(view, 2, 128, 16, 4096, 1 << 20)
    yield view
    R.rimuru_view_destroy(view)
    R.rimuru_pool_destroy(pool)


def test_children_have_the_pages_of_the_tokens_and_no_others(kv):
    """A parent may hold pages past its tokens; no child is given an entry for them."""
    pages = [R.rimuru_page_alloc(kv) for _ in range(6)]
    assert R.rimuru_kv_fork(kv, pages[1:], 32, 3) == [pages[1:3]] * 3
    assert [R.rimuru_page_refs(kv, p) for p in pages] == [1, 4, 4, 1, 1, 1]
    assert R.rimuru_kv_fork(kv, pages, 0, 2) == [[], []]
    assert R.rimuru_kv_fork(kv, [], 0, 2) == [[], []]
    assert R.rimuru_kv_fork(kv, pages, 16, 0) == []
