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


NO_MEMORY = """
import ctypes, resource, sys
sys.path.insert(0, {root!r})
from paged_moe_shared_gb300 import rimuru as R
page, n = 2 * 64 * 16, 1 << 18
pool = R.rimuru_pool_create(64 << 20, n * page, 16 * page)
kv = R.rimuru_view_create(pool, page)
R.rimuru_view_set_kv_shape(kv, 1, 64, 16, 4096, R.rimuru_kv_scale_bytes(kv, 1))
pages = (ctypes.c_int32 * n)(*[R.rimuru_page_alloc(kv) for _ in range(n)])
kids = (ctypes.c_int32 * n)()
at = lambda a: ctypes.cast(a, ctypes.c_void_p)
R.lib.rimuru_kv_fork(kv, at(pages), 16, 1, at(kids), n, None)   # every path has run once
R.rimuru_page_free(kv, pages[0])
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (4 << 20), resource.RLIM_INFINITY))
st = R.lib.rimuru_kv_fork(kv, at(pages), 16 * n, 1, at(kids), n, None)
resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
assert st == R.ERR_OOM, st
assert all(R.rimuru_page_refs(kv, p) == 1 for p in pages)
assert R.lib.rimuru_kv_fork(kv, at(pages), 16 * n, 1, at(kids), n, None) == 0
assert list(kids) == list(pages) and all(R.rimuru_page_refs(kv, p) == 2 for p in pages)
print("fine")
"""


def test_fork_without_host_memory_is_an_error_and_changes_nothing():
    """A host allocation that fails inside the call ends in a status, not in the process's end."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", NO_MEMORY.format(root=root)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "fine" in r.stdout, (r.returncode, r.stderr[-500:])


def refused(status, fn, *args):
    with pytest.raises(R.RimuruError) as e:
        fn(*args)
    assert e.value.status == status, str(e.value)


@pytest.mark.parametrize("big", [1e39, -1e300])
def test_factors_that_are_not_finite_in_fp32_are_refused(kv, big):
    h = R.Heads(4096, 256, 128, 2, R.BF16)
    refused(R.ERR_ARG, R.rimuru_kv_attention, kv, h, h, 0, 0, 16, 1, 1, 1, 16, 4, big, 0, 4096, 1 << 30)
    refused(R.ERR_ARG, R.rimuru_rope_create, 128, R.ROPE_HALF, 1e4, R.ROPE_PLAIN, 1.0, 0.0, 0.0, 0.0, big)


def test_frequencies_that_are_not_finite_are_refused():
    refused(R.ERR_ARG, R.rimuru_rope_create, 128, R.ROPE_HALF, 1e4, R.ROPE_LINEAR, 5e-324)
    refused(R.ERR_ARG, R.rimuru_rope_create, 128, R.ROPE_HALF, 1e4, R.ROPE_BY_PARTS, 5e-324, 8192.0, 1.0, 4.0)
    refused(R.ERR_ARG, R.rimuru_rope_create, 128, R.ROPE_HALF, 1e4, R.ROPE_BY_PARTS, 4.0, 1e308, -1e308, 1e308)
