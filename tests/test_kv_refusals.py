"""Arguments that the KV-cache and rotary entry points refuse, without touching a device."""
import ctypes

import pytest

from paged_moe_shared_gb300 import rimuru as R

BASE = 64 << 20  # a 2 MiB aligned address that is never dereferenced


def refused(status, fn, *args):
    with pytest.raises(R.RimuruError) as e:
        fn(*args)
    assert e.value.status == status, str(e.value)


@pytest.fixture
def views():
    page = 2 * 2 * 128 * 16
    pool = R.rimuru_pool_create(BASE, 64 * page, 16 * page)
    kv, other = R.rimuru_view_create(pool, page), R.rimuru_view_create(pool, 16 * page)
    yield pool, kv, other, page
    R.rimuru_view_destroy(kv)
    R.rimuru_view_destroy(other)
    R.rimuru_pool_destroy(pool)


def shape(view, heads=2, dim=128, tokens=16, scales=4096, nbytes=1 << 20):
    R.rimuru_view_set_kv_shape(view, heads, dim, tokens, scales, nbytes)


def heads(data=4096, ts=256, hs=128, n=2, dtype=R.BF16):
    return R.Heads(data, ts, hs, n, dtype)


def test_kv_shape(views):
    _, kv, other, page = views
    for kw, st in ((dict(heads=0), R.ERR_ARG), (dict(dim=-1), R.ERR_ARG), (dict(scales=0), R.ERR_ARG),
                   (dict(scales=4100), R.ERR_ALIGN), (dict(dim=96), R.ERR_UNSUPPORTED),
                   (dict(tokens=24), R.ERR_UNSUPPORTED), (dict(heads=3), R.ERR_UNSUPPORTED),
                   (dict(tokens=32), R.ERR_UNSUPPORTED), (dict(nbytes=64 * 2 * 2 * 4 - 1), R.ERR_ARG)):
        with pytest.raises(R.RimuruError) as e:
            shape(kv, **kw)
        assert e.value.status == st, kw
    assert R.rimuru_kv_scale_bytes(kv, 2) == 64 * 2 * 2 * 4
    assert R.rimuru_kv_scale_bytes(kv, 0) == 0
    shape(kv)
    refused(R.ERR_STATE, shape, kv)
    refused(R.ERR_STATE, R.rimuru_view_set_moe_shape, kv, 1, 8, 256, 128, 2, 1)
    assert R.rimuru_get_device_error(kv) == R.DEV_OK


def test_operators_need_the_shape(views):
    _, kv, _, _ = views
    refused(R.ERR_STATE, R.rimuru_kv_append, kv, heads(), heads(), 16, 16, 1, 1, 16, 4)
    refused(R.ERR_STATE, R.rimuru_kv_attention, kv, heads(), heads(), 0, 0, 16, 1, 1, 1, 16, 4, 1.0, 0, 1024, 1024)
    refused(R.ERR_STATE, R.rimuru_kv_copy_pages, kv, 16, 16, 1)
    refused(R.ERR_STATE, R.rimuru_kv_fork, kv, [0], 16, 1)
    refused(R.ERR_STATE, R.rimuru_kv_compact, kv, [0], 1)
    assert R.rimuru_kv_attention_workspace_bytes(kv, 2, 1, 1, 1) == 0


def test_append(views):
    _, kv, _, _ = views
    shape(kv)

    def go(k=None, v=None, cu=16, lens=16, seqs=1, tokens=1, table=16, stride=4):
        R.rimuru_kv_append(kv, k or heads(), v or heads(), cu, lens, seqs, tokens, table, stride)

    for kw, st in ((dict(seqs=-1), R.ERR_ARG), (dict(tokens=-1), R.ERR_ARG), (dict(k=heads(n=3)), R.ERR_ARG),
                   (dict(v=heads(dtype=R.F16)), R.ERR_ARG), (dict(k=heads(dtype=9)), R.ERR_ARG),
                   (dict(k=heads(data=0)), R.ERR_ARG), (dict(k=heads(data=4104)), R.ERR_ALIGN),
                   (dict(v=heads(ts=260)), R.ERR_ALIGN), (dict(v=heads(hs=4)), R.ERR_ALIGN),
                   (dict(v=heads(ts=-256)), R.ERR_ARG), (dict(cu=0), R.ERR_ARG), (dict(lens=0), R.ERR_ARG),
                   (dict(table=0), R.ERR_ARG), (dict(stride=0), R.ERR_ARG)):
        with pytest.raises(R.RimuruError) as e:
            go(**kw)
        assert e.value.status == st, kw
    go(seqs=0, tokens=0)
    go(tokens=0)


def test_attention(views):
    _, kv, _, _ = views
    shape(kv)
    need = R.rimuru_kv_attention_workspace_bytes(kv, 8, 1, 1, 1)
    assert need > 0
    assert R.rimuru_kv_attention_workspace_bytes(kv, 7, 1, 1, 1) == 0

    def go(q=None, out=None, cu=0, lens=16, seqs=1, rows=1, max_q=1, table=16, stride=4, scale=1.0,
           window=0, ws=4096, nbytes=need):
        R.rimuru_kv_attention(kv, q or heads(n=8), out or heads(n=8), 0, cu, lens, seqs, rows, max_q,
                              table, stride, scale, window, ws, nbytes)

    for kw, st in ((dict(seqs=-1), R.ERR_ARG), (dict(rows=-1), R.ERR_ARG), (dict(max_q=-1), R.ERR_ARG),
                   (dict(window=-1), R.ERR_ARG), (dict(scale=float("nan")), R.ERR_ARG),
                   (dict(scale=float("inf")), R.ERR_ARG), (dict(rows=2), R.ERR_ARG),
                   (dict(q=heads(n=8, dtype=R.F32), out=heads(n=8, dtype=R.F32)), R.ERR_UNSUPPORTED),
                   (dict(out=heads(n=8, dtype=R.F16)), R.ERR_ARG), (dict(out=heads(n=4)), R.ERR_ARG),
                   (dict(q=heads(n=7), out=heads(n=7)), R.ERR_UNSUPPORTED), (dict(lens=0), R.ERR_ARG),
                   (dict(table=0), R.ERR_ARG), (dict(stride=0), R.ERR_ARG), (dict(ws=0), R.ERR_ARG),
                   (dict(ws=4112), R.ERR_ALIGN), (dict(nbytes=need - 1), R.ERR_WORKSPACE),
                   (dict(q=heads(n=8, data=4098)), R.ERR_ALIGN),
                   (dict(q=heads(n=258), out=heads(n=258)), R.ERR_UNSUPPORTED),
                   (dict(stride=1 << 40), R.ERR_UNSUPPORTED)):
        with pytest.raises(R.RimuruError) as e:
            go(**kw)
        assert e.value.status == st, kw
    go(seqs=0, rows=0)


def test_pages(views):
    _, kv, _, _ = views
    shape(kv)
    refused(R.ERR_ARG, R.rimuru_kv_copy_pages, kv, 16, 16, -1)
    refused(R.ERR_ARG, R.rimuru_kv_copy_pages, kv, 0, 16, 1)
    R.rimuru_kv_copy_pages(kv, 0, 0, 0)
    a, b = R.rimuru_page_alloc(kv), R.rimuru_page_alloc(kv)
    refused(R.ERR_STATE, R.rimuru_kv_fork, kv, [a, 63], 32, 1)
    refused(R.ERR_RANGE, R.rimuru_kv_fork, kv, [a, 64], 32, 1)
    refused(R.ERR_ARG, R.rimuru_kv_fork, kv, [a], 32, 1)  # rows shorter than the sequence
    refused(R.ERR_ARG, R.rimuru_kv_fork, kv, [a], -1, 1)
    assert R.rimuru_kv_fork(kv, [a, b], 32, 2) == [[a, b], [a, b]]  # full pages: nothing to copy
    assert R.rimuru_page_refs(kv, a) == 3
    for _ in range(3):
        R.rimuru_page_free(kv, a)
    refused(R.ERR_STATE, R.rimuru_page_free, kv, a)
    refused(R.ERR_STATE, R.rimuru_page_share, kv, a)
    refused(R.ERR_RANGE, R.rimuru_page_share, kv, 64)
    refused(R.ERR_RANGE, R.rimuru_page_refs, kv, -1)
    assert R.rimuru_page_refs(kv, a) == 0
    refused(R.ERR_ARG, R.rimuru_kv_compact, kv, [b], -1)
    assert R.rimuru_kv_compact(kv, [b], 0) == ([b], 0)
    assert R.rimuru_kv_compact(kv, [], 5) == ([], 0)


def test_rope():
    ok = (128, R.ROPE_HALF, 10000.0, R.ROPE_PLAIN, 1.0, 0.0, 0.0, 0.0, 1.0)

    def with_(i, x):
        return ok[:i] + (x,) + ok[i + 1:]

    nan = float("nan")
    for args, st in ((with_(0, 0), R.ERR_UNSUPPORTED), (with_(0, 258), R.ERR_UNSUPPORTED),
                     (with_(0, 24), R.ERR_UNSUPPORTED), (with_(1, 2), R.ERR_ARG), (with_(2, 1.0), R.ERR_ARG),
                     (with_(2, nan), R.ERR_ARG), (with_(3, 4), R.ERR_ARG), (with_(8, nan), R.ERR_ARG),
                     ((128, 0, 1e4, R.ROPE_LINEAR, 0.0, 0, 0, 0, 1.0), R.ERR_ARG),
                     ((128, 0, 1e4, R.ROPE_BY_PARTS, 2.0, 0.0, 1, 4, 1.0), R.ERR_ARG),
                     ((128, 0, 1e4, R.ROPE_BY_PARTS, 2.0, 8192, 4, 4, 1.0), R.ERR_ARG)):
        refused(st, R.rimuru_rope_create, *args)
    r = R.rimuru_rope_create(*ok)

    def go(i=None, o=None, pos=16, T=1, dim=128):
        R.rimuru_rope_apply(r, pos, T, dim, [i or heads()], [o or heads()])

    for kw, st in ((dict(T=-1), R.ERR_ARG), (dict(pos=0), R.ERR_ARG), (dict(dim=64), R.ERR_UNSUPPORTED),
                   (dict(dim=132), R.ERR_UNSUPPORTED), (dict(pos=18), R.ERR_ALIGN),
                   (dict(o=heads(n=3)), R.ERR_ARG), (dict(o=heads(dtype=R.F16)), R.ERR_ARG),
                   (dict(i=heads(data=0)), R.ERR_ARG), (dict(o=heads(data=4104)), R.ERR_ALIGN),
                   (dict(i=heads(ts=100)), R.ERR_ALIGN)):
        with pytest.raises(R.RimuruError) as e:
            go(**kw)
        assert e.value.status == st, kw
    go(T=0)
    refused(R.ERR_ARG, R.rimuru_rope_apply, r, 16, 1, 128, [], [])
    refused(R.ERR_ARG, R.rimuru_rope_apply, r, 16, 1, 128, [heads()] * 5, [heads()] * 5)
    R.rimuru_rope_destroy(r)
    refused(R.ERR_ARG, R.rimuru_rope_destroy, None)


def test_heads_struct_matches_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(R.__file__), "..", "include", "rimuru.h")).read()
    body = re.search(r"typedef struct rimuru_heads \{(.*?)\} rimuru_heads;", text, re.S).group(1)
    names = re.findall(r"(\w+)\s*;", re.sub(r"/\*.*?\*/", "", body))
    assert names == [n for n, _ in R.Heads._fields_]
    assert ctypes.sizeof(R.Heads) == 32
