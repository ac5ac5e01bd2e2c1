"""Arguments that the norm, linear-attention and beam entry points refuse, without touching a device."""
import math

import pytest
import torch

from paged_moe_shared_gb300 import rimuru as R

BASE = 64 << 20  # a 2 MiB aligned address that is never dereferenced


def refused(status, fn, *args, **kw):
    with pytest.raises(R.RimuruError) as e:
        fn(*args, **kw)
    assert e.value.status == status, (str(e.value), kw)


def heads(data=4096, ts=512, hs=128, n=4, dtype=R.BF16):
    return R.Heads(data, ts, hs, n, dtype)


def norm(weight=4096, eps=1e-6, offset=0.0, dtype=R.BF16):
    return R.HeadNorm(weight, eps, offset, dtype)


@pytest.fixture
def views():
    page = 4 * 128 * 128 * 4
    pool = R.rimuru_pool_create(BASE, 64 * page, page)
    made = [R.rimuru_view_create(pool, page) for _ in range(3)]
    yield made
    for v in made:
        R.rimuru_view_destroy(v)
    R.rimuru_pool_destroy(pool)


def test_norm_rope():
    rope = R.rimuru_rope_create(64)

    def go(x=None, y=None, n=None, tokens=1, dim=128, pos=4096, rope=rope, count=1):
        R.rimuru_norm_rope_apply(rope, pos, tokens, dim, [x or heads()] * count, [y or heads()] * count,
                                 [n or norm()] * count, 0)

    for kw, st in ((dict(tokens=-1), R.ERR_ARG), (dict(dim=56), R.ERR_UNSUPPORTED), (dict(dim=100), R.ERR_UNSUPPORTED),
                   (dict(dim=1032), R.ERR_UNSUPPORTED), (dict(dim=0), R.ERR_UNSUPPORTED),
                   (dict(dim=0, rope=None), R.ERR_UNSUPPORTED), (dict(pos=0), R.ERR_ARG), (dict(pos=4098), R.ERR_ALIGN),
                   (dict(x=heads(data=0)), R.ERR_ARG), (dict(x=heads(data=4104)), R.ERR_ALIGN),
                   (dict(x=heads(ts=4)), R.ERR_ALIGN), (dict(y=heads(hs=-8)), R.ERR_ARG), (dict(y=heads(n=3)), R.ERR_ARG),
                   (dict(y=heads(dtype=R.F16)), R.ERR_ARG), (dict(x=heads(dtype=7)), R.ERR_ARG),
                   (dict(n=norm(eps=0.0)), R.ERR_ARG), (dict(n=norm(eps=1e-30)), R.ERR_ARG),
                   (dict(n=norm(eps=math.nan)), R.ERR_ARG), (dict(n=norm(eps=2.0)), R.ERR_ARG),
                   (dict(n=norm(offset=math.inf)), R.ERR_ARG), (dict(n=norm(offset=1e39)), R.ERR_ARG),
                   (dict(n=norm(weight=4104)), R.ERR_ALIGN), (dict(n=norm(dtype=5)), R.ERR_ARG),
                   (dict(count=5), R.ERR_ARG), (dict(x=heads(n=1 << 21), y=heads(n=1 << 21)), R.ERR_UNSUPPORTED)):
        refused(st, go, **kw)
    go(tokens=0)
    with pytest.raises(ValueError):
        R.rimuru_norm_rope_apply(rope, 4096, 1, 128, [heads()], [heads()], [])
    R.rimuru_rope_destroy(rope)


def test_state_shape(views):
    a, b, c = views
    shape = R.rimuru_view_set_state_shape
    for args, st in (((0, 128, 128), R.ERR_ARG), ((4, -1, 128), R.ERR_ARG), ((4, 96, 128), R.ERR_UNSUPPORTED),
                     ((4, 128, 256), R.ERR_UNSUPPORTED), ((5, 128, 128), R.ERR_UNSUPPORTED),
                     ((1025, 64, 64), R.ERR_UNSUPPORTED)):
        refused(st, shape, a, *args)
    shape(a, 4, 128, 128)
    refused(R.ERR_STATE, shape, a, 4, 128, 128)
    refused(R.ERR_STATE, R.rimuru_view_set_moe_shape, a, 1, 8, 256, 128, 2, 1)
    refused(R.ERR_STATE, R.rimuru_view_set_kv_shape, a, 2, 128, 16, 4096, 1 << 20)
    refused(R.ERR_STATE, R.rimuru_kv_copy_pages, a, 16, 16, 1)
    R.rimuru_view_set_moe_shape(b, 1, 8, 256, 128, 2, 1)
    refused(R.ERR_STATE, shape, b, 4, 128, 128)
    R.rimuru_view_set_kv_shape(c, 2, 128, 16, 4096, 1 << 20)
    refused(R.ERR_STATE, shape, c, 4, 128, 128)
    assert R.rimuru_get_device_error(a) == R.DEV_OK


def test_linear_attention(views):
    view, other, _ = views
    assert R.rimuru_linear_attention_workspace_bytes(view, 1, 1, 1) == 0
    R.rimuru_view_set_state_shape(view, 4, 128, 128)
    assert R.rimuru_linear_attention_workspace_bytes(view, -1, 1, 1) == 0
    assert R.rimuru_linear_attention_workspace_bytes(view, 1, 1, -1) == 0

    def go(view=view, q=None, k=None, v=None, o=None, g=4096, gts=4, ghs=1, cu=4096, seqs=1, tokens=8, most=8, sin=4096,
           sout=4096, scale=1.0, ws=4096, nbytes=1 << 40):
        R.rimuru_linear_attention(view, q or heads(), k or heads(), v or heads(), o or heads(), g, gts, ghs, cu, seqs,
                                  tokens, most, sin, sout, scale, ws, nbytes)

    bad = [(dict(view=other), R.ERR_STATE), (dict(seqs=-1), R.ERR_ARG), (dict(tokens=-1), R.ERR_ARG),
           (dict(most=-1), R.ERR_ARG), (dict(scale=math.nan), R.ERR_ARG), (dict(scale=1e39), R.ERR_ARG),
           (dict(q=heads(n=3), k=heads(n=3)), R.ERR_UNSUPPORTED), (dict(q=heads(n=2)), R.ERR_ARG),
           (dict(v=heads(n=2)), R.ERR_ARG), (dict(o=heads(n=8)), R.ERR_ARG), (dict(q=heads(dtype=R.F32)), R.ERR_UNSUPPORTED),
           (dict(v=heads(dtype=R.F16)), R.ERR_ARG), (dict(o=heads(data=4100)), R.ERR_ALIGN),
           (dict(k=heads(ts=12)), R.ERR_ALIGN), (dict(g=0), R.ERR_ARG), (dict(g=4098), R.ERR_ALIGN),
           (dict(gts=-1), R.ERR_ARG), (dict(ghs=-1), R.ERR_ARG), (dict(cu=0), R.ERR_ARG), (dict(cu=4097), R.ERR_ALIGN),
           (dict(sin=0), R.ERR_ARG), (dict(sout=0), R.ERR_ARG), (dict(sout=4099), R.ERR_ALIGN), (dict(ws=0), R.ERR_ARG),
           (dict(ws=4096 + 512), R.ERR_ALIGN), (dict(nbytes=0), R.ERR_WORKSPACE),
           (dict(seqs=1 << 29, tokens=1 << 29, most=1), R.ERR_UNSUPPORTED), (dict(q=heads(ts=0)), R.ERR_UNSUPPORTED),
           (dict(v=heads(ts=0)), R.ERR_UNSUPPORTED), (dict(o=heads(ts=0)), R.ERR_UNSUPPORTED),
           (dict(o=heads(hs=0)), R.ERR_UNSUPPORTED)]
    for kw, st in bad:
        refused(st, go, **kw)
    go(seqs=0)


def test_beam_select():
    assert R.rimuru_beam_select_workspace_bytes(1, 0, 10, 1) == 0
    assert R.rimuru_beam_select_workspace_bytes(-1, 1, 10, 1) == 0
    assert R.rimuru_beam_select_workspace_bytes(1, 1, 0, 1) == 0

    def go(data=4096, stride=1000, cols=1000, dtype=R.BF16, scores=4096, done=0, groups=2, beams=4, pad=0, k=8, a=4096,
           b=4096, c=4096, ws=4096, nbytes=1 << 40):
        R.rimuru_beam_select(R.Rows(data, stride, cols, dtype), scores, done, groups, beams, pad, k, a, b, c, ws, nbytes)

    bad = [(dict(groups=-1), R.ERR_ARG), (dict(beams=0), R.ERR_ARG), (dict(k=0), R.ERR_ARG), (dict(cols=0), R.ERR_ARG),
           (dict(beams=129), R.ERR_UNSUPPORTED), (dict(k=129), R.ERR_UNSUPPORTED), (dict(dtype=3), R.ERR_ARG),
           (dict(cols=2 ** 31 - 1), R.ERR_UNSUPPORTED), (dict(groups=1 << 25), R.ERR_UNSUPPORTED),
           (dict(data=0), R.ERR_ARG), (dict(data=4097), R.ERR_ALIGN), (dict(stride=-1), R.ERR_ARG),
           (dict(scores=0), R.ERR_ARG), (dict(scores=4098), R.ERR_ALIGN), (dict(a=0), R.ERR_ARG), (dict(b=0), R.ERR_ARG),
           (dict(c=0), R.ERR_ARG), (dict(c=4097), R.ERR_ALIGN), (dict(done=4096, pad=-1), R.ERR_ARG),
           (dict(done=4096, pad=1000), R.ERR_ARG), (dict(ws=0), R.ERR_ARG), (dict(ws=4608), R.ERR_ALIGN),
           (dict(nbytes=100), R.ERR_WORKSPACE)]
    for kw, st in bad:
        refused(st, go, **kw)
    go(groups=0)


def test_kv_reorder(views):
    kv, other, _ = views
    R.rimuru_view_set_kv_shape(kv, 2, 128, 16, 4096, 1 << 20)

    def go(view=kv, parents=4096, n=2, lens=4096, n_parents=2, a=4096, b=8192, layers=1, stride=4, fresh=4096, out=8192):
        R.rimuru_kv_reorder(view, parents, n, lens, n_parents, a, b, layers, stride, fresh, out)

    bad = [(dict(view=other), R.ERR_STATE), (dict(n=-1), R.ERR_ARG), (dict(n_parents=-1), R.ERR_ARG),
           (dict(layers=-1), R.ERR_ARG), (dict(parents=0), R.ERR_ARG), (dict(lens=0), R.ERR_ARG), (dict(a=0), R.ERR_ARG),
           (dict(b=0), R.ERR_ARG), (dict(fresh=0), R.ERR_ARG), (dict(out=0), R.ERR_ARG), (dict(stride=0), R.ERR_ARG),
           (dict(layers=65536), R.ERR_UNSUPPORTED), (dict(b=4096), R.ERR_ARG), (dict(out=4096), R.ERR_ARG),
           (dict(parents=4097), R.ERR_ALIGN)]
    for kw, st in bad:
        refused(st, go, **kw)
    go(n=0)
    go(layers=0)


def test_descriptors_of_the_wrong_kind_are_refused():
    x = torch.zeros(2, 3, 64)
    heads, norm = R.heads_of(x), R.head_norm_of(None)
    for ins, outs, norms in (([heads], [norm], [norm]), ([heads], [heads], [heads]), ([x], [heads], [norm])):
        with pytest.raises(TypeError):
            R.rimuru_norm_rope_apply(None, 0, 2, 64, ins, outs, norms)
    with pytest.raises(ValueError):
        R.head_norm_of(torch.zeros(128)[::2])
    with pytest.raises(ValueError):
        R.rows_of(torch.zeros(64, 4).t())
