"""Outputs that lie on inputs or on one another are refused, without touching a device."""
import pytest

from paged_moe_shared_gb300 import rimuru as R
from test_hybrid_refusals import heads, norm, refused, views  # noqa: F401


@pytest.fixture(autouse=True)
def no_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses that a device must not see")


def test_norm_rope_outputs_on_one_another():
    def go(x, y, tokens=2):
        R.rimuru_norm_rope_apply(None, 0, tokens, 128, [x], [y], [norm()], 0)

    refused(R.ERR_UNSUPPORTED, go, heads(), heads(ts=0))
    refused(R.ERR_UNSUPPORTED, go, heads(), heads(hs=0))
    refused(R.ERR_UNSUPPORTED, go, heads(ts=0), heads(ts=0))
    # one token, or one head, lies on nothing, and inputs may: these get as far as the device
    for x, y, tokens in ((heads(), heads(data=1 << 20, ts=0), 1), (heads(n=1), heads(data=1 << 20, n=1, hs=0), 2),
                         (heads(ts=0, hs=0), heads(data=1 << 20), 2)):
        refused(R.ERR_CUDA, go, x, y, tokens)


def test_selection_over_its_scores():
    def go(scores, out, n_select, beams=4):
        R.rimuru_beam_select(R.Rows(4096, 1000, 1000, R.BF16), scores, 0, 2, beams, 0, n_select, out, 1 << 20, 2 << 20,
                             4096, 1 << 30)

    refused(R.ERR_ARG, go, 8192, 8192, 8)   # another entry's scores would be overwritten
    refused(R.ERR_ARG, go, 8192, 8192, 3)
    refused(R.ERR_ARG, go, 8192, 8192 + 16, 4)
    refused(R.ERR_ARG, go, 8192, 8192 - 28, 4)
    refused(R.ERR_CUDA, go, 8192, 8192, 4)  # each entry's own: gets as far as the device
    refused(R.ERR_CUDA, go, 8192, 8192 + 32, 4)
    refused(R.ERR_CUDA, go, 8192, 8192 - 32, 4)


def test_linear_attention_over_its_inputs(views):  # noqa: F811
    view = views[0]
    R.rimuru_view_set_state_shape(view, 4, 128, 128)

    def go(q, k, v, o):
        R.rimuru_linear_attention(view, q, k, v, o, 4096, 4, 1, 4096, 1, 8, 8, 4096, 4096, 1.0, 4096, 1 << 40)

    a, b, c, d = (heads(data=i << 20) for i in range(1, 5))
    for which in (a, b, c):
        refused(R.ERR_ARG, go, a, b, c, which)
    refused(R.ERR_CUDA, go, a, b, c, d)
    refused(R.ERR_CUDA, go, a, a, a, d)  # inputs may be one array
