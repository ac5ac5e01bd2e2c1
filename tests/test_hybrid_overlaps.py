"""Outputs that lie on inputs or on one another are refused, without touching a device."""
import pytest

from paged_moe_shared_gb300 import rimuru as R
from test_hybrid_refusals import heads, norm, refused


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
