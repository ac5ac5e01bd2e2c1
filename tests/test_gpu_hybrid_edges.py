"""Norms, linear attention and beam selection where they can go wrong: many CTAs beside other work, ties
over rows that begin anywhere, tokens that are not finite, histories that are forgotten."""
import math

import pytest
import torch

from paged_moe_shared_gb300 import rimuru as R
from test_gpu_beam import TYPES, check, plain, select
from test_gpu_linear import Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


# ------------------------------------------------------------------ selection
@pytest.mark.parametrize("V,N,K", [(5000, 3, 5), (1001, 4, 8), (70, 2, 3)])
def test_every_entry_beside_other_work(V, N, K):
    """Many entries, again and again while another stream keeps the SMs and their caches busy: no
    candidate is lost where some warps of an entry are late."""
    g = torch.Generator(device=DEV).manual_seed(V)
    logits = torch.randn(2000 * N, V, generator=g, device=DEV).bfloat16()
    scores = -torch.rand(2000, N, generator=g, device=DEV)
    want, rows, tokens = plain(logits, scores, None, 0, K)
    ws = torch.empty(R.rimuru_beam_select_workspace_bytes(2000, N, V, K) + 1024, dtype=torch.uint8, device=DEV)
    busy, other = torch.randn(1 << 24, device=DEV), torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        with torch.cuda.stream(other):
            busy.mul_(1.0)
        best, r, t = select(logits, scores, K=K, ws=ws)
        assert torch.equal(r, rows) and torch.equal(t, tokens)
        assert bool(((best.double() - want).abs() <= 2.0 ** -24 * want.abs() + 2.0 ** -18).all())


# ------------------------------------------------------------------ linear attention
@pytest.mark.parametrize("new", [[1000, 700], [64 * 20] * 9])
def test_f16_prompts_beside_other_work(new):
    """Many chunks while another stream takes issue slots and caches: every pass ends in time and is the same."""
    c = Case(new, 16, 8, 128, 128, kind="f16", rate=0.02)
    c.run()
    torch.cuda.synchronize()
    out, states = c.out.clone(), c.mem[c.state_out.long()].clone()
    assert bool(out.isfinite().all())
    busy, other = torch.randn(1 << 24, device=DEV), torch.cuda.Stream()
    for _ in range(30):
        with torch.cuda.stream(other):
            busy.mul_(1.0)
        c.out.zero_()
        c.run(ws=c.ws)
        assert torch.equal(c.out, out) and torch.equal(c.mem[c.state_out.long()], states)
    assert R.rimuru_get_device_error(c.view) == R.DEV_OK


def in_order(row, beams, K):
    """The K best of equal beams with equal scores: by the logit, then the beam, then the token."""
    x = row.double().nan_to_num(nan=-math.inf).expand(beams, -1).flatten()
    at = torch.sort(x, descending=True, stable=True)[1][:K]
    return (at // len(row)).int(), (at % len(row)).int()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V,N,stride", [(50257, 9, 50257), (1001, 12, 1001), (151935, 8, 151937), (7, 16, 7), (2049, 8, 2050),
                                        (1024, 8, 1027), (8191, 9, 8193)])
def test_equal_beams_tie_wherever_their_rows_begin(V, N, stride, kind):
    """Beams that are alike have sums that are alike to the last bit: a first step from one prompt selects
    by beam and token, not by where a row lies."""
    g = torch.Generator(device=DEV).manual_seed(V)
    for first in range(2):
        x = torch.full((1 + 2 * N * stride,), math.inf, dtype=TYPES[kind], device=DEV)[first:first + 2 * N * stride].view(2 * N, stride)[:, :V]
        K = min(3 * N, 128)
        for e in range(2):
            x[e * N:(e + 1) * N] = (torch.randn(V, generator=g, device=DEV) * 3).to(x.dtype)
        best, rows, tokens = select(x, torch.full((2, N), -1.5, device=DEV), K=K)
        for e in range(2):
            want_b, want_t = in_order(x[e * N], N, K)
            assert torch.equal(rows[e, :len(want_b)], want_b + e * N) and torch.equal(tokens[e, :len(want_b)], want_t)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(4, 2, 128, 128), (2, 1, 64, 128), (2, 2, 128, 64)])
@pytest.mark.parametrize("new", [[5, 3], [64, 40], [17, 200], [1300]])
def test_a_history_that_is_forgotten_leaves_nothing(new, shape, kind):
    """States far larger than what comes, and decays that forget them in one token, over a few or not at
    all: what is left of them in the outputs is what the formula leaves, also far below 2^-64."""
    c = Case(new, *shape, kind=kind, rate=0.02)
    c.mem *= 1e25
    c.g[:] = torch.where(torch.rand(c.T, c.H, generator=c.gen, device=DEV) < 0.15,
                         -torch.rand(c.T, c.H, generator=c.gen, device=DEV) * 120, c.g)
    first = 0
    for b, n in enumerate(new):
        c.g[first] = torch.linspace(-48, -90, c.H, device=DEV)  # 1e25 becomes 10^4 to 10^-14
        c.g[first + min(n - 1, 2), 0] = -math.inf
        c.g[first + n // 2, -1] = -math.inf
        first += n
    want = c.plain()
    c.run()
    c.check(want, max(new) > 16)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(4, 2, 128, 128), (2, 1, 64, 128), (2, 2, 128, 64)])
@pytest.mark.parametrize("new", [[64], [9, 100, 33], [63, 130], [1300, 40]])
def test_a_value_that_is_not_finite_reaches_no_earlier_token(new, shape, kind):
    """A NaN or an infinity among the values makes its column of the head NaN or infinite from its token
    on; the tokens before it, other columns, heads and sequences are what they are without it."""
    c = Case(new, *shape, kind=kind, rate=0.02)
    chunked = max(new) > 16
    heads, dv = shape[0], shape[3]
    g = torch.Generator().manual_seed(sum(new))
    hurt = torch.zeros(c.T, heads, dv, dtype=torch.bool, device=DEV)
    lost = {}
    clean, first = c.v.clone(), 0
    for b, n in enumerate(new):
        for k in range(6):
            t = [0, n - 1, n // 2, 5 % n][k] if k < 4 else int(torch.randint(0, n, (1,), generator=g))
            h, col = k % heads, int(torch.randint(0, dv, (1,), generator=g))
            c.v[first + t, h, col] = [math.nan, math.inf, -math.inf][k % 3]
            clean[first + t, h, col] = 0
            hurt[first + t:first + n, h, col] = True
            lost.setdefault(int(c.state_out[b]), set()).add((h, col))
        first += n
    bad, c.v = c.v, clean
    want = c.plain()
    c.v = bad
    c.run()
    torch.cuda.synchronize()
    assert not bool(c.out[hurt].isfinite().any())
    c.out = torch.where(hurt, want[0].to(c.out.dtype), c.out)
    for page, places in lost.items():
        for h, col in places:
            assert not bool(c.states()[page, h, :, col].isfinite().any())
            c.states()[page, h, :, col] = want[2][page][0][h, :, col].float()
    c.check(want, chunked)
