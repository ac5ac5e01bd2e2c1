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


@pytest.mark.parametrize("kind,V", [("bf16", 151936), ("f32", 151935)])
def test_more_chunks_than_shared_memory_keeps(kind, V):
    """40 beams: 5960 chunk maxima, which are read again from the workspace."""
    g = torch.Generator(device=DEV).manual_seed(V)
    x = (torch.randn(2 * 40, V, generator=g, device=DEV) * 3).to(TYPES[kind])
    scores = -3 * torch.rand(2, 40, generator=g, device=DEV)
    check(x, scores, K=40)
    check(x, scores, K=128)
    check(x, scores, (torch.rand(2, 40, generator=g, device=DEV) < 0.5).to(torch.uint8), 7, K=80)
    scores[:, 1:] = -math.inf
    check(x, scores, K=16)


@pytest.mark.parametrize("N,K", [(8, 16), (8, 128), (40, 128)])
@pytest.mark.parametrize("kind,V", [("bf16", 151936), ("f32", 151935)])
def test_more_alike_chunks_than_the_list_holds(kind, V, N, K):
    """More than 1024 chunks whose leaders are the same: the first ones by beam and token."""
    x, scores = torch.zeros(N, V, dtype=TYPES[kind], device=DEV), torch.full((1, N), -0.5, device=DEV)
    want = torch.arange(K, dtype=torch.int32, device=DEV)
    _, rows, tokens = select(x, scores, K=K)
    assert torch.equal(rows[0], want * 0) and torch.equal(tokens[0], want)
    x[3, 5000], x[1, V - 1], x[1, 70000] = 1.0, 1.0, 1.0  # a few better ones in beams that this makes different
    scores[0, 2] = -math.inf
    check(x, scores, K=K)
    x[:] = 0
    x[:, ::1024] = 2.0  # a leader in every chunk, better than the rest of it
    _, rows, tokens = select(x, scores * 0, K=K)
    n = (V + 1023) // 1024
    assert torch.equal(rows[0], want // n) and torch.equal(tokens[0], want % n * 1024)


@pytest.mark.parametrize("N,V", [(4, 5003), (16, 300), (128, 77)])
def test_scores_in_place(N, V):
    """The selected sums replace the scores, as a loop over steps may have it; all entries at once."""
    g = torch.Generator(device=DEV).manual_seed(N)
    x, scores = torch.randn(500 * N, V, generator=g, device=DEV).bfloat16(), -torch.rand(500, N, generator=g, device=DEV)
    want = select(x, scores, K=N)
    rows, tokens = (torch.empty(500, N, dtype=torch.int32, device=DEV) for _ in range(2))
    nbytes = R.rimuru_beam_select_workspace_bytes(500, N, V, N)
    ws = torch.empty(nbytes + 1024, dtype=torch.uint8, device=DEV)
    R.rimuru_beam_select(R.rows_of(x), scores.data_ptr(), 0, 500, N, 0, N, scores.data_ptr(), rows.data_ptr(), tokens.data_ptr(),
                         (ws.data_ptr() + 1023) // 1024 * 1024, nbytes, torch.cuda.current_stream().cuda_stream)
    assert all(torch.equal(a, b) for a, b in zip((scores, rows, tokens), want))


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


@pytest.mark.parametrize("what", ["in", "out", "low", "long", "back", "past"])
@pytest.mark.parametrize("max_new", [1, 40, 900])
def test_bystanders_of_bad_tables(max_new, what):
    """Sequences beside one with a bad page or bad offsets are computed as if it were not there; what it
    would have read or written stays, pages as well as rows."""
    new = [1, 1, 1] if max_new == 1 else [max_new, 30, 17]
    c = Case(new, 4, 2, 64, 64, rate=0.02)
    (want, size, states), before, out = c.plain(), c.mem.clone(), c.out.clone()
    hurt, code = [1], R.DEV_BAD_PAGE if what in ("in", "out", "low") else R.DEV_BAD_SHAPE
    pages = c.state_out.tolist()
    if what in ("in", "low"):
        c.state_in[1] = c.pages if what == "in" else -2
    elif what == "out":
        c.state_out[1] = -1
    elif what == "long":  # longer than max_new, and the third one begins past the rows
        c.cu[2] += 2 * max_new
        c.cu[3] = c.cu[2]
        hurt = [1, 2]
    elif what == "back":  # the third one ends before it begins
        c.cu[3] = c.cu[2] - 1
        hurt = [2]
    else:
        c.cu[3] = c.T + 1
        hurt = [2]
    c.run(max_new=max_new)
    torch.cuda.synchronize()
    assert R.rimuru_get_device_error(c.view, True) == code
    rows = torch.tensor([0] + new).cumsum(0).tolist()
    for b in hurt:
        at = slice(rows[b], rows[b + 1])
        assert torch.equal(c.out[at], out[at]) and torch.equal(c.mem[pages[b]], before[pages[b]])
        c.out[at] = want[at].to(c.out.dtype)
        states.pop(pages[b])
    c.check((want, size, states), max_new > 16)


def test_states_pass_on_without_tokens():
    """No tokens at all, in every form of the call: pages are copied, zeros for -1, nothing else changes."""
    for new, max_new in (([0], 0), ([0, 0, 0], 5), ([0] * 5, 1000)):
        c = Case(new, 3, 1, 64, 128, pages=12)
        before = c.mem.clone()
        c.state_in[0] = -1
        c.run(max_new=max_new)
        torch.cuda.synchronize()
        assert R.rimuru_get_device_error(c.view) == R.DEV_OK
        for b in range(c.B):
            want = before[c.state_in[b]] if b else torch.zeros_like(before[0])
            assert torch.equal(c.mem[c.state_out[b]], want)
        others = [p for p in range(12) if p not in c.state_out.tolist()]
        assert torch.equal(c.mem[others], before[others])


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(4, 2, 128, 128), (2, 1, 64, 64)])
@pytest.mark.parametrize("where", ["scores", "state"])
def test_what_parts_of_a_factor_lose(where, shape, kind):
    """Outputs that are the difference of two almost equal products show what each of them has lost.  A factor
    of 2^e to 2^(e + 1) less its nearest bf16 is 2^(e - 8) at most, and a number below that, to the nearest
    bf16, 2^(e - 17) off: 2^-17 of the factor (cut off instead of rounded, the first part would leave twice
    that).  Queries and keys are 1, one part.  fp32's own roundings (a decay, two products, sums) stay
    below 2^-20."""
    c = Case([64, 50, 900], *shape, kind=kind)
    heads, key_heads, dk, dv = shape
    c.scale = 1.0
    c.q.zero_(), c.k.zero_(), c.v.zero_(), c.mem.zero_()
    if where == "scores":  # one key of 1, one of -1 a moment later; what the decays leave of both
        c.q[..., 0] = 1.0
        c.g[:] = -torch.rand(c.T, heads, generator=c.gen, device=DEV) * 0.01
        at = 0
        for n in c.new:
            for first in range(0, n - 1, 64):
                c.k[at + first:at + first + 2, :, 0] = 1.0
                c.v[at + first], c.v[at + first + 1] = 1.0, -1.0
                c.g[at + first + 1] = -2.0 ** -11 * torch.rand(heads, generator=c.gen, device=DEV)
            at += n
        c.g[::64] -= 12.0  # chunks before have little left to say
    else:  # queries that add two rows of the state
        c.q[..., 0] = c.q[..., 1] = 1.0
        c.g.zero_()
        x = torch.rand(c.pages, heads, dv, generator=c.gen, device=DEV) + 1
        c.states()[:, :, 0] = x
        c.states()[:, :, 1] = -x * (1 + 2.0 ** -11 * torch.rand(x.shape, generator=c.gen, device=DEV))
    want, size, _ = c.plain()
    c.run()
    torch.cuda.synchronize()
    tol = torch.finfo(c.out.dtype).eps / 2 * want.abs() + (2.0 ** -17 + 2.0 ** -20) * size
    tol += 2.0 ** -25 if kind == "f16" else 0
    err = (c.out.double() - want).abs()
    assert bool((err <= tol).all()), float((err / (tol + 1e-30)).max())
    assert R.rimuru_get_device_error(c.view) == R.DEV_OK
