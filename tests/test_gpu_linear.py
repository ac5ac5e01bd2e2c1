"""Linear attention on state pages against the recurrence in 64 bits, token by token."""
import math

import pytest
import torch

from paged_moe_shared_gb300 import rimuru as R
from paged_moe_shared_gb300.device_pool import DevicePool

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


class Case:
    """A pool of state pages and one call's tensors."""

    def __init__(self, new, heads, key_heads, dk, dv, kind="bf16", seed=0, pages=None, spare=0, rate=0.3):
        g = self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.new, self.B, self.H, self.Hk, self.dk, self.dv = list(new), len(new), heads, key_heads, dk, dv
        self.T = sum(new)
        self.pages = pages or 2 * self.B + 2
        self.page_bytes = heads * dk * dv * 4 + spare
        self.pool = DevicePool(self.pages * self.page_bytes, self.page_bytes, DEV)
        self.view = self.pool.view(self.page_bytes)
        R.rimuru_view_set_state_shape(self.view, heads, dk, dv)
        self.mem = self.pool.mem.view(torch.float32).view(self.pages, -1)
        self.mem.normal_(generator=g)
        dt = TYPES[kind]
        self.q, self.k = (self.rand(self.T, key_heads, dk) * dk ** -0.5).to(dt), (self.rand(self.T, key_heads, dk) * dk ** -0.5).to(dt)
        self.v = self.rand(self.T, heads, dv).to(dt)
        self.out = torch.full((self.T, heads, dv), 7.0, dtype=dt, device=DEV)
        self.g = -rate * self.rand(self.T, heads).exp()
        self.cu = torch.tensor([0] + self.new).cumsum(0).to(torch.int32).to(DEV)
        order = torch.randperm(self.pages, generator=g, device=DEV).to(torch.int32)
        self.state_in, self.state_out = order[:self.B].clone(), order[self.B:2 * self.B].clone()
        self.scale = 0.7

    def rand(self, *shape):
        return torch.randn(shape, generator=self.gen, device=DEV)

    def states(self):
        return self.mem[:, :self.H * self.dk * self.dv].view(self.pages, self.H, self.dk, self.dv)

    def run(self, max_new=None, cu=True, stream=None, ws=None):
        max_new = max(self.new + [0]) if max_new is None else max_new
        nbytes = R.rimuru_linear_attention_workspace_bytes(self.view, self.B, self.T, max_new)
        if ws is None:
            ws = torch.full((nbytes + 1024,), 0xFF, dtype=torch.uint8, device=DEV)
        self.ws = ws
        gs = self.g.stride() if self.g.dim() == 2 else (0, self.g.stride(0))
        R.rimuru_linear_attention(self.view, R.heads_of(self.q), R.heads_of(self.k), R.heads_of(self.v),
                                  R.heads_of(self.out), self.g.data_ptr(), *gs, self.cu.data_ptr() if cu else 0,
                                  self.B, self.T, max_new, self.state_in.data_ptr(), self.state_out.data_ptr(),
                                  self.scale, (ws.data_ptr() + 1023) // 1024 * 1024, nbytes,
                                  (stream or torch.cuda.current_stream()).cuda_stream)

    def plain(self):
        """(out, {page: state}) in 64 bits, and the same of the magnitudes, which bound the rounding."""
        per = self.H // self.Hk
        got, size = (torch.zeros(self.T, self.H, self.dv, dtype=torch.float64, device=DEV) for _ in range(2))
        states, first = {}, 0
        start = self.states().double().clone()
        g = self.g.expand(self.T, self.H).double()
        for b, n in enumerate(self.new):
            p = int(self.state_in[b])
            S = start[p].clone() if p >= 0 else torch.zeros_like(start[0])
            A = S.abs()
            for t in range(first, first + n):
                q, k = (x[t].double().repeat_interleave(per, 0) for x in (self.q, self.k))
                v, f = self.v[t].double(), g[t].exp()[:, None, None]
                S = torch.where(f > 0, S * f, 0.0) + k[:, :, None] * v[:, None]
                A = torch.where(f > 0, A * f, 0.0) + k[:, :, None].abs() * v[:, None].abs()
                got[t] = self.scale * (q[:, :, None] * S).sum(1)
                size[t] = self.scale * (q[:, :, None].abs() * A).sum(1)
            states[int(self.state_out[b])] = (S, A)
            first += n
        return got, size, states

    def check(self, plain, chunked):
        """Recurrent: a state element takes 2 roundings a token, which later decays only shrink, and the
        dot product at most 28 (the key rows of a thread, then partial sums): 2^-24 (2 n + 28) of the sum
        of magnitudes.  Chunked: every factor that is split is good to 2^-16, a product of two of
        them and the fp32 sums of a chunk stay below 2^-14; a state's factors to 2^-21 with its sums."""
        out, size, states = plain
        n = max(self.new + [1])
        e_out = 2.0 ** -14 if chunked else 2.0 ** -24 * (2 * n + 28)
        tol = torch.finfo(self.out.dtype).eps / 2 * out.abs() + e_out * size + (2.0 ** -25 if self.out.dtype == torch.float16 else 0)
        err = (self.out.double() - out).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
        e_state = 2.0 ** -20 if chunked else 2.0 ** -23 * (n + 2)
        for page, (S, A) in states.items():
            err = (self.states()[page].double() - S).abs()
            assert bool((err <= e_state * A + 1e-30).all()), float((err / (A + 1e-30)).max())
        torch.cuda.synchronize()
        assert R.rimuru_get_device_error(self.view) == R.DEV_OK


SHAPES = [(4, 2, 128, 128), (3, 1, 64, 128), (2, 2, 128, 64), (6, 3, 64, 64)]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("new", [[1], [1] * 9, [3, 0, 1, 5], [16, 2], [8], [9]])
def test_steps(new, shape, kind):
    c = Case(new, *shape, kind=kind, seed=len(new))
    c.state_in[0] = -1
    want, before = c.plain(), c.mem.clone()
    c.run()
    c.check(want, False)
    others = [p for p in range(c.pages) if p not in want[2]]
    assert torch.equal(c.mem[others], before[others])


@pytest.mark.parametrize("B,heads", [(80, 8), (3, 152)])
def test_many_states(B, heads):
    c = Case([1] * B, heads, heads // 2, 128, 128)
    want = c.plain()
    c.run(cu=False)
    c.check(want, False)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("new", [[17], [64], [65, 1, 0, 130], [128, 127, 129], [300], [33, 513, 18]])
def test_chunks(new, shape, kind):
    c = Case(new, *shape, kind=kind, seed=len(new))
    c.state_in[-1] = -1
    want, before = c.plain(), c.mem.clone()
    c.run()
    c.check(want, True)
    others = [p for p in range(c.pages) if p not in want[2]]
    assert torch.equal(c.mem[others], before[others])


@pytest.mark.parametrize("new", [[1500], [700, 1, 1100, 40]])
def test_long_sequences(new):
    c = Case(new, 2, 1, 128, 128, rate=0.01)
    want = c.plain()
    c.run()
    c.check(want, True)


@pytest.mark.parametrize("new", [[2], [7, 1], [200, 31]])
def test_in_place(new):
    c = Case(new, 4, 4, 128, 128)
    c.state_out = c.state_in
    want = c.plain()
    c.run()
    c.check(want, max(new) > 16)


@pytest.mark.parametrize("new", [[4, 1], [150, 40]])
@pytest.mark.parametrize("decay", ["none", "head", "one", "resets", "strong", "mixed"])
def test_decays(new, decay):
    c = Case(new, 4, 2, 64, 128)
    if decay == "none":
        c.g = torch.zeros(4, device=DEV)
    elif decay == "head":
        c.g = -torch.tensor([1e-4, 0.1, 3.0, 60.0], device=DEV)
    elif decay == "one":
        c.g = torch.full((1,), -0.2, device=DEV).expand(4)
    elif decay == "resets":
        c.g[torch.rand(c.T, 4, generator=c.gen, device=DEV) < 0.2] = -math.inf
    elif decay == "strong":
        c.g = -300 * torch.rand(c.T, 4, generator=c.gen, device=DEV)
    else:  # tiny ones after a huge one: differences of their sums keep the tiny ones
        c.g = -1e-3 * torch.rand(c.T, 4, generator=c.gen, device=DEV)
        c.g[::7] = -9e4
    want = c.plain()
    c.run()
    c.check(want, max(new) > 16)


@pytest.mark.parametrize("new", [[3, 2], [70, 140]])
def test_strides_and_rows_of_a_larger_batch(new):
    c = Case(new, 4, 2, 128, 64)
    want = c.plain()
    fused = torch.full((c.T + 5, 2, 2, 136), math.nan, dtype=c.q.dtype, device=DEV)
    fused[2:2 + c.T, 0, :, :128], fused[2:2 + c.T, 1, :, :128] = c.q, c.k
    values = torch.full((4, c.T + 5, 64), math.nan, dtype=c.q.dtype, device=DEV)  # heads outermost
    values[:, 2:2 + c.T] = c.v.transpose(0, 1)
    out = torch.full((c.T + 5, 4, 72), 3.0, dtype=c.q.dtype, device=DEV)
    decay = torch.full((4, c.T + 5), math.nan, device=DEV)
    decay[:, 2:2 + c.T] = c.g.T
    c.q, c.k, c.v, c.out, c.g = fused[:, 0, :, :128], fused[:, 1, :, :128], values.transpose(0, 1), out[:, :, :64], decay.T
    c.cu += 2
    c.T += 5
    c.run()
    c.T -= 5
    c.out = out[2:2 + c.T, :, :64]
    c.check(want, max(new) > 16)
    assert bool((out[:2] == 3).all()) and bool((out[2 + c.T:] == 3).all()) and bool((out[..., 64:] == 3).all())


def test_beams_share_a_parents_state():
    c = Case([1, 1, 1, 1], 4, 2, 128, 128, pages=8)
    c.state_in = torch.tensor([2, 2, 5, 2], dtype=torch.int32, device=DEV)
    c.state_out = torch.tensor([0, 1, 3, 4], dtype=torch.int32, device=DEV)
    want = c.plain()
    c.run()
    c.check(want, False)


@pytest.mark.parametrize("max_new", [1, 40])
def test_bad_tables(max_new):
    """Bad pages and offsets are recorded; their sequences are left alone, the others are computed."""
    new = [1, 1, 1] if max_new == 1 else [40, 30, 17]
    for what, code in (("in", R.DEV_BAD_PAGE), ("out", R.DEV_BAD_PAGE), ("low", R.DEV_BAD_PAGE),
                       ("long", R.DEV_BAD_SHAPE), ("back", R.DEV_BAD_SHAPE), ("past", R.DEV_BAD_SHAPE)):
        c = Case(new, 4, 2, 64, 64)
        want, before, out = c.plain(), c.mem.clone(), c.out.clone()
        hurt = [1]
        page = int(c.state_out[1])
        if what == "in":
            c.state_in[1] = c.pages
        elif what == "out":
            c.state_out[1] = -1
        elif what == "low":
            c.state_in[1] = -2
        elif what == "long":  # longer than max_new
            c.cu[2] += 60
            c.cu[3] = c.cu[2]
            hurt = [1, 2]
        elif what == "back":  # the third one then begins in the second's rows
            c.cu[2] = c.cu[1] - 1
            hurt = [1, 2]
        else:
            c.cu[3] = c.T + 1
            hurt = [2]
        c.run(max_new=max_new)
        torch.cuda.synchronize()
        assert R.rimuru_get_device_error(c.view, True) == code, what
        if what == "back":
            continue
        rows = torch.tensor([0] + new).cumsum(0).tolist()
        for b in range(3):
            at = slice(rows[b], rows[b + 1])
            if b in hurt:
                if what != "long":
                    assert torch.equal(c.out[at], out[at]), what
            else:
                assert float((c.out[at].double() - want[0][at]).abs().max()) < 0.1
        if what in ("in", "low"):
            assert torch.equal(c.mem[page], before[page])


@pytest.mark.parametrize("new", [[], [0, 0], [1], [60]])
def test_nothing_to_do(new):
    """No sequences or no tokens: states pass from page to page."""
    c = Case(new, 2, 1, 64, 128, pages=5)
    if c.T:
        return
    c.run()
    torch.cuda.synchronize()
    for b in range(c.B):
        assert torch.equal(c.mem[c.state_in[b]], c.mem[c.state_out[b]])


@pytest.mark.parametrize("new", [[1, 1], [200, 90, 3], [1500]])
def test_streams_graphs_and_repetition(new):
    c = Case(new, 4, 2, 128, 128)
    c.run()
    torch.cuda.synchronize()
    out, mem = c.out.clone(), c.mem.clone()
    s = torch.cuda.Stream()
    c.out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    s.synchronize()
    assert torch.equal(c.out, out) and torch.equal(c.mem, mem)
    graph = torch.cuda.CUDAGraph()
    ws = torch.empty(R.rimuru_linear_attention_workspace_bytes(c.view, c.B, c.T, max(new)) + 1024, dtype=torch.uint8, device=DEV)
    with torch.cuda.graph(graph):
        c.run(ws=ws)
    c.out.zero_()
    for _ in range(3):
        ws.fill_(0xFF)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, out) and torch.equal(c.mem, mem)


def test_prompt_then_steps_equals_the_whole():
    """A prompt in one call, then tokens one by one, against the recurrence over all of them."""
    c = Case([90], 4, 2, 128, 128)
    want = c.plain()
    q, k, v, g, out = c.q, c.k, c.v, c.g, c.out
    c.T, c.new = 80, [80]
    c.cu = torch.tensor([0, 80], dtype=torch.int32, device=DEV)
    c.run()
    c.state_in = c.state_out
    c.T, c.new = 1, [1]
    for t in range(80, 90):
        c.q, c.k, c.v, c.g, c.out = (x[t:t + 1] for x in (q, k, v, g, out))
        c.run(cu=False)
    c.T, c.new, c.out = 90, [90], out
    c.check(want, True)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(2, 1, 64, 128), (1, 1, 128, 64), (2, 2, 128, 128)])
def test_pieces(shape, kind):
    """Sequences long enough to be cut into pieces, in place, one from zeros, one that is short."""
    c = Case([1300, 40, 2000], *shape, kind=kind, rate=0.02)
    c.state_out = c.state_in.clone()
    c.state_in[0] = -1
    c.state_out[0] = [p for p in range(c.pages) if p not in c.state_in.tolist()][0]
    want = c.plain()
    c.run()
    c.check(want, True)


@pytest.mark.parametrize("new", [[1, 1, 1], [5, 3, 2], [70, 30, 65], [1200, 17, 700]])
def test_a_sequence_of_nan_stays_alone(new):
    """NaN and infinities in one sequence's tokens, and in the rows around the call's, reach no other."""
    for hurt in range(3):
        c = Case(new, 4, 2, 64, 128, rate=0.02)
        want = c.plain()
        rows = torch.tensor([0] + new).cumsum(0).tolist()
        at = slice(rows[hurt], rows[hurt + 1])
        for t, x in ((c.q, math.nan), (c.k, math.inf), (c.v, math.nan), (c.g, math.nan)):
            t[at] = x
        c.run()
        torch.cuda.synchronize()
        assert bool(c.out[at].isnan().all()) and bool(c.states()[c.state_out[hurt]].isnan().all())
        for b in range(3):
            if b != hurt:
                at = slice(rows[b], rows[b + 1])
                assert float((c.out[at].double() - want[0][at]).abs().max()) < 0.05
                assert float((c.states()[c.state_out[b]].double() - want[2][int(c.state_out[b])][0]).abs().max()) < 1e-3
        assert R.rimuru_get_device_error(c.view) == R.DEV_OK


@pytest.mark.parametrize("new", [[3], [100]])
def test_decays_above_zero_count_as_zero(new):
    c = Case(new, 2, 1, 64, 64)
    c.g[::3] = 0.0
    want = c.plain()
    c.g[::3] = 5.0
    c.g[0, 1] = math.inf
    c.run()
    c.check(want, max(new) > 16)


def test_many_sequences_equal_their_halves():
    """More units than one CTA lists; what a sequence gives does not depend on the others of the call."""
    g = torch.Generator().manual_seed(0)
    new = torch.randint(0, 24, (1400,), generator=g).tolist()
    new[7], new[1300] = 130, 64
    c = Case(new, 8, 4, 64, 64)
    c.run()
    torch.cuda.synchronize()
    out, states = c.out.clone(), c.mem[c.state_out.long()].clone()
    assert bool(out.isfinite().all())
    n = c.T
    c.out.zero_()
    c.mem[c.state_out.long()] = 0
    cu, si, so = c.cu, c.state_in, c.state_out
    for at in (slice(0, 500), slice(500, 1400)):
        c.cu, c.state_in, c.state_out = cu[at.start:at.stop + 1].contiguous(), si[at].contiguous(), so[at].contiguous()
        c.B = at.stop - at.start
        c.run(max_new=130)
    torch.cuda.synchronize()
    assert c.T == n and torch.equal(c.out, out) and torch.equal(c.mem[so.long()], states)
    assert R.rimuru_get_device_error(c.view) == R.DEV_OK


def test_few_tokens_of_many_sequences():
    """Where every SM has many states the chunked form begins at fewer tokens."""
    for new, chunked in ([4] * 96, False), ([7] * 96, True):
        c = Case(new, 8, 4, 128, 128)
        want = c.plain()
        c.run()
        c.check(want, chunked)


@pytest.mark.parametrize("new", [[3, 2], [70, 140]])
def test_heads_that_lie_on_one_another(new):
    """Queries, keys and values broadcast over their heads, by a stride of 0."""
    c = Case(new, 4, 2, 64, 128)
    c.q, c.k = c.q[:, :1].expand(-1, 2, -1), c.k[:, 1:].expand(-1, 2, -1)
    c.v = c.v[:, 2:3].expand(-1, 4, -1)
    want = c.plain()
    c.run()
    c.check(want, max(new) > 16)


def test_inputs_of_one_projection():
    """q, k and v as neighbouring slices of one array, as a fused projection leaves them."""
    for new in ([1, 1], [40, 25]):
        c = Case(new, 4, 2, 64, 64, kind="f16")
        fused = torch.cat([c.q.flatten(1), c.k.flatten(1), c.v.flatten(1)], 1)
        c.q, c.k = (fused[:, 128 * i:128 * i + 128].view(c.T, 2, 64) for i in range(2))
        c.v = fused[:, 256:].view(c.T, 4, 64)
        want = c.plain()
        c.run()
        c.check(want, max(new) > 16)
