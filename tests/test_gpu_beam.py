"""Beam selection and the reordering of the paged cache, against plain implementations in 64 bits."""
import math

import pytest
import torch

from paged_moe_shared_gb300 import rimuru as R
from paged_moe_shared_gb300.device_pool import DevicePool

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def plain(logits, scores, done, pad, K):
    G, N = scores.shape
    V = logits.shape[1]
    x = logits.double()
    x = torch.where(x.isnan(), -math.inf, x).clamp(max=float(torch.finfo(torch.float32).max)).view(G, N, V)
    top = x.amax(-1, keepdim=True)
    safe = torch.where(top > -math.inf, top, 0.0)
    x = x - safe - (x - safe).exp().sum(-1, keepdim=True).log()
    x = torch.where(x.isnan(), -math.inf, x) + scores.double()[..., None]
    x = torch.where(top > -math.inf, x, -math.inf)
    if done is not None:
        only = torch.full_like(x, -math.inf)
        only[..., pad] = scores.double()
        x = torch.where(done[..., None] != 0, only, x)
    value, at = torch.sort(x.view(G, -1), dim=-1, descending=True, stable=True)
    if value.shape[1] < K:
        more = K - value.shape[1]
        value, at = torch.nn.functional.pad(value, (0, more), value=-math.inf), torch.nn.functional.pad(at, (0, more))
    value, at = value[:, :K], at[:, :K]
    live = value > -math.inf
    rows = torch.arange(G, device=DEV)[:, None] * N + at // V
    return value, torch.where(live, rows, -1).int(), torch.where(live, at % V, -1).int()


def select(logits, scores, done=None, pad=0, K=8, stream=None, ws=None):
    G, N = scores.shape
    nbytes = R.rimuru_beam_select_workspace_bytes(G, N, logits.shape[1], K)
    ws = torch.full((nbytes + 1024,), 0xFF, dtype=torch.uint8, device=DEV) if ws is None else ws
    best = torch.empty(G, K, device=DEV)
    rows, tokens = (torch.empty(G, K, dtype=torch.int32, device=DEV) for _ in range(2))
    R.rimuru_beam_select(R.rows_of(logits), scores.data_ptr(), 0 if done is None else done.data_ptr(), G, N, pad, K,
                         best.data_ptr(), rows.data_ptr(), tokens.data_ptr(), (ws.data_ptr() + 1023) // 1024 * 1024,
                         nbytes, (stream or torch.cuda.current_stream()).cuda_stream)
    select.keep = ws
    return best, rows, tokens


def check(logits, scores, done=None, pad=0, K=8):
    best, rows, tokens = select(logits, scores, done, pad, K)
    want, w_rows, w_tokens = plain(logits, scores, done, pad, K)
    assert torch.equal(tokens, w_tokens) and torch.equal(rows, w_rows)
    live = want > -math.inf
    assert bool((best[~live] == -math.inf).all())
    # the worth's own rounding to fp32, and a sum of exponentials of 2^-22 each added up in fp32: 2^-18 of it
    tol = 2.0 ** -24 * want[live].abs() + 2.0 ** -18
    assert bool(((best[live].double() - want[live]).abs() <= tol).all())


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("G,N,V,K", [(1, 4, 50257, 8), (3, 5, 1001, 10), (2, 1, 128000, 1), (1, 12, 32003, 25),
                                     (4, 3, 63, 6), (2, 2, 65, 128), (1, 7, 1, 4), (5, 2, 8193, 4), (1, 128, 300, 128)])
def test_values(G, N, V, K, kind):
    g = torch.Generator(device=DEV).manual_seed(V)
    logits = (torch.randn(G * N, V, generator=g, device=DEV) * 3).to(TYPES[kind])
    scores = -10 * torch.rand(G, N, generator=g, device=DEV)
    check(logits, scores, K=K)
    done = (torch.rand(G, N, generator=g, device=DEV) < 0.4).to(torch.uint8)
    check(logits, scores, done, min(2, V - 1), K)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_ties_go_to_the_lowest(kind):
    dt = TYPES[kind]
    scores = torch.zeros(2, 3, device=DEV)
    check(torch.zeros(6, 5000, dtype=dt, device=DEV), scores, K=20)           # all alike: the list overflows
    few = torch.randint(0, 3, (6, 5000), device=DEV).to(dt)                   # a third of them at the top
    few[1], few[2] = few[0], few[0]                                           # beams that are alike
    check(few, scores, K=40)
    x = torch.full((6, 40000), -1.0, dtype=dt, device=DEV)
    x[:, 39999] = x[:, 17] = x[:, 64] = 2.0
    check(x, scores, K=5)
    check(torch.randn(4, 3000, device=DEV).to(dt).repeat(2, 1)[:8], torch.zeros(2, 4, device=DEV), K=16)


def test_first_step_scores():
    """All beams but the first are out, by -inf or by a very low score."""
    x = torch.randn(8, 30000, device=DEV).bfloat16()
    for low in (-math.inf, -1e9, -1e30):
        scores = torch.full((2, 4), low, device=DEV)
        scores[:, 0] = 0
        best, rows, _ = select(x, scores, K=8)
        assert rows.tolist() == [[0] * 8, [4] * 8]
        check(x, scores, K=8)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_masks(kind):
    dt, V = TYPES[kind], 9001
    x = torch.randn(6, V, device=DEV).to(dt)
    lowest = torch.finfo(dt).min
    x[0] = -math.inf                      # a row without a token
    x[1, 3:] = -math.inf                  # three tokens left
    x[2, :V - 1] = lowest                 # masked by the type's lowest value
    x[3, 5:900] = math.nan
    x[4] = math.nan
    x[5, 77] = math.inf
    check(x, torch.zeros(1, 6, device=DEV), K=30)
    check(x, torch.zeros(6, 1, device=DEV), K=5)
    check(x, torch.zeros(2, 3, device=DEV), K=12)
    x[5, 9000] = math.inf                 # two of them share the row
    check(x, torch.zeros(6, 1, device=DEV), K=3)
    check(torch.full((2, 100), lowest, dtype=dt, device=DEV), torch.zeros(1, 2, device=DEV), K=4)
    check(x, torch.full((1, 6), math.nan, device=DEV), K=4)


def test_far_logits():
    x = torch.randn(4, 20000, device=DEV) * 1e4
    check(x, -torch.rand(1, 4, device=DEV), K=8)
    x = torch.randn(4, 20000, device=DEV) * 1e30
    check(x, -torch.rand(4, 1, device=DEV), K=8)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("first", range(0, 9, 3))
def test_rows_anywhere(kind, first):
    """Rows of a wider array that begin off the 16-byte boundaries; what lies around them is not read."""
    x = torch.full((7, 2600), math.inf, dtype=TYPES[kind], device=DEV)
    x[:, first:first + 2501] = torch.randn(7, 2501, device=DEV).to(x.dtype)
    scores = -torch.rand(1, 6, device=DEV)
    check(x.view(-1)[:6 * 2600].view(6, 2600)[:, first:first + 2501], scores, K=12)
    wide = x.view(-1)[:7 * 2599].view(7, 2599)  # an odd stride
    wide[:] = math.inf
    wide[:, first:first + 2501] = torch.randn(7, 2501, device=DEV).to(x.dtype)
    check(wide[:6, first:first + 2501], scores, K=12)


def test_many_entries():
    x = torch.randn(70000, 70, device=DEV).bfloat16()
    check(x, -torch.rand(35000, 2, device=DEV), K=3)


def test_streams_graphs_and_repetition():
    x, scores = torch.randn(8, 50000, device=DEV).bfloat16(), -torch.rand(2, 4, device=DEV)
    want = select(x, scores)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = select(x, scores, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = torch.empty(R.rimuru_beam_select_workspace_bytes(2, 4, 50000, 8) + 1024, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = select(x, scores, ws=ws)
        b = select(x, scores, ws=ws)
    for _ in range(3):
        ws.fill_(0xFF)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, want)) and all(torch.equal(p, q) for p, q in zip(b, want))


# ------------------------------------------------------------------ reordering
class Cache:
    def __init__(self, pages, Hk=2, D=64, P=16, extra=0):
        self.page_bytes = 2 * Hk * P * D + extra
        self.pages, self.shape = pages, (pages, 2, Hk)
        self.pool = DevicePool(pages * self.page_bytes, self.page_bytes, DEV)
        self.view = self.pool.view(self.page_bytes)
        self.scales = torch.exp2(torch.randint(-9, 9, self.shape, device=DEV).float())
        R.rimuru_view_set_kv_shape(self.view, Hk, D, P, self.scales.data_ptr(), self.scales.numel() * 4)
        self.codes = self.pool.mem.view(pages, self.page_bytes)
        self.codes.copy_(torch.randint(0, 255, self.codes.shape, dtype=torch.uint8, device=DEV))
        self.P, self.used = P, 2 * Hk * P * D

    def reorder(self, parents, lens, table, out, fresh, stream=None):
        i32 = lambda x: x.to(torch.int32).to(DEV)  # noqa: E731
        self.args = parents, lens = i32(parents), i32(lens)
        got = torch.full((len(parents),), 99, dtype=torch.int32, device=DEV)
        R.rimuru_kv_reorder(self.view, parents.data_ptr(), len(parents), lens.data_ptr(), len(lens), table.data_ptr(),
                            out.data_ptr(), table.shape[0], table.shape[2], fresh.data_ptr(), got.data_ptr(),
                            (stream or torch.cuda.current_stream()).cuda_stream)
        return got


@pytest.mark.parametrize("layers,n,children,width,P,D", [(1, 1, 1, 1, 16, 64), (3, 4, 4, 5, 16, 128), (2, 3, 7, 9, 32, 64),
                                                         (1, 8, 2, 300, 64, 256), (5, 2, 2, 3, 16, 256)])
def test_reorder(layers, n, children, width, P, D):
    g = torch.Generator().manual_seed(n)
    c = Cache(layers * (n + children) + layers * n * (width - 1) + 3, D=D, P=P, extra=P * D)
    order = torch.randperm(c.pages, generator=g).int()
    fresh = order[:layers * children].view(layers, children).to(DEV)
    table = order[layers * children:layers * children + layers * n * width].view(layers, n, width).to(DEV)
    lens = torch.randint(0, width * P + 1, (n,), generator=g)
    lens[0] = width * P if n > 1 else max(1, width * P - 3)
    if n > 2:
        lens[1], lens[2] = 0, P
    parents = torch.randint(0, n, (children,), generator=g)
    out = torch.full((layers, children, width), -7, dtype=torch.int32, device=DEV)
    codes, scales = c.codes.clone(), c.scales.clone()
    got = c.reorder(parents, lens, table, out, fresh)
    torch.cuda.synchronize()
    assert R.rimuru_get_device_error(c.view) == R.DEV_OK
    assert got.tolist() == lens[parents].tolist()
    for layer in range(layers):
        for i, p in enumerate(parents.tolist()):
            full, part = divmod(int(lens[p]), P)
            row = table[layer, p].tolist()
            want = row[:full] + ([int(fresh[layer, i])] if part else [])
            assert out[layer, i].tolist() == want + [-7] * (width - len(want))
            if part:
                codes[fresh[layer, i], :c.used] = codes[row[full], :c.used]
                scales[fresh[layer, i]] = scales[row[full]]
    assert torch.equal(c.codes, codes) and torch.equal(c.scales, scales)


def test_reorder_of_bad_tables():
    c = Cache(16)
    table = torch.tensor([[[0, 1], [2, 99], [3, 4]]], dtype=torch.int32, device=DEV)
    fresh = torch.tensor([[8, 9, 10, 16]], dtype=torch.int32, device=DEV)
    codes = c.codes.clone()

    def go(parents, lens, code):
        out = torch.full((1, len(parents), 2), -7, dtype=torch.int32, device=DEV)
        got = c.reorder(torch.tensor(parents), torch.tensor(lens), table, out, fresh)
        torch.cuda.synchronize()
        assert R.rimuru_get_device_error(c.view, True) == code
        return got.tolist(), out[0].tolist()

    assert go([-1, 0], [16, 16, 16], R.DEV_OK) == ([0, 16], [[-7, -7], [0, -7]])
    assert go([3, 0], [16, 16, 16], R.DEV_BAD_SHAPE) == ([0, 16], [[-7, -7], [0, -7]])
    assert go([-2], [16, 16, 16], R.DEV_BAD_SHAPE) == ([0], [[-7, -7]])
    assert go([0, 2], [33, 16, 32], R.DEV_BAD_SHAPE) == ([0, 32], [[-7, -7], [3, 4]])
    assert go([0], [-1, 16, 32], R.DEV_BAD_SHAPE) == ([0], [[-7, -7]])
    assert go([1], [16, 20, 16], R.DEV_BAD_PAGE) == ([20], [[2, -1]])          # the source
    assert go([0, 0, 0, 0], [32, 16, 16], R.DEV_OK) == ([32] * 4, [[0, 1]] * 4)  # full: fresh pages are not named
    assert torch.equal(c.codes, codes)
    assert go([2, 2, 2, 2], [16, 16, 5], R.DEV_BAD_PAGE) == ([5] * 4, [[8, -7], [9, -7], [10, -7], [-1, -7]])


def test_reorder_captured_on_another_stream():
    c = Cache(32)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 2, 2)
    fresh = torch.arange(8, 12, dtype=torch.int32, device=DEV).view(2, 2)
    out = torch.full((2, 2, 2), -1, dtype=torch.int32, device=DEV)
    parents, lens = torch.tensor([1, 1], dtype=torch.int32, device=DEV), torch.tensor([32, 20], dtype=torch.int32, device=DEV)
    c.reorder(parents, lens, table, out, fresh)  # makes the error word
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        got = c.reorder(parents, lens, table, out, fresh)
    out.fill_(-1)
    c.codes[8:12] = 0
    graph.replay()
    torch.cuda.synchronize()
    assert out.tolist() == [[[2, 8], [2, 9]], [[6, 10], [6, 11]]] and got.tolist() == [20, 20]
    assert torch.equal(c.codes[8:12, :c.used], c.codes[[3, 3, 7, 7], :c.used])
