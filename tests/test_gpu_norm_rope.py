"""Norms of heads with their rotation in one pass, against the formula in 64 bits."""
import math

import pytest
import torch

from paged_moe_shared_gb300 import rimuru as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def plain(x, w, offset, eps, pos, rot, interleaved, base, mscale=1.0):
    """The formula in 64 bits, and for each element what its rounding errors are relative to."""
    y = x.double()
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * (w.double() + offset)
    size = y.abs().clone()
    if rot:
        n = rot // 2
        f = torch.tensor([base ** (-2.0 * i / rot) for i in range(n)], dtype=torch.float64, device=x.device)
        ang = pos.double()[:, None, None] * f
        c, s = ang.cos() * mscale, ang.sin() * mscale
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, n), slice(n, rot))
        u, v = y[..., a].clone(), y[..., b].clone()
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
        size[..., a] = size[..., b] = (u.abs() + v.abs()) * abs(mscale)
    return y, size


def check(got, want, size):
    # half a step of the type (f16: and of its smallest numbers), and fp32: a sum of up to 1024 squares in
    # chains of 32 and five shuffles, the root, three products, an angle rounded to 2^-24 of half a turn
    t = got.dtype
    tol = torch.finfo(t).eps / 2 * want.abs() + 2.0 ** -19 * size + (2.0 ** -25 if t == torch.float16 else 1e-37)
    assert bool(((got.double() - want).abs() <= tol).all()), float(((got.double() - want).abs() / tol).max())


def run(ins, norms, pos, D, rope, outs=None, stream=None):
    outs = [torch.empty_like(x) for x in ins] if outs is None else outs
    R.rimuru_norm_rope_apply(rope, pos.data_ptr() if pos is not None else 0, ins[0].shape[0], D,
                             [R.heads_of(x) for x in ins], [R.heads_of(x) for x in outs], norms,
                             (stream or torch.cuda.current_stream()).cuda_stream)
    return outs


CASES = [  # tokens, heads of the arrays, head_dim, rot, interleaved, type
    (1, (32, 4), 128, 128, False, "bf16"), (1, (1,), 8, 8, True, "f32"), (3, (5, 2, 1), 64, 32, False, "f16"),
    (17, (16, 2), 256, 64, False, "bf16"), (130, (7, 1), 96, 48, False, "bf16"), (9, (3, 3), 80, 40, True, "f16"),
    (5, (2, 1), 1024, 256, False, "f32"), (4, (3, 1, 2, 2), 520, 16, False, "bf16"), (33, (4, 4), 192, 8, True, "f32"),
    (2500, (8, 1), 128, 64, True, "bf16"), (700, (40, 8), 128, 128, False, "f16"), (6, (1, 1), 1000, 248, True, "bf16"),
    (2, (300, 1), 16, 16, False, "bf16"), (1000, (2,), 24, 16, False, "bf16"),
]


@pytest.mark.parametrize("T,heads,D,rot,inter,kind", CASES)
def test_values(T, heads, D, rot, inter, kind):
    g = torch.Generator(device=DEV).manual_seed(T + D)
    dt = TYPES[kind]
    fused = torch.randn(T, sum(heads) + 1, D, generator=g, device=DEV) * torch.exp(torch.randn(T, 1, 1, generator=g, device=DEV) * 3)
    fused = fused.clamp(-6e4, 6e4).to(dt)
    ins = list(fused.split(list(heads) + [1], 1)[:len(heads)])
    pos = torch.randint(-5, 200000, (T,), generator=g, device=DEV).to(torch.int32)
    rope = R.rimuru_rope_create(rot, R.ROPE_INTERLEAVED if inter else R.ROPE_HALF, 1e5, mscale=1.25)
    weights = [torch.randn(D, generator=g, device=DEV).to(t) for t in (dt, torch.float32, torch.float16, torch.bfloat16)]
    offsets = [0.0, 1.0, 0.5, 1.0]
    norms = [R.head_norm_of(w, 1e-6, o) for w, o in zip(weights, offsets)][:len(ins)]
    for x, w, o, y in zip(ins, weights, offsets, run(ins, norms, pos, D, rope)):
        check(y, *plain(x, w, o, 1e-6, pos, rot, inter, 1e5, 1.25))
    # in place, on the slices of the fused projection: the rest of it stays
    rest, wants = fused[:, -1].clone(), [plain(x, w, o, 1e-6, pos, rot, inter, 1e5, 1.25)
                                         for x, w, o in zip(ins, weights, offsets)]
    run(ins, norms, pos, D, rope, ins)
    for x, want in zip(ins, wants):
        check(x, *want)
    assert torch.equal(rest, fused[:, -1])
    R.rimuru_rope_destroy(rope)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_without_rotation_or_weight_and_other_orders(kind):
    dt = TYPES[kind]
    x = torch.randn(6, 11, 128, device=DEV).to(dt).transpose(0, 1)  # heads outermost
    y = torch.zeros(11, 9, 160, dtype=dt, device=DEV)[:, :6, :128]  # padded rows
    run([x], [R.head_norm_of(None, 1e-5)], None, 128, None, [y])
    check(y, *plain(x, None, 0, 1e-5, None, 0, False, 1.0))


def test_far_values():
    """Zeros, squares that leave fp32, and heads with a NaN or an infinity beside ordinary ones."""
    rope = R.rimuru_rope_create(32, R.ROPE_INTERLEAVED, 1e4)
    for dt in (torch.bfloat16, torch.float32):
        x = torch.randn(3, 8, 64, device=DEV).to(dt)
        x[0, 0] = 0
        x[0, 1] *= 1e30
        x[0, 2] *= 1e-30
        x[1, 3, 5] = 3e38
        x[1, 4, 40] = math.nan
        x[2, 5, 50] = math.inf
        x[2, 6] = 3.0e38
        pos = torch.tensor([0, 7, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
        y = run([x], [R.head_norm_of(None, 1e-6)], pos, 64, rope)[0]
        want, size = plain(x, None, 0, 1e-6, pos, 32, True, 1e4)
        ok = torch.ones(3, 8, dtype=torch.bool, device=DEV)
        ok[1, 4] = ok[2, 5] = False
        size = size + 0.0
        # at 2^31 positions the frequencies, doubles, leave 2^-22 of a turn
        check(y[ok], want[ok], size[ok] * 4)
        assert bool(y[1, 4].isnan().all())
        assert bool(y[2, 5, 50].isnan()) and float(y[2, 5, :50].abs().max()) == 0
    R.rimuru_rope_destroy(rope)


@pytest.mark.parametrize("T,heads,D,rot,inter,kind", [
    (20001, (3, 2), 64, 32, False, "bf16"), (6001, (1,), 1024, 256, False, "f32"), (3001, (1, 1, 1), 256, 256, True, "f16"),
    (4097, (7, 6, 1, 3), 72, 16, False, "bf16"), (41000, (1,), 8, 8, True, "f32"), (9000, (2, 2), 1024, 16, False, "f16"),
    (301, (64, 8), 128, 128, False, "bf16"),
])
def test_runs_of_heads_over_many_tokens(T, heads, D, rot, inter, kind):
    """A group's heads begin and end inside tokens and pass over several of them."""
    test_values(T, heads, D, rot, inter, kind)


@pytest.mark.parametrize("scale,weight", [(1e38, 1e-6), (1e-12, 1e30)])
def test_the_norm_times_the_weight_may_leave_fp32(scale, weight):
    """1 / rms times the weight is below fp32's normal numbers (or above them all); the result is not."""
    x = (torch.rand(5, 3, 96, device=DEV) + 1) * scale
    w = (torch.rand(96, device=DEV) + 1) * weight
    y = run([x], [R.head_norm_of(w, 1e-20)], None, 96, None)[0]
    check(y, *plain(x, w, 0, 1e-20, None, 0, False, 1.0))


def test_equals_the_rotation_alone_after_a_norm_of_ones():
    """Heads of magnitude 1 everywhere have a norm of 1: what is left is rimuru_rope_apply, bit for bit
    but for the norm's own rounding (eps is far below a half step)."""
    x = torch.where(torch.rand(40, 6, 128, device=DEV) < 0.5, -1.0, 1.0).bfloat16()
    pos = torch.arange(40, dtype=torch.int32, device=DEV) * 999
    rope = R.rimuru_rope_create(128, R.ROPE_HALF, 1e6)
    y, z = run([x], [R.head_norm_of(None, 1e-20)], pos, 128, rope)[0], torch.empty_like(x)
    R.rimuru_rope_apply(rope, pos.data_ptr(), 40, 128, [R.heads_of(x)], [R.heads_of(z)],
                        torch.cuda.current_stream().cuda_stream)
    assert torch.equal(y, z)
    R.rimuru_rope_destroy(rope)


def test_streams_and_graphs():
    x = torch.randn(64, 12, 128, device=DEV).bfloat16()
    pos = torch.arange(64, dtype=torch.int32, device=DEV)
    rope = R.rimuru_rope_create(128)
    w = torch.randn(128, device=DEV)
    want = run([x], [R.head_norm_of(w)], pos, 128, rope)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run([x], [R.head_norm_of(w)], pos, 128, rope, stream=s)[0]
    s.synchronize()
    assert torch.equal(got, want)
    out, graph = torch.zeros_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run([x], [R.head_norm_of(w)], pos, 128, rope, [out])
    R.rimuru_rope_destroy(rope)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
