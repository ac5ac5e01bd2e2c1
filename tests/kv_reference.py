"""Plain 64-bit restatements of the rotary, KV-cache and attention operators, for the tests, and
a small cache on the device.  Nothing here shares code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

from paged_moe_shared_gb300 import rimuru as R
from paged_moe_shared_gb300.device_pool import DevicePool

DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_ULP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # relative, per rounding


# ------------------------------------------------------------------ rotary positions
def inv_freq(rot, base, scaling, factor=1.0, orig_len=0.0, low=0.0, high=0.0):
    if scaling == R.ROPE_BASE:
        base = base * factor ** (rot / (rot - 2))
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == R.ROPE_LINEAR:
        f = f / factor
    if scaling == R.ROPE_BY_PARTS:
        g = np.clip((orig_len * f / (2 * math.pi) - low) / (high - low), 0, 1)
        f = (1 - g) * f / factor + g * f
    return f


def rope(x, positions, f, interleaved, mscale=1.0):
    """x [T, heads, dim] -> float64 [T, heads, dim]."""
    y = x.double().cpu().numpy().copy()
    n = len(f)
    # angles modulo one turn in extended steps: positions are below 2^31, f below 1
    ang = np.mod(positions.cpu().numpy().astype(np.float64)[:, None] * f, 2 * math.pi)
    c, s = (np.cos(ang) * mscale)[:, None], (np.sin(ang) * mscale)[:, None]
    iu, iv = (np.arange(n) * 2, np.arange(n) * 2 + 1) if interleaved else (np.arange(n), np.arange(n) + n)
    u, v = y[..., iu].copy(), y[..., iv].copy()
    y[..., iu] = u * c - v * s
    y[..., iv] = v * c + u * s
    return y


# ------------------------------------------------------------------ the cache
class Cache:
    """A KV view of a small pool, every byte a NaN code, with scales of NaN."""

    def __init__(self, kv_heads, dim, page_tokens, pages, per_parent=8, extra_bytes=0):
        self.Hk, self.D, self.P = kv_heads, dim, page_tokens
        self.page_bytes = 2 * kv_heads * dim * page_tokens + extra_bytes
        self.pages = -(-pages // per_parent) * per_parent
        self.pool = DevicePool(self.pages * self.page_bytes, per_parent * self.page_bytes, DEV)
        self.pool.mem.fill_(0x7F)
        self.view = self.pool.view(self.page_bytes)
        self.scales = torch.full((self.pages, 2, kv_heads), float("nan"), device=DEV)
        R.rimuru_view_set_kv_shape(self.view, kv_heads, dim, page_tokens, self.scales.data_ptr(),
                                   self.scales.numel() * 4)

    def codes(self):
        """uint8 [pages, 2, kv_heads, page_tokens, dim], a view of the pool."""
        used = 2 * self.Hk * self.P * self.D
        return self.pool.mem.view(self.pages, self.page_bytes)[:, :used].unflatten(
            1, (2, self.Hk, self.P, self.D))

    def values(self):
        """float64 [pages, 2, kv_heads, page_tokens, dim] on the CPU."""
        c = self.codes().contiguous().view(E4M3).cpu().double()
        return c * self.scales.cpu().double()[..., None, None]

    def tables(self, lens, seed=0, spare=2):
        """A page table with scattered pages for sequences of these lengths; unused entries are -1."""
        need = [-(-n // self.P) for n in lens]
        assert sum(need) <= self.pages
        order = np.random.default_rng(seed).permutation(self.pages)
        t = np.full((max(1, len(lens)), max(need + [0]) + spare), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            t[b, :n] = order[at:at + n]
            at += n
        return torch.from_numpy(t).to(DEV)

    def fill(self, table, lens, seed=0, spread=3, loud=1.0):
        """Random codes in the live slots of each sequence and scales 2^(-8 .. -8 + spread)."""
        g = torch.Generator().manual_seed(seed)
        codes, t = self.codes(), table.cpu()
        for b, n in enumerate(lens):
            for c in range(-(-n // self.P)):
                page, m = int(t[b, c]), min(self.P, n - c * self.P)
                x = (torch.randn(2, self.Hk, m, self.D, generator=g) * 64 * loud).clamp(-448, 448)
                codes[page, :, :, :m] = x.to(E4M3).view(torch.uint8).to(DEV)
                k = torch.randint(-8, -8 + spread, (2, self.Hk), generator=g)
                self.scales[page] = torch.exp2(k.float()).to(DEV)

    def close(self):
        self.pool.close()


def rne_e4m3(x):
    """float64 array (|x| <= 448) -> nearest e4m3 value, ties to even."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)                     # |x| in [2^(e-1), 2^e)
    q = np.exp2(np.maximum(e - 1, -6) - 3.0)  # spacing: 3 mantissa bits, subnormal below 2^-6
    return np.clip(np.rint(x / q) * q, -448, 448)


def pow2_scale(amax):
    if amax == 0:
        return 2.0 ** -60
    m, e = math.frexp(amax / 448.0)
    k = e - 1 if m == 0.5 else e
    return 2.0 ** max(-60, min(60, k))


def append(values, scales, table, cu, lens, k, v, P):
    """In place on float64 values [pages, 2, Hk, P, D] and scales [pages, 2, Hk]."""
    x = np.stack([k.double().cpu().numpy(), v.double().cpu().numpy()], 1)  # [T, 2, Hk, D]
    for b, n_all in enumerate(lens):
        n = cu[b + 1] - cu[b]
        start = n_all - n
        for c in range(start // P, -(-n_all // P)):
            lo, hi = max(start, c * P), min(n_all, (c + 1) * P)
            if hi <= lo:
                continue
            page = int(table[b][c])
            for w in range(2):
                for h in range(values.shape[2]):
                    new = x[cu[b] + lo - start:cu[b] + hi - start, w, h]
                    fin = np.abs(new[np.isfinite(new)])
                    s = pow2_scale(float(fin.max()) if fin.size else 0.0)
                    old = values[page, w, h, :lo - c * P]
                    if lo > c * P:
                        s = max(s, float(scales[page, w, h]))
                        values[page, w, h, :lo - c * P] = rne_e4m3(old / s) * s
                    scales[page, w, h] = s
                    y = np.where(np.isnan(new), 0.0, new)
                    with np.errstate(over="ignore"):
                        values[page, w, h, lo - c * P:hi - c * P] = rne_e4m3(np.clip(y / s, -448, 448)) * s
    return values, scales


# ------------------------------------------------------------------ attention
def attention(values, table, lens, q, cu, scale, window, P):
    """float64: out [rows, Hq, D], lse [rows, Hq], and for the tolerances sum p |v| and the
    largest scale * sum |q k| of each row."""
    q = q.double().cpu()
    rows, Hq, D = q.shape
    Hk = values.shape[2]
    G = Hq // Hk
    out, mag = torch.zeros(rows, Hq, D, dtype=torch.float64), torch.zeros(rows, Hq, D, dtype=torch.float64)
    lse, top = torch.full((rows, Hq), -math.inf, dtype=torch.float64), torch.zeros(rows, Hq, dtype=torch.float64)
    for b, L in enumerate(lens):
        r0, r1 = (cu[b], cu[b + 1]) if cu is not None else (b, b + 1)
        n = r1 - r0
        if L == 0 or n == 0:
            continue
        ids = [int(t) for t in table[b][:-(-L // P)]]
        kv = values[ids]  # [M, 2, Hk, P, D]
        pos = torch.arange(L - n, L)[:, None]
        j = torch.arange(L)
        see = j <= pos
        if window:
            see &= j > pos - window
        for h in range(Hk):
            k, v = (kv[:, w, h].reshape(-1, D)[:L] for w in (0, 1))
            for g in range(G):
                qq = q[r0:r1, h * G + g]
                x = (qq @ k.T * scale).masked_fill(~see, -math.inf)
                some = see.any(1)
                p = torch.where(some[:, None], torch.softmax(x, -1), 0.0)
                out[r0:r1, h * G + g] = p @ v
                mag[r0:r1, h * G + g] = p @ v.abs()
                lse[r0:r1, h * G + g] = torch.where(some, torch.logsumexp(x, -1), -math.inf)
                top[r0:r1, h * G + g] = torch.where(see, qq.abs() @ k.abs().T * abs(scale), 0.0).amax(1)
    return out, lse, mag, top
