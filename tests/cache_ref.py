"""References in 64 bits for the page-cache operators: the e4m3 and e2m1 roundings, the norm and
rotation of a row, and helpers that lay tokens out in a paged pool."""
from __future__ import annotations

import numpy as np
import torch

E2M1_GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3_GRID = np.array([m * 2.0 ** -9 for m in range(8)] +
                     [(1 + m / 8) * 2.0 ** p for p in range(-6, 9) for m in range(8)])[:-1]


def nearest(x, grid):
    """Code (index into grid) nearest to |x|, ties to the even code, at most the last."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    mid = (grid[1:] + grid[:-1]) / 2
    lo = np.searchsorted(mid, a, side="left")   # borders below |x|
    hi = np.searchsorted(mid, a, side="right")  # borders at or below |x|
    return np.where((lo != hi) & (lo % 2 == 1), hi, lo)


def to_e4m3(x):
    """e4m3 values of x, saturating; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    v = E4M3_GRID[nearest(np.nan_to_num(x, nan=0.0), E4M3_GRID)]
    return np.where(np.isnan(x), np.nan, np.copysign(v, x))


def quantise(x, scale):
    """Rows [.., D] of a 4-bit cache: (values with their scales, scales [.., D / 16])."""
    b = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, 16)
    nan = np.isnan(b).any(-1)
    top = np.abs(np.nan_to_num(b, nan=0.0, posinf=np.inf, neginf=-np.inf)).max(-1)
    s = E4M3_GRID[nearest(top / (6.0 * scale), E4M3_GRID)]
    by = (s * scale)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(by > 0, np.nan_to_num(b, nan=0.0, posinf=np.inf, neginf=-np.inf) / by, 0.0)
    v = np.copysign(E2M1_GRID[nearest(t, E2M1_GRID)], t)
    s = np.where(nan, np.nan, s)
    return (v * s[..., None]).reshape(x.shape), s


def dequantise(data, scales):
    """Values of packed codes (uint8 [.., D / 2]) with e4m3 scales [.., D / 16], times no scale."""
    data = data.view(torch.uint8).cpu().numpy()
    code = np.stack([data & 15, data >> 4], axis=-1).reshape(*data.shape[:-1], -1)
    v = np.where(code & 8, -1.0, 1.0) * E2M1_GRID[code & 7]
    s = scales.view(torch.float8_e4m3fn).cpu().double().numpy()
    return v * np.repeat(s, 16, axis=-1), s


def norm_rotate(x, weight=None, eps=1e-6, cos_sin=None, positions=None, interleaved=False):
    """Rows x [tokens, heads, D] normed and rotated; also the sums of the terms' magnitudes."""
    x = np.asarray(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    terms = np.abs(x)
    if cos_sin is not None:
        r = cos_sin.shape[1]
        cs = cos_sin[positions].astype(np.float64)[:, None, :]
        c, s = cs[..., :r // 2], cs[..., r // 2:]
        x, terms = x.copy(), terms.copy()
        i, j = (np.arange(0, r, 2), np.arange(1, r, 2)) if interleaved else \
            (np.arange(r // 2), np.arange(r // 2, r))
        a, b = x[..., i].copy(), x[..., j].copy()
        x[..., i], x[..., j] = a * c - b * s, b * c + a * s
        terms[..., i], terms[..., j] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return x, terms


def half_step(dtype):
    return float(torch.finfo(dtype).eps) / 2


def assert_rounded(got, ref, terms, dtype, what):
    """got is ref rounded once to dtype, computed in 32 bits from terms of the given magnitudes:
    half a step of the value, and 16 roundings of 2^-24 on the terms (norm 12.5, rotation 2).
    Values below the normal range have the step of its lower end."""
    got = got.double().cpu().numpy()
    tiny = float(torch.finfo(dtype).tiny)
    tol = half_step(dtype) * np.maximum(np.abs(ref), tiny) + 2.0 ** -20 * terms * (1 + half_step(dtype))
    with np.errstate(invalid="ignore"):
        off = np.where(got == ref, 0.0, np.abs(got - ref))  # an infinity is itself
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, max {np.nanmax(off):.3e}"


class Pages:
    """A pool and the page table of sequences of the given lengths, pages in random order."""

    def __init__(self, lens, page, hkv, d, kv, layout, seed=0, dtype=torch.bfloat16, device="cuda",
                 spare=3):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.page, self.hkv, self.d, self.kv, self.layout, self.dtype = page, hkv, d, kv, layout, dtype
        lens = np.asarray(lens, dtype=np.int64)
        n = -(-lens // page)
        indptr = np.zeros(len(lens) + 1, dtype=np.int32)
        np.cumsum(n, out=indptr[1:])
        self.num_pages = int(indptr[-1]) + spare
        indices = rng.permutation(self.num_pages)[:indptr[-1]].astype(np.int32)
        self.lens, self.host_indptr, self.host_indices = lens, indptr, indices
        self.last = np.where(lens > 0, lens - (n - 1) * page, 0).astype(np.int32)
        self.indptr, self.indices = (torch.from_numpy(x).to(device) for x in (indptr, indices))
        if kv == "e2m1":
            self.pool = torch.randint(0, 256, self.shape(d // 2), generator=g, dtype=torch.uint8).to(device)
            x = torch.rand(self.shape(d // 16), generator=g) + 0.25
            self.scales = x.to(torch.float8_e4m3fn).to(device)
        else:
            td = {"same": dtype, "e4m3": torch.float8_e4m3fn}[kv]
            self.pool = torch.randn(self.shape(d), generator=g).to(td).to(device)
            self.scales = None

    def shape(self, width):
        inner = (self.page, self.hkv) if self.layout == "NHD" else (self.hkv, self.page)
        return (self.num_pages, 2) + inner + (width,)

    def where(self, b, pos):
        """(page, slot) of tokens, as host arrays."""
        b, pos = np.asarray(b), np.asarray(pos)
        return self.host_indices[self.host_indptr[b] + pos // self.page], pos % self.page

    def rows(self, pool, kv, b, pos):
        """[tokens, hkv, width] rows of K (0) or V (1)."""
        page, slot = (torch.from_numpy(np.asarray(x).astype(np.int64)).to(pool.device)
                      for x in self.where(b, pos))
        return pool[page, kv, slot] if self.layout == "NHD" else pool[page, kv, :, slot]

    def values16(self):
        """The pool as fp16 values without k_scale / v_scale (exact for 4 bits), on the host."""
        if self.kv != "e2m1":
            return self.pool.cpu()
        v, _ = dequantise(self.pool, self.scales)
        h = torch.from_numpy(v).half()
        assert torch.equal(h.double(), torch.from_numpy(v)) or np.isnan(v).any()
        return h

    def status(self):
        return torch.zeros(1, dtype=torch.int32, device=self.pool.device)
