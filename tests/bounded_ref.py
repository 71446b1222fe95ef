"""References in 64 bits for the operators that keep a cache bounded: decode over a window and sinks
with every key's weight, and eviction, both written from their definitions."""
from __future__ import annotations

import math

import numpy as np
import torch

from cache_ref import Pages, dequantise, half_step


def values(pool, scales=None):
    """What a pool (codes with `scales`) holds, in fp64 on the host."""
    if scales is not None:
        return torch.from_numpy(dequantise(pool, scales)[0])
    return pool.float().cpu().double()


def sequence(pg: Pages, pool64, b, n):
    """K and V of sequence b's first n tokens, [n, kv heads, d]."""
    page, slot = (torch.from_numpy(np.asarray(x).astype(np.int64)) for x in pg.where(np.full(n, b), np.arange(n)))
    if pg.layout == "NHD":
        return pool64[page, 0, slot], pool64[page, 1, slot]
    return pool64[page, 0, :, slot], pool64[page, 1, :, slot]


def attended(last, window, sinks):
    """Positions that a row at position `last` attends."""
    t = np.arange(last + 1)
    return t if window < 0 else t[(t >= last - window) | (t < sinks)]


def _rope(x, pos, theta=1e4):
    d = x.shape[-1]
    a = torch.as_tensor(pos, dtype=torch.float64).reshape(-1, 1) * theta ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    c, s = a.cos().unsqueeze(1), a.sin().unsqueeze(1)
    x, y = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([x * c - y * s, y * c + x * s], dim=-1)


def decode_ref(pg: Pages, pool64, q, lens=None, q_len=1, window=-1, sinks=0, cap=0.0, k_scale=1.0, v_scale=1.0,
               pos=None):
    """o, sum p |v|, lse of every row, and {sequence: [kv heads, n] sums of the keys' weights}.
    pos: None, "ROPE_LLAMA" or "ALIBI" (a power of two of heads)."""
    lens = pg.lens if lens is None else lens
    q64 = q.double().cpu()
    rows, hq, d = q64.shape
    group = hq // pg.hkv
    o, mag = torch.zeros(rows, hq, d, dtype=torch.float64), torch.zeros(rows, hq, d, dtype=torch.float64)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64)
    sums = {}
    for b, n in enumerate(lens):
        n = int(n)
        k, v = sequence(pg, pool64, b, n)
        if pos == "ROPE_LLAMA":
            k = _rope(k, np.arange(n))
        sums[b] = torch.zeros(pg.hkv, n, dtype=torch.float64)
        for j in range(q_len):
            last, r = n - q_len + j, b * q_len + j
            if last < 0:
                continue
            t = torch.from_numpy(attended(last, window, sinks))
            x = q64[r:r + 1]
            x = (_rope(x, [last]) if pos == "ROPE_LLAMA" else x)[0].view(pg.hkv, group, d)
            s = torch.einsum("hgd,thd->hgt", x, k[t]) * k_scale / math.sqrt(d)
            if pos == "ALIBI":
                slope = 2.0 ** (-8.0 * (torch.arange(hq, dtype=torch.float64) + 1) / hq)
                s = s + slope.view(pg.hkv, group, 1) * (t - last).double()
            if cap:
                s = cap * torch.tanh(s / cap)
            z = torch.logsumexp(s, dim=2)
            p = torch.exp(s - z[..., None])
            lse[r] = z.reshape(-1)
            o[r] = torch.einsum("hgt,thd->hgd", p, v[t]).reshape(hq, d) * v_scale
            mag[r] = torch.einsum("hgt,thd->hgd", p, v[t].abs()).reshape(hq, d) * abs(v_scale)
            sums[b][:, t] += p.sum(1)
    return o.numpy(), mag.numpy(), lse.numpy(), sums


def assert_decode(q, o, lse, ref, pool64, longest, v_scale=1.0, rope=False, what=""):
    """o: half a step of its type; half a step of fp16 on every weight (2^-11 of sum p |v|, and 2^-25
    of the largest |v| for each weight below fp16's normal range); and the 32-bit arithmetic, 1e-4 of
    sum p |v|: scores off by 16 roundings of their terms, below 1e-5 each, move every weight by that
    much, twice.  With RoPE in the kernel the operands are rotated in fp16: each logit is off by
    three roundings of 2^-11 on terms whose root of squares is below 2, below 4e-3 at the worst of
    some 1e4 keys, which moves a weight by 4e-3, twice."""
    ref_o, mag, ref_l, _ = ref
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    logit = 4e-3 if rope else 1e-5
    vmax = float(pool64.nan_to_num(0.0).abs().max()) * abs(v_scale)
    tol = half_step(q.dtype) * np.abs(ref_o) + (2.0 ** -11 + 8 * logit + 2e-5) * mag + 2.0 ** -25 * max(1, longest) * vmax
    bad = ~(np.abs(o - ref_o) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} o off, max {np.abs(o - ref_o).max():.3e}"
    empty = np.isneginf(ref_l)
    assert np.array_equal(np.isneginf(lse), empty) and (o[empty] == 0).all(), what
    assert np.abs(lse[~empty] - ref_l[~empty]).max(initial=0.0) <= max(1e-4, logit), what


def decoder(pg: Pages, hq, dtype, ws=64 << 20, graph=None, cls=None, indices=None, **plan):
    """A planned BatchDecodePagedKV over pg's page table."""
    from paged_kv_decode_23_gb300 import BatchDecodePagedKV
    dec = BatchDecodePagedKV(torch.zeros(ws, dtype=torch.uint8, device="cuda"), pg.layout)
    kv = {"same": dtype, "e4m3": torch.float8_e4m3fn, "e2m1": "e2m1"}[pg.kv]
    ix = pg.indices if indices is None else indices
    dec.plan(torch.from_numpy(pg.host_indptr), ix if len(ix) else torch.zeros(1, dtype=torch.int32, device="cuda"),
             torch.from_numpy(pg.last), hq, pg.hkv, pg.d, pg.page, q_data_type=dtype, kv_data_type=kv, **plan)
    return dec


def evict_ref(weights, n, budget, sinks, recent):
    """For one sequence and head: weights [n] -> (kept [budget], weights after [n]).  kept[j] is the
    slot whose row ends in slot j, -1 past the sequence's end."""
    kept = np.full(budget, -1, dtype=np.int64)
    if n <= budget:
        kept[:n] = np.arange(n)
        return kept, weights.copy()
    kept[:] = np.arange(budget)
    # NaN first, then descending, equal weights by slot
    key = [(0 if math.isnan(w) else 1, 0.0 if math.isnan(w) else -float(w), t)
           for t, w in zip(range(sinks, n - recent), weights[sinks:n - recent])]
    chosen = sorted(t for _, _, t in sorted(key)[:budget - sinks - recent])
    holes = sorted(set(range(sinks, budget - recent)) - set(chosen))
    movers = [t for t in chosen if t >= budget - recent]
    assert len(holes) == len(movers)
    for hole, t in zip(holes, movers):
        kept[hole] = t
    kept[budget - recent:] = np.arange(n - recent, n)
    after = np.zeros_like(weights)
    after[:budget] = weights[kept]
    return kept, after
