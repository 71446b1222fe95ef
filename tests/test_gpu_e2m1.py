"""Decode over a 4-bit cache against the fp64 oracle (on the cache's exact values), its refusals,
and the operators around it run together."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from cache_ref import Pages, half_step, quantise
from helpers import ORACLE_CODE

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
NAME = {BF16: "bf16", F16: "f16"}


def _ref(pg, q, hq, q_len=1, cap=0.0, window=-1, scales=(1.0, 1.0), magnitudes=False, **pos):
    """Oracle o and lse on the cache's values, which fp16 holds exactly."""
    pool = pg.values16().half()
    if magnitudes:
        pool[:, 1] = pool[:, 1].abs()
    return oracle.batch_decode_pool(pg.host_indptr, pg.host_indices, pg.last, W.raw_bits(q.cpu()), ORACLE_CODE[NAME[q.dtype]],
                                    W.raw_bits(pool), oracle.F16, pg.layout, sm_scale=1 / np.sqrt(pg.d), logits_soft_cap=cap,
                                    window_left=window, k_scale=scales[0], v_scale=scales[1], q_len=q_len, **pos)


def assert_decode(pg, q, o, lse, hq, scales=(1.0, 1.0), **kw):
    """o: half a step of its type, half a step of fp16 on every weight (2^-11 of sum p |v|, and 2^-25
    for each weight below fp16's normal range, of a sum of weights of at least 1), and the 32-bit
    arithmetic: scores off by 16 roundings of their terms, below 1e-5 each, move every weight by
    that much, twice (numerator and sum), with exp2 and the sums' own errors inside 1e-4 in all."""
    ref_o, ref_l = _ref(pg, q, hq, scales=scales, **kw)
    mag, _ = _ref(pg, q, hq, scales=scales, magnitudes=True, **kw)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    vmax = float(pg.values16().double().abs().nan_to_num(0.0).max()) * scales[1]
    tol = half_step(q.dtype) * np.abs(ref_o) + (2.0 ** -11 + 1e-4) * mag + 2.0 ** -25 * max(1, pg.lens.max()) * vmax
    bad = ~(np.abs(o - ref_o) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} o off, max {np.abs(o - ref_o).max():.3e}"
    empty = np.isneginf(ref_l)
    assert np.array_equal(np.isneginf(lse), empty) and (o[empty] == 0).all()
    assert np.abs(lse[~empty] - ref_l[~empty]).max(initial=0.0) <= 1e-4


def _dec(pg, hq, dtype, ws=None, **plan):
    from paged_kv_decode_23_gb300 import BatchDecodePagedKV
    dec = BatchDecodePagedKV(torch.zeros(ws or (64 << 20), dtype=torch.uint8, device="cuda"), pg.layout)
    dec.plan(torch.from_numpy(pg.host_indptr), pg.indices if len(pg.indices) else torch.zeros(1, dtype=torch.int32, device="cuda"),
             torch.from_numpy(pg.last), hq, pg.hkv, pg.d, pg.page, q_data_type=dtype, kv_data_type="e2m1", **plan)
    return dec


def _q(rows, hq, d, dtype, seed=0):
    return torch.randn(rows, hq, d, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


# dtype, layout, hq, hkv, d, page, lens, options
CASES = [
    (BF16, "HND", 32, 8, 128, 16, [1, 15, 16, 17, 500, 0, 1300], {}),
    (F16, "NHD", 8, 8, 64, 8, [3, 129, 128, 127, 2000], {}),
    (BF16, "NHD", 16, 2, 256, 32, [1, 63, 64, 65, 3000], dict(logits_soft_cap=30.0, window_left=100)),
    (F16, "HND", 24, 2, 128, 64, [700, 5], dict(window_left=0)),        # 12 heads a kv head: two slices
    (BF16, "HND", 6, 1, 64, 256, [4000, 1, 256], dict(fixed_split_size=1)),
    (F16, "NHD", 3, 3, 256, 16, [777] * 3, dict(disable_split_kv=True)),
    (BF16, "HND", 40, 8, 128, 16, [9000], {}),
    (F16, "HND", 8, 1, 256, 128, [5000, 130], dict(logits_soft_cap=5.0)),
    (BF16, "NHD", 32, 4, 64, 16, [333, 40, 1000], dict(pos_encoding_mode="ALIBI")),
]


@pytest.mark.parametrize("dtype,layout,hq,hkv,d,page,lens,opt", CASES)
def test_decode_matches_the_oracle(dtype, layout, hq, hkv, d, page, lens, opt):
    pg = Pages(lens, page, hkv, d, "e2m1", layout, seed=d + hq)
    q = _q(len(lens), hq, d, dtype)
    scales = (0.4, 1.7)
    dec = _dec(pg, hq, dtype, **opt)
    o, lse = dec.run(q, pg.pool, kv_block_scales=pg.scales, k_scale=scales[0], v_scale=scales[1], return_lse=True)
    torch.cuda.synchronize()
    assert dec.check_status() == 0
    kw = dict(cap=opt.get("logits_soft_cap", 0.0), window=opt.get("window_left", -1))
    if "pos_encoding_mode" in opt:
        kw["pos_encoding_mode"] = opt["pos_encoding_mode"]
    assert_decode(pg, q, o, lse, hq, scales=tuple(float(np.float32(s)) for s in scales), **kw)
    # a (k, v) pair of the same pool, float4 codes where torch has them, raw scale bytes: same bits
    pool = (pg.pool[:, 0], pg.pool[:, 1])
    if hasattr(torch, "float4_e2m1fn_x2"):
        pool = tuple(t.view(torch.float4_e2m1fn_x2) for t in pool)
    sf = pg.scales.view(torch.uint8)
    again = dec.run(q, pool, kv_block_scales=(sf[:, 0], sf[:, 1]), k_scale=scales[0], v_scale=scales[1])
    assert torch.equal(again, o)


@pytest.mark.parametrize("q_len", [2, 5])
def test_decode_several_queries_a_sequence(q_len):
    pg = Pages([5, 300, 64, 1000], 16, 2, 128, "e2m1", "HND", seed=1)
    q = _q(4 * q_len, 16, 128, BF16)
    dec = _dec(pg, 16, BF16, q_len_per_req=q_len)
    o, lse = dec.run(q, pg.pool, kv_block_scales=pg.scales, return_lse=True)
    assert_decode(pg, q, o, lse, 16, q_len=q_len)


def test_batches_of_nothing():
    """No sequence at all, and sequences without tokens: o = 0, lse = -inf."""
    pg = Pages([], 16, 2, 128, "e2m1", "NHD")
    o, lse = _dec(pg, 8, BF16).run(_q(0, 8, 128, BF16), pg.pool, kv_block_scales=pg.scales, return_lse=True)
    assert o.shape == (0, 8, 128) and lse.shape == (0, 8)
    pg = Pages([0, 0, 0], 16, 2, 128, "e2m1", "NHD")
    o, lse = _dec(pg, 8, BF16).run(_q(3, 8, 128, BF16), pg.pool, kv_block_scales=pg.scales, return_lse=True)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_unattended_slots_hold_anything():
    """NaN scales and any codes behind the last token, before the window and in foreign pages."""
    lens, window = [50, 9, 200, 16], 70
    pg = Pages(lens, 16, 2, 128, "e2m1", "NHD", seed=2)
    q = _q(4, 8, 128, BF16)
    dec = _dec(pg, 8, BF16, window_left=window)
    want = dec.run(q, pg.pool, kv_block_scales=pg.scales, return_lse=True)
    keep = torch.zeros(pg.num_pages, 16, dtype=torch.bool)
    for i, n in enumerate(lens):
        page, slot = pg.where([i] * n, np.arange(n))
        seen = np.arange(n) >= n - 1 - window
        keep[torch.from_numpy(page.astype(np.int64))[seen], torch.from_numpy(slot.astype(np.int64))[seen]] = True
    gone = ~keep.cuda().view(pg.num_pages, 1, 16, 1, 1)
    sf = pg.scales.view(torch.uint8)
    sf = torch.where(gone, torch.full_like(sf, 0x7f), sf)
    pool = torch.where(gone, torch.full_like(pg.pool, 0xff), pg.pool)
    got = dec.run(q, pool, kv_block_scales=sf, return_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # ... while an attended NaN shows
    page, slot = pg.where([0], [49])
    sf[int(page[0]), 0, int(slot[0]), 1, 3] = 0x7f
    o = dec.run(q, pool, kv_block_scales=sf)
    assert torch.isnan(o[0, 4:]).all() and not torch.isnan(o[0, :4]).any() and not torch.isnan(o[1:]).any()


def test_queries_of_any_range():
    """A bf16 head far outside fp16's range, and one far below it, beside ordinary ones."""
    pg = Pages([300, 40], 16, 1, 128, "e2m1", "HND", seed=4)
    q = _q(2, 8, 128, BF16)
    factor = torch.tensor([1.0, 1e-6, 3e4, 1e-3, 1.0, 1e-12, 60.0, 0.0], device="cuda").view(1, 8, 1)
    q = (q.float() * factor).to(BF16)
    scale = 1e-4  # keeps the largest scores in a range where the softmax says something
    dec = _dec(pg, 8, BF16)
    o, lse = dec.run(q, pg.pool, kv_block_scales=pg.scales, k_scale=scale, return_lse=True)
    assert_decode(pg, q, o, lse, 8, scales=(float(np.float32(scale)), 1.0))
    # tiny queries with a scale that makes up for them: their own bits decide the softmax
    q2 = (_q(2, 8, 128, BF16).float() * 1e-20).to(BF16)
    o, lse = _dec(pg, 8, BF16).run(q2, pg.pool, kv_block_scales=pg.scales, k_scale=1e20, return_lse=True)
    assert_decode(pg, q2, o, lse, 8, scales=(float(np.float32(1e20)), 1.0))


def test_bad_page_ids_are_reported_and_read_as_zeros():
    from paged_kv_decode_23_gb300 import _lib as L
    pg = Pages([64, 30], 16, 2, 128, "e2m1", "HND", seed=6)
    q = _q(2, 8, 128, BF16)
    ids = pg.indices.clone()
    ids[1] = pg.num_pages + 5
    dec = _dec(pg, 8, BF16)
    dec.plan(torch.from_numpy(pg.host_indptr), ids, torch.from_numpy(pg.last), 8, 2, 128, 16, q_data_type=BF16, kv_data_type="e2m1")
    got = dec.run(q, pg.pool, kv_block_scales=pg.scales)
    assert dec.check_status() == L.STATUS_BAD_PAGE
    pg.scales.view(torch.uint8)[int(pg.host_indices[1])] = 0
    want = _dec(pg, 8, BF16).run(q, pg.pool, kv_block_scales=pg.scales)
    assert torch.equal(got, want)


def test_wait_limit_reports_a_timeout():
    from paged_kv_decode_23_gb300 import _lib as L
    pg = Pages([3000] * 4, 16, 8, 128, "e2m1", "HND", seed=6)
    q = _q(4, 32, 128, BF16)
    dec = _dec(pg, 32, BF16)
    want = dec.run(q, pg.pool, kv_block_scales=pg.scales)
    dec.set_wait_limit(0)
    dec.run(q, pg.pool, kv_block_scales=pg.scales)
    assert dec.check_status() & L.STATUS_TIMEOUT
    dec.set_wait_limit(2_000_000_000)
    assert torch.equal(dec.run(q, pg.pool, kv_block_scales=pg.scales), want) and dec.check_status() == 0


def test_strided_pools():
    """Codes and scales as slices of wider tensors; the scales in a layout order of their own."""
    pg = Pages([100, 33], 16, 2, 128, "e2m1", "NHD", seed=3)
    q = _q(2, 4, 128, F16)
    dec = _dec(pg, 4, F16)
    want = dec.run(q, pg.pool, kv_block_scales=pg.scales)
    wide = torch.zeros(pg.num_pages, 2, 20, 3, 96, dtype=torch.uint8, device="cuda")
    wide[:, :, 2:18, 1:, 16:80] = pg.pool
    sf = torch.zeros(pg.num_pages, 2, 2, 17, 16, dtype=torch.uint8, device="cuda")[:, :, :, :16, 8:].transpose(2, 3)
    sf.copy_(pg.scales.view(torch.uint8))
    assert torch.equal(dec.run(q, wide[:, :, 2:18, 1:, 16:80], kv_block_scales=sf), want)


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("page", [8, 32, 128])
@pytest.mark.parametrize("first", ["k", "v"])
def test_k_and_v_in_buffers_of_their_own(layout, page, first):
    """A (k, v) pair of separate tensors, K's buffer below V's and above it."""
    pg = Pages([1000, 1, 333, 64], page, 2, 128, "e2m1", layout, seed=6)
    q = _q(4, 8, 128, BF16)
    dec = _dec(pg, 8, BF16)
    want = dec.run(q, pg.pool, kv_block_scales=pg.scales)

    def apart(x):
        b = torch.empty((2, x.shape[0]) + x.shape[2:], dtype=torch.uint8, device="cuda")
        at = (0, 1) if first == "k" else (1, 0)
        for i, j in enumerate(at):
            b[j] = x.view(torch.uint8)[:, i]
        return b[at[0]], b[at[1]]
    got = dec.run(q, apart(pg.pool), kv_block_scales=apart(pg.scales))
    torch.cuda.synchronize()
    assert dec.check_status() == 0 and torch.equal(got, want)


@pytest.mark.parametrize("cap", [1.0, 50.0])
def test_soft_cap_of_small_logits(cap):
    """Logits far below the cap pass it unchanged but for their cube: lse is good to its own
    rounding (2^-21 near 7) and the 32-bit sums' (16 roundings), below 2e-6; five times that."""
    pg = Pages([1000, 40], 16, 2, 128, "e2m1", "HND", seed=2)
    q = (_q(2, 8, 128, F16).float() * 1e-3).to(F16)
    dec = _dec(pg, 8, F16, logits_soft_cap=cap)
    o, lse = dec.run(q, pg.pool, kv_block_scales=pg.scales, return_lse=True)
    assert_decode(pg, q, o, lse, 8, cap=cap)
    _, ref = _ref(pg, q, 8, cap=cap)
    assert np.abs(lse.double().cpu().numpy() - ref).max() <= 1e-5


def test_two_plans_on_two_streams():
    """Two handles with workspaces of their own, their appends, runs and gathers in flight at once."""
    from paged_kv_decode_23_gb300 import append_paged_kv, gather_paged_kv
    sides = []
    for i, (hq, d) in enumerate(((8, 128), (24, 64))):
        pg = Pages([2000 + i, 700, 1], 16, 2, d, "e2m1", "NHD", seed=20 + i)
        g = torch.Generator().manual_seed(i)
        rows = [torch.randn(3, h, d, generator=g).to(BF16).cuda() for h in (hq, 2, 2)]
        b = torch.arange(3, dtype=torch.int32, device="cuda")
        pos = torch.from_numpy(pg.lens.astype(np.int32) - 1).cuda()
        sides.append((pg, _dec(pg, hq, BF16), rows, b, pos, torch.cuda.Stream()))

    def step(side, stream):
        pg, dec, rows, b, pos, _ = side
        table = dict(kv_indptr=pg.indptr, kv_indices=pg.indices, kv_layout="NHD", kv_block_scales=pg.scales)
        q = append_paged_kv(*rows, b, pos, pg.pool, stream=stream, **table)
        o = dec.run(q, pg.pool, kv_block_scales=pg.scales, stream=stream)
        return (o,) + gather_paged_kv(b, pos, pg.pool, stream=stream, **table)
    want = [step(s, None) for s in sides]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [step(s, s[5]) for s in sides]
    torch.cuda.synchronize()
    for s, g, w in zip(sides, got, want):
        assert s[1].check_status() == 0 and all(torch.equal(x, y) for x, y in zip(g, w))


def test_refusals():
    from paged_kv_decode_23_gb300 import PkdError
    pg = Pages([40], 16, 2, 128, "e2m1", "NHD", seed=3)
    q = _q(1, 4, 128, BF16)
    dec = _dec(pg, 4, BF16)
    sf = pg.scales
    for pool, scales in ((pg.pool, None), (pg.pool, sf[..., :4]), (pg.pool, sf.half()), (pg.pool, sf[:-1]),
                         (pg.pool, sf.transpose(2, 3)), (pg.pool[..., :32], sf), (pg.pool.to(F16), sf), (pg.pool, sf.cpu())):
        with pytest.raises(ValueError):
            dec.run(q, pool, kv_block_scales=scales)
    odd = torch.zeros(pg.num_pages, 2, 16, 2, 12, dtype=torch.uint8, device="cuda")[..., 4:]
    with pytest.raises(PkdError):
        dec.run(q, pg.pool, kv_block_scales=odd)
    with pytest.raises(PkdError):
        _dec(pg, 4, BF16, pos_encoding_mode="ROPE_LLAMA")
    with pytest.raises(PkdError):
        _dec(pg, 4, BF16, use_tensor_cores=False)
    same = Pages([40], 16, 2, 128, "same", "NHD", seed=3)
    from paged_kv_decode_23_gb300 import BatchDecodePagedKV
    plain = BatchDecodePagedKV(torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"))
    plain.plan(torch.from_numpy(same.host_indptr), same.indices, torch.from_numpy(same.last), 4, 2, 128, 16, q_data_type=BF16)
    with pytest.raises(ValueError):
        plain.run(q, same.pool, kv_block_scales=sf)
    assert plain.run(q, same.pool).shape == q.shape


def test_graph_replays_across_plans():
    """One captured launch serves later plans of the same batch size."""
    from paged_kv_decode_23_gb300 import CUDAGraphBatchDecodePagedKV
    pg = Pages([3000, 3000, 3000], 16, 2, 128, "e2m1", "HND", seed=8)
    dev = "cuda"
    bufs = [torch.zeros(n, dtype=torch.int32, device=dev) for n in (4, len(pg.indices), 3)]
    dec = CUDAGraphBatchDecodePagedKV(torch.zeros(64 << 20, dtype=torch.uint8, device=dev), *bufs, kv_layout="HND")
    q, o = _q(3, 8, 128, BF16), torch.zeros(3, 8, 128, dtype=BF16, device=dev)
    lse = torch.zeros(3, 8, device=dev)
    graph = None
    full = pg.host_indices.copy()
    for lens in ([3000, 17, 250], [1, 0, 2999], [16, 32, 48]):
        n = -(-np.array(lens) // 16)
        pg.host_indptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        pg.host_indices, pg.lens = full[:pg.host_indptr[-1]], np.array(lens)
        pg.last = np.where(pg.lens > 0, pg.lens - (n - 1) * 16, 0).astype(np.int32)
        dec.plan(torch.from_numpy(pg.host_indptr), torch.from_numpy(pg.host_indices).cuda(), torch.from_numpy(pg.last), 8, 2, 128, 16,
                 q_data_type=BF16, kv_data_type="e2m1")
        if graph is None:
            dec.run(q, pg.pool, kv_block_scales=pg.scales, out=o, lse=lse)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                dec.run(q, pg.pool, kv_block_scales=pg.scales, out=o, lse=lse)
        o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert dec.check_status() == 0
        assert_decode(pg, q, o, lse, 8)


def test_offsets_past_32_bits():
    """Pages whose codes and scales start past 2^32 bytes into their pools."""
    from paged_kv_decode_23_gb300 import append_paged_kv, copy_pages, gather_paged_kv
    hkv, page, d = 8, 256, 128
    per_page = 2 * page * hkv * d // 2  # 256 KiB
    pages = (1 << 32) // per_page + 8
    pool = torch.zeros(pages, 2, hkv, page, d // 2, dtype=torch.uint8, device="cuda")
    # scale pages spread far apart
    sf = torch.zeros(pages * (2 << 18), dtype=torch.uint8, device="cuda")
    sf = sf.as_strided((pages, 2, hkv, page, 8), (2 << 18, 1 << 18, page * 8, 8, 1))
    lens = [300]
    ids = np.array([pages - 1, pages - 3], dtype=np.int32)
    b, pos = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0] * 300, list(range(300))))
    indptr, indices = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 2], ids.tolist()))
    k, v = _q(300, hkv, d, BF16, 1), _q(300, hkv, d, BF16, 2)
    append_paged_kv(None, k, v, b, pos, pool, indptr, indices, "HND", kv_block_scales=sf)
    kb, vb = gather_paged_kv(b, pos, pool, indptr, indices, "HND", kv_block_scales=sf)
    for x, back in ((k, kb), (v, vb)):
        assert np.array_equal(quantise(x.double().cpu().numpy(), 1.0)[0], back.double().cpu().numpy())
    assert not pool[:pages - 3].any() and not pool[pages - 2].any()
    copy_pages([pool, sf[:, 0], sf[:, 1]], ids, [pages - 2, 1])
    kc, vc = gather_paged_kv(b, pos, pool, indptr, torch.tensor([pages - 2, 1], dtype=torch.int32, device="cuda"), "HND", kv_block_scales=sf)
    assert torch.equal(kc, kb) and torch.equal(vc, vb)
    from paged_kv_decode_23_gb300 import BatchDecodePagedKV
    q = _q(1, 8, d, BF16)
    outs = []
    for table in (ids, np.array([pages - 2, 1], dtype=np.int32)):
        dec = BatchDecodePagedKV(torch.zeros(8 << 20, dtype=torch.uint8, device="cuda"), "HND")
        dec.plan(torch.tensor([0, 2], dtype=torch.int32), torch.from_numpy(table).cuda(), torch.tensor([44], dtype=torch.int32), 8, hkv,
                 d, page, q_data_type=BF16, kv_data_type="e2m1")
        outs.append(dec.run(q, pool, kv_block_scales=sf))
    assert torch.equal(outs[0], outs[1])
    s = np.einsum("hd,thd->ht", q[0].double().cpu().numpy(), kb.double().cpu().numpy()) / np.sqrt(d)
    p = np.exp(s - s.max(1, keepdims=True))
    ref = np.einsum("ht,thd->hd", p / p.sum(1, keepdims=True), vb.double().cpu().numpy())
    assert np.abs(outs[0][0].double().cpu().numpy() - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 2e-3


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("kv", ["same", "e4m3", "e2m1"])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
def test_serving_sequences_from_prompt_to_fork_to_compaction(kv, layout):
    """Prompts are appended, steps decoded, a sequence forks, one ends, the pool is compacted: after
    each, every sequence decodes to what its own tokens, kept apart, give."""
    from paged_kv_decode_23_gb300 import (BatchDecodePagedKV, PageAllocator, append_paged_kv, copy_pages, gather_paged_kv,
                                          make_cos_sin_cache)
    hq, hkv, d, page, pages = 8, 2, 128, 16, 64
    dev = "cuda"
    dt = {"same": BF16, "e4m3": torch.float8_e4m3fn, "e2m1": torch.uint8}[kv]

    def pool(width, dtype):
        inner = (page, hkv) if layout == "NHD" else (hkv, page)
        return torch.zeros((pages, 2) + inner + (width,), dtype=torch.uint8 if dtype.itemsize == 1 else dtype, device=dev).view(dtype)
    data = pool(d // 2 if kv == "e2m1" else d, dt)
    scales = pool(d // 16, torch.float8_e4m3fn) if kv == "e2m1" else None
    pools = [data] if scales is None else [data, scales]
    sc = dict(k_scale=0.5, v_scale=0.25) if kv != "same" else {}
    alloc, table = PageAllocator(pages), make_cos_sin_cache(400, d)
    g = torch.Generator().manual_seed(11)
    weights = [(1 + 0.1 * torch.randn(d, generator=g)).to(BF16).to(dev) for _ in range(2)]
    seqs, kept = {}, {}  # name -> [pages, length]; name -> (k rows, v rows) as gathered

    def csr(names):
        ids = [np.asarray(seqs[n][0]) for n in names]
        indptr = np.concatenate([[0], np.cumsum([len(x) for x in ids])]).astype(np.int32)
        return indptr, np.concatenate(ids).astype(np.int32)

    def step(new):  # {name: tokens to append}
        names = list(new)
        for n in names:
            need = -(-(seqs[n][1] + new[n]) // page) - len(seqs[n][0])
            seqs[n][0] = np.concatenate([seqs[n][0], alloc.alloc(max(0, need))]).astype(np.int32)
        indptr, ids = csr(names)
        b = np.repeat(np.arange(len(names)), list(new.values())).astype(np.int32)
        pos = np.concatenate([np.arange(seqs[n][1], seqs[n][1] + new[n]) for n in names]).astype(np.int32)
        t = len(b)
        qkv = torch.randn(t, hq + 2 * hkv, d, generator=g).to(BF16).to(dev)
        q, k, v = qkv.split([hq, hkv, hkv], dim=1)
        bi, po, ip, ix = (torch.from_numpy(x).to(dev) for x in (b, pos, indptr, ids))
        qr = append_paged_kv(q, k, v, bi, po, data, ip, ix, layout, q_weight=weights[0], k_weight=weights[1],
                             cos_sin_cache=table, kv_block_scales=scales, **sc)
        back = gather_paged_kv(bi, po, data, ip, ix, layout, kv_block_scales=scales, **sc)
        for i, n in enumerate(names):
            mine = torch.from_numpy(b == i).to(dev)
            old = kept.get(n, (back[0][:0], back[1][:0]))
            kept[n] = tuple(torch.cat([o, x[mine]]) for o, x in zip(old, back))
            seqs[n][1] += new[n]
        return qr, b

    def check(names, q):
        indptr, ids = csr(names)
        lens = np.array([seqs[n][1] for n in names])
        last = (lens - 1) % page + 1
        dec = BatchDecodePagedKV(torch.zeros(16 << 20, dtype=torch.uint8, device=dev), layout)
        dec.plan(torch.from_numpy(indptr), torch.from_numpy(ids).to(dev), torch.from_numpy(last.astype(np.int32)), hq, hkv, d, page,
                 q_data_type=BF16, kv_data_type={"same": BF16, "e4m3": torch.float8_e4m3fn, "e2m1": "e2m1"}[kv])
        o = dec.run(q, data, **({} if scales is None else dict(kv_block_scales=scales)), **sc)
        assert dec.check_status() == 0
        for i, n in enumerate(names):
            k, v = (x.double().repeat_interleave(hq // hkv, dim=1) for x in kept[n])
            assert k.shape[0] == seqs[n][1]
            s = torch.einsum("hd,thd->ht", q[i].double(), k) / d ** 0.5
            p = torch.softmax(s, dim=1)
            want, mag = torch.einsum("ht,thd->hd", p, v), torch.einsum("ht,thd->hd", p, v.abs())
            # the gathered rows are rounded to bf16 (exactly, but for e4m3 and e2m1 times a scale: powers of two here)
            tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 1e-4) * mag + 1e-6
            assert ((o[i].double() - want).abs() <= tol).all(), n

    for n in "abc":
        seqs[n] = [np.zeros(0, dtype=np.int32), 0]
    step({"a": 37, "b": 100, "c": 5})
    for _ in range(3):
        q, _ = step({"a": 1, "b": 1, "c": 1})
        check(["a", "b", "c"], q)
    child, src, dst = alloc.fork(seqs["b"][0], seqs["b"][1], page)  # 103 tokens: 6 pages shared, one copied
    assert len(src) == 1 and child[:6].tolist() == seqs["b"][0][:6].tolist()
    copy_pages(pools, src, dst)
    seqs["d"], kept["d"] = [child, seqs["b"][1]], kept["b"]
    q, _ = step({"b": 1, "d": 1, "a": 1})  # the two diverge
    check(["b", "d", "a"], q)
    alloc.free(seqs.pop("a")[0])
    alloc.free(seqs.pop("b")[0])  # d keeps the shared pages
    src, dst, remap = alloc.compact()
    assert len(src) > 0
    copy_pages(pools, src, dst)
    for n in seqs:
        seqs[n][0] = remap[seqs[n][0]]
    assert max(max(s[0]) for s in seqs.values()) == int((alloc.uses() > 0).sum()) - 1
    q, _ = step({"c": 1, "d": 20})
    check(["c", "d"], q[[0, 20]])


def test_rotated_keys_match_rope_in_the_decode_kernel():
    """Keys rotated as they are appended, decoded without RoPE, against unrotated keys decoded with
    ROPE_LLAMA (both from q's own position): the same scores up to roundings."""
    from paged_kv_decode_23_gb300 import BatchDecodePagedKV, append_paged_kv, make_cos_sin_cache
    n, hq, hkv, d, page = 200, 8, 2, 128, 16
    pg = Pages([n], page, hkv, d, "same", "NHD", seed=1, dtype=F16)
    raw = torch.zeros_like(pg.pool)
    q, k, v = (torch.randn(n, h, d, generator=torch.Generator().manual_seed(h)).half().cuda() for h in (hq, hkv, hkv + 1))
    v = v[:, :hkv]
    b = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    qr = append_paged_kv(q, k, v, b, pos, pg.pool, pg.indptr, pg.indices, cos_sin_cache=make_cos_sin_cache(n, d))
    append_paged_kv(None, k, v, b, pos, raw, pg.indptr, pg.indices)
    outs = []
    for pool, query, mode in ((pg.pool, qr[-1:], "NONE"), (raw, q[-1:], "ROPE_LLAMA")):
        dec = BatchDecodePagedKV(torch.zeros(8 << 20, dtype=torch.uint8, device="cuda"))
        dec.plan(torch.from_numpy(pg.host_indptr), pg.indices, torch.from_numpy(pg.last), hq, hkv, d, page, pos_encoding_mode=mode,
                 q_data_type=F16)
        outs.append(dec.run(query.contiguous(), pool).double())
    # rotated q and k are rounded to fp16 in both: scores of std 1 with terms of up to ~8 differ by
    # some 2^-11 * 8 * 2, weights by that, o (|o| < 1, weights of 200 tokens) by less than 2e-2
    assert (outs[0] - outs[1]).abs().max() <= 2e-2


@pytest.mark.parametrize("dtype,hq,hkv,d,layout", [(F16, 4, 1, 128, "HND"), (BF16, 8, 1, 128, "NHD"), (F16, 16, 2, 64, "NHD"),
                                                   (BF16, 3, 3, 64, "HND"), (F16, 8, 2, 256, "NHD"), (BF16, 6, 1, 256, "HND")])
@pytest.mark.parametrize("depth", [14, 20, 25.5, 29])
def test_weights_far_below_a_dominant_key_count(dtype, hq, hkv, d, layout, depth):
    """A long row of keys `depth` bits below a few dominant ones, which weigh nothing in V: all of o comes
    from the small weights.  A weight is held to 11 bits, and to 2^-32 of the largest."""
    n = 65536
    pg = Pages([n], 64, hkv, d, "e2m1", layout, seed=1)
    pg.scales.fill_(1.0)
    pg.pool.zero_()
    codes = pg.pool if layout == "NHD" else pg.pool.transpose(2, 3)  # [pages, 2, slot, head, d / 2]
    codes[:, 1] = 0x57  # V: 6 and 3
    top = [3, 19, 35, 51]  # one key in every 16 of the first page
    codes[int(pg.host_indices[0]), 0, top, :, 0] = 0x07  # K: 6 in dim 0
    codes[int(pg.host_indices[0]), 1, top] = 0
    q = torch.zeros(1, hq, d)
    q[..., 0] = depth * np.log(2.0) * np.sqrt(d) / 6.0
    q[:, 1::2] *= 0.75
    q = q.to(dtype).cuda()
    o = _dec(pg, hq, dtype, disable_split_kv=True).run(q, pg.pool, kv_block_scales=pg.scales)
    ref_o, _ = _ref(pg, q, hq)
    o = o.double().cpu().numpy()
    # the weights sum to 4 at least where the largest is 1
    tol = (half_step(dtype) + 2.0 ** -11 + 1e-4) * np.abs(ref_o) + 2.0 ** -32 * n * 6.0 / 4 + float(torch.finfo(dtype).tiny) * half_step(dtype)
    assert (np.abs(o - ref_o) <= tol).all(), f"off by up to {(np.abs(o - ref_o) / np.abs(ref_o)).max():.3f} of o"


@pytest.mark.parametrize("hq,d", [(4, 128), (8, 128), (4, 64), (8, 256)])
@pytest.mark.parametrize("depth", [19.3, 20.4, 21.8])
def test_the_sum_of_small_weights_next_to_a_dominant_one(hq, d, depth):
    """lse of a long row whose small weights all round the same way when they are added to a large sum.
    Of n tokens a lane adds up n / 128 steps of four, each rounded to 2^-24 of the sum at most; scores,
    exp2 and the joining of the lanes stay within 1e-5 here (one product a score)."""
    n = 131072
    pg = Pages([n], 64, 1, d, "e2m1", "HND", seed=1)
    pg.scales.fill_(1.0)
    pg.pool.zero_()
    pg.pool[int(pg.host_indices[0]), 0, 0, [3, 19, 35, 51], 0] = 0x07  # K: 6 in dim 0 of one key in every 16
    q = torch.zeros(1, hq, d)
    q[..., 0] = depth * np.log(2.0) * np.sqrt(d) / 6.0 * (1 + torch.arange(hq) / 64)
    q = q.to(F16).cuda()
    _, lse = _dec(pg, hq, F16, disable_split_kv=True).run(q, pg.pool, kv_block_scales=pg.scales, return_lse=True)
    _, ref = _ref(pg, q, hq)
    assert np.abs(lse.double().cpu().numpy() - ref).max() <= n / 128 * 2.0 ** -24 + 1e-5


def test_derivatives_are_refused_not_dropped():
    import torch.autograd.forward_ad as fwAD
    pg = Pages([50], 16, 2, 128, "e2m1", "NHD", seed=2)
    q = _q(1, 8, 128, BF16)
    dec = _dec(pg, 8, BF16)
    want = dec.run(q, pg.pool, kv_block_scales=pg.scales)
    leaf = q.clone().requires_grad_()
    with pytest.raises(NotImplementedError, match="backward"):
        dec.run(leaf, pg.pool, kv_block_scales=pg.scales)
    with torch.no_grad():
        assert torch.equal(dec.run(leaf, pg.pool, kv_block_scales=pg.scales), want)
    with fwAD.dual_level():
        dual = fwAD.make_dual(q.clone(), torch.ones_like(q))
        with pytest.raises(NotImplementedError, match="forward"):
            dec.run(dual, pg.pool, kv_block_scales=pg.scales)
