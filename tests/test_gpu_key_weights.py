"""Decode that sums its keys' softmax weights, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from bounded_ref import assert_decode, decode_ref, decoder, values
from cache_ref import Pages

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def _q(rows, hq, d, dtype, seed=0):
    return torch.randn(rows, hq, d, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _weights(pg, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.rand(pg.num_pages, pg.hkv, pg.page, generator=g).cuda()


def assert_weights(pg, got, before, sums, lens=None, what=""):
    """Each added weight is off by what its score is (below 1e-5, see assert_decode), twice, with exp2
    and the sums inside 1e-4 of it in all; the addition rounds once, the sum of rows and heads before it
    is counted.  Entries of keys that no row attends keep their bits."""
    got, want = got.cpu().double(), before.cpu().double()
    add = torch.zeros_like(want)
    for b, s in sums.items():
        n = s.shape[1]
        page, slot = (torch.from_numpy(np.asarray(x).astype(np.int64)) for x in pg.where(np.full(n, b), np.arange(n)))
        for i in range(n):
            add[page[i], :, slot[i]] += s[:, i]
    off = (got - want - add).abs()
    tol = 1e-4 * add + 2.0 ** -23 * (want + add).abs()
    assert (off <= tol).all(), f"{what}: {int((off > tol).sum())} weights off, max {float(off.max()):.3e}"
    same = add == 0
    assert torch.equal(got[same], want[same]), what


# dtype, kv, layout, hq, hkv, d, page, lens, options
CASES = [
    (BF16, "same", "NHD", 32, 8, 128, 16, [1, 15, 16, 17, 500, 0, 1300], {}),
    (F16, "same", "HND", 8, 8, 64, 8, [3, 129, 128, 255, 256, 257, 2000], {}),
    (BF16, "same", "NHD", 16, 2, 256, 32, [3000, 64, 1], dict(logits_soft_cap=30.0, window_left=500)),
    (F16, "same", "HND", 24, 2, 128, 64, [700, 5], dict(window_left=0)),              # 12 heads a kv head
    (BF16, "same", "HND", 6, 1, 64, 256, [4000, 1, 256], dict(fixed_split_size=1)),
    (F16, "same", "NHD", 3, 3, 256, 16, [777] * 3, dict(disable_split_kv=True)),
    (BF16, "same", "HND", 32, 8, 128, 16, [9000], {}),                                # one row over the GPU
    (BF16, "same", "NHD", 8, 2, 128, 16, [2000, 103, 102, 4], dict(window_left=100, num_sink_tokens=4)),
    (F16, "same", "NHD", 8, 2, 128, 16, [40, 41, 300], dict(window_left=33, num_sink_tokens=6)),  # both in one page
    (BF16, "same", "NHD", 8, 2, 128, 16, [600, 40], dict(pos_encoding_mode="ALIBI")),
    (F16, "same", "HND", 8, 1, 128, 64, [9000, 8000], dict(window_left=3000, num_sink_tokens=1000)),  # sinks in chunks
    (BF16, "e2m1", "HND", 8, 1, 128, 8, [4000], dict(window_left=100, num_sink_tokens=520, fixed_split_size=16)),
    (BF16, "e4m3", "HND", 32, 8, 128, 64, [5000, 129, 0, 2], dict(window_left=1023, num_sink_tokens=100)),
    (F16, "e4m3", "NHD", 16, 2, 256, 32, [3000, 77], dict(logits_soft_cap=20.0)),
    (BF16, "e2m1", "HND", 32, 8, 128, 16, [1, 15, 500, 0, 1300, 5000], {}),
    (F16, "e2m1", "NHD", 8, 8, 64, 8, [3, 129, 2000], dict(window_left=128, num_sink_tokens=40)),
    (BF16, "e2m1", "NHD", 16, 2, 256, 32, [1, 63, 3000], dict(logits_soft_cap=30.0)),
    (F16, "e2m1", "HND", 12, 1, 128, 128, [3000, 9], {}),
]


@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_key_weights_match_the_definition(case, q_len):
    dtype, kv, layout, hq, hkv, d, page, lens, opt = CASES[case]
    pg = Pages(lens, page, hkv, d, kv, layout, seed=case, dtype=dtype)
    pool64 = values(pg.pool, pg.scales)
    q = _q(len(lens) * q_len, hq, d, dtype, seed=case)
    scales = (0.4, 1.7) if kv != "same" else (1.0, 1.0)
    run = dict(kv_block_scales=pg.scales, k_scale=scales[0], v_scale=scales[1], return_lse=True)
    dec = decoder(pg, hq, dtype, q_len_per_req=q_len, key_weights=True, **opt)
    before = _weights(pg, case)
    got = before.clone()
    o, lse = dec.run(q, pg.pool, key_weights=got, **run)
    torch.cuda.synchronize()
    assert dec.check_status() == 0
    ref = decode_ref(pg, pool64, q, q_len=q_len, window=opt.get("window_left", -1), sinks=opt.get("num_sink_tokens", 0),
                     cap=opt.get("logits_soft_cap", 0.0), k_scale=scales[0], v_scale=scales[1],
                     pos=opt.get("pos_encoding_mode"))
    assert_decode(q, o, lse, ref, pool64, max(lens), scales[1])
    assert_weights(pg, got, before, ref[3])
    # the same bits again, and those of a run without the weights
    again = before.clone()
    o2, lse2 = dec.run(q, pg.pool, key_weights=again, **run)
    assert torch.equal(got, again) and torch.equal(o, o2) and torch.equal(lse, lse2)
    o3, lse3 = decoder(pg, hq, dtype, q_len_per_req=q_len, **opt).run(q, pg.pool, **run)
    assert torch.equal(o, o3) and torch.equal(lse, lse3)


def test_lse_may_be_left_out_and_weights_may_have_strides():
    pg = Pages([300, 40], 16, 2, 128, "same", "NHD", seed=1)
    q = _q(2, 8, 128, BF16)
    dec = decoder(pg, 8, BF16, key_weights=True)
    a = torch.zeros(pg.num_pages, 2, 16, device="cuda")
    dec.run(q, pg.pool, key_weights=a)
    big = torch.full((pg.num_pages, 16, 5), 7.0, device="cuda")  # [pages, slots, heads and more]
    b = big[:, :, 1:3].transpose(1, 2)
    b.zero_()
    dec.run(q, pg.pool, key_weights=b)
    assert torch.equal(a, b) and (big[:, :, 0] == 7).all() and (big[:, :, 3:] == 7).all()
    for off in (1, 2, 3):  # an address that is no multiple of 16
        flat = torch.zeros(a.numel() + 8, device="cuda")
        mine = flat[off:off + a.numel()].view(a.shape)
        dec.run(q, pg.pool, key_weights=mine)
        assert torch.equal(a, mine) and (flat[:off] == 0).all() and (flat[off + a.numel():] == 0).all()
    k, v = pg.pool[:, 0].contiguous(), pg.pool[:, 1].contiguous()
    c = torch.zeros_like(a)
    dec.run(q, (k, v), key_weights=c)
    assert torch.equal(a, c)


def test_requests_that_share_pages_add_up():
    pg = Pages([160, 160, 160], 16, 2, 128, "same", "HND", seed=2)
    # the three requests share their first five pages
    for b in (1, 2):
        pg.host_indices[pg.host_indptr[b]:pg.host_indptr[b] + 5] = pg.host_indices[:5]
    pg.indices = torch.from_numpy(pg.host_indices).cuda()
    q = _q(3, 8, 128, F16)
    pg.pool = pg.pool.half()
    dec = decoder(pg, 8, F16, key_weights=True)
    before = _weights(pg)
    got = before.clone()
    dec.run(q, pg.pool, key_weights=got)
    ref = decode_ref(pg, values(pg.pool), q)
    assert_weights(pg, got, before, ref[3])


def test_dominant_and_far_keys():
    """One key with nearly all the weight, its neighbours 2^-100 and less below it; and logits so far
    apart that all but one weight is 0."""
    pg = Pages([64, 64], 16, 1, 128, "same", "NHD", seed=3)
    pg.pool.zero_()
    for b, big in ((0, 8.0), (1, 300.0)):
        page, slot = pg.where(np.array([b]), np.array([37]))
        pg.pool[int(page[0]), 0, int(slot[0]), 0, 0] = big
    q = torch.zeros(2, 4, 128, dtype=BF16, device="cuda")
    q[:, :, 0] = 100.0
    dec = decoder(pg, 4, BF16, key_weights=True)
    before = torch.zeros(pg.num_pages, 1, 16, device="cuda")
    got = before.clone()
    dec.run(q, pg.pool, key_weights=got)
    assert_weights(pg, got, before, decode_ref(pg, values(pg.pool), q)[3])


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows_of_infinitely_low_scores_have_no_weights(dtype):
    """Requests whose every score is -inf (one task, and split into several), and one with some such keys: no
    weight and no NaN is added for them."""
    lens = [40, 9000, 300]
    pg = Pages(lens, 16, 2, 128, "same", "NHD", seed=21, dtype=dtype)
    low = {0: range(40), 1: range(9000), 2: (0, 17, 18, 299)}
    for b, tokens in low.items():
        page, slot = pg.where(np.full(len(tokens), b), np.array(tokens))
        pg.pool[torch.from_numpy(page).long().cuda(), 0, torch.from_numpy(slot).long().cuda(), :, 0] = -float("inf")
    q = _q(3, 8, 128, dtype)
    q[..., 0] = 1.0
    dec = decoder(pg, 8, dtype, key_weights=True)
    before = _weights(pg)
    got = before.clone()
    o, lse = dec.run(q, pg.pool, key_weights=got, return_lse=True)
    assert dec.check_status() == 0
    assert (o[:2] == 0).all() and torch.isneginf(lse[:2]).all() and torch.isfinite(lse[2]).all()
    ref = decode_ref(pg, values(pg.pool), q)
    assert_weights(pg, got, before, {2: ref[3][2]})


def test_bad_pages_have_no_weights():
    pg = Pages([100, 30], 16, 2, 128, "same", "NHD", seed=4)
    ids = pg.host_indices.copy()
    gone = int(ids[2])
    ids[2] = pg.num_pages  # keys 32..47 of request 0: read as zeros, no entry
    dec = decoder(pg, 8, BF16, key_weights=True, indices=torch.from_numpy(ids).cuda())
    got = torch.zeros(pg.num_pages, 2, 16, device="cuda")
    q = _q(2, 8, 128, BF16)
    dec.run(q, pg.pool, key_weights=got)
    from paged_kv_decode_23_gb300 import _lib as L
    assert dec.check_status() == L.STATUS_BAD_PAGE
    zeroed = pg.pool.clone()
    zeroed[gone] = 0
    ref = decode_ref(pg, values(zeroed), q)[3]
    ref[0][:, 32:48] = 0
    assert_weights(pg, got, torch.zeros_like(got), ref)


def test_nothing_is_added_after_a_timeout():
    pg = Pages([3000], 16, 2, 128, "same", "NHD", seed=5)
    dec = decoder(pg, 8, BF16, key_weights=True)
    q = _q(1, 8, 128, BF16)
    got = torch.zeros(pg.num_pages, 2, 16, device="cuda")
    dec.run(q, pg.pool, key_weights=got)
    want = got.clone()
    dec.set_wait_limit(0)
    torch.zeros(300 << 20, dtype=torch.uint8, device="cuda")  # (a cold L2)
    dec.run(q, pg.pool, key_weights=got)
    from paged_kv_decode_23_gb300 import _lib as L
    status = dec.check_status()
    if status == L.STATUS_TIMEOUT:
        assert torch.equal(got, want)
    dec.set_wait_limit(2 * 10 ** 9)
    got.zero_()
    dec.run(q, pg.pool, key_weights=got)
    assert dec.check_status() == 0 and torch.equal(got, want)


def test_a_captured_run_replays_across_plans():
    from paged_kv_decode_23_gb300 import CUDAGraphBatchDecodePagedKV, graph_workspace_bytes
    page, batch, dtype = 16, 4, BF16
    pg = Pages([4000] * batch, page, 2, 128, "e4m3", "NHD", seed=6)
    pool64 = values(pg.pool)
    pages, items = len(pg.host_indices), batch + 2 * 152
    i32 = dict(dtype=torch.int32, device="cuda")
    fb, ib = graph_workspace_bytes(items, 16, 2, 128, key_weights_pages=pages, page_size=page, max_batch=batch)
    dec = CUDAGraphBatchDecodePagedKV(torch.zeros(fb, dtype=torch.uint8, device="cuda"), torch.zeros(batch + 1, **i32),
                                      torch.zeros(pages, **i32), torch.zeros(batch, **i32), "NHD", max_items=items,
                                      int_workspace_buffer=torch.zeros(ib, dtype=torch.uint8, device="cuda"))
    q = torch.zeros(batch, 16, 128, dtype=dtype, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros(batch, 16, device="cuda")
    w = torch.zeros(pg.num_pages, 2, page, device="cuda")
    graph = None
    for step, (lens, opt) in enumerate([([4000, 17, 900, 1], dict(window_left=800, num_sink_tokens=4)),
                                        ([1, 0, 3999, 2500], dict(window_left=2000, num_sink_tokens=300)),
                                        ([4000] * 4, {}), ([0, 0, 0, 5], {})]):
        part = Pages(lens, page, 2, 128, "e4m3", "NHD", seed=6 + step, spare=pages)
        at = np.random.default_rng(step).permutation(pg.num_pages)
        part.host_indices = at[:len(part.host_indices)].astype(np.int32)
        part.num_pages = pg.num_pages
        ix = torch.from_numpy(part.host_indices).cuda()
        dec.plan(torch.from_numpy(part.host_indptr), ix, torch.from_numpy(part.last), 16, 2, 128, page,
                 q_data_type=dtype, kv_data_type=torch.float8_e4m3fn, key_weights=True, **opt)
        q.copy_(_q(batch, 16, 128, dtype, seed=step))
        if graph is None:
            dec.run(q, pg.pool, out=o, lse=lse, key_weights=w)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                dec.run(q, pg.pool, out=o, lse=lse, key_weights=w)
        before = w.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert dec.check_status() == 0
        ref = decode_ref(part, pool64, q, window=opt.get("window_left", -1), sinks=opt.get("num_sink_tokens", 0))
        assert_decode(q, o, lse, ref, pool64, 4000, what=str(step))
        assert_weights(part, w, before, ref[3], what=str(step))
    with pytest.raises(Exception, match="key_weights is fixed"):
        dec.plan(torch.from_numpy(part.host_indptr), ix, torch.from_numpy(part.last), 16, 2, 128, page,
                 q_data_type=dtype, kv_data_type=torch.float8_e4m3fn)


def test_two_handles_on_two_streams():
    pg = Pages([2000, 300], 16, 2, 128, "same", "NHD", seed=7)
    q = _q(2, 8, 128, BF16)
    decs = [decoder(pg, 8, BF16, key_weights=True) for _ in range(2)]
    outs = [torch.zeros(pg.num_pages, 2, 16, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for dec, w, s in zip(decs, outs, streams):
            dec.run(q, pg.pool, key_weights=w, stream=s)
    torch.cuda.synchronize()
    one = torch.zeros_like(outs[0])
    for _ in range(5):
        decs[0].run(q, pg.pool, key_weights=one)
    assert torch.equal(outs[0], one) and torch.equal(outs[1], one)


def test_refusals():
    from paged_kv_decode_23_gb300 import PkdError
    pg = Pages([300, 40], 16, 2, 128, "same", "NHD", seed=8)
    q = _q(2, 8, 128, BF16)
    w = torch.zeros(pg.num_pages, 2, 16, device="cuda")
    plain, dec = decoder(pg, 8, BF16), decoder(pg, 8, BF16, key_weights=True)
    with pytest.raises(ValueError, match="key_weights"):
        plain.run(q, pg.pool, key_weights=w)
    with pytest.raises(ValueError, match="key_weights"):
        dec.run(q, pg.pool)
    for bad in (w.half(), w[:-1], w.transpose(1, 2), w.cpu(), w.view(-1), 5):
        with pytest.raises(ValueError, match="key_weights"):
            dec.run(q, pg.pool, key_weights=bad)
    with pytest.raises(PkdError, match="overlap"):
        dec.run(q, pg.pool, key_weights=w[:1].expand(pg.num_pages, -1, -1))
    with pytest.raises(NotImplementedError):
        dec.run(q, pg.pool, key_weights=w.clone().requires_grad_())
    with pytest.raises(NotImplementedError):
        dec.run(q.clone().requires_grad_(), pg.pool, key_weights=w)
    with pytest.raises(ValueError):
        dec.run(q, pg.pool[:, :, :8], key_weights=w)
    for opt in (dict(use_tensor_cores=False), dict(pos_encoding_mode="ROPE_LLAMA")):
        with pytest.raises(PkdError, match="UNSUPPORTED"):
            decoder(pg, 8, BF16, key_weights=True, **opt)
    with pytest.raises(PkdError, match="workspace too small"):
        decoder(pg, 8, BF16, ws=20000, key_weights=True)
    assert (w == 0).all()


def test_workspace_bytes_are_enough():
    from paged_kv_decode_23_gb300 import BatchDecodePagedKV, workspace_bytes
    pg = Pages([3000, 40, 0, 700], 16, 2, 128, "same", "NHD", seed=9)
    for opt in ({}, dict(window_left=300, num_sink_tokens=20, q_len_per_req=2)):
        fb, ib = workspace_bytes(pg.host_indptr, pg.last, 8, 2, 128, 16, kv_dtype=1, key_weights=True, **opt)
        dec = BatchDecodePagedKV(torch.zeros(fb, dtype=torch.uint8, device="cuda"), "NHD",
                                 int_workspace_buffer=torch.zeros(ib, dtype=torch.uint8, device="cuda"))
        dec.plan(torch.from_numpy(pg.host_indptr), pg.indices, torch.from_numpy(pg.last), 8, 2, 128, 16, q_data_type=BF16,
                 key_weights=True, **opt)
        w = torch.zeros(pg.num_pages, 2, 16, device="cuda")
        q = _q(4 * opt.get("q_len_per_req", 1), 8, 128, BF16)
        dec.run(q, pg.pool, key_weights=w)
        # every row with a key adds a weight of 1 per qo head (4 of them a kv head)
        rows = 3 * opt.get("q_len_per_req", 1)
        assert abs(float(w.double().sum()) - rows * 8) < 1e-4 * rows * 8


def test_a_cache_whose_gradient_would_be_lost_is_refused():
    pg = Pages([300, 40], 16, 2, 128, "same", "NHD", seed=10)
    q = _q(2, 8, 128, BF16)
    w = torch.zeros(pg.num_pages, 2, 16, device="cuda")
    dec = decoder(pg, 8, BF16, key_weights=True)
    k, v = pg.pool[:, 0].contiguous(), pg.pool[:, 1].contiguous()
    for cache in (pg.pool.clone().requires_grad_(), (k.clone().requires_grad_(), v), (k, v.clone().requires_grad_())):
        with pytest.raises(NotImplementedError, match="no backward pass"):
            dec.run(q, cache, key_weights=w)
        with torch.no_grad():
            dec.run(q, cache, key_weights=torch.zeros_like(w))
    assert (w == 0).all()


@pytest.mark.parametrize("opt", [dict(sm_scale=1e300), dict(logits_soft_cap=1e39), dict(pos_encoding_mode="ROPE_LLAMA", rope_theta=1e39),
                                 dict(pos_encoding_mode="ROPE_LLAMA", rope_scale=float("inf"))])
def test_infinite_numbers_are_refused(opt):
    from paged_kv_decode_23_gb300 import PkdError
    pg = Pages([30], 16, 2, 128, "same", "NHD", seed=11)
    with pytest.raises(PkdError, match="finite"):
        decoder(pg, 8, BF16, **opt)


def test_more_keys_than_the_second_kernels_grid_holds():
    """So many (tile of keys, kv head)s that its CTAs (16 an SM at most) take several, with and without sinks; and
    the same plan in CUDA-graph mode, replayed."""
    from paged_kv_decode_23_gb300 import CUDAGraphBatchDecodePagedKV, graph_workspace_bytes
    hkv, hq, d, page = 8, 16, 64, 8
    ctas = 16 * torch.cuda.get_device_properties(0).multi_processor_count
    batch = 2 * ctas // hkv + 10  # a tile each at least
    lens = np.random.default_rng(5).integers(1, 65, batch)
    lens[5], lens[-1], lens[17] = 1700, 2000, 0
    pg = Pages(lens.tolist(), page, hkv, d, "same", "NHD", seed=12, dtype=F16)
    pool64 = values(pg.pool)
    q = _q(batch, hq, d, F16)
    for opt in ({}, dict(window_left=9, num_sink_tokens=5)):
        ref = decode_ref(pg, pool64, q, window=opt.get("window_left", -1), sinks=opt.get("num_sink_tokens", 0))
        before = _weights(pg)
        got = before.clone()
        dec = decoder(pg, hq, F16, key_weights=True, **opt)
        dec.run(q, pg.pool, key_weights=got)
        assert dec.check_status() == 0
        assert_weights(pg, got, before, ref[3])
        i32 = dict(dtype=torch.int32, device="cuda")
        items, pages = batch + 2 * 152, len(pg.host_indices)
        fb, ib = graph_workspace_bytes(items, hq, hkv, d, key_weights_pages=pages, page_size=page, max_batch=batch)
        dec = CUDAGraphBatchDecodePagedKV(torch.zeros(fb, dtype=torch.uint8, device="cuda"), torch.zeros(batch + 1, **i32),
                                          torch.zeros(pages, **i32), torch.zeros(batch, **i32), "NHD", max_items=items,
                                          int_workspace_buffer=torch.zeros(ib, dtype=torch.uint8, device="cuda"))
        dec.plan(torch.from_numpy(pg.host_indptr), pg.indices, torch.from_numpy(pg.last), hq, hkv, d, page, q_data_type=F16,
                 key_weights=True, **opt)
        o, w = torch.zeros_like(q), before.clone()
        dec.run(q, pg.pool, out=o, key_weights=w)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dec.run(q, pg.pool, out=o, key_weights=w)
        w.copy_(before)
        graph.replay()
        torch.cuda.synchronize()
        assert dec.check_status() == 0
        assert_weights(pg, w, before, ref[3], what="replayed")


def test_a_run_that_timed_out_adds_nothing():
    """Waits that give up at once, over keys that are not in L2: the status says so, and no entry changes."""
    from paged_kv_decode_23_gb300 import _lib as L
    pg = Pages([3000, 17, 2000, 4000, 1000, 700, 0, 2500] * 4, 16, 2, 128, "same", "NHD", seed=13)
    dec = decoder(pg, 8, BF16, key_weights=True, fixed_split_size=8)
    q = _q(32, 8, 128, BF16)
    before = _weights(pg)
    want = before.clone()
    dec.run(q, pg.pool, key_weights=want)
    assert dec.check_status() == 0
    got = before.clone()
    dec.set_wait_limit(0)
    torch.zeros(300 << 20, dtype=torch.uint8, device="cuda")
    dec.run(q, pg.pool, key_weights=got)
    dec.set_wait_limit(2 * 10 ** 9)
    dec.run(q, pg.pool, key_weights=got)  # (the word is still set)
    assert dec.check_status() & L.STATUS_TIMEOUT
    assert torch.equal(got, before)
    dec.run(q, pg.pool, key_weights=got)
    assert dec.check_status() == 0 and torch.equal(got, want)
