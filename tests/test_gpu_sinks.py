"""Decode over a sliding window and the first tokens of each request (sinks) against its definition in
64 bits."""
import numpy as np
import pytest
import torch

from bounded_ref import assert_decode, decode_ref, decoder, values
from cache_ref import Pages

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16

# dtype, kv, layout, hq, hkv, d, page, lens, window, sinks, options
CASES = [
    (BF16, "same", "NHD", 32, 8, 128, 16, [1, 4, 5, 6, 100, 101, 102, 0, 1300], 100, 4, {}),
    (F16, "same", "HND", 8, 8, 64, 8, [700, 3, 64, 65, 66], 63, 1, {}),
    (BF16, "same", "NHD", 16, 2, 256, 32, [3000, 200, 1], 150, 33, dict(logits_soft_cap=30.0)),
    (BF16, "same", "HND", 24, 2, 128, 64, [9000, 8000], 3000, 1000, {}),             # sinks cut into chunks
    (F16, "same", "NHD", 4, 1, 128, 16, [20000], 9000, 128, {}),                     # one row over the GPU
    (BF16, "same", "NHD", 6, 1, 64, 256, [4000, 1, 256, 700], 300, 17, dict(fixed_split_size=1)),
    (F16, "same", "NHD", 3, 3, 256, 16, [777] * 3, 0, 5, dict(disable_split_kv=True)),
    (BF16, "same", "HND", 8, 2, 128, 16, [500, 2000], 64, 600, dict(fixed_split_size=8)),
    (BF16, "same", "NHD", 8, 2, 128, 16, [600, 40], 100, 10, dict(pos_encoding_mode="ALIBI")),
    (BF16, "e4m3", "HND", 32, 8, 128, 64, [5000, 129, 0, 128, 2], 1023, 100, {}),
    (F16, "e4m3", "NHD", 16, 2, 256, 32, [4000, 77], 500, 4, dict(logits_soft_cap=20.0)),
    (BF16, "e2m1", "HND", 32, 8, 128, 16, [1, 15, 500, 0, 1300, 9000], 250, 4, {}),
    (F16, "e2m1", "NHD", 8, 8, 64, 8, [3, 129, 2000], 128, 40, {}),
    (BF16, "e2m1", "NHD", 16, 2, 256, 32, [1, 63, 3000], 100, 700, dict(logits_soft_cap=30.0)),
    (F16, "e2m1", "HND", 8, 1, 128, 256, [3000, 9], 511, 300, dict(pos_encoding_mode="ALIBI")),
    (BF16, "e2m1", "HND", 8, 1, 128, 8, [4000], 3, 520, dict(fixed_split_size=16)),
    # the fp32 CUDA-core kernel and the rotating ones
    (BF16, "same", "NHD", 8, 2, 128, 16, [900, 33, 0], 100, 4, dict(use_tensor_cores=False)),
    (F16, "same", "HND", 8, 8, 64, 8, [500, 20], 63, 30, dict(use_tensor_cores=False)),
    (F16, "e4m3", "NHD", 16, 2, 256, 32, [900, 77], 200, 4, dict(use_tensor_cores=False)),
    (F16, "same", "NHD", 8, 2, 128, 16, [900, 33], 100, 4, dict(pos_encoding_mode="ROPE_LLAMA")),
    (BF16, "e4m3", "HND", 8, 2, 128, 32, [900, 133], 100, 65, dict(pos_encoding_mode="ROPE_LLAMA")),
    (F16, "same", "NHD", 8, 2, 128, 16, [900, 33], 100, 4, dict(pos_encoding_mode="ROPE_LLAMA", use_tensor_cores=False)),
]


def _q(rows, hq, d, dtype, seed=0):
    return torch.randn(rows, hq, d, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _ref(pg, pool64, q, opt, window, sinks, scales, q_len=1):
    return decode_ref(pg, pool64, q, q_len=q_len, window=window, sinks=sinks, cap=opt.get("logits_soft_cap", 0.0),
                      k_scale=scales[0], v_scale=scales[1], pos=opt.get("pos_encoding_mode"))


@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_sinks_match_the_definition(case, q_len):
    dtype, kv, layout, hq, hkv, d, page, lens, window, sinks, opt = CASES[case]
    pg = Pages(lens, page, hkv, d, kv, layout, seed=case, dtype=dtype)
    pool64 = values(pg.pool, pg.scales)
    q = _q(len(lens) * q_len, hq, d, dtype, seed=case)
    scales = (0.4, 1.7) if kv != "same" else (1.0, 1.0)
    # what no row attends: NaN in the pages' slots, and page ids of whole pages in between that are none
    indices = pg.host_indices.copy()
    pool, sf = pg.pool.clone(), None if pg.scales is None else pg.scales.clone()
    dead = sf if sf is not None else pool
    seen = np.zeros((pg.num_pages, page), dtype=bool)
    for b, n in enumerate(lens):
        for j in range(q_len):
            last = n - q_len + j
            if last >= 0:
                t = [t for t in range(last + 1) if t >= last - window or t < sinks]
                pid, slot = pg.where(np.full(len(t), b), np.array(t, dtype=np.int64))
                seen[pid, slot] = True
    off = torch.from_numpy(~seen).cuda()
    nan = 0x7f if sf is not None or kv == "e4m3" else None
    view = dead.view(torch.uint8) if nan else dead
    for i in (0, 1):
        x = view[:, i] if layout == "NHD" else view[:, i].transpose(1, 2)
        x[off] = nan if nan else float("nan")
    for i in range(len(indices)):
        if not seen[pg.host_indices[i]].any():
            indices[i] = (-1, 2 ** 31 - 1, pg.num_pages)[i % 3]
    dec = decoder(pg, hq, dtype, indices=torch.from_numpy(indices).cuda(), window_left=window, num_sink_tokens=sinks,
                  q_len_per_req=q_len, **opt)
    o, lse = dec.run(q, pool, kv_block_scales=sf, k_scale=scales[0], v_scale=scales[1], return_lse=True)
    torch.cuda.synchronize()
    assert dec.check_status() == 0
    assert_decode(q, o, lse, _ref(pg, pool64, q, opt, window, sinks, scales, q_len), pool64, max(lens), scales[1],
                  rope=opt.get("pos_encoding_mode") == "ROPE_LLAMA")
    o2, lse2 = dec.run(q, pool, kv_block_scales=sf, k_scale=scales[0], v_scale=scales[1], return_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kv", ["same", "e4m3", "e2m1"])
def test_sinks_that_reach_the_window_are_no_window_at_all(kv):
    pg = Pages([900, 40, 333], 16, 2, 128, kv, "NHD", seed=3)
    q = _q(3, 8, 128, BF16)
    got = []
    for opt in (dict(window_left=100, num_sink_tokens=800), dict(window_left=-1), dict(window_left=-1, num_sink_tokens=5)):
        dec = decoder(pg, 8, BF16, **opt)
        got.append(dec.run(q, pg.pool, kv_block_scales=pg.scales, return_lse=True))
    for o, lse in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])


def test_a_fixed_split_gives_a_row_the_same_bits_in_every_batch():
    lens = [3000, 77, 1500]
    pg = Pages(lens, 16, 2, 128, "same", "NHD", seed=4)
    q = _q(3, 8, 128, BF16)
    opt = dict(window_left=700, num_sink_tokens=90, fixed_split_size=4)
    o, lse = decoder(pg, 8, BF16, **opt).run(q, pg.pool, return_lse=True)
    from paged_kv_decode_23_gb300 import BatchDecodePagedKV
    for b, n in enumerate(lens):
        one = BatchDecodePagedKV(torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"), "NHD")
        ix = pg.indices[int(pg.host_indptr[b]):int(pg.host_indptr[b + 1])].contiguous()
        one.plan(torch.tensor([0, len(ix)], dtype=torch.int32), ix, torch.from_numpy(pg.last[b:b + 1]), 8, 2, 128, 16,
                 q_data_type=BF16, **opt)
        o1, l1 = one.run(q[b:b + 1].contiguous(), pg.pool, return_lse=True)
        assert torch.equal(o1[0], o[b]) and torch.equal(l1[0], lse[b])


def test_a_captured_run_with_sinks_replays_across_plans():
    from paged_kv_decode_23_gb300 import CUDAGraphBatchDecodePagedKV
    page, batch, dtype = 16, 4, BF16
    pg = Pages([4000] * batch, page, 2, 128, "same", "NHD", seed=5)
    pool64 = values(pg.pool)
    i32 = dict(dtype=torch.int32, device="cuda")
    dec = CUDAGraphBatchDecodePagedKV(torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"), torch.zeros(batch + 1, **i32),
                                      torch.zeros(len(pg.host_indices), **i32), torch.zeros(batch, **i32), "NHD")
    q = torch.zeros(batch, 16, 128, dtype=dtype, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros(batch, 16, device="cuda")
    graph = None
    for step, (lens, window, sinks) in enumerate([([4000, 17, 900, 1], 800, 4), ([1, 0, 3999, 2500], 2000, 300),
                                                  ([3900, 3000, 3000, 3000], -1, 9)]):
        part = Pages(lens, page, 2, 128, "same", "NHD", seed=6 + step, spare=len(pg.host_indices))
        part.host_indices %= pg.num_pages  # (pages shared between requests are read alike)
        dec.plan(torch.from_numpy(part.host_indptr), torch.from_numpy(part.host_indices).cuda(),
                 torch.from_numpy(part.last), 16, 2, 128, page, q_data_type=dtype, window_left=window, num_sink_tokens=sinks)
        q.copy_(_q(batch, 16, 128, dtype, seed=step))
        if graph is None:
            dec.run(q, pg.pool, out=o, lse=lse)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                dec.run(q, pg.pool, out=o, lse=lse)
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert dec.check_status() == 0
        assert_decode(q, o, lse, decode_ref(part, pool64, q, window=window, sinks=sinks), pool64, 4000, what=str(step))


def test_captured_runs_without_sinks_take_none_later():
    from paged_kv_decode_23_gb300 import CUDAGraphBatchDecodePagedKV, PkdError
    i32 = dict(dtype=torch.int32, device="cuda")
    dec = CUDAGraphBatchDecodePagedKV(torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"), torch.zeros(2, **i32),
                                      torch.zeros(64, **i32), torch.zeros(1, **i32), "NHD")
    pg = Pages([900], 16, 2, 128, "same", "NHD", seed=9)
    args = (torch.from_numpy(pg.host_indptr), pg.indices, torch.from_numpy(pg.last), 8, 2, 128, 16)
    dec.plan(*args, q_data_type=BF16, window_left=100)
    with pytest.raises(PkdError, match="no sinks"):
        dec.plan(*args, q_data_type=BF16, window_left=100, num_sink_tokens=4)
    dec.plan(*args, q_data_type=BF16, window_left=50)
    # the CUDA-core kernel takes them anyway
    dec = CUDAGraphBatchDecodePagedKV(torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"), torch.zeros(2, **i32),
                                      torch.zeros(64, **i32), torch.zeros(1, **i32), "NHD", use_tensor_cores=False)
    dec.plan(*args, q_data_type=BF16, window_left=100)
    dec.plan(*args, q_data_type=BF16, window_left=100, num_sink_tokens=4)


@pytest.mark.parametrize("pos", ["NONE", "ROPE_LLAMA"])
@pytest.mark.parametrize("kv,d", [("same", 64), ("same", 128), ("same", 256), ("e4m3", 128), ("e4m3", 256)])
def test_instances_with_and_without_sinks_agree(kv, d, pos):
    """A plan whose sinks leave no gap runs an instance that takes sinks, one without them (mostly) another:
    the same bits, for every group of query heads of either kernel."""
    for dtype in (BF16, F16):
        pg = Pages([900, 1, 40, 0, 1333], 16, 2, d, kv, "NHD", seed=12, dtype=dtype)
        for group, tc in ((1, False), (2, False), (3, False), (8, False), (4, True)):
            q = _q(5, 2 * group, d, dtype)
            got = []
            for opt in (dict(num_sink_tokens=5), {}):
                dec = decoder(pg, 2 * group, dtype, use_tensor_cores=tc, pos_encoding_mode=pos, **opt)
                got.append(dec.run(q, pg.pool, return_lse=True))
                assert dec.check_status() == 0
            assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]), (dtype, group, tc)


@pytest.mark.parametrize("tc,pos", [(False, "NONE"), (False, "ROPE_LLAMA"), (True, "ROPE_LLAMA")])
def test_runs_captured_without_sinks_take_them_later_on_these_kernels(tc, pos):
    from paged_kv_decode_23_gb300 import CUDAGraphBatchDecodePagedKV
    i32 = dict(dtype=torch.int32, device="cuda")
    pg = Pages([900, 133], 16, 2, 128, "same", "NHD", seed=14)
    dec = CUDAGraphBatchDecodePagedKV(torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"), torch.zeros(3, **i32),
                                      torch.zeros(128, **i32), torch.zeros(2, **i32), "NHD", use_tensor_cores=tc)
    q = _q(2, 8, 128, BF16)
    o, lse = torch.zeros_like(q), torch.zeros(2, 8, device="cuda")
    graph = None
    for opt in ({}, dict(window_left=100, num_sink_tokens=9), dict(window_left=50), dict(window_left=300, num_sink_tokens=200)):
        dec.plan(torch.from_numpy(pg.host_indptr), pg.indices, torch.from_numpy(pg.last), 8, 2, 128, 16, q_data_type=BF16,
                 pos_encoding_mode=pos, **opt)
        if graph is None:
            dec.run(q, pg.pool, out=o, lse=lse)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                dec.run(q, pg.pool, out=o, lse=lse)
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert dec.check_status() == 0
        ref = decode_ref(pg, values(pg.pool), q, window=opt.get("window_left", -1), sinks=opt.get("num_sink_tokens", 0),
                         pos=None if pos == "NONE" else pos)
        assert_decode(q, o, lse, ref, values(pg.pool), 900, rope=pos != "NONE", what=str(opt))
