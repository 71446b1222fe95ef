"""Eviction from a paged cache against its definition, bit for bit, and the operators of a bounded cache
run together."""
import numpy as np
import pytest
import torch

from bounded_ref import assert_decode, decode_ref, decoder, evict_ref, values
from cache_ref import Pages

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def _weights(pg, lens, seed=0, kind="normal"):
    """Weights of the sequences' tokens; 0 in slots without one."""
    g = torch.Generator().manual_seed(seed)
    shape = (pg.num_pages, pg.hkv, pg.page)
    w = torch.exp(2 * torch.randn(shape, generator=g))
    if kind == "ties":
        w = torch.randint(0, 4, shape, generator=g).float() / 4
    elif kind == "zero":
        w = torch.zeros(shape)
    elif kind == "odd":  # what no sum of weights should hold, but may
        pick = torch.randint(0, 9, shape, generator=g)
        odd = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, -1.0, 1e-42, -1e-42])
        w = torch.where(pick < 8, odd[pick.clamp(max=7)], w)
    keep = torch.zeros(pg.num_pages, 1, pg.page)
    for b, n in enumerate(lens):
        if n > 0:
            page, slot = (torch.from_numpy(np.asarray(x).astype(np.int64)) for x in pg.where(np.full(n, b), np.arange(n)))
            keep[page, 0, slot] = 1
    return torch.where(keep > 0, w, torch.zeros(())).cuda()


def _view(pg, x, b, n):
    """x's entries of sequence b's first n slots: [kv heads, n, ...] from pools [pages, heads, slots, ...]."""
    page, slot = (torch.from_numpy(np.asarray(y).astype(np.int64)) for y in pg.where(np.full(n, b), np.arange(n)))
    return x[page, :, slot].transpose(0, 1)


def _bits(x):
    return x.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


def _pools(pg):
    """Every pool as bits, [pages, kv heads, slots, width], K and V apart."""
    got = []
    for x in (pg.pool, pg.scales):
        if x is not None:
            for kv in (0, 1):
                y = _bits(x.cpu())[:, kv]
                got.append(y if pg.layout == "HND" else y.transpose(1, 2))
    return got


def check_evicted(pg, lens, before, w0, after, w1, kept, budget, sinks, recent, skip=()):
    want_w = w0.cpu().clone()
    want = [x.clone() for x in before]
    for b, n in enumerate(lens):
        if b in skip:
            assert kept is None or (kept[b] == -1).all()
            continue
        full = max(n, min(budget, n))
        rows = _view(pg, w0.cpu(), b, full).numpy()
        for h in range(pg.hkv):
            k, w = evict_ref(rows[h], n, budget, sinks, recent)
            if kept is not None:
                assert np.array_equal(kept[b, h].cpu().numpy(), k), (b, h, n)
            page, slot = pg.where(np.full(n, b), np.arange(n))
            want_w[page, h, slot] = torch.from_numpy(w)
            new = min(n, budget)
            for x, y in zip(before, want):
                src = k[:new]
                y[page[:new], h, slot[:new]] = x[page[src], h, slot[src]]
    assert torch.equal(_bits(w1.cpu()), _bits(want_w))
    for x, y in zip(after, want):
        assert torch.equal(x, y)


def _evict(pg, lens, w, budget, sinks, recent, **kw):
    from paged_kv_decode_23_gb300 import evict_paged_kv
    return evict_paged_kv(pg.pool, w, torch.tensor(lens, dtype=torch.int32, device="cuda"), pg.indptr, pg.indices, budget,
                          pg.layout, num_sink_tokens=sinks, num_recent=recent, kv_block_scales=pg.scales, **kw)


# kv, layout, hkv, d, page, lens, budget, sinks, recent
CASES = [
    ("same", "NHD", 2, 128, 16, [100, 64, 65, 63, 1, 0, 300], 64, 4, 16),
    ("same", "HND", 3, 64, 8, [513, 512, 2000], 512, 0, 0),
    ("same", "NHD", 1, 256, 32, [2049, 2064], 2048, 4, 128),          # the newest overlap their new places
    ("same", "HND", 8, 128, 64, [5000], 700, 1, 699),                 # nothing to choose
    ("same", "NHD", 2, 128, 256, [3000, 299], 300, 300, 0),           # the first tokens alone
    ("e4m3", "NHD", 2, 256, 32, [900, 33, 500], 100, 0, 100),         # the newest alone
    ("e4m3", "HND", 4, 128, 16, [20000], 1, 0, 0),
    ("e4m3", "HND", 1, 64, 16, [400], 399, 5, 33),
    ("e2m1", "NHD", 2, 64, 8, [100, 600, 77], 76, 3, 9),
    ("e2m1", "HND", 2, 128, 16, [1500, 40], 1000, 4, 600),
    ("e2m1", "NHD", 1, 256, 128, [700], 130, 128, 1),
    ("same", "NHD", 2, 64, 16, [40000, 30000], 9000, 4, 1000),
    ("same", "HND", 2, 128, 16, [1025] * 5, 1024, 4, 1000),           # one token more, each
    ("same", "NHD", 2, 64, 16, [40000] + [9] * 40, 9000, 4, 100),     # far longer than the others
    ("e4m3", "HND", 1, 128, 8, [70000, 8, 8], 300, 0, 7),             # and over several CTAs
]


@pytest.mark.parametrize("kind", ["normal", "ties", "zero", "odd"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_eviction_matches_the_definition(case, kind):
    kv, layout, hkv, d, page, lens, budget, sinks, recent = CASES[case]
    pg = Pages(lens, page, hkv, d, kv, layout, seed=case, spare=3)
    w = _weights(pg, lens, seed=case, kind=kind)
    before, w0 = _pools(pg), w.clone()
    status = pg.status()
    kept = _evict(pg, lens, w, budget, sinks, recent, return_kept=True, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    check_evicted(pg, lens, before, w0, _pools(pg), w, kept, budget, sinks, recent)


@pytest.mark.parametrize("seed", range(40))
def test_drawn_evictions(seed):
    rng = np.random.default_rng(seed)
    page, d = int(rng.choice([8, 16, 64])), int(rng.choice([64, 128, 256]))
    top = int(rng.choice([3, 40, 700, 3000]))
    lens = rng.integers(0, top + 1, int(rng.integers(1, 7))).tolist()
    budget = int(rng.integers(1, top + 2))
    sinks = int(rng.integers(0, budget + 1)) if seed % 3 else 0
    recent = int(rng.integers(0, budget - sinks + 1)) if seed % 4 else 0
    kv, layout = ("same", "e4m3", "e2m1")[seed % 3], ("NHD", "HND")[seed // 3 % 2]
    pg = Pages(lens, page, int(rng.choice([1, 2, 3])), d, kv, layout, seed=seed)
    w = _weights(pg, lens, seed=seed, kind=("normal", "ties")[seed % 2])
    before, w0 = _pools(pg), w.clone()
    kept = _evict(pg, lens, w, budget, sinks, recent, return_kept=True)
    check_evicted(pg, lens, before, w0, _pools(pg), w, kept, budget, sinks, recent)


def test_pairs_strides_and_no_kept():
    """K and V apart, a pool inside a larger one, weights with strides."""
    from paged_kv_decode_23_gb300 import evict_paged_kv
    lens, budget, sinks, recent = [300, 90], 80, 4, 20
    pg = Pages(lens, 16, 2, 128, "same", "NHD", seed=1)
    w = _weights(pg, lens)
    before, w0 = _pools(pg), w.clone()
    wide = torch.full((pg.num_pages, 16, 3, 160), 5.0, dtype=BF16, device="cuda")
    k = wide[:, :, 1:, 16:144]
    k.copy_(pg.pool[:, 0])
    v = torch.empty_strided(k.shape, k.stride(), dtype=BF16, device="cuda")
    v.copy_(pg.pool[:, 1])
    big = torch.full((16, pg.num_pages, 2), 7.0, device="cuda")
    ws = big.permute(1, 2, 0)
    ws.copy_(w)
    assert evict_paged_kv((k, v), ws, torch.tensor(lens, dtype=torch.int32, device="cuda"), pg.indptr, pg.indices, budget,
                          num_sink_tokens=sinks, num_recent=recent) is None
    pg.pool[:, 0], pg.pool[:, 1] = k, v
    check_evicted(pg, lens, before, w0, _pools(pg), ws.contiguous(), None, budget, sinks, recent)
    assert (wide[:, :, 0] == 5).all() and (wide[..., :16] == 5).all() and (wide[..., 144:] == 5).all()


@pytest.mark.parametrize("off", [1, 2, 3])
def test_weights_whose_address_is_no_multiple_of_16(off):
    from paged_kv_decode_23_gb300 import evict_paged_kv
    lens = [500, 77, 2000]
    pg = Pages(lens, 8, 3, 64, "e4m3", "HND", seed=off)
    w = _weights(pg, lens, seed=off)
    before, w0 = _pools(pg), w.clone()
    flat = torch.full((w.numel() + 8,), 3.0, device="cuda")
    mine = flat[off:off + w.numel()].view(w.shape)
    mine.copy_(w)
    kept = evict_paged_kv(pg.pool, mine, torch.tensor(lens, dtype=torch.int32, device="cuda"), pg.indptr, pg.indices, 70,
                          "HND", num_sink_tokens=off, num_recent=9, return_kept=True)
    check_evicted(pg, lens, before, w0, _pools(pg), mine, kept, 70, off, 9)
    assert (flat[:off] == 3).all() and (flat[off + w.numel():] == 3).all()


def test_sequences_that_cannot_be_evicted_are_left_alone():
    from paged_kv_decode_23_gb300 import _lib as L
    lens = [300, 200, 250, 100]
    for bad in ("long", "negative", "page", "page below", "table"):
        pg = Pages(lens, 16, 2, 128, "same", "HND", seed=2)
        w = _weights(pg, lens)
        before, w0, status = _pools(pg), w.clone(), pg.status()
        said, want = list(lens), L.STATUS_BAD_TOKEN
        if bad == "long":
            said[1] = 16 * 13 + 1  # one more than its pages hold
        elif bad == "negative":
            said[1] = -5
        elif bad == "table":
            ptr = pg.host_indptr.copy()
            pg.indices = pg.indices[:int(ptr[2]) - 1].contiguous()  # sequence 1 ends behind the list
            said, want = [300, 200, 0, 0], L.STATUS_BAD_TOKEN
        else:
            ids = pg.host_indices.copy()
            ids[pg.host_indptr[1] + 3] = pg.num_pages if bad == "page" else -1
            pg.indices, want = torch.from_numpy(ids).cuda(), L.STATUS_BAD_PAGE
        kept = _evict(pg, said, w, 90, 4, 30, return_kept=True, status=status)
        torch.cuda.synchronize()
        assert int(status) == want, bad
        after = [n if n > 0 else 0 for n in said]
        check_evicted(pg, after, before, w0, _pools(pg), w, kept, 90, 4, 30, skip=(1,))


def test_a_captured_eviction_reads_the_lengths_of_its_replay():
    lens = [500, 300, 400]
    pg = Pages(lens, 16, 2, 128, "e4m3", "NHD", seed=3)
    from paged_kv_decode_23_gb300 import evict_paged_kv
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    w = _weights(pg, lens)
    pool0, w0 = pg.pool.clone(), w.clone()

    def call():
        return evict_paged_kv(pg.pool, w, n, pg.indptr, pg.indices, 128, num_sink_tokens=2, num_recent=40, return_kept=True)

    call()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs, each with its own workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kept = call()
        graphs.append((g, kept))
    for said, (g, kept) in zip(([500, 128, 400], [129, 300, 5]), graphs):
        pg.pool.view(torch.uint8).copy_(pool0.view(torch.uint8))
        w.copy_(w0)
        n.copy_(torch.tensor(said, dtype=torch.int32))
        before = _pools(pg)
        g.replay()
        torch.cuda.synchronize()
        check_evicted(pg, said, before, w0, _pools(pg), w, kept, 128, 2, 40)


def test_two_streams():
    sets = []
    for i in range(2):
        lens = [700 + i, 300]
        pg = Pages(lens, 16, 2, 128, "same", "NHD", seed=4 + i)
        w = _weights(pg, lens, seed=i)
        sets.append((pg, lens, w, _pools(pg), w.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    kept = [_evict(pg, lens, w, 200, 4, 50, return_kept=True, stream=s) for pg, lens, w, _, _, s in sets]
    torch.cuda.synchronize()
    for k, (pg, lens, w, before, w0, _) in zip(kept, sets):
        check_evicted(pg, lens, before, w0, _pools(pg), w, k, 200, 4, 50)


def test_calls_of_different_sizes_from_two_threads():
    """Calls that ask for more and less shared memory, at the same time."""
    import threading
    sets = []
    for i, n in enumerate((30000, 3500)):
        lens = [n] * (2 if i == 0 else 6)
        pg = Pages(lens, 16, 2, 64, "same", "NHD", seed=20 + i)
        w = _weights(pg, lens, seed=i)
        sets.append((pg, lens, w, _pools(pg), w.clone(), pg.pool.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    errors = []

    def work(pg, lens, w, before, w0, pool0, stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(40):
                    pg.pool.copy_(pool0)
                    w.copy_(w0)
                    _evict(pg, lens, w, 1000, 4, 100)
        except Exception as e:  # pragma: no cover
            errors.append(e)

    threads = [threading.Thread(target=work, args=s) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for pg, lens, w, before, w0, _, _ in sets:
        check_evicted(pg, lens, before, w0, _pools(pg), w, None, 1000, 4, 100)


def test_refusals():
    from paged_kv_decode_23_gb300 import PkdError, evict_paged_kv
    lens = [300, 40]
    pg = Pages(lens, 16, 2, 128, "same", "NHD", seed=5)
    w = _weights(pg, lens)
    before, w0 = _pools(pg), w.clone()
    for budget, sinks, recent in ((0, 0, 0), (-1, 0, 0), (10, 11, 0), (10, 5, 6), (10, -1, 0), (10, 0, -1), (2 ** 31, 0, 0), (2 ** 30 + 1, 0, 0),
                                  (10, 2 ** 31 - 1, 2 ** 31 - 1)):
        with pytest.raises(ValueError):
            _evict(pg, lens, w, budget, sinks, recent)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def call(pool=pg.pool, weights=w, lens=n, **kw):
        return evict_paged_kv(pool, weights, lens, pg.indptr, pg.indices, 50, **kw)

    for bad in (w.half(), w[:-1], w.transpose(1, 2), w.cpu(), 3, None):
        with pytest.raises(ValueError):
            call(weights=bad)
    for bad in (n.long(), n[:1], n.cpu(), n.repeat(2)):
        with pytest.raises(ValueError):
            call(lens=bad)
    with pytest.raises(ValueError):
        call(pool=pg.pool.cpu())
    with pytest.raises(ValueError):
        call(pool=pg.pool.view(torch.uint8)[..., :64])
    with pytest.raises(ValueError):
        call(kv_layout="HNS")
    with pytest.raises(PkdError, match="overlap"):
        call(weights=w[:1].expand(pg.num_pages, -1, -1))
    with pytest.raises(PkdError, match="strides"):
        call(pool=pg.pool[:1].expand(pg.num_pages, -1, -1, -1, -1))
    with pytest.raises(PkdError, match="one"):
        call(pool=(pg.pool[:, 0], pg.pool[:, 0]))
    with pytest.raises(NotImplementedError):
        call(weights=w.clone().requires_grad_())
    for x, y in zip(before, _pools(pg)):
        assert torch.equal(x, y)
    assert torch.equal(w, w0)
    # nothing to do
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert evict_paged_kv(pg.pool, w, n[:0], none, pg.indices, 50, return_kept=True).shape == (0, 2, 50)


@pytest.mark.parametrize("kv", ["same", "e4m3", "e2m1"])
def test_a_bounded_cache_step_after_step(kv):
    """Prompts enter, steps decode with key weights and append, the cache is cut back to its budget and
    its pages are given back: attention stays that over the tokens that were kept, whose weights stay
    the sums of what each step gave them."""
    from paged_kv_decode_23_gb300 import PageAllocator, append_paged_kv, evict_paged_kv, make_cos_sin_cache
    dev, page, hq, hkv, d, dtype = torch.device("cuda"), 16, 8, 2, 128, BF16
    budget, sinks, recent, slack = 96, 4, 24, 8
    prompts = [150, 97, 30]
    batch, num_pages = len(prompts), 40
    alloc = PageAllocator(num_pages)
    g = torch.Generator().manual_seed(11)
    shape = (num_pages, 2, page, hkv)
    if kv == "e2m1":
        pool = torch.zeros(shape + (d // 2,), dtype=torch.uint8, device=dev)
        scales = torch.zeros(shape + (d // 16,), dtype=torch.float8_e4m3fn, device=dev)
    else:
        pool, scales = torch.zeros(shape + (d,), dtype=dtype if kv == "same" else torch.float8_e4m3fn, device=dev), None
    weights = torch.zeros(num_pages, hkv, page, device=dev)
    table = [alloc.alloc(-(-n // page)) for n in prompts]
    lens, seen = list(prompts), list(prompts)  # tokens in the cache, tokens so far
    cos_sin = make_cos_sin_cache(400, d)
    from paged_kv_decode_23_gb300 import BatchDecodePagedKV
    dec = BatchDecodePagedKV(torch.zeros(64 << 20, dtype=torch.uint8, device=dev), "NHD")

    def put(counts):
        """New tokens of every sequence behind its others, rotated at their own positions."""
        rows = sum(counts)
        q, k, v = (torch.randn(rows, h, d, generator=g).to(dtype).to(dev) for h in (hq, hkv, hkv))
        seq = np.repeat(np.arange(batch), counts)
        slot = np.concatenate([np.arange(n - c, n) for n, c in zip(lens, counts)])
        true = np.concatenate([np.arange(n - c, n) for n, c in zip(seen, counts)])
        i32 = [torch.from_numpy(x.astype(np.int32)).to(dev) for x in (seq, slot, true)]
        return append_paged_kv(q, k, v, i32[0], i32[1], pool, indptr, indices, cos_sin_cache=cos_sin,
                               rope_positions=i32[2], kv_block_scales=scales)

    def tables():
        ptr = np.zeros(batch + 1, dtype=np.int32)
        np.cumsum([len(t) for t in table], out=ptr[1:])
        return ptr, torch.from_numpy(ptr).to(dev), torch.from_numpy(np.concatenate(table).astype(np.int32)).to(dev)

    host_ptr, indptr, indices = tables()
    put(prompts)
    mine = [np.zeros((hkv, n)) for n in prompts]  # each token's weight, by the reference
    for step in range(3 * slack):
        for b in range(batch):
            if lens[b] % page == 0:
                table[b] = np.concatenate([table[b], alloc.alloc(1)])
            lens[b] += 1
            seen[b] += 1
            mine[b] = np.concatenate([mine[b], np.zeros((hkv, 1))], axis=1)
        host_ptr, indptr, indices = tables()
        q = put([1] * batch)
        last = np.array([(n - 1) % page + 1 for n in lens], dtype=np.int32)
        pg = Pages([1] * batch, page, hkv, d, kv, "NHD")  # (its table and pool are replaced)
        pg.host_indptr, pg.host_indices, pg.last = host_ptr, indices.cpu().numpy(), last
        pg.lens, pg.pool, pg.scales, pg.num_pages = np.array(lens), pool, scales, num_pages
        kv_dt = {"same": dtype, "e4m3": torch.float8_e4m3fn, "e2m1": "e2m1"}[kv]
        dec.plan(host_ptr, indices, last, hq, hkv, d, page, q_data_type=dtype, kv_data_type=kv_dt, key_weights=True)
        o, lse = dec.run(q, pool, kv_block_scales=scales, return_lse=True, key_weights=weights)
        pool64 = values(pool, scales)
        ref = decode_ref(pg, pool64, q)
        assert dec.check_status() == 0
        assert_decode(q, o, lse, ref, pool64, max(lens), what=str(step))
        for b in range(batch):
            mine[b] = mine[b] + ref[3][b].numpy()
        if step % slack == slack - 1:
            before, w0 = _pools(pg), weights.clone()
            n = torch.tensor(lens, dtype=torch.int32, device=dev)
            kept = evict_paged_kv(pool, weights, n, indptr, indices, budget, num_sink_tokens=sinks, num_recent=recent,
                                  kv_block_scales=scales, return_kept=True)
            check_evicted(pg, lens, before, w0, _pools(pg), weights, kept, budget, sinks, recent)
            for b in range(batch):
                new = min(lens[b], budget)
                src = kept[b, :, :new].cpu().numpy()
                mine[b] = np.take_along_axis(mine[b], src, axis=1)
                own = -(-new // page)
                alloc.free(table[b][own:])
                table[b], lens[b] = table[b][:own], new
            # (the weights that moved are the sums, within what the steps' additions rounded off)
            pg.host_indptr, _, ix = tables()
            pg.host_indices = ix.cpu().numpy()
            for b in range(batch):
                got = _view(pg, weights.cpu(), b, lens[b]).numpy()
                assert (np.abs(got - mine[b]) <= 2e-4 * mine[b] + 1e-7).all()
    assert max(lens) == budget and min(lens) < budget  # the short one never reached it
    assert alloc.num_free == num_pages - sum(len(t) for t in table)
    used = torch.zeros(num_pages, page, dtype=torch.bool)
    for t, n in zip(table, lens):
        for i in range(n):
            used[t[i // page], i % page] = True
    assert (weights.cpu().transpose(1, 2)[~used] == 0).all()  # slots without a token hold no weight


def _many(heads, extra=2):
    """So many sequences of `heads` kv heads that a (sequence, kv head) of each would fill two CTAs an SM, and `extra`."""
    return 2 * torch.cuda.get_device_properties(0).multi_processor_count // heads + extra


@pytest.mark.parametrize("kind", ["normal", "ties", "odd"])
@pytest.mark.parametrize("kv,layout", [("same", "NHD"), ("e4m3", "HND"), ("e2m1", "NHD")])
def test_more_sequences_than_the_gpu_holds(kv, layout, kind):
    """CTAs of 256 threads, one a (sequence, kv head): ragged lengths, one sequence past the keys that a CTA can
    hold (8,192) and many past those that it does hold for the average length."""
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 700, _many(8)).tolist()
    lens[0], lens[1], lens[7], lens[-1] = 9500, 8200, 2300, 3000
    pg = Pages(lens, 16, 8, 64, kv, layout, seed=30)
    w = _weights(pg, lens, seed=31, kind=kind)
    before, w0 = _pools(pg), w.clone()
    kept = _evict(pg, lens, w, 256, 4, 37, return_kept=True)
    check_evicted(pg, lens, before, w0, _pools(pg), w, kept, 256, 4, 37)


@pytest.mark.parametrize("kind", ["normal", "ties"])
def test_many_sequences_cut_back_after_a_few_steps(kind):
    """The same CTAs, their keys all in shared memory."""
    lens = np.random.default_rng(2).integers(2049, 2065, _many(8)).tolist()
    pg = Pages(lens, 16, 8, 64, "same", "NHD", seed=32)
    w = _weights(pg, lens, seed=33, kind=kind)
    before, w0 = _pools(pg), w.clone()
    kept = _evict(pg, lens, w, 2048, 4, 128, return_kept=True)
    check_evicted(pg, lens, before, w0, _pools(pg), w, kept, 2048, 4, 128)


def test_more_long_sequences_than_the_gpu_holds():
    """Above 6,000 tokens a sequence (by the pages that the table lists) CTAs of 512 threads, in several waves."""
    from paged_kv_decode_23_gb300 import evict_paged_kv
    lens = np.random.default_rng(3).integers(0, 700, _many(8, 200)).tolist()
    lens[3] = 9000
    pg = Pages(lens, 16, 8, 64, "same", "HND", seed=34)
    w = _weights(pg, lens, seed=35)
    before, w0 = _pools(pg), w.clone()
    indices = torch.cat([pg.indices, torch.zeros(6100 * len(lens) // 16, dtype=torch.int32, device="cuda")])
    kept = evict_paged_kv(pg.pool, w, torch.tensor(lens, dtype=torch.int32, device="cuda"), pg.indptr, indices, 200, "HND",
                          num_sink_tokens=3, num_recent=30, return_kept=True)
    check_evicted(pg, lens, before, w0, _pools(pg), w, kept, 200, 3, 30)


def test_calls_of_one_kernel_that_need_less_and_more_shared_memory_from_two_threads(monkeypatch):
    """Both take the CTAs of a cluster, with 32 and 64 KiB of keys: more than a launch may ask for before its
    kernel's limit is raised, so that a call that lowered it would fail the other's launch.  The threads make the
    library's call alone, over and over, so that the calls meet (sequences inside the budget: nothing moves)."""
    import threading
    from paged_kv_decode_23_gb300 import _lib as L, cache
    sets, packed = [], []
    for i, n in enumerate((30000, 60000)):
        pg = Pages([n], 16, 2, 64, "same", "NHD", seed=40 + i)
        w = _weights(pg, [n], seed=i)
        sets.append((pg, n, w, _pools(pg), w.clone(), torch.tensor([1000], dtype=torch.int32, device="cuda")))
        with monkeypatch.context() as m:
            m.setattr(cache, "_launch", lambda call, dev, stream, *args: packed.append(args))
            cache.evict_paged_kv(pg.pool, w, sets[-1][-1], pg.indptr, pg.indices, 1000, num_sink_tokens=4, num_recent=100)
    torch.cuda.synchronize()
    failed = []
    start = threading.Barrier(len(sets))

    def work(args, stream):
        start.wait()
        for _ in range(20000):
            if L.lib().pkd_evict(*args, stream.cuda_stream):
                failed.append(L.lib().pkd_last_error())
                return

    threads = [threading.Thread(target=work, args=(a, torch.cuda.Stream())) for a in packed]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for pg, n, w, before, w0, _ in sets:
        assert torch.equal(w, w0) and all(torch.equal(x, y) for x, y in zip(before, _pools(pg)))
        _evict(pg, [n], w, 1000, 4, 100)
        check_evicted(pg, [n], before, w0, _pools(pg), w, None, 1000, 4, 100)
