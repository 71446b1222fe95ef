"""Page-cache operators on the GPU against references in 64 bits: append (norm, rotation, every
cache type), gather, page copies."""
import numpy as np
import pytest
import torch

from cache_ref import (Pages, assert_rounded, dequantise, half_step, norm_rotate, quantise, to_e4m3)

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def _qkv(n, hq, hkv, d, dtype, seed, fused=True):
    g = torch.Generator().manual_seed(seed)
    if fused:  # views of one projection's output
        x = torch.randn(n, hq + 2 * hkv, d, generator=g).to(dtype).cuda()
        return x.split([hq, hkv, hkv], dim=1)
    return [torch.randn(n, h, d, generator=g).to(dtype).cuda() for h in (hq, hkv, hkv)]


def _f64(t):
    return t.double().cpu().numpy()


def _table(positions, rotary, seed=3):
    """Any float32 table will do as cos and sin; a real one keeps the values in range."""
    from paged_kv_decode_23_gb300 import make_cos_sin_cache
    return make_cos_sin_cache(positions, rotary, rope_theta=1e4)


def _idx(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def check_append(pg, q, k, v, b, pos, q_weight=None, k_weight=None, cos_sin=None, interleaved=False,
                 k_scale=None, v_scale=None, rope_positions=None, eps=1e-6, stream=None, call=None):
    """Runs append on pool `pg` and compares q, the written slots and every other slot."""
    from paged_kv_decode_23_gb300 import append_paged_kv
    b, pos = np.asarray(b), np.asarray(pos)
    live = b >= 0
    pool0 = pg.pool.clone()
    scales0 = pg.scales.clone() if pg.scales is not None else None
    status = pg.status()
    out = torch.full_like(q, 7.0) if q is not None else None
    kw = dict(q_weight=q_weight, k_weight=k_weight, eps=eps, cos_sin_cache=cos_sin, interleaved=interleaved,
              kv_block_scales=pg.scales, k_scale=k_scale, v_scale=v_scale, out=out, status=status,
              rope_positions=None if rope_positions is None else _idx(rope_positions), stream=stream)
    args = (q, k, v, _idx(b), _idx(pos), pg.pool, pg.indptr, pg.indices, pg.layout)
    got = append_paged_kv(*args, **kw) if call is None else call(args, kw)
    torch.cuda.synchronize()
    assert status.item() == 0 and (got is out)
    cs = None if cos_sin is None else cos_sin.cpu().numpy()
    rp = (pos if rope_positions is None else np.asarray(rope_positions))[live]

    def ref(x, w):
        return norm_rotate(_f64(x)[live], None if w is None else _f64(w), eps, cs, rp, interleaved)
    if q is not None:
        want, terms = ref(q, q_weight)
        assert_rounded(out[torch.from_numpy(live).cuda()], want, terms, q.dtype, "q")
        assert (out[torch.from_numpy(~live).cuda()] == 7.0).all(), "padding rows of q were written"
    if k is None:
        return
    kr, kt = ref(k, k_weight)
    vr = _f64(v)[live]
    for i, (x, terms, sc, name) in enumerate(((kr, kt, k_scale, "k"), (vr, np.abs(vr), v_scale, "v"))):
        sc = 1.0 if sc is None else float(np.float32(sc))
        rows = pg.rows(pg.pool, i, b[live], pos[live])
        if pg.kv == "same":
            assert_rounded(rows, x, terms, k.dtype, name)
            if i == 1:
                assert torch.equal(rows, v[torch.from_numpy(live).cuda()])
        elif pg.kv == "e4m3":
            want = to_e4m3(x / sc)
            assert np.array_equal(_f64(rows), want), f"{name}: {(_f64(rows) != want).sum()} codes differ"
        else:
            want, s = quantise(x, sc)
            have, hs = dequantise(rows, pg.rows(pg.scales, i, b[live], pos[live]))
            assert np.array_equal(hs, s), f"{name}: {(hs != s).sum()} scales differ"
            assert np.array_equal(have, want), f"{name}: {(have != want).sum()} codes differ"
    # nothing else changed
    page, slot = pg.where(b[live], pos[live])
    keep = torch.ones(pg.num_pages, pg.page, dtype=torch.bool)
    keep[torch.from_numpy(page.astype(np.int64)), torch.from_numpy(slot.astype(np.int64))] = False
    for now, then in ((pg.pool, pool0), (pg.scales, scales0)):
        if now is None:
            continue
        a, c = (x.view(torch.uint8) if x.element_size() == 1 else x.view(torch.int16) for x in (now, then))
        a, c = (x.movedim(2 if pg.layout == "NHD" else 3, 1)[keep.cuda()] for x in (a, c))
        assert torch.equal(a, c), "a slot that no row names has changed"


# dtype, cache, layout, hq, hkv, d, page, rotary, interleaved, norm
CASES = [
    (BF16, "same", "NHD", 32, 8, 128, 16, 128, False, True),
    (F16, "same", "HND", 5, 1, 64, 8, 64, True, True),
    (BF16, "same", "HND", 4, 4, 256, 32, 48, False, False),
    (F16, "same", "NHD", 0, 3, 128, 64, 0, False, False),
    (BF16, "e4m3", "NHD", 16, 2, 256, 32, 64, True, True),
    (F16, "e4m3", "HND", 6, 3, 128, 16, 128, False, True),
    (BF16, "e4m3", "NHD", 3, 3, 64, 256, 16, False, False),
    (F16, "e4m3", "HND", 2, 1, 128, 8, 0, False, True),
    (BF16, "e2m1", "HND", 32, 8, 128, 16, 128, False, True),
    (F16, "e2m1", "NHD", 12, 3, 64, 8, 64, False, True),
    (BF16, "e2m1", "NHD", 8, 2, 256, 64, 96, True, True),
    (F16, "e2m1", "HND", 1, 1, 128, 16, 32, True, False),
    (BF16, "e2m1", "HND", 0, 5, 128, 32, 0, False, False),
    (F16, "e2m1", "NHD", 7, 7, 256, 16, 256, False, True),
]


@pytest.mark.parametrize("dtype,kv,layout,hq,hkv,d,page,rotary,inter,norm", CASES)
@pytest.mark.parametrize("shape", ["one", "step", "prompts"])
def test_append(dtype, kv, layout, hq, hkv, d, page, rotary, inter, norm, shape):
    rng = np.random.default_rng(hq * 1000 + d + page)
    if shape == "one":
        lens, new = [37], [1]
    elif shape == "step":  # a batch padded behind and, once, within
        lens = rng.integers(1, 300, 13)
        new = [1] * 13
    else:
        lens, new = [700, 1, page, 0, 333], [690, 1, page, 0, 5]
    b = np.repeat(np.arange(len(lens)), new)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)]).astype(np.int64)
    if shape == "step":
        b, pos = np.concatenate([b[:4], [-1], b[4:], [-1, -7]]), np.concatenate([pos[:4], [5], pos[4:], [0, -3]])
    pg = Pages(lens, page, hkv, d, kv, layout, seed=page + d, dtype=dtype)
    q, k, v = _qkv(len(b), hq, hkv, d, dtype, seed=d + hq)
    w = [(1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(i))).cuda() for i in (1, 2)]
    w = [x.to(dtype) if page % 16 == 0 else x for x in w]  # weights of the rows' type, or float32
    scale = dict(k_scale=0.1, v_scale=1.25) if kv != "same" else {}
    check_append(pg, q if hq else None, k, v, b, pos, *(w if norm else (None, None)),
                 cos_sin=_table(int(max(lens)) + 1, rotary) if rotary else None, interleaved=inter, **scale)


@pytest.mark.parametrize("kv", ["e4m3", "e2m1"])
def test_append_codes_of_many_values_are_exact(kv):
    """Enough computed keys that some lie within 32-bit error of a border between two codes (about
    one row in a thousand), and values that lie on borders: v is k's exact codes' borders times
    their scale, and rotation by position 0 leaves exact values in the computed path."""
    n, hkv, d, page = 3000, 8, 128, 16
    pg = Pages([n], page, hkv, d, kv, "NHD", seed=5)
    q, k, v = _qkv(n, 1, hkv, d, BF16, seed=6)
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 2, device="cuda")
    v = v.clone().view(n, hkv, d // 16, 16)
    v[::2] = (border * torch.sign(v[::2].float())).to(BF16) * 0.5 ** (torch.arange(d // 16, device="cuda") % 5).view(-1, 1).to(BF16)
    v = v.view(n, hkv, d)
    w = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(8))).cuda()
    check_append(pg, q, k, v, np.zeros(n, int), np.arange(n), w, w, cos_sin=_table(n, d), k_scale=0.37, v_scale=0.75)
    # without norm, at rotation angle 0: exact values through the computed path
    check_append(pg, q, v.clone(), v, np.zeros(n, int), np.arange(n), cos_sin=_table(n, d),
                 rope_positions=np.zeros(n, int), k_scale=1.0, v_scale=1.0)
    check_append(pg, q, v.clone(), v, np.zeros(n, int), np.arange(n), cos_sin=_table(n, 32), k_scale=1.0, v_scale=1.0)


@pytest.mark.parametrize("kv", ["e4m3", "e2m1"])
@pytest.mark.parametrize("scale", [1 / 17, 1 / 19, 1 / 7, 1 / 5, 1 / 3, 0.1, 1 / 27])
def test_append_codes_next_to_borders(kv, scale):
    """Values of few bits over scales whose rounding puts the quotient within 2^-24 of a border
    between two codes, on either side: 1 / float32(1 / 17) against 17, and the like."""
    n, hkv, d = 400, 4, 128
    pg = Pages([n], 16, hkv, d, kv, "NHD", seed=5)
    g = torch.Generator().manual_seed(3)
    q, k, v = (((torch.randint(-15, 16, (n, h, d), generator=g) * 2.0 ** torch.randint(-3, 4, (n, h, 1), generator=g))
                .to(BF16).cuda()) for h in (2, hkv, hkv))
    check_append(pg, q, k, v, np.zeros(n, int), np.arange(n), k_scale=scale, v_scale=scale)
    # the same values of k through the computed path
    check_append(pg, q, k, v, np.zeros(n, int), np.arange(n), cos_sin=_table(n, d), rope_positions=np.zeros(n, int),
                 k_scale=scale, v_scale=scale)


@pytest.mark.parametrize("kv", ["same", "e4m3", "e2m1"])
def test_append_special_values(kv):
    """Zeros, the type's extremes, subnormals, infinities and NaNs stay in their own rows."""
    n, hkv, d = 12, 2, 128
    pg = Pages([n], 16, hkv, d, kv, "HND", seed=1)
    q, k, v = _qkv(n, 2, hkv, d, BF16, seed=2, fused=False)
    v[0] = 0.0
    v[1] = 3e38
    v[2] = 1e-38
    v[3, 0, 5] = float("inf")
    v[4, 1, 100] = float("-inf")
    v[5] *= 1e-30
    v[6] *= 1e30
    k[0] = 0.0
    k[7, 1, 3] = 3e38
    k[8, 0, 16:32] = 0.0
    check_append(pg, q, k, v, np.zeros(n, int), np.arange(n), k_scale=None if kv == "same" else 0.5)
    v[7, 0, 33] = float("nan")
    k[9, 1, 64] = float("nan")
    from paged_kv_decode_23_gb300 import append_paged_kv
    append_paged_kv(q, k, v, _idx(np.zeros(n)), _idx(np.arange(n)), pg.pool, pg.indptr, pg.indices, "HND",
                    kv_block_scales=pg.scales, k_weight=torch.ones(d, device="cuda"))
    torch.cuda.synchronize()
    for i, (row, head, d0, wide) in enumerate(((9, 1, 64, True), (7, 0, 33, False))):  # k, v
        rows = pg.rows(pg.pool, i, np.zeros(n, int), np.arange(n))
        vals = dequantise(rows, pg.rows(pg.scales, i, np.zeros(n, int), np.arange(n)))[0] if kv == "e2m1" else _f64(rows)
        nan = np.isnan(vals)
        want = np.zeros_like(nan)
        if wide:  # the norm spreads a NaN over its head
            want[row, head] = True
        elif kv == "e2m1":
            want[row, head, d0 // 16 * 16:d0 // 16 * 16 + 16] = True
        else:
            want[row, head, d0] = True
        assert np.array_equal(nan, want)


@pytest.mark.parametrize("kv", ["same", "e4m3", "e2m1"])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_append_norm_of_any_magnitude(kv, eps):
    """bf16 rows whose squares leave the 32-bit range, at either end, and rows of mixed magnitudes."""
    power = [-126, -110, -100, -70, -62, -50, -40, -20, 0, 30, 50, 58, 62, 63, 64, 80, 100, 125]
    n, hkv, d = len(power) + 2, 3, 64
    pg = Pages([n], 16, hkv, d, kv, "NHD", seed=4)
    q, k, v = _qkv(n, 5, hkv, d, BF16, seed=9, fused=False)
    for x in (q, k):
        x.clamp_(-4, 4)  # (times 2^125 that is the type's range)
        for i, p in enumerate(power):
            x[i] = (x[i].double() * 2.0 ** p).to(BF16)
        x[n - 2, :, 3] = 2.0 ** 120
        x[n - 1] = (x[n - 1].double() * 2.0 ** -120).to(BF16)
        x[n - 1, :, 40] = 2.0 ** -70
    w = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(8))).cuda()
    check_append(pg, q, k, v, np.zeros(n, int), np.arange(n), w, w, cos_sin=_table(n, 32), eps=eps,
                 k_scale=None if kv == "same" else 0.4)


def test_append_strides_alignment_and_in_place():
    """Rows and pools that are views: every other token, sliced heads, a pool that is a slice of a
    wider one, one of a (k, v) pair, and q rotated in place."""
    from paged_kv_decode_23_gb300 import append_paged_kv
    n, hq, hkv, d, page = 21, 6, 2, 64, 8
    pg = Pages([30, 9], page, hkv, d, "same", "NHD", seed=3)
    wide = torch.zeros(pg.num_pages, 2, 2 * page, hkv + 1, d, dtype=BF16, device="cuda")
    pg.pool = wide[:, :, 3:3 + page, 1:]
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(2 * n, h + 3, d + 8, generator=g).to(BF16).cuda()[::2, 1:1 + h, 8:] for h in (hq, hkv, hkv))
    b = [0] * 15 + [1] * 6
    pos = list(range(15, 30)) + list(range(3, 9))
    check_append(pg, q, k, v, b, pos, cos_sin=_table(40, d))
    # the same with K and V as two tensors
    kc, vc = (torch.zeros(pg.num_pages, page, hkv, d, dtype=BF16, device="cuda") for _ in range(2))
    want, _ = norm_rotate(_f64(q), cos_sin=_table(40, d).cpu().numpy(), positions=np.array(pos))
    qc = q.clone()
    got = append_paged_kv(qc, k, v, _idx(b), _idx(pos), (kc, vc), pg.indptr, pg.indices, cos_sin_cache=_table(40, d), out=qc)
    assert got is qc
    assert_rounded(qc, want, np.abs(want) + 8, BF16, "in place")
    assert torch.equal(kc, pg.pool[:, 0]) and torch.equal(vc, pg.pool[:, 1])


def test_append_q_alone():
    from paged_kv_decode_23_gb300 import append_paged_kv
    q = torch.randn(5, 3, 128, generator=torch.Generator().manual_seed(0)).half().cuda()
    b, pos = _idx([0, 0, -1, 0, 3]), _idx([4, 1, 2, 0, 3])
    out = torch.zeros_like(q)
    append_paged_kv(q, None, None, b, pos, None, None, None, q_weight=torch.ones(128, device="cuda"), out=out,
                    cos_sin_cache=_table(5, 128))
    want, terms = norm_rotate(_f64(q), np.ones(128), 1e-6, _table(5, 128).cpu().numpy(), np.array([4, 1, 2, 0, 3]))
    live = [0, 1, 3, 4]
    assert_rounded(out[live], want[live], terms[live], F16, "q")
    assert (out[2] == 0).all()


@pytest.mark.parametrize("kv", ["same", "e2m1"])
def test_rows_without_a_slot_are_reported_and_left_out(kv):
    """Bad tokens are found by the kernels' own checks: nothing of them is read or written."""
    from paged_kv_decode_23_gb300 import append_paged_kv, gather_paged_kv
    from paged_kv_decode_23_gb300 import _lib as L
    n, hkv, d, page = 6, 2, 128, 16
    pg = Pages([20, 40], page, hkv, d, kv, "NHD", seed=9)
    q, k, v = _qkv(n, 4, hkv, d, BF16, seed=1)
    good_b, good_pos = [0, 1, 1, 0, 1, 0], [3, 4, 39, 19, 0, 7]

    def run(b, pos, indices=None, **kw):
        st = pg.status()
        pool0 = pg.pool.clone()
        out = torch.full_like(q, 9.0)
        append_paged_kv(q, k, v, _idx(b), _idx(pos), pg.pool, pg.indptr, pg.indices if indices is None else indices,
                        kv_block_scales=pg.scales, out=out, status=st, **kw)
        st2 = pg.status()
        ko = torch.full((n, hkv, d), 5.0, dtype=BF16, device="cuda")
        gather_paged_kv(_idx(b), _idx(pos), pg.pool, pg.indptr, pg.indices if indices is None else indices,
                        kv_block_scales=pg.scales, out=(ko, ko.clone()), status=st2)
        torch.cuda.synchronize()
        changed = (pg.pool.view(torch.uint8) != pool0.view(torch.uint8)).flatten(1).any(1).cpu().numpy()
        pg.pool.copy_(pool0)
        return st.item(), st2.item(), changed, out, ko
    st, st2, changed, out, ko = run(good_b, good_pos)
    assert st == st2 == 0 and set(np.flatnonzero(changed)) == set(pg.where(good_b, good_pos)[0])
    # all rows but row 2 of these have no slot: past the pages, negative, no such sequence
    for b, pos in (([0, 1, 1, 2, 0, 100], [32, 48, 5, 0, -1, 0]), ([1, 0, 1, 2 ** 31 - 1, 1, 0], [2 ** 31 - 1, 1000, 5, 0, 64, 2 ** 30])):
        st, st2, changed, out, ko = run(b, pos)
        assert st == st2 == L.STATUS_BAD_TOKEN
        assert set(np.flatnonzero(changed)) == {pg.where([1], [5])[0][0]}
        assert torch.equal(out, q), "q is written all the same"
        assert (ko[[0, 1, 3, 4, 5]] == 5.0).all() and not (ko[2] == 5.0).all()
    # page ids outside the pool
    ids = pg.indices.clone()
    ids[pg.host_indptr[1]:] = torch.tensor([pg.num_pages, -1, 2 ** 31 - 1], dtype=torch.int32)
    st, st2, changed, out, ko = run([0, 1, 1, 1, 0, 1], [3, 4, 20, 39, 19, 0], indices=ids)
    assert st == st2 == L.STATUS_BAD_PAGE and set(np.flatnonzero(changed)) == set(pg.where([0, 0], [3, 19])[0])
    assert (ko[[1, 2, 3, 5]] == 5.0).all()
    # a rotation position outside the table leaves the whole row out
    st, _, changed, out, _ = run(good_b, good_pos, cos_sin_cache=_table(20, d))
    assert st == L.STATUS_BAD_TOKEN and (out[2] == 9.0).all() and not (out[[0, 1, 3, 4, 5]] == 9.0).any()
    st, _, _, out, _ = run(good_b, good_pos, cos_sin_cache=_table(20, d), rope_positions=_idx([0, -1, 1, 2, 19, 20]))
    assert st == L.STATUS_BAD_TOKEN and (out[[1, 5]] == 9.0).all() and not (out[[0, 2, 3, 4]] == 9.0).any()
    # without a status word the same rows are left out in silence
    append_paged_kv(q, k, v, _idx([7] * n), _idx(good_pos), pg.pool, pg.indptr, pg.indices, kv_block_scales=pg.scales)
    torch.cuda.synchronize()


def test_append_refusals():
    from paged_kv_decode_23_gb300 import PkdError, append_paged_kv
    n, hq, hkv, d = 3, 4, 2, 128
    pg = Pages([10], 16, hkv, d, "same", "NHD")
    q, k, v = _qkv(n, hq, hkv, d, BF16, seed=1)
    b, pos = _idx([0, 0, 0]), _idx([0, 1, 2])

    def run(q=q, k=k, v=v, b=b, pos=pos, pool=pg.pool, indptr=pg.indptr, indices=pg.indices, layout="NHD", **kw):
        append_paged_kv(q, k, v, b, pos, pool, indptr, indices, layout, **kw)
    run()
    bad = [dict(q=q.float()), dict(k=k.half()), dict(v=v[:2]), dict(b=b.long()), dict(pos=pos[:2]), dict(b=b[::2]),
           dict(layout="DNH"), dict(pool=pg.pool.half()), dict(pool=pg.pool[..., :64]), dict(pool=pg.pool[:, :1]),
           dict(indptr=pg.indptr.cpu()), dict(indices=pg.indices.long()), dict(k=None), dict(out=q[:2]),
           dict(q_weight=torch.ones(64, device="cuda")), dict(k_weight=torch.ones(d)), dict(q=q.cpu()),
           dict(q_weight=torch.ones(d, device="cuda"), k_weight=torch.ones(d, device="cuda", dtype=BF16)),
           dict(cos_sin_cache=torch.zeros(9, 64, device="cuda", dtype=F16)), dict(rope_positions=pos),
           dict(cos_sin_cache=torch.zeros(64, 9, device="cuda").T), dict(status=torch.zeros(2, device="cuda", dtype=torch.int32)),
           dict(status=torch.zeros(1, dtype=torch.int32)), dict(pool=pg.pool.view(torch.uint8)),
           dict(kv_block_scales=torch.zeros(pg.shape(8), dtype=torch.uint8, device="cuda")),
           dict(q=None, out=q), dict(q=None, k=None, v=None), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))]
    for kw in bad:
        with pytest.raises(ValueError):
            run(**kw)
    for kw in (dict(cos_sin_cache=torch.zeros(9, 8, device="cuda")), dict(eps=-1.0), dict(q=torch.randn(3, 4, 132, device="cuda").to(BF16)[..., 4:]),
               dict(k=torch.randn(3, 2, 129, device="cuda").to(BF16)[..., :128])):
        with pytest.raises(PkdError):
            run(**kw)
    with pytest.raises(NotImplementedError):
        run(q=q.clone().requires_grad_())


@pytest.mark.parametrize("kv", ["same", "e4m3", "e2m1"])
def test_append_on_another_stream_and_in_a_graph(kv):
    """A captured step replays with new rows, positions and page table in the same tensors."""
    from paged_kv_decode_23_gb300 import append_paged_kv
    lens = [50, 3, 129]
    pg = Pages(lens, 16, 2, 128, kv, "HND", seed=2)
    q, k, v = _qkv(4, 4, 2, 128, BF16, seed=3, fused=False)
    table = _table(200, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check_append(pg, q, k, v, [0, 1, 2, -1], [49, 2, 128, 0], cos_sin=table, stream=side)
    bi, po = _idx([0, 1, 2, -1]), _idx([0, 0, 0, 0])
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    kw = dict(cos_sin_cache=table, kv_block_scales=pg.scales, k_scale=0.75, v_scale=0.5, out=out) if kv != "same" else \
        dict(cos_sin_cache=table, out=out)
    with torch.cuda.graph(graph):
        append_paged_kv(q, k, v, bi, po, pg.pool, pg.indptr, pg.indices, "HND", **kw)
    for seed in (7, 8):
        q2, k2, v2 = _qkv(4, 4, 2, 128, BF16, seed=seed, fused=False)
        b, pos = np.array([2, -1, 0, 1]), np.array([100 + seed, 0, seed, 1])

        def replay(args, kws):
            for t, x in ((q, q2), (k, k2), (v, v2), (bi, _idx(b)), (po, _idx(pos))):
                t.copy_(x)
            out.fill_(7.0)
            graph.replay()
            kws["out"].copy_(out)
            return kws["out"]
        check_append(pg, q2, k2, v2, b, pos, cos_sin=table, call=replay,
                     **({} if kv == "same" else dict(k_scale=0.75, v_scale=0.5)))


# ------------------------------------------------------------------------------ gather
@pytest.mark.parametrize("kv,layout,hkv,d,page,out_dtype", [
    ("same", "NHD", 8, 128, 16, BF16), ("same", "HND", 1, 64, 8, BF16), ("e4m3", "NHD", 2, 256, 32, BF16),
    ("e4m3", "HND", 3, 64, 16, F16), ("e2m1", "HND", 8, 128, 16, BF16), ("e2m1", "NHD", 3, 64, 8, F16),
    ("e2m1", "NHD", 5, 256, 256, F16)])
@pytest.mark.parametrize("scales", [(None, None), (0.3, 2.7)])
def test_gather(kv, layout, hkv, d, page, out_dtype, scales):
    from paged_kv_decode_23_gb300 import gather_paged_kv
    lens = [1, 300, page, 77]
    pg = Pages(lens, page, hkv, d, kv, layout, seed=4)
    rng = np.random.default_rng(1)
    b = np.concatenate([np.repeat(np.arange(4), lens), rng.integers(0, 4, 50), [-1, -1]])
    pos = np.concatenate([np.arange(n) for n in lens] + [rng.integers(0, np.array(lens)[b[-52:-2]]), [0, 9]])
    n = len(b)
    out = tuple(torch.full((n, hkv, d), 5.0, dtype=out_dtype, device="cuda") for _ in range(2))
    got = gather_paged_kv(_idx(b), _idx(pos), pg.pool, pg.indptr, pg.indices, layout, kv_block_scales=pg.scales,
                          k_scale=scales[0], v_scale=scales[1], out=out)
    fresh = gather_paged_kv(_idx(b[:-2]), _idx(pos[:-2]), pg.pool, pg.indptr, pg.indices, layout, kv_block_scales=pg.scales,
                            k_scale=scales[0], v_scale=scales[1], out_dtype=out_dtype)
    torch.cuda.synchronize()
    vals = pg.values16().double().cuda()
    for i in range(2):
        assert got[i] is out[i] and (got[i][-2:] == 5.0).all()
        assert torch.equal(fresh[i], got[i][:-2])
        want = _f64(pg.rows(vals, i, b[:-2], pos[:-2])) * (1.0 if scales[i] is None else float(np.float32(scales[i])))
        # one rounding to the type, one of the product to 32 bits
        tol = (half_step(out_dtype) + 2.0 ** -24) * np.maximum(np.abs(want), float(torch.finfo(out_dtype).tiny))
        assert (np.abs(_f64(got[i][:-2]) - want) <= tol).all()


def test_gather_into_strided_rows():
    from paged_kv_decode_23_gb300 import PkdError, gather_paged_kv
    pg = Pages([40], 16, 2, 128, "same", "NHD", seed=4)
    b, pos = _idx([0] * 40), _idx(np.arange(40))
    want = gather_paged_kv(b, pos, pg.pool, pg.indptr, pg.indices)
    both = torch.zeros(40, 4, 128, dtype=BF16, device="cuda")
    gather_paged_kv(b, pos, pg.pool, pg.indptr, pg.indices, out=(both[:, :2], both[:, 2:]))
    assert torch.equal(both, torch.cat(want, dim=1))
    empty = gather_paged_kv(b[:0], pos[:0], pg.pool, pg.indptr, pg.indices)
    assert empty[0].shape == (0, 2, 128)
    odd = torch.zeros(40, 2, 132, dtype=BF16, device="cuda")
    for bad in (dict(out_dtype=torch.float32), dict(out=(both[:, :3], both[:, :2])), dict(kv_layout="X"),
                dict(out=(both[:, :2].half(), both[:, 2:].half())), dict(out=want, out_dtype=F16)):
        with pytest.raises(ValueError):
            gather_paged_kv(b, pos, pg.pool, pg.indptr, pg.indices, **bad)
    with pytest.raises(PkdError):
        gather_paged_kv(b, pos, pg.pool, pg.indptr, pg.indices, out=(odd[..., :128], odd[..., 4:]))


def test_append_then_gather_returns_what_was_written():
    from paged_kv_decode_23_gb300 import append_paged_kv, gather_paged_kv
    pg = Pages([100, 7], 8, 3, 128, "same", "HND", seed=1)
    q, k, v = _qkv(107, 1, 3, 128, BF16, seed=3)
    b, pos = _idx([0] * 100 + [1] * 7), _idx(list(range(100)) + list(range(7)))
    append_paged_kv(None, k, v, b, pos, pg.pool, pg.indptr, pg.indices, "HND")
    got = gather_paged_kv(b, pos, pg.pool, pg.indptr, pg.indices, "HND")
    assert torch.equal(got[0], k) and torch.equal(got[1], v)


# ------------------------------------------------------------------------------ page copies
@pytest.mark.parametrize("n_pairs,n_pools", [(0, 1), (1, 1), (1, 70), (65, 3), (2100, 2), (300, 258)])
def test_copy_pages(n_pairs, n_pools):
    """Pools of several types and page sizes in one call, more pairs and pools than a launch holds."""
    from paged_kv_decode_23_gb300 import copy_pages
    rng = np.random.default_rng(n_pairs + n_pools)
    pages = 2 * n_pairs + 5
    order = rng.permutation(pages).astype(np.int32)
    src, dst = order[:n_pairs], order[pages - n_pairs:]
    g = torch.Generator().manual_seed(1)
    shapes = [(2, 16, 2, 64), (5, 3), (17,), (2, 8, 4), (4096 + 16,)]
    pools = []
    for i in range(n_pools):
        size = int(np.prod(shapes[i % 5])) if n_pools < 100 or i % 5 else 16
        raw = torch.randint(0, 256, (pages, size), generator=g, dtype=torch.uint8)
        kind = (torch.uint8, BF16, torch.float8_e4m3fn)[i % 3 if size % 2 == 0 else 0]
        pools.append(raw.view(kind).cuda() if kind != torch.float8_e4m3fn else raw.cuda().view(kind))
    want = []
    for t in pools:
        w = t.view(torch.uint8).clone()
        w[torch.from_numpy(dst).long().cuda()] = w[torch.from_numpy(src).long().cuda()]
        want.append(w)
    copy_pages(pools, src, torch.from_numpy(dst))
    torch.cuda.synchronize()
    for t, w in zip(pools, want):
        assert torch.equal(t.view(torch.uint8), w)


def test_copy_pages_of_views_and_refusals():
    from paged_kv_decode_23_gb300 import PkdError, copy_pages
    pool = torch.randn(10, 2, 8, 2, 64, device="cuda")
    before = pool.clone()
    copy_pages(pool[:, 1], [3, 9], [0, 4])  # V alone
    want = before.clone()
    want[[0, 4], 1] = want[[3, 9], 1]
    assert torch.equal(pool, want)
    odd = torch.zeros(10, 33, dtype=torch.uint8, device="cuda")
    odd.copy_(torch.arange(330).view(10, 33) % 251)
    view = odd[:, 1:32]
    keep = odd.clone()
    copy_pages([view], [2], [7])
    keep[7, 1:32] = keep[2, 1:32]
    assert torch.equal(odd, keep)
    for bad in (([0], [0]), ([0, 1], [1, 2]), ([10], [0]), ([0, 1], [3, 3])):
        with pytest.raises(PkdError):
            copy_pages(pool, *bad)
    for pools in ([pool, pool[:9]], [pool.transpose(2, 3)], [pool, pool.cpu()]):
        with pytest.raises(ValueError):
            copy_pages(pools, [0], [1])
    assert torch.equal(pool, want)


def test_copy_pages_in_a_graph_and_on_a_stream():
    from paged_kv_decode_23_gb300 import copy_pages
    pool = torch.arange(40, device="cuda", dtype=torch.int32).view(10, 4).clone()
    src, dst = np.array([1, 2], dtype=np.int32), np.array([8, 9], dtype=np.int32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        copy_pages(pool, src, dst)
    src[:], dst[:] = 0, 0  # the captured launch holds its own lists
    pool[1:3] = -1
    graph.replay()
    torch.cuda.synchronize()
    assert (pool[8:] == -1).all() and pool[0].tolist() == [0, 1, 2, 3]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    copy_pages(pool, [0], [5], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(pool[5], pool[0])


def test_appends_and_copies_queued_on_two_streams_and_in_two_graphs():
    """Two captured steps over pools of their own, replayed on two streams at once: nothing is shared."""
    from paged_kv_decode_23_gb300 import append_paged_kv, copy_pages, gather_paged_kv
    sides = []
    for i, kv in enumerate(("e4m3", "e2m1")):
        pg = Pages([500, 300], 16, 2, 128, kv, "HND", seed=30 + i)
        q, k, v = _qkv(800, 4, 2, 128, BF16, seed=40 + i)
        b, pos = _idx([0] * 500 + [1] * 300), _idx(list(range(500)) + list(range(300)))
        pools = [pg.pool] + ([pg.scales] if pg.scales is not None else [])
        src, dst = pg.host_indices[:2].copy(), np.setdiff1d(np.arange(pg.num_pages), pg.host_indices)[:2]
        sides.append((pg, q, k, v, b, pos, pools, src, dst, torch.cuda.Stream()))

    def step(side):
        pg, q, k, v, b, pos, pools, src, dst, _ = side
        kw = dict(kv_indptr=pg.indptr, kv_indices=pg.indices, kv_layout=pg.layout, kv_block_scales=pg.scales)
        out = append_paged_kv(q, k, v, b, pos, pg.pool, **kw)
        copy_pages(pools, src, dst)
        return (out,) + gather_paged_kv(b, pos, pg.pool, **kw)
    want = [[t.clone() for t in step(s)] for s in sides]
    torch.cuda.synchronize()
    graphs = []
    for s in sides:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step(s)
        graphs.append((g, got))
    for s in sides:
        s[6][0].view(torch.uint8).zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for s, (g, _) in zip(sides, graphs):
            with torch.cuda.stream(s[9]):
                g.replay()
    torch.cuda.synchronize()
    for s, (_, got), w in zip(sides, graphs, want):
        assert all(torch.equal(x, y) for x, y in zip(got, w))
        for t in s[6]:
            raw = t.view(torch.uint8)
            assert torch.equal(raw[torch.from_numpy(s[8]).long()], raw[torch.from_numpy(s[7]).long()])


# ------------------------------------------------------------------------------ scales of a 16-bit cache
def nearest16(x, dtype):
    """fp64 x rounded once to dtype (ties to even), as fp64; exact where x is within 2^-48 of its true
    value and that is no closer to a border."""
    fi = torch.finfo(dtype)
    bits = {BF16: 8, F16: 11}[dtype]
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.maximum(np.frexp(np.where(np.isfinite(x), x, 1.0))[1], np.frexp(fi.tiny)[1])
        step = np.ldexp(1.0, e - bits)
        r = np.rint(x / step) * step
        return np.where(np.abs(r) > fi.max, np.copysign(np.inf, x), r)


@pytest.mark.parametrize("dtype,layout,d", [(BF16, "NHD", 128), (F16, "HND", 64), (BF16, "HND", 256), (F16, "NHD", 128)])
@pytest.mark.parametrize("scales", [(0.5, 4.0), (0.3, 2.7), (1 / 17, 1 / 3)])
def test_append_divides_into_a_16_bit_cache(dtype, layout, d, scales):
    """A 16-bit cache holds k / k_scale and v / v_scale: copied values rounded once from the exact
    quotient, computed ones within their 32-bit error; gather and decode multiply them back."""
    from paged_kv_decode_23_gb300 import BatchDecodePagedKV, append_paged_kv, gather_paged_kv
    n, hq, hkv, page = 45, 4, 2, 16
    ks, vs = (float(np.float32(s)) for s in scales)
    q, k, v = _qkv(n, hq, hkv, d, dtype, seed=d)
    b, pos = [0] * n, np.arange(n)
    w = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(8))).cuda()
    table = _table(n, d // 2)
    pools = []
    for kw, ref in ((dict(), (_f64(k), None)),
                    (dict(cos_sin_cache=table), norm_rotate(_f64(k), None, 0, table.cpu().numpy(), pos)),
                    (dict(k_weight=w, cos_sin_cache=table, interleaved=True),
                     norm_rotate(_f64(k), _f64(w), 1e-6, table.cpu().numpy(), pos, True))):
        pg = Pages([n], page, hkv, d, "same", layout, seed=2, dtype=dtype)
        out = append_paged_kv(q, k, v, _idx(b), _idx(pos), pg.pool, pg.indptr, pg.indices, layout, k_scale=scales[0],
                              v_scale=scales[1], **kw)
        kc, vc = (pg.rows(pg.pool, i, b, pos) for i in range(2))
        assert np.array_equal(_f64(vc), nearest16(_f64(v) / vs, dtype))
        x, terms = ref
        if terms is None:
            assert np.array_equal(_f64(kc), nearest16(x / ks, dtype)) and torch.equal(out, q)
        else:
            assert_rounded(kc, x / ks, terms / ks, dtype, "k")
            flat = slice(d // 2, None)  # dims that are not rotated
            if "k_weight" not in kw:
                assert np.array_equal(_f64(kc)[..., flat], nearest16(x[..., flat] / ks, dtype))
        gk, gv = gather_paged_kv(_idx(b), _idx(pos), pg.pool, pg.indptr, pg.indices, layout, k_scale=scales[0], v_scale=scales[1])
        # two roundings to the type, one of them of the quotient
        for got, want, t in ((gk, x, 0 if terms is None else 2.0 ** -20 * terms), (gv, _f64(v), 0)):
            assert (np.abs(_f64(got) - want) <= 2.01 * half_step(dtype) * np.abs(want) + t + 1e-6).all()
        pools.append(pg)
    if scales == (0.5, 4.0):  # powers of two: the same bits as without scales
        outs = []
        for ks, vs in ((None, None), scales):
            pg = pools[0]
            append_paged_kv(None, k, v, _idx(b), _idx(pos), pg.pool, pg.indptr, pg.indices, layout, k_scale=ks, v_scale=vs)
            dec = BatchDecodePagedKV(torch.zeros(32 << 20, dtype=torch.uint8, device="cuda"), layout)
            dec.plan(torch.from_numpy(pg.host_indptr), pg.indices, torch.from_numpy(pg.last), hq, hkv, d, page, q_data_type=dtype)
            outs.append(dec.run(q[-1:].contiguous(), pg.pool, k_scale=ks, v_scale=vs, return_lse=True))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("scale", [2.0 ** -64, 1e-9, 1 / 17, 0.999, 3.0, 1e9, 2.0 ** 64])
def test_append_into_16_bits_over_any_scale(dtype, scale):
    """Quotients of every magnitude: into the subnormals, past the largest value, and those whose
    32-bit rounding is a border of the 16-bit type; infinities, NaNs and signed zeros."""
    from paged_kv_decode_23_gb300 import append_paged_kv
    n, hkv, d = 300, 2, 64
    g = torch.Generator().manual_seed(3)
    raw = torch.randint(-32768, 32768, (2, n, hkv, d), generator=g, dtype=torch.int32).to(torch.int16).view(dtype).cuda()
    k, v = raw[0], raw[1].clone()
    # few bits over a scale that rounds a simple fraction: quotients next to borders
    v[: n // 2] = (torch.randint(-4095, 4096, (n // 2, hkv, d), generator=g) * 2.0 ** -6).to(dtype).cuda()
    pg = Pages([n], 16, hkv, d, "same", "NHD", seed=2, dtype=dtype)
    append_paged_kv(None, k, v, _idx([0] * n), _idx(np.arange(n)), pg.pool, pg.indptr, pg.indices, k_scale=scale, v_scale=scale)
    s = float(np.float32(scale))
    for i, x in enumerate((k, v)):
        got, want = _f64(pg.rows(pg.pool, i, [0] * n, np.arange(n))), nearest16(_f64(x) / s, dtype)
        assert np.array_equal(got, want, equal_nan=True), f"{(got != want).sum()} differ"
        assert np.array_equal(np.signbit(got[~np.isnan(want)]), np.signbit(want[~np.isnan(want)]))


# ------------------------------------------------------------------------------ large calls
def _large_tokens(lens, n, seed):
    """n rows over the sequences, each token at most once, with one row in nine padding."""
    rng = np.random.default_rng(seed)
    every = np.concatenate([np.stack([np.full(m, i), np.arange(m)], axis=1) for i, m in enumerate(lens)])
    rows = every[rng.permutation(len(every))[:n]]
    b, pos = rows[:, 0].copy(), rows[:, 1].copy()
    b[rng.random(n) < 1 / 9] = -1
    return b, pos


LARGE = {64: (21, 11, 3700, 16), 128: (13, 5, 3400, 32), 256: (7, 3, 3000, 8)}  # hq, hkv, rows, page


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kv", ["same", "e4m3", "e2m1"])
@pytest.mark.parametrize("dtype,layout,inter", [(BF16, "NHD", False), (F16, "HND", True)])
def test_append_of_large_calls(dtype, layout, inter, kv, d):
    """Calls above the size from which groups of lanes take two heads each and warps several items:
    head counts that leave a warp's last heads empty, padding rows all over."""
    hq, hkv, n, page = LARGE[d]
    assert n * (hq + 2 * hkv) * (d // 8) >= 4 * 152 * 2048
    lens = [1500, 1, 2000, 900]
    b, pos = _large_tokens(lens, n, seed=d)
    pg = Pages(lens, page, hkv, d, kv, layout, seed=3, dtype=dtype)
    q, k, v = _qkv(n, hq, hkv, d, dtype, seed=d)
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(i))).cuda() for i in (1, 2))
    rotary = {64: 64, 128: 96, 256: 64}[d]
    scales = {} if kv == "same" else dict(k_scale=0.1, v_scale=1.25)
    check_append(pg, q, k, v, b, pos, qw, kw, cos_sin=_table(2000, rotary), interleaved=inter, **scales)
    if kv != "same":  # copied and computed values in one row
        check_append(pg, q, k, v, b, pos, cos_sin=_table(2000, 16), interleaved=inter, **scales)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype,layout", [(BF16, "HND"), (F16, "NHD")])
def test_append_of_large_calls_over_scales(dtype, layout, d):
    from paged_kv_decode_23_gb300 import append_paged_kv
    hq, hkv, n, page = LARGE[d]
    lens = [1500, 1, 2000, 900]
    b, pos = _large_tokens(lens, n, seed=d + 1)
    live = b >= 0
    pg = Pages(lens, page, hkv, d, "same", layout, seed=3, dtype=dtype)
    q, k, v = _qkv(n, hq, hkv, d, dtype, seed=d)
    w = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(1))).cuda()
    table = _table(2000, 32)
    out = append_paged_kv(q, k, v, _idx(b), _idx(pos), pg.pool, pg.indptr, pg.indices, layout, q_weight=w, k_weight=w,
                          cos_sin_cache=table, k_scale=0.3, v_scale=2.7)
    cs = table.cpu().numpy()
    (wq, tq), (wk, tk) = (norm_rotate(_f64(x)[live], _f64(w), 1e-6, cs, pos[live]) for x in (q, k))
    ks, vs = float(np.float32(0.3)), float(np.float32(2.7))
    assert_rounded(out[torch.from_numpy(live).cuda()], wq, tq, dtype, "q")
    assert_rounded(pg.rows(pg.pool, 0, b[live], pos[live]), wk / ks, tk / ks, dtype, "k")
    assert np.array_equal(_f64(pg.rows(pg.pool, 1, b[live], pos[live])), nearest16(_f64(v)[live] / vs, dtype))


# ------------------------------------------------------------------------------ gather rounds once
def _false_ties(values, dtype, count):
    """float32 scales whose product with one of `values` rounds to a border of dtype in 32 bits, while the
    exact product lies beside it."""
    bits = {BF16: 8, F16: 11}[dtype]
    rng = np.random.default_rng(bits)
    found = []
    while len(found) < count:
        c = float(rng.choice(values))
        border = (2 * int(rng.integers(2 ** (bits - 1), 2 ** bits)) + 1) * 2.0 ** -bits
        s = np.float32(border / c)
        if np.float32(c) * s == np.float32(border) and c * float(s) != border:
            found.append(float(s))
    return found


@pytest.mark.parametrize("kv,out_dtype", [("same", BF16), ("same", F16), ("e4m3", BF16), ("e4m3", F16), ("e2m1", BF16), ("e2m1", F16)])
def test_gather_rounds_once(kv, out_dtype):
    """Every stored value times the scale, rounded once from the exact product."""
    from paged_kv_decode_23_gb300 import gather_paged_kv
    n, hkv, d = 64, 2, 128
    pg = Pages([n], 16, hkv, d, kv, "NHD", seed=4, dtype=out_dtype)
    if kv == "same":  # values of few bits, so that they occur
        pg.pool.copy_((torch.randint(-63, 64, pg.pool.shape, generator=torch.Generator().manual_seed(1)) * 0.125).cuda())
    elif kv == "e4m3":
        pg.pool.copy_((torch.randint(-15, 16, pg.pool.shape, generator=torch.Generator().manual_seed(1)) * 0.25).cuda())
    vals = pg.values16().double().cuda()
    stored = np.unique(np.abs(_f64(vals[pg.indices.long()])))
    b, pos = _idx([0] * n), _idx(np.arange(n))
    want = [_f64(pg.rows(vals, i, [0] * n, np.arange(n))) for i in range(2)]
    scales = _false_ties(stored[stored > 0], out_dtype, 40)
    for ks, vs in zip(scales[::2], scales[1::2]):
        got = gather_paged_kv(b, pos, pg.pool, pg.indptr, pg.indices, kv_block_scales=pg.scales, k_scale=ks, v_scale=vs,
                              out_dtype=out_dtype)
        for x, w, s in zip(got, want, (ks, vs)):
            bad = _f64(x) != nearest16(w * s, out_dtype)
            assert not bad.any(), f"{bad.sum()} of {bad.size} rounded twice at scale {s}"


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("scale", [2.0 ** -64, 1e-13, 0.3, 1.0, 3.3, 1e10, 2.0 ** 64])
def test_gather_of_any_16_bit_value(dtype, scale):
    """Products of every magnitude: into the subnormals and past the largest value; infinities and NaNs."""
    from paged_kv_decode_23_gb300 import gather_paged_kv
    n, hkv, d = 256, 2, 64
    pg = Pages([n], 16, hkv, d, "same", "HND", seed=2, dtype=dtype)
    raw = torch.randint(-32768, 32768, pg.pool.shape, generator=torch.Generator().manual_seed(7), dtype=torch.int32)
    pg.pool = raw.to(torch.int16).view(dtype).cuda()
    got = gather_paged_kv(_idx([0] * n), _idx(np.arange(n)), pg.pool, pg.indptr, pg.indices, "HND", k_scale=scale, v_scale=scale)
    for i in range(2):
        want = nearest16(_f64(pg.rows(pg.pool, i, [0] * n, np.arange(n))) * float(np.float32(scale)), dtype)
        assert np.array_equal(_f64(got[i]), want, equal_nan=True), f"{(_f64(got[i]) != want).sum()} differ"


# ------------------------------------------------------------------------------ derivatives
def test_derivatives_are_refused_not_dropped():
    """Inputs that need a gradient, and dual tensors of forward mode, wherever they come in."""
    import torch.autograd.forward_ad as fwAD
    from paged_kv_decode_23_gb300 import append_paged_kv, gather_paged_kv
    n, d = 3, 128
    pg = Pages([10], 16, 2, d, "same", "NHD")
    q, k, v = _qkv(n, 4, 2, d, BF16, seed=1, fused=False)
    b, pos = _idx([0] * n), _idx(np.arange(n))
    w, table = torch.ones(d, device="cuda"), _table(10, d)

    def append(**kw):
        a = dict(q=q, k=k, v=v, pool=pg.pool, qw=w, kw=w, cs=table, out=torch.zeros_like(q))
        a.update(kw)
        return append_paged_kv(a["q"], a["k"], a["v"], b, pos, a["pool"], pg.indptr, pg.indices, q_weight=a["qw"],
                               k_weight=a["kw"], cos_sin_cache=a["cs"], out=a["out"])

    def gather(pool):
        return gather_paged_kv(b, pos, pool, pg.indptr, pg.indices)
    calls = [(lambda t, x=x: append(**{x: t}), t) for x, t in
             (("q", q), ("k", k), ("v", v), ("qw", w), ("kw", w), ("cs", table))]
    kc, vc = (pg.pool[:, i].clone() for i in range(2))
    calls += [(gather, pg.pool), (lambda t: gather((t, vc)), kc), (lambda t: gather((kc, t)), vc)]
    before = pg.pool.clone()
    for call, t in calls:
        leaf = t.detach().clone().requires_grad_()
        with pytest.raises(NotImplementedError, match="backward"):
            call(leaf)
        with fwAD.dual_level():
            dual = fwAD.make_dual(t.detach().clone(), torch.ones_like(t))
            with pytest.raises(NotImplementedError, match="forward"):
                call(dual)
            with torch.no_grad(), pytest.raises(NotImplementedError, match="forward"):
                call(dual)  # (no_grad does not switch forward mode off)
            call(fwAD.unpack_dual(dual).primal)
        pg.pool.copy_(before)
    with torch.no_grad():
        got = append(q=q.clone().requires_grad_())
    assert torch.equal(got, append())
